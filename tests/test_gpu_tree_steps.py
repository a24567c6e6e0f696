"""Steps of trees on the device: the order of TreeDecode's calls, trees of more than
64 nodes, calls of many sequences."""

import numpy as np
import pytest
import torch

import mla_chunked_context_gb300 as M
from oracle import tree as TR

from test_gpu_decode import (DEV, LARGE, SMALL, _cuda, _no_device_errors, i32, loc,  # noqa: F401
                             make_cache, make_dims, normal)
from test_gpu_tree import chain, check_tree, drafted, run_tree, same, tree

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("own_stream", [False, True])
def test_a_captured_verification_between_an_eager_plan_and_commit(own_stream):
    """Two steps, the graph of one verification replayed in each: the second commits
    what it kept of its own trees.  A fresh plan without one is not committed."""
    rng = np.random.default_rng(3)
    dims, _ = make_dims(SMALL, 2, 16, "f32")
    ql, lens, V = [6, 4], [30, 21], 50
    qsl, qsl_d, lens_d, new = loc(ql), i32(loc(ql)), i32(lens), i32([0, 0])
    cache, table = make_cache(rng, lens, 16, SMALL[0] + SMALL[1], dims.dtype)
    cache_d, table_d = cache.to(DEV), table.to(DEV)
    dec = M.TreeDecode(dims, 10, 2, device=DEV)
    p, parents, tokens = torch.zeros(10, V, device=DEV), i32([-1] * 10), i32([0] * 10)
    dec.plan(parents, qsl_d, lens_d)
    dec.verify(p, tokens)
    dec.plan(parents, qsl_d, lens_d)
    with pytest.raises(ValueError, match="verify comes before commit"):
        dec.commit([cache_d], table_d, new)
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        dec.verify(p, tokens, stream=s if own_stream else None)
    ref = cache.double().numpy()
    for k in range(2):
        a = drafted(np.random.default_rng(20 + k), "greedy", ql, V, torch.float32)
        p.copy_(a[0])
        tokens.copy_(i32(a[2]))
        par = i32(a[3])
        parents.copy_(par)
        dec.plan(parents, qsl_d, lens_d)
        graph.replay()
        dec.commit([cache_d], table_d, new)
        torch.cuda.synchronize()
        path, kept = dec.path.cpu().numpy(), dec.num_kept.tolist()
        for r in range(2):
            lo, hi = qsl[r], qsl[r + 1]
            line, nxt = TR.verify(a[0][lo:hi].cpu().double().numpy(), None, a[2][lo:hi], a[3][lo:hi], None, None, 16)
            assert path[r, :kept[r]].tolist() == line and dec.next_tokens[r].item() == nxt
        assert new.tolist() == TR.commit(ref, table.numpy(), qsl, lens, path, kept, 16)
        assert same(cache_d.cpu(), torch.from_numpy(ref).float())


def test_a_tree_of_more_than_64_nodes_keeps_its_masks():
    """Without a word about masks, and a step's attention over them."""
    rng = np.random.default_rng(4)
    dims, od = make_dims(SMALL, 2, 16, "f32")
    L, P, Dn, Dv = SMALL
    ql, lens = [100, 3], [130, 40]
    T, qsl = sum(ql), loc(ql)
    parents = tree(rng, 100) + chain(3)
    cache, table = make_cache(rng, lens, 16, L + P, dims.dtype)
    dec, status = M.TreeDecode(dims, T, 2, device=DEV), i32([0])
    dec.plan(i32(parents), i32(qsl), i32(lens), status)
    mask, pos = TR.layout(parents, qsl, lens, 2)
    assert (dec.tree_mask.cpu().numpy() == mask).all() and (dec.positions.cpu().numpy() == pos).all()
    q, w = normal(rng, T, 2, Dn + P, std=0.5), normal(rng, 2 * (Dn + Dv), L, std=0.1)
    out, lse = torch.empty(T, 2, Dv, device=DEV), torch.empty(2, T, device=DEV)
    after = cache.to(DEV)
    dec(q.to(DEV), normal(rng, T, L + P).to(DEV), None, after, table.to(DEV), w.to(DEV), out, lse, dev_status=status)
    assert status.item() == 0
    check_tree(dims, od, qsl, lens, mask, dec.q_latent, after.cpu(), table, dec.o_latent, lse)


@pytest.mark.parametrize("H,bs", [(48, 64), (48, 16), (4, 64)])
def test_attention_of_more_sequences_than_a_block_has_threads(H, bs):
    """500 sequences, some without tokens: pairs (72 rows a sequence) and single CTAs."""
    rng = np.random.default_rng(H + bs)
    dims, od = make_dims(LARGE, H, bs, "bf16")
    ql = [int(x) for x in rng.integers(0, 4, size=500)]
    lens = [int(x) for x in rng.integers(3, 150, size=500)]
    qsl = loc(ql)
    mask, _ = TR.layout(sum((tree(rng, n) for n in ql), []), qsl, lens, 1)
    cache, table = make_cache(rng, lens, bs, 576, dims.dtype)
    q = normal(rng, qsl[-1], H, 576, std=0.4, dtype=dims.dtype)
    o, lse = run_tree(dims, qsl, lens, mask, q, cache, table)
    check_tree(dims, od, qsl, lens, mask, q, cache, table, o, lse)


def test_layout_and_commit_of_many_sequences():
    rng = np.random.default_rng(12)
    dims, _ = make_dims(SMALL, 1, 16, "f32")
    R = 3000
    ql, lens = [int(x) for x in rng.integers(0, 9, R)], [int(x) for x in rng.integers(9, 40, R)]
    qsl, parents = loc(ql), sum((tree(rng, n) for n in ql), [])
    mask, pos = torch.zeros(qsl[-1], 1, dtype=torch.int64, device=DEV), i32([0] * qsl[-1])
    M.mla_tree_layout(i32(parents), i32(qsl), i32(lens), mask, pos)
    ref, rpos = TR.layout(parents, qsl, lens, 1)
    assert (mask.cpu().numpy() == ref).all() and (pos.cpu().numpy() == rpos).all()
    paths = [TR.ancestors(parents[qsl[r]:qsl[r + 1]])[-1] if n else [] for r, n in enumerate(ql)]
    paths = [p if not p or p[0] == 0 else [0] for p in paths]
    path = torch.tensor([p + [-1] * (8 - len(p)) for p in paths], dtype=torch.int32)
    kept = [len(p) for p in paths]
    cache, table = make_cache(rng, lens, 16, SMALL[0] + SMALL[1], dims.dtype)
    layers, new = [cache.to(DEV), (cache + 1).to(DEV)], i32([0] * R)
    M.mla_commit_tree(dims, path.to(DEV), i32(kept), i32(qsl), i32(lens), layers, table.to(DEV), new)
    for got, first in zip(layers, (cache, cache + 1)):
        want = first.numpy().copy()
        assert new.tolist() == TR.commit(want, table.numpy(), qsl, lens, path.numpy(), kept, 16)
        assert same(got.cpu(), torch.from_numpy(want))
