"""Calls on drafted trees at the edges of what their documentation allows: masks
shorter and longer than the trees, rows that are no probabilities, the largest
vocabulary, two calls at once, repeated calls, guarded outputs.  Tolerances as in
test_gpu_tree.py, whose helpers these are."""

import math

import numpy as np
import pytest
import torch

import mla_chunked_context_gb300 as M
from oracle import tree as TR

from test_gpu_decode import (DEV, LARGE, ODD, SMALL, _cuda, _no_device_errors, i32, loc,  # noqa: F401
                             make_cache, make_dims, normal)
from test_gpu_tree import (chain, check_tree, check_verify, drafted, masks, rows, run_tree, run_verify, same,
                           status_word, tree, words)

pytestmark = [pytest.mark.gpu,
              pytest.mark.filterwarnings("ignore::RuntimeWarning")]


# -------------------------------------------------------------- attention --
@pytest.mark.parametrize("W", [1, 2, 40])
@pytest.mark.parametrize("shape,dtype,H", [(LARGE, "bf16", 128), (LARGE, "bf16", 2), (SMALL, "f32", 3)])
def test_masks_of_other_lengths_than_the_trees(shape, dtype, H, W):
    """Bits that a mask has no words for count as 0; words beyond the tree count
    for nothing, whatever they hold."""
    rng = np.random.default_rng(W)
    dims, od = make_dims(shape, H, 64, dtype)
    ql, lens = [100, 30, 1], [150, 30, 7]
    qsl = loc(ql)
    mask = rng.integers(-(1 << 63), (1 << 63) - 1, size=(qsl[-1], W), dtype=np.int64)
    cache, table = make_cache(rng, lens, 64, shape[0] + shape[1], dims.dtype)
    q = normal(rng, qsl[-1], H, shape[0] + shape[1], std=0.4, dtype=dims.dtype)
    o, lse = run_tree(dims, qsl, lens, mask, q, cache, table)
    check_tree(dims, od, qsl, lens, mask, q, cache, table, o, lse)


@pytest.mark.parametrize("H", [128, 24])
def test_many_ragged_trees(H):
    """Several units a cluster, several clusters a unit, slots without tokens."""
    rng = np.random.default_rng(H)
    dims, od = make_dims(LARGE, H, 32, "bf16")
    ql = [int(x) for x in rng.integers(0, 12, size=70)]
    lens = [int(x) for x in rng.integers(0, 400, size=70)]
    lens[7] = 3000
    qsl = [x + 1 for x in loc(ql)]
    T = qsl[-1] + 2
    mask = np.full((T, 1), -1, dtype=np.int64)
    mask[1:-2] = masks(rng, "tree", ql)
    cache, table = make_cache(rng, lens, 32, 576, dims.dtype)
    q = normal(rng, T, H, 576, std=0.4, dtype=dims.dtype)
    o, lse = run_tree(dims, qsl, lens, mask, q, cache, table)
    check_tree(dims, od, qsl, lens, mask, q, cache, table, o, lse)
    o2, lse2 = run_tree(dims, qsl, lens, mask, q, cache, table)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_locations_beyond_the_tokens_and_none():
    """Locations are clamped to the tokens; lse may be left out."""
    rng = np.random.default_rng(1)
    dims, od = make_dims(LARGE, 16, 16, "bf16")
    lens, qsl = [40, 50], [0, 4, 7]
    mask = masks(rng, "tree", [4, 3])
    cache, table = make_cache(rng, lens, 16, 576, dims.dtype)
    q = normal(rng, 7, 16, 576, std=0.4, dtype=dims.dtype)
    o, lse = run_tree(dims, [0, 4, 99], lens, mask, q, cache, table)
    check_tree(dims, od, qsl, lens, mask, q, cache, table, o, lse)
    o2 = torch.empty_like(o)
    ws = torch.empty(M.mla_latent_attn_workspace_bytes(dims, 7, 2), dtype=torch.uint8, device=DEV)
    M.mla_tree_attn(dims, i32(qsl), i32(lens), words(mask), q.to(DEV), cache.to(DEV), table.to(DEV), ws, o2)
    assert torch.equal(o, o2)


# ----------------------------------------------------------------- verify --
@pytest.mark.parametrize("mode", ["draft", "point", "greedy"])
def test_verify_the_largest_vocabulary(mode):
    rng = np.random.default_rng(3)
    V = 1 << 24
    p = np.zeros((3, V), np.float32)
    p[:, rng.integers(0, V, 1000)] = 1e-3
    p[:, [0, V - 1, 12345678]] = [0.25, 0.5, 0.125]
    q = np.roll(p, 1, axis=1)
    pd, qd = torch.from_numpy(p).to(DEV), torch.from_numpy(q).to(DEV)
    for u in ([0.1, 0.2, 0.3], [0.99, 0.98, 0.97]):
        for un in (0.0, 0.3, 0.7, 1 - 2.0 ** -24):
            args = (pd, qd if mode == "draft" else None, [0, V - 1, 12345678], [-1, 0, 0], [0, 3],
                    *((None, None) if mode == "greedy" else (np.float32(u), [un])))
            check_verify(run_verify(*args, 3), *args, 3)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf, -1.0, 5.0, 1e30])
@pytest.mark.parametrize("mode", ["draft", "point"])
def test_verify_of_rows_that_are_no_probabilities(mode, bad):
    """What such rows give is not specified, but the call ends and its results are
    nodes of the tree and tokens of the vocabulary."""
    rng = np.random.default_rng(4)
    V, sizes = 5000, [12] * 40
    p, q, tokens, parents, qsl, u, un = drafted(rng, mode, sizes, V, torch.float32)
    for t in (p, q):
        if t is not None:
            t[torch.rand(t.shape, device=DEV) < 0.01] = bad
    p[24:36] = bad
    for uu, unn in ((u, un), (np.full_like(u, bad), np.full_like(un, bad))):
        path, kept, nxt = run_verify(p, q, tokens, parents, qsl, uu, unn, 6)
        assert ((nxt >= 0) & (nxt < V)).all() and ((kept >= 1) & (kept <= 6)).all()
        for r in range(40):
            line = path[r, :kept[r]].tolist()
            assert line[0] == 0 and (path[r, kept[r]:] == -1).all()
            assert all(parents[12 * r + b] == a for a, b in zip(line, line[1:]))


def test_verify_twice_and_without_tokens():
    rng = np.random.default_rng(5)
    args = drafted(rng, "draft", [7] * 30, 3001, torch.float32)
    a, b = run_verify(*args, 5), run_verify(*args, 5)
    assert all((x == y).all() for x, y in zip(a, b))
    p = torch.zeros(0, 100, device=DEV)
    path, kept, nxt = run_verify(p, p, [], [], [0, 0, 0], np.zeros(0), [0.5, 0.5], 4)
    assert (path == -1).all() and (kept == 0).all() and (nxt == -1).all()
    none = torch.zeros(0, 4, dtype=torch.int32, device=DEV)
    M.mla_verify_tree(args[0], None, i32(args[2]), i32(args[3]), i32([0]), None, None, none, i32([]), i32([]))


# -------------------------------------------------------------- all calls --
def guarded(shape, dtype, fill, guard=64):
    """A tensor inside a larger one, whose ends a test looks at."""
    n = int(np.prod(shape))
    whole = torch.full((n + 2 * guard,), fill, dtype=dtype, device=DEV)
    return whole[guard:guard + n].view(shape), whole


def intact(whole, n, fill, guard=64):
    ends = torch.cat([whole[:guard], whole[guard + n:]])
    return bool((ends == fill).all())


@pytest.mark.parametrize("shape,dtype,H", [(LARGE, "bf16", 128), (LARGE, "bf16", 6), (ODD, "bf16", 5), (SMALL, "f32", 3)])
def test_nothing_is_written_beside_the_outputs(shape, dtype, H):
    rng = np.random.default_rng(H)
    dims, od = make_dims(shape, H, 16, dtype)
    L, P = shape[:2]
    ql, lens = [9, 0, 70, 3], [40, 5, 200, 3]
    qsl, T, R, V = loc(ql), sum(ql), 4, 333
    parents = sum((tree(rng, n) for n in ql), [])
    mask, mask_w = guarded((T, 2), torch.int64, 5)
    pos, pos_w = guarded((T,), torch.int32, 5)
    M.mla_tree_layout(i32(parents), i32(qsl), i32(lens), mask, pos)
    cache, table = make_cache(rng, lens, 16, L + P, dims.dtype)
    cache_g, cache_w = guarded(tuple(cache.shape), dims.dtype, 5.0, 1024)
    cache_g.copy_(cache)
    o, o_w = guarded((T, H, L), dims.dtype, 5.0, 1024)
    lse, lse_w = guarded((H, T), torch.float32, 5.0)
    need = M.mla_latent_attn_workspace_bytes(dims, T, R)
    ws, ws_w = guarded((need,), torch.uint8, 5, 4096)
    q = normal(rng, T, H, L + P, std=0.4, dtype=dims.dtype)
    M.mla_tree_attn(dims, i32(qsl), i32(lens), mask, q.to(DEV), cache_g, table.to(DEV), ws, o, lse)
    p, qd, tokens, _, _, u, un = drafted(rng, "draft", ql, V, torch.float32)
    path, path_w = guarded((R, 5), torch.int32, 5)
    kept, kept_w = guarded((R,), torch.int32, 5)
    nxt, nxt_w = guarded((R,), torch.int32, 5)
    new, new_w = guarded((R,), torch.int32, 5)
    f = lambda x: torch.from_numpy(x).to(DEV)  # noqa: E731
    M.mla_verify_tree(p, qd, i32(tokens), i32(parents), i32(qsl), f(u), f(un), path, kept, nxt)
    M.mla_commit_tree(dims, path, kept, i32(qsl), i32(lens), [cache_g], table.to(DEV), new)
    torch.cuda.synchronize()
    assert intact(mask_w, 2 * T, 5) and intact(pos_w, T, 5) and intact(cache_w, cache.numel(), 5.0, 1024)
    assert intact(o_w, T * H * L, 5.0, 1024) and intact(lse_w, H * T, 5.0) and intact(ws_w, need, 5, 4096)
    assert intact(path_w, 5 * R, 5) and all(intact(w, R, 5) for w in (kept_w, nxt_w, new_w))
    ref = cache.double().numpy()
    TR.commit(ref, table.numpy(), qsl, lens, path.cpu().numpy(), kept.tolist(), 16)
    assert same(cache_g.cpu(), torch.from_numpy(ref).to(dims.dtype))


def test_two_streams_at_once():
    """Steps of two batches on two streams, each with its own instance, many times:
    as one after the other."""
    rng = np.random.default_rng(9)
    H, V = 32, 20000
    dims, _ = make_dims(LARGE, H, 64, "bf16")

    class Side:
        def __init__(self, ql, lens):
            self.qsl, self.lens, T = i32(loc(ql)), i32(lens), sum(ql)
            self.cache, self.table = (x.to(DEV) for x in make_cache(rng, lens, 64, 576, dims.dtype))
            self.first = self.cache.clone()
            self.q = normal(rng, T, H, 576, std=0.4, dtype=dims.dtype).to(DEV)
            self.p, self.d, tok, par, _, u, un = drafted(rng, "draft", ql, V, torch.float32)
            self.tok, self.par = i32(tok), i32(par)
            self.u, self.un = torch.from_numpy(u).to(DEV), torch.from_numpy(un).to(DEV)
            self.dec = M.TreeDecode(dims, T, len(ql), device=DEV)
            self.o = torch.zeros(T, H, 512, dtype=dims.dtype, device=DEV)
            self.new = i32([0] * len(ql))

        def step(self):
            d = self.dec
            d.plan(self.par, self.qsl, self.lens)
            M.mla_tree_attn(dims, self.qsl, self.lens, d.tree_mask[:self.q.shape[0]], self.q, self.cache,
                            self.table, d.workspace, self.o)
            d.verify(self.p, self.tok, self.u, self.un, draft=self.d)
            d.commit([self.cache], self.table, self.new)

        def results(self):
            d = self.dec
            return [t.clone() for t in (self.o, self.cache, self.new, d.path, d.num_kept, d.next_tokens)]

    a, b = Side([9] * 20, [300] * 20), Side([16, 3, 30], [2000, 70, 90])
    alone = []
    for side in (a, b):
        side.step()
        torch.cuda.synchronize()
        alone.append(side.results())
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(10):
        for side in (a, b):
            side.cache.copy_(side.first)
            side.o.zero_()
        torch.cuda.synchronize()
        for side, s in zip((a, b), streams):
            with torch.cuda.stream(s):
                side.step()
        torch.cuda.synchronize()
        for side, ref in zip((a, b), alone):
            for x, y in zip(side.results(), ref):
                assert same(x, y) if x.is_floating_point() else torch.equal(x, y)


def test_chained_calls_back_to_back():
    """The calls of a step follow each other without a pause, twenty steps deep, and
    each step starts from what the one before left."""
    rng = np.random.default_rng(11)
    dims, od = make_dims(SMALL, 4, 16, "f32")
    n, R, V = 6, 5, 400
    lens = [int(x) for x in rng.integers(10, 60, R)]
    cache, table = make_cache(rng, [x + 200 for x in lens], 16, 80, dims.dtype)
    ref, ref_lens = cache.double().numpy(), list(lens)
    cache, table_d = cache.to(DEV), table.to(DEV)
    qsl = loc([n] * R)
    len_d = [i32([x + n for x in lens]), i32([0] * R)]
    steps = []
    for _ in range(20):
        steps.append(drafted(rng, "point", [n] * R, V, torch.float32))
    on_device = [(p, i32(t), i32(par), torch.from_numpy(u).to(DEV), torch.from_numpy(un).to(DEV))
                 for p, _, t, par, _, u, un in steps]
    dec = M.TreeDecode(dims, n * R, R, max_path=n, device=DEV)
    kv = [normal(rng, n * R, 80) for _ in steps]
    kv_d = [x.to(DEV) for x in kv]
    qsl_d, got = i32(qsl), []
    torch.cuda.synchronize()
    for (p, t, par, u, un), x in zip(on_device, kv_d):
        dec.plan(par, qsl_d, len_d[0])
        M.mla_append_latent(dims, x, qsl_d, len_d[0], None, cache, table_d)
        dec.verify(p, t, u, un)
        dec.commit(cache, table_d, len_d[1])
        got.append((dec.path.clone(), dec.num_kept.clone(), dec.next_tokens.clone()))
        len_d[0] = len_d[1] + n                        # the next step's new tokens behind the kept ones
        len_d[1] = torch.empty_like(len_d[1])
    torch.cuda.synchronize()
    for (p, _, t, par, _, u, un), x, (path, kept, nxt) in zip(steps, kv, got):
        full = [v + n for v in ref_lens]
        for r in range(R):
            for i in range(n):
                j = ref_lens[r] + i
                ref[table[r, j // 16], j % 16] = x[qsl[r] + i].double().numpy()
        check_verify((path.cpu().numpy(), kept.cpu().numpy(), nxt.cpu().numpy()), p, None, t, par, qsl, u, un, n)
        ref_lens = TR.commit(ref, table.numpy(), qsl, full, path.cpu().numpy(), kept.tolist(), 16)
    assert len_d[0].tolist() == [v + n for v in ref_lens]
    assert same(cache.cpu(), torch.from_numpy(ref).float())


@pytest.mark.parametrize("n,W", [(16384, 256), (16385, 257), (40000, 1)])
def test_layout_of_long_chains(n, W):
    """Nodes from 16384 on count as without a parent."""
    mask = torch.full((n, W), 0x0707, dtype=torch.int64, device=DEV)
    pos, status = i32([-77] * n), status_word()
    M.mla_tree_layout(i32(chain(n)), i32([0, n]), i32([n + 5]), mask, pos, status)
    most = min(n, 16384)
    assert status.item() == (M.MLA_STATUS_BAD_TREE if n > 16384 else 0)
    assert pos.tolist() == list(range(5, 5 + most)) + [5] * (n - most)
    bits = np.arange(64 * W)
    for i in (0, 1, 63, 64, 1023, 1024, 1025, 9999, most - 1, n - 1):
        want = bits <= i if i < most else bits == i
        got = np.unpackbits(mask[i].cpu().numpy().view(np.uint8), bitorder="little").astype(bool)
        assert (got == want).all()


def test_commit_takes_layers_in_any_order_but_none_twice():
    """Views of one allocation, in an order that neither rises nor falls; a cache
    listed twice, whose rows would move twice, is refused and stays as it was."""
    rng = np.random.default_rng(29)
    dims, _ = make_dims(SMALL, 2, 16, "f32")
    cache, table = make_cache(rng, [40], 16, SMALL[0] + SMALL[1], dims.dtype)
    whole = torch.stack([cache + l for l in range(4)]).to(DEV)
    before, new = whole.clone(), i32([0])
    path, kept, qsl, lens = i32([[0, 2, 4, 5]]), i32([4]), i32([0, 8]), i32([40])
    for bad in ([whole[0], whole[0]], [whole[2], whole[1], whole[3], whole[1]]):
        with pytest.raises(M.MlaError, match="invalid argument"):
            M.mla_commit_tree(dims, path, kept, qsl, lens, bad, table.to(DEV), new)
    assert torch.equal(whole.view(torch.int32), before.view(torch.int32)) and new.item() == 0
    M.mla_commit_tree(dims, path, kept, qsl, lens, [whole[l] for l in (2, 0, 3, 1)], table.to(DEV), new)
    for l in range(4):
        ref = before[l].cpu().numpy()
        TR.commit(ref, table.numpy(), [0, 8], [40], [[0, 2, 4, 5]], [4], 16)
        assert (whole[l].cpu().numpy().view(np.int32) == ref.view(np.int32)).all()
    assert new.item() == 36
