"""TreeDecode's order of calls on the device."""

import numpy as np
import pytest
import torch

import mla_chunked_context_gb300 as M
from oracle import tree as TR

from test_gpu_decode import DEV, SMALL, _cuda, _no_device_errors, i32, loc, make_cache, make_dims  # noqa: F401
from test_gpu_tree import drafted, same

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
