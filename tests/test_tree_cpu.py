"""Trees of drafted tokens without a GPU: what the calls refuse (before anything
touches a device), and the oracle's own properties."""

import ctypes as C

import numpy as np
import pytest
import torch

import mla_chunked_context_gb300 as M
from mla_chunked_context_gb300 import _lib
from oracle import mla as O
from oracle import tree as T

from test_abi_cpu import built_library  # noqa: F401  (builds the library when it is stale)
from test_decode_cpu import HALF, INVALID, ODD, SMALL_WS, TC, UNSUPPORTED, X, dims

FOUR = C.c_void_p(4100)     # 4-byte aligned


def layout(T=3, R=2, qsl=X, lens=X, parents=X, words=1, mask=X, pos=X):
    return _lib.lib().mla_tree_layout(T, R, qsl, lens, parents, words, mask, pos, None, None)


@pytest.mark.parametrize("change,code", [
    (dict(T=-1), INVALID), (dict(R=-1), INVALID), (dict(words=0), INVALID), (dict(qsl=None), INVALID),
    (dict(lens=None), INVALID), (dict(parents=None), INVALID), (dict(mask=None), INVALID),
    (dict(mask=FOUR), INVALID), (dict(parents=ODD), INVALID), (dict(pos=ODD), INVALID),
    (dict(T=0, parents=None, mask=None), 0), (dict(R=0, qsl=None), 0),
])
def test_layout_refuses(change, code):
    assert layout(**change) == code


def attn(d, R=2, qsl=X, lens=X, mask=X, words=1, T=3, q=X, cache=X, blocks=4, table=X, stride=2, ws=X,
         wsb=1 << 40, o=X, lse=X):
    return _lib.lib().mla_tree_attn(C.byref(d), R, qsl, lens, mask, words, T, q, cache, blocks, table,
                                    stride, ws, wsb, o, lse, None, None)


@pytest.mark.parametrize("shape", [dict(), TC])
@pytest.mark.parametrize("change,code", [
    (dict(R=-1), INVALID), (dict(T=-1), INVALID), (dict(blocks=-1), INVALID), (dict(stride=0), INVALID),
    (dict(words=0), INVALID), (dict(mask=None), INVALID), (dict(mask=FOUR), INVALID),
    (dict(qsl=None), INVALID), (dict(lens=None), INVALID), (dict(q=None), INVALID),
    (dict(cache=None), INVALID), (dict(table=None), INVALID), (dict(o=None), INVALID),
    (dict(T=1 << 23), UNSUPPORTED), (dict(q=ODD), INVALID), (dict(o=ODD), INVALID),
    (dict(lse=ODD), INVALID), (dict(cache=HALF), INVALID), (dict(T=0, q=None), 0), (dict(R=0, q=None), 0),
])
def test_attention_refuses(change, code, shape):
    assert attn(dims(**shape), **change) == code


def test_attention_refuses_workspaces():
    d = dims(**TC)
    need = C.c_size_t(0)
    assert _lib.lib().mla_latent_attn_workspace_bytes(C.byref(d), 3, 2, C.byref(need)) == 0
    assert attn(d, wsb=need.value - 1) == SMALL_WS
    assert attn(d, ws=None) == INVALID
    assert attn(dims(L=1024, P=16)) == UNSUPPORTED
    if not torch.cuda.is_available():
        assert attn(d) == UNSUPPORTED


def verify(dtype=0, T=3, R=2, V=10, p=X, p_ld=10, q=X, q_ld=10, tokens=X, parents=X, qsl=X, u=X, un=X,
           path=X, path_ld=4, kept=X, nxt=X):
    return _lib.lib().mla_verify_tree(dtype, T, R, V, p, p_ld, q, q_ld, tokens, parents, qsl, u, un, path,
                                      path_ld, kept, nxt, None, None)


@pytest.mark.parametrize("change,code", [
    (dict(dtype=2), INVALID), (dict(T=-1), INVALID), (dict(R=-1), INVALID), (dict(V=0), INVALID),
    (dict(p_ld=9), INVALID), (dict(q_ld=9), INVALID), (dict(path_ld=0), INVALID), (dict(p=None), INVALID),
    (dict(tokens=None), INVALID), (dict(parents=None), INVALID), (dict(qsl=None), INVALID),
    (dict(u=None), INVALID), (dict(un=None), INVALID), (dict(path=None), INVALID),
    (dict(kept=None), INVALID), (dict(nxt=None), INVALID), (dict(p=ODD), INVALID), (dict(q=ODD), INVALID),
    (dict(tokens=ODD), INVALID), (dict(path=ODD), INVALID), (dict(u=ODD), INVALID),
    (dict(V=(1 << 24) + 1, p_ld=1 << 25, q_ld=1 << 25), UNSUPPORTED),
    (dict(T=(1 << 24) + 1), UNSUPPORTED), (dict(R=(1 << 24) + 1), UNSUPPORTED), (dict(R=0, qsl=None), 0),
])
def test_verify_refuses(change, code):
    assert verify(**change) == code


def commit(d, R=2, T=3, path=X, path_ld=4, kept=X, qsl=X, lens=C.c_void_p(8192), caches=(4096, 8192),
           layers=2, blocks=4, table=X, stride=2, new=X):
    arr = (C.c_void_p * 2)(*caches) if caches else None
    return _lib.lib().mla_commit_tree(C.byref(d), R, T, path, path_ld, kept, qsl, lens, arr, layers,
                                      blocks, table, stride, new, None, None)


@pytest.mark.parametrize("change,code", [
    (dict(R=-1), INVALID), (dict(T=-1), INVALID), (dict(path_ld=0), INVALID), (dict(layers=-1), INVALID),
    (dict(blocks=-1), INVALID), (dict(stride=0), INVALID), (dict(path=None), INVALID),
    (dict(kept=None), INVALID), (dict(qsl=None), INVALID), (dict(lens=None), INVALID),
    (dict(lens=X), INVALID), (dict(caches=None), INVALID), (dict(caches=(4096, None)), INVALID),
    (dict(caches=(4104, 8192)), INVALID), (dict(table=None), INVALID), (dict(R=0, path=None), 0),
])
def test_commit_refuses(change, code):
    assert commit(dims(), **change) == code


@pytest.mark.parametrize("caches,blocks,code", [
    # a cache has blocks * 16 rows of 80 float32, blocks * 5120 bytes
    ((4096, 4096), 4, INVALID), ((4096, 4096 + 4 * 5120 - 16), 4, INVALID), ((4 * 5120, 4096), 4, INVALID),
    ((4096, 4096 + 4 * 5120), 4, None), ((4096 + 4 * 5120, 4096), 4, None), ((4096, 4096), 0, None),
    ((1 << 20, 0x7FFFFFF0), 1 << 30, INVALID),
])
def test_commit_refuses_caches_that_share_memory(caches, blocks, code):
    if code is None and torch.cuda.is_available():
        pytest.skip("would launch on these addresses")
    rc = commit(dims(), caches=caches, blocks=blocks)
    assert rc == code if code is not None else rc != INVALID


def test_bindings_refuse():
    d, z, i = M.Dims(2, 64, 16, 32, 32, 16, 0.1, torch.float32), torch.zeros, dict(dtype=torch.int32)
    m = z(3, 1, dtype=torch.int64)
    with pytest.raises(ValueError, match="current device"):
        M.mla_tree_layout(z(3, **i), z(2, **i), z(1, **i), m)
    with pytest.raises(ValueError, match="tree_mask has to have 2 dimensions"):
        M.mla_tree_layout(z(3, **i), z(2, **i), z(1, **i), m[:, 0])
    with pytest.raises(ValueError, match="current device"):
        M.mla_tree_attn(d, z(2, **i), z(1, **i), m, z(3, 2, 80), z(4, 16, 80), z(1, 2, **i), None,
                        z(3, 2, 64))
    v = (z(3, **i), z(3, **i), z(2, **i))
    out = (z(1, 4, **i), z(1, **i), z(1, **i))
    with pytest.raises(ValueError, match="current device"):
        M.mla_verify_tree(z(3, 10), None, *v, None, None, *out)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        M.mla_verify_tree(z(3, 10).half(), None, *v, None, None, *out)
    with pytest.raises(ValueError, match="target has to have 2 dimensions"):
        M.mla_verify_tree(z(10), None, *v, None, None, *out)
    with pytest.raises(ValueError, match="current device"):
        M.mla_commit_tree(d, z(1, 4, **i), z(1, **i), z(2, **i), z(1, **i), [z(4, 16, 80)], z(1, 2, **i))
    with pytest.raises(ValueError, match="path has to be a tensor"):
        M.mla_commit_tree(d, None, z(1, **i), z(2, **i), z(1, **i), [], z(1, 2, **i))


def test_tree_decode_refuses():
    d, z, i = M.Dims(2, 64, 16, 32, 32, 16, 0.1, torch.float32), torch.zeros, dict(dtype=torch.int32)
    dec = M.TreeDecode(d, 2, 2, device="cpu")
    for n, r in ((3, 2), (2, 3)):
        with pytest.raises(ValueError, match="room"):
            dec.plan(z(n, **i), z(r + 1, **i), z(r, **i))
    for call in (lambda: dec.verify(z(2, 10), z(2, **i)), lambda: dec.commit([], z(2, 2, **i)),
                 lambda: dec(z(2, 2, 48), z(2, 80), None, z(4, 16, 80), z(2, 2, **i), z(128, 64),
                             z(2, 2, 32))):
        with pytest.raises(ValueError, match="plan comes first"):
            call()


# ------------------------------------------------------------------ oracle --
def test_oracle_chain_is_causal():
    rng = np.random.default_rng(0)
    od = O.MlaDims(3, 12, 4, 6, 5, 4, 0.37)
    lens, qsl = [9, 5, 2], [0, 3, 4, 7]             # the last: 3 new tokens, 2 tokens
    cache, table = rng.normal(size=(8, 4, 16)), np.array([[3, 1, 6], [2, 5, 0], [7, 0, 0]])
    q = rng.normal(size=(7, 3, 16))
    mask, pos = T.layout([-1, 0, 1, -1, -1, 0, 1], qsl, lens, 1)
    assert pos.tolist() == [6, 7, 8, 4, -1, 0, 1]
    a = O.latent_attention(q, cache, table, qsl, lens, od, True)
    b = T.tree_attention(q, cache, table, qsl, lens, mask, od)
    for x, y in zip(a, b):
        np.testing.assert_array_equal(x, y)


@pytest.mark.parametrize("kids", [1, 2, 3])
@pytest.mark.parametrize("drawn", [True, False])
def test_oracle_tokens_follow_the_target(kids, drawn):
    """The first token behind the root (a kept child's or the next token) has the
    target's probabilities: 40000 walks, each share within 5 standard
    deviations."""
    rng = np.random.default_rng(kids)
    V, N = 5, 40000
    p, q = rng.dirichlet(np.ones(V)), rng.dirichlet(np.ones(V))
    count = np.zeros(V)
    target, draft = np.tile(p, (kids + 1, 1)), np.tile(q, (kids + 1, 1))
    for _ in range(N):
        x = rng.choice(V, kids, p=q) if drawn else np.argsort(-q)[:kids]
        tokens = [0] + [int(v) for v in x]
        path, nxt = T.verify(target, draft if drawn else None, tokens, [-1] + [0] * kids,
                             rng.random(kids + 1), rng.random(), 2)
        count[tokens[path[1]] if len(path) > 1 else nxt] += 1
    assert (np.abs(count / N - p) < 5 * np.sqrt(p * (1 - p) / N)).all()


def test_oracle_commit():
    cache = np.arange(24.0).reshape(4, 3, 2)
    lens = T.commit(cache, [[2, 0], [3, 1]], [0, 4, 5], [6, 2], [[0, 2, 3], [0, -1, -1]], [3, 1], 3)
    assert lens == [5, 2]
    # positions 2, 4, 5 -> 2, 3, 4: rows 2 of block 2, then 1 and 2 of block 0 to 0 and 1
    assert cache[0].tolist() == [[2.0, 3.0], [4.0, 5.0], [4.0, 5.0]]
    assert cache[3].tolist() == [[18.0, 19.0], [20.0, 21.0], [22.0, 23.0]]
