"""Decode calls without a GPU: what they refuse (before anything touches a
device), and the oracle's decode formulas against the expanded form."""

import ctypes as C
import math

import numpy as np
import pytest
import torch

import mla_chunked_context_gb300 as M
from mla_chunked_context_gb300 import _lib
from oracle import mla as O

from test_abi_cpu import built_library  # noqa: F401  (builds the library when it is stale)

INVALID, SMALL_WS, UNSUPPORTED = (_lib.MLA_ERR_INVALID, _lib.MLA_ERR_TOO_SMALL,
                                  _lib.MLA_ERR_UNSUPPORTED)
X = C.c_void_p(4096)        # a pointer that no refused call may follow
ODD = C.c_void_p(4097)
HALF = C.c_void_p(4104)     # 8-byte aligned


def dims(H=4, L=64, P=16, Dn=32, Dv=32, bs=16, dtype=torch.float32, scale=0.1):
    return M.Dims(H, L, P, Dn, Dv, bs, scale, dtype).c()


TC = dict(L=512, P=64, Dn=128, Dv=128, bs=64, dtype=torch.bfloat16)


def append(d, kv_a=X, ld=80, w=X, eps=1e-6, T=3, R=2, qsl=X, lens=X, pos=None, rope=X, n_pos=9,
           inter=0, cache=X, blocks=4, table=X, stride=2, lat=None, q=None, pe=None, pe_ld=16):
    return _lib.lib().mla_append_latent(C.byref(d), kv_a, ld, w, eps, T, R, qsl, lens, pos, rope,
                                        n_pos, inter, cache, blocks, table, stride, lat, q, pe,
                                        pe_ld, None, None)


@pytest.mark.parametrize("change,code", [
    (dict(T=-1), INVALID), (dict(R=-1), INVALID), (dict(blocks=-1), INVALID),
    (dict(stride=0), INVALID), (dict(n_pos=-1), INVALID), (dict(ld=79), INVALID),
    (dict(inter=2), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=math.nan), INVALID),
    (dict(eps=math.inf), INVALID), (dict(kv_a=None), INVALID), (dict(qsl=None), INVALID),
    (dict(lens=None), INVALID), (dict(cache=None), INVALID), (dict(table=None), INVALID),
    (dict(q=X), INVALID), (dict(pe=X), INVALID), (dict(q=X, pe=X, pe_ld=15), INVALID),
    (dict(cache=HALF), INVALID), (dict(lat=HALF), INVALID), (dict(kv_a=ODD), INVALID),
    (dict(w=ODD), INVALID), (dict(rope=ODD), INVALID), (dict(q=ODD, pe=X), INVALID),
    (dict(q=X, pe=ODD), INVALID), (dict(T=1 << 23), UNSUPPORTED),
])
def test_append_refuses(change, code):
    assert append(dims(), **change) == code


def test_append_refuses_shapes_and_takes_nothing():
    assert append(dims(L=63, P=17), ld=80) == UNSUPPORTED      # odd rope with a table
    assert append(dims(H=70000)) == UNSUPPORTED
    assert append(dims(), T=0, kv_a=None) == _lib.MLA_OK
    assert append(dims(), R=0, qsl=None) == _lib.MLA_OK


def attn(d, causal=1, R=2, qsl=X, lens=X, T=3, q=X, cache=X, blocks=4, table=X, stride=2, ws=X,
         wsb=1 << 40, o=X, lse=X):
    return _lib.lib().mla_latent_attn(C.byref(d), causal, R, qsl, lens, T, q, cache, blocks, table,
                                      stride, ws, wsb, o, lse, None, None)


@pytest.mark.parametrize("shape", [dict(), TC])
@pytest.mark.parametrize("change,code", [
    (dict(causal=2), INVALID), (dict(R=-1), INVALID), (dict(T=-1), INVALID),
    (dict(blocks=-1), INVALID), (dict(stride=0), INVALID), (dict(qsl=None), INVALID),
    (dict(lens=None), INVALID), (dict(q=None), INVALID), (dict(cache=None), INVALID),
    (dict(table=None), INVALID), (dict(o=None), INVALID), (dict(T=1 << 23), UNSUPPORTED),
    (dict(q=ODD), INVALID), (dict(o=ODD), INVALID), (dict(lse=ODD), INVALID),
    (dict(cache=HALF), INVALID),
])
def test_latent_attn_refuses(change, code, shape):
    assert attn(dims(**shape), **change) == code


def test_latent_attn_refuses_shapes_and_workspaces():
    assert attn(dims(L=1024, P=16)) == UNSUPPORTED
    d = dims(**TC)
    need = C.c_size_t(0)
    assert _lib.lib().mla_latent_attn_workspace_bytes(C.byref(d), 3, 2, C.byref(need)) == 0
    assert need.value > 0
    assert attn(d, wsb=need.value - 1) == SMALL_WS
    assert attn(d, ws=None) == INVALID
    assert attn(d, ws=HALF) == INVALID
    if not torch.cuda.is_available():
        assert attn(d) == UNSUPPORTED          # no tcgen05 GPU: not handed to other kernels
    assert attn(d, T=0, q=None) == _lib.MLA_OK
    assert attn(d, R=0, q=None) == _lib.MLA_OK
    for bad in (dict(T=-1), dict(R=-1)):
        a = dict(T=1, R=1, **{})
        a.update(bad)
        assert _lib.lib().mla_latent_attn_workspace_bytes(C.byref(d), a["T"], a["R"],
                                                          C.byref(need)) == INVALID
    assert _lib.lib().mla_latent_attn_workspace_bytes(C.byref(d), 1, 1, None) == INVALID


@pytest.mark.parametrize("shape", [dict(), TC])
def test_head_products_refuse(shape):
    L = _lib.lib()
    d = dims(**shape)
    r = C.byref(d)
    for a in ((None, 3, X, 1, X), (X, 3, None, 1, X), (X, 3, X, 1, None), (X, -1, X, 1, X),
              (X, 3, X, 2, X), (ODD, 3, X, 1, X), (X, 3, ODD, 1, X), (X, 3, X, 1, ODD)):
        assert L.mla_absorb_query(r, *a, None) == INVALID
    assert L.mla_absorb_query(r, X, 1 << 23, X, 1, X, None) == UNSUPPORTED
    assert L.mla_absorb_query(r, None, 0, None, 1, None, None) == _lib.MLA_OK
    for a in ((None, 3, X, X), (X, 3, None, X), (X, 3, X, None), (X, -1, X, X), (ODD, 3, X, X),
              (X, 3, ODD, X), (X, 3, X, ODD)):
        assert L.mla_expand_output(r, *a, None) == INVALID
    assert L.mla_expand_output(r, X, 1 << 23, X, X, None) == UNSUPPORTED
    assert L.mla_expand_output(r, None, 0, None, None, None) == _lib.MLA_OK
    if shape:
        assert L.mla_absorb_query(r, HALF, 3, X, 1, X, None) == UNSUPPORTED
        assert L.mla_expand_output(r, X, 3, HALF, X, None) == UNSUPPORTED


def test_bindings_refuse_host_tensors():
    d = M.Dims(2, 64, 16, 32, 32, 16, 0.1, torch.float32)
    z = torch.zeros
    i = dict(dtype=torch.int32)
    with pytest.raises(ValueError, match="current device"):
        M.mla_absorb_query(d, z(1, 2, 48), z(128, 64), z(1, 2, 80))
    with pytest.raises(ValueError, match="current device"):
        M.mla_expand_output(d, z(1, 2, 64), z(128, 64), z(1, 2, 32))
    with pytest.raises(ValueError, match="current device"):
        M.mla_latent_attn(d, True, z(2, **i), z(1, **i), z(1, 2, 80), z(4, 16, 80), z(1, 2, **i),
                          None, z(1, 2, 64))
    with pytest.raises(ValueError, match="current device"):
        M.mla_append_latent(d, z(1, 80), z(2, **i), z(1, **i), None, z(4, 16, 80), z(1, 2, **i))


def test_bindings_refuse_what_is_no_tensor():
    d = M.Dims(2, 64, 16, 32, 32, 16, 0.1, torch.float32)
    z = torch.zeros
    with pytest.raises(ValueError, match="q has to be a tensor"):
        M.mla_absorb_query(d, None, z(128, 64), z(1, 2, 80))
    with pytest.raises(ValueError, match="o_latent has to have 3 dimensions"):
        M.mla_expand_output(d, z(2, 64), z(128, 64), z(1, 2, 32))
    with pytest.raises(ValueError, match="kv_a has to be"):
        M.mla_append_latent(d, z(1, 79), z(2), z(1), None, z(4, 16, 80), z(1, 2))
    for dtype in (torch.int8, "float32"):
        with pytest.raises(ValueError, match="unsupported dtype"):
            M.mla_absorb_query(M.Dims(2, 64, 16, 32, 32, 16, 0.1, dtype), z(1, 2, 48), z(128, 64),
                               z(1, 2, 80))
    with pytest.raises(AttributeError):
        M.mla_absorb_query(object(), z(1, 2, 48), z(128, 64), z(1, 2, 80))


def test_more_than_an_instance_has_room_for():
    d = M.Dims(2, 64, 16, 32, 32, 16, 0.1, torch.float32)
    dec, z = M.LatentDecode(d, 2, 2, device="cpu"), torch.zeros
    i = dict(dtype=torch.int32)
    for T, R in ((3, 2), (2, 3)):
        with pytest.raises(ValueError, match="room"):
            dec(z(T, 2, 48), z(T, 80), z(R + 1, **i), z(R, **i), None, z(4, 16, 80), z(R, 2, **i),
                z(128, 64), z(T, 2, 32))


def test_largest_calls_that_are_taken():
    """One token more than the grids hold is refused, whatever the pointers."""
    n = C.c_size_t(1)
    f = lambda d, T: _lib.lib().mla_latent_attn_workspace_bytes(C.byref(d), T, 1, C.byref(n))
    assert f(dims(H=1), 65535 * 64) == _lib.MLA_OK
    assert f(dims(H=1), 65535 * 64 + 1) == UNSUPPORTED
    assert f(dims(H=65535), 16384) == _lib.MLA_OK
    assert f(dims(H=65535), 16385) == UNSUPPORTED
    assert f(dims(H=65536), 1) == UNSUPPORTED


# ------------------------------------------------------------------ oracle --
def test_oracle_absorbed_equals_expanded():
    """Absorbed attention with the two head products is the expanded
    attention, on ragged requests with several new tokens and one without
    tokens."""
    rng = np.random.default_rng(0)
    od = O.MlaDims(3, 12, 4, 6, 5, 4, 0.37)
    lens, qsl = [9, 0, 5, 2], [0, 2, 3, 4, 7]       # the last: 3 new tokens, 2 tokens
    cache, table = rng.normal(size=(8, 4, 16)), np.array([[3, 1, 6], [0, 0, 0], [2, 5, 0], [7, 0, 0]])
    q, w = rng.normal(size=(7, 3, 10)), rng.normal(size=(3 * 11, 12))
    for causal in (True, False):
        o, lse, mass, size = O.latent_attention(O.absorb_query(q, w, od), cache, table, qsl, lens, od,
                                                causal)
        out = O.expand_output(o, w, od)
        for r, n in enumerate(lens):
            lo, hi = qsl[r], qsl[r + 1]
            rows = np.array([O.context_row(cache, table, r, j, 4) for j in range(n)]).reshape(n, 16)
            kn, v = O.up_project(rows, w, od)
            last = n - (hi - lo) + np.arange(hi - lo)
            vis = np.arange(n)[None, :] <= (last if causal else np.full(hi - lo, n))[:, None]
            ro, rl = O.attention_with_lse(q[lo:hi], kn, rows[:, 12:], v, 0.37, vis)
            np.testing.assert_allclose(out[lo:hi], ro, atol=1e-12)
            np.testing.assert_allclose(lse[:, lo:hi], rl, atol=1e-12)
        assert (mass >= np.abs(np.nan_to_num(o)) - 1e-12).all()


def test_oracle_rotation():
    """Rotations keep norms and depend on the difference of positions only;
    the two pairings are one permutation apart."""
    rng = np.random.default_rng(1)
    tab = O.rope_table(50, 8)
    a, b = rng.normal(size=8), rng.normal(size=8)
    for inter in (False, True):
        d = [O.rotate(a, tab[i + 7], inter) @ O.rotate(b, tab[i], inter) for i in (0, 11, 42)]
        np.testing.assert_allclose(d, d[0], atol=1e-12)
        np.testing.assert_allclose(np.linalg.norm(O.rotate(a, tab[13], inter)), np.linalg.norm(a))
    perm = np.arange(8).reshape(4, 2).T.ravel()
    np.testing.assert_allclose(O.rotate(a, tab[5], True)[perm], O.rotate(a[perm], tab[5], False))
    od = O.MlaDims(1, 4, 8, 1, 1, 4, 1.0)
    x = rng.normal(size=12)
    row = O.latent_row(x, od, np.full(4, 2.0), 0.0, None, False)
    np.testing.assert_allclose(np.mean(row[:4] ** 2), 4.0)
    np.testing.assert_allclose(row[4:], x[4:])
