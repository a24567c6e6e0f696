"""What tokens get that see a cache row with an infinity: NaN where its score is
+inf; where it is -inf, what the other keys give, but for the infinite column of the
output, which may be NaN.  Tolerances as in test_gpu_tree.py."""

import math

import numpy as np
import pytest
import torch

from oracle import mla as O
from oracle import tree as TR

from test_gpu_decode import (F, LARGE, SMALL, _cuda, _no_device_errors, f64, loc, make_cache, make_dims,  # noqa: F401
                             normal, run_attn, unit, within)
from test_gpu_tree import chain, run_tree, tree

pytestmark = [pytest.mark.gpu, pytest.mark.filterwarnings("ignore::RuntimeWarning")]


def attend(q, cache, table, sees, r, od):
    """One token over the positions `sees`: (o, lse, sum p|c|, largest sum |q||c|)."""
    L = od.kv_lora_rank
    if not sees:
        return np.zeros((len(q), L)), np.full(len(q), -np.inf), np.zeros((len(q), L)), np.zeros(len(q))
    c = np.stack([O.context_row(cache, table, r, j, od.block_size) for j in sees]).astype(np.float64)
    s = q @ c.T * od.softmax_scale
    mx = s.max(axis=1, keepdims=True)
    e = np.exp(s - mx)
    tot = e.sum(axis=1, keepdims=True)
    size = (np.abs(q) @ np.abs(c).T).max(axis=1) * od.softmax_scale
    return (e / tot) @ c[:, :L], (mx + np.log(tot))[:, 0], (e / tot) @ np.abs(c[:, :L]), size


@pytest.mark.parametrize("shape,dtype,H,bs", [(LARGE, "bf16", 128, 64), (LARGE, "bf16", 128, 16), (LARGE, "bf16", 6, 64),
                                              (SMALL, "f32", 3, 16)])
@pytest.mark.parametrize("value", [math.inf, -math.inf])
@pytest.mark.parametrize("rope", [False, True])
@pytest.mark.parametrize("kind", ["tree", "causal"])
def test_rows_with_an_infinity(kind, rope, value, shape, dtype, H, bs):
    rng = np.random.default_rng(8)
    dims, od = make_dims(shape, H, bs, dtype)
    L, P = shape[:2]
    col = L + 3 if rope else 37
    ql, lens = [9, 20, 70, 1], [120, 70, 200, 1]
    qsl, T = loc(ql), sum(ql)
    parents = sum((tree(rng, n) if kind == "tree" else chain(n) for n in ql), [])
    mask, _ = TR.layout(parents, qsl, lens, 2)
    cache, table = make_cache(rng, lens, bs, L + P, dims.dtype)
    q = normal(rng, T, H, L + P, std=0.4, dtype=dims.dtype)
    sign = torch.tensor([1.0, -1.0]).repeat(T)[:T, None].expand(T, H)
    sign = torch.where(torch.arange(T)[:, None] == T - 1, -torch.sign(torch.tensor(value)), sign)
    q[..., col] = 0.5 * sign
    # a cached row, new ones, and a sequence's only row
    bad = {(0, 30), (0, 115), (1, 53), (2, 131), (2, 164), (3, 0)}
    finite = f64(cache)
    for r, j in bad:
        cache[table[r, j // bs], j % bs, col] = value
    if kind == "tree":
        o, lse = run_tree(dims, qsl, lens, mask, q, cache, table)
    else:
        o, lse = run_attn(dims, True, qsl, lens, q, cache, table)
    go, gl, q64, tab = f64(o), f64(lse), f64(q), table.numpy()
    tc, u, n, plain, nans = dtype == "bf16", unit(dims.dtype), max(lens), 0, 0
    for r, m in enumerate(ql):
        base = lens[r] - m
        for t in range(qsl[r], qsl[r + 1]):
            sees = [j for j in range(lens[r]) if j < base or TR.bit(mask[t], j - base)]
            hit = [j for j in sees if (r, j) in bad]
            if hit and sign[t, 0].item() * value > 0:
                assert np.isnan(go[t]).all() and np.isnan(gl[:, t]).all()
                nans += 1
                continue
            plain += len(hit) > 0
            ro, rl, mass, size = attend(q64[t], finite, tab, [j for j in sees if j not in hit], r, od)
            E = (L + P + 8) * F * size + 2.0 ** -22
            tol = u * np.abs(ro) + (2 * E[:, None] + (n / 8 + 64) * F + (u if tc else 0)) * mass
            got = go[t].copy()
            if hit and not rope:                     # the infinite column
                got[:, col] = np.where(np.isnan(got[:, col]), ro[:, col], got[:, col])
            within(got, ro, tol, "o")
            within(gl[:, t], rl, E + (n / 8 + 16) * F + F * np.abs(rl), "lse")
    assert min(plain, nans) >= 10
