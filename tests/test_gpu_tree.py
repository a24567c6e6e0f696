"""Parity of the calls on trees of drafted tokens with the float64 oracle.
Attention tolerances as in test_gpu_decode.py (the same arithmetic); layout,
verification and commit are whole numbers and moved rows, which have to be
equal but where a random number is next to a border (slack below)."""

import math

import numpy as np
import pytest
import torch

import mla_chunked_context_gb300 as M
from oracle import mla as O
from oracle import tree as TR

from test_gpu_decode import (DEV, F, LARGE, ODD, SMALL, _cuda, _no_device_errors, f64, i32,  # noqa: F401
                             loc, make_cache, make_dims, normal, run_attn, unit, within)

pytestmark = [pytest.mark.gpu,
              pytest.mark.filterwarnings("ignore::RuntimeWarning")]


def tree(rng, n):
    """Parents of a random tree, every parent before its children."""
    return [-1] + [int(rng.integers(max(0, i - 6), i)) for i in range(1, n)] if n else []


def chain(n):
    return list(range(-1, n - 1))


def words(x):
    return torch.from_numpy(np.asarray(x, dtype=np.int64)).to(DEV)


def status_word():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


# ----------------------------------------------------------------- layout --
def run_layout(parents, qsl, lens, W, status=None):
    T = len(parents)
    mask = torch.full((T, W), 0x0707, dtype=torch.int64, device=DEV)
    pos = torch.full((T,), -77, dtype=torch.int32, device=DEV)
    M.mla_tree_layout(i32(parents), i32(qsl), i32(lens), mask, pos, status)
    return mask.cpu().numpy(), pos.cpu().numpy()


@pytest.mark.parametrize("sizes,W", [([1], 1), ([8], 1), ([64], 1), ([65], 2), ([130, 3], 3), ([5, 0, 1, 40], 1),
                                     ([33] * 70, 1), ([200], 7), ([1100, 1500], 24)])
@pytest.mark.parametrize("kind", ["tree", "chain", "star"])
def test_layout(sizes, W, kind):
    rng = np.random.default_rng(sum(sizes))
    make = {"tree": lambda n: tree(rng, n), "chain": chain, "star": lambda n: [-1] + [0] * (n - 1) if n else []}[kind]
    parents = sum((make(n) for n in sizes), [])
    qsl, lens = loc(sizes), [int(x) for x in rng.integers(0, 5000, len(sizes))]
    status = status_word()
    mask, pos = run_layout(parents, qsl, lens, W, status)
    ref, rpos = TR.layout(parents, qsl, lens, W)
    assert (mask == ref).all() and (pos == rpos).all() and status.item() == 0


def test_layout_of_what_is_no_tree():
    """Parents that are no earlier node count as none; nodes beyond the mask's
    words have no bit; rows of no sequence stay as they were."""
    status = status_word()
    bad = [0, 0, 9, -5, 3, 2, 4]
    mask, pos = run_layout([0] + bad + [0], [1, 8], [20], 1, status)
    ref, rpos = TR.layout(bad, [0, 7], [20], 1)
    assert (mask[1:8] == ref).all() and (pos[1:8] == rpos).all()
    assert (mask[[0, 8]] == 0x0707).all() and (pos[[0, 8]] == -77).all()
    assert status.item() == M.MLA_STATUS_BAD_TREE
    status.zero_()
    mask, pos = run_layout(chain(70), [0, 70], [70], 1, status)
    ref, rpos = TR.layout(chain(70), [0, 70], [70], 1)
    assert (mask == ref).all() and (pos == rpos).all() and status.item() == M.MLA_STATUS_BAD_TREE
    status.zero_()                                   # locations beyond the tokens are clamped
    mask, _ = run_layout(chain(3), [0, 9], [9], 1, status)
    assert mask[:, 0].tolist() == [1, 3, 7] and status.item() == 0
    m = torch.zeros(3, 1, dtype=torch.int64, device=DEV)   # without positions
    M.mla_tree_layout(i32(chain(3)), i32([0, 3]), i32([3]), m)
    assert m[:, 0].tolist() == [1, 3, 7]


# -------------------------------------------------------------- attention --
def run_tree(dims, qsl, lens, mask, q, cache, table, status=None, stream=None):
    T = q.shape[0]
    o = torch.full((T, dims.num_heads, dims.kv_lora_rank), 7.0, dtype=dims.dtype, device=DEV)
    lse = torch.full((dims.num_heads, T), 7.0, device=DEV)
    ws = torch.full((M.mla_latent_attn_workspace_bytes(dims, T, len(lens)),), 0xFF, dtype=torch.uint8, device=DEV)
    M.mla_tree_attn(dims, i32(qsl), i32(lens), words(mask), q.to(DEV), cache.to(DEV), table.to(DEV), ws, o, lse,
                    status, stream)
    torch.cuda.synchronize()
    return o, lse


def check_tree(dims, od, qsl, lens, mask, q, cache, table, o, lse):
    ro, rl, mass, size = TR.tree_attention(f64(q), f64(cache), table.numpy(), qsl, lens, mask, od)
    own = ~np.isnan(rl[0])
    n = max([1] + list(lens))
    tc = dims.dtype == torch.bfloat16 and dims.kv_lora_rank == 512
    E = (od.kv_lora_rank + od.qk_rope_dim + 8) * F * size + 2.0 ** -22
    u = unit(dims.dtype)
    go, gl = f64(o), f64(lse)
    within(gl[:, own], rl[:, own], (E + (n / 8 + 16) * F + F * np.abs(rl))[:, own], "lse")
    tol = u * np.abs(ro) + (2 * E.T[:, :, None] + (n / 8 + 64) * F + (u if tc else 0)) * mass
    within(go[own], ro[own], tol[own], "o")
    assert (go[~own] == 7.0).all() and (gl[:, ~own] == 7.0).all()


CASES = {
    # lens, new tokens per request
    "root": ([70], [1]),
    "no context": ([8, 1, 64, 65], [8, 1, 64, 65]),
    "tile edges": ([63, 64, 65, 127, 128, 129, 130], [5, 6, 7, 8, 9, 64, 2]),
    "gaps": ([300, 17, 0, 5, 200], [0, 9, 3, 0, 12]),
    "more new tokens than tokens": ([3, 0, 70], [6, 2, 75]),
    "two words": ([400, 129], [100, 129]),
    "long": ([2900, 900], [20, 3]),
}
MASKS = ["tree", "random", "none"]


def masks(rng, kind, ql):
    W = -(-max(ql + [1]) // 64)
    T = sum(ql)
    if kind == "tree":
        return TR.layout(sum((tree(rng, n) for n in ql), []), loc(ql), [0] * len(ql), W)[0]
    if kind == "none":
        return np.zeros((T, W), dtype=np.int64)
    m = rng.integers(-(1 << 63), (1 << 63) - 1, size=(T, W), dtype=np.int64)
    m[rng.random(T) < 0.2] = 0
    return m


@pytest.mark.parametrize("kind", MASKS)
@pytest.mark.parametrize("H,bs", [(128, 64), (128, 16), (32, 64), (5, 16), (1, 64)])
@pytest.mark.parametrize("case", list(CASES))
def test_attention_large(case, H, bs, kind):
    lens, ql = CASES[case]
    rng = np.random.default_rng(len(case) * 1000 + H + bs)
    dims, od = make_dims(LARGE, H, bs, "bf16")
    qsl, mask = loc(ql), masks(rng, kind, ql)
    cache, table = make_cache(rng, lens, bs, 576, dims.dtype)
    q = torch.cat([normal(rng, qsl[-1], H, 512, std=0.3), normal(rng, qsl[-1], H, 64)], 2).to(dims.dtype)
    o, lse = run_tree(dims, qsl, lens, mask, q, cache, table)
    check_tree(dims, od, qsl, lens, mask, q, cache, table, o, lse)


@pytest.mark.parametrize("kind", MASKS)
@pytest.mark.parametrize("shape,dtype,bs", [(SMALL, "f32", 16), (ODD, "bf16", 7), (LARGE, "f32", 64),
                                            (SMALL, "bf16", 1), ((960, 64, 16, 8), "f32", 8)])
@pytest.mark.parametrize("case", ["no context", "gaps", "more new tokens than tokens", "two words"])
def test_attention_other_shapes(case, shape, dtype, bs, kind):
    lens, ql = CASES[case]
    rng = np.random.default_rng(bs + len(case))
    dims, od = make_dims(shape, 3, bs, dtype)
    qsl, mask = loc(ql), masks(rng, kind, ql)
    cache, table = make_cache(rng, lens, bs, shape[0] + shape[1], dims.dtype)
    q = normal(rng, qsl[-1], 3, shape[0] + shape[1], std=0.5, dtype=dims.dtype)
    o, lse = run_tree(dims, qsl, lens, mask, q, cache, table)
    check_tree(dims, od, qsl, lens, mask, q, cache, table, o, lse)


@pytest.mark.parametrize("bs", [1, 5, 8, 24, 32, 96, 100, 256])
@pytest.mark.parametrize("H", [128, 4])
def test_attention_block_sizes(H, bs):
    lens, ql = [301, 30, 130], [12, 9, 8]
    rng = np.random.default_rng(bs)
    dims, od = make_dims(LARGE, H, bs, "bf16")
    qsl, mask = loc(ql), masks(rng, "tree", ql)
    cache, table = make_cache(rng, lens, bs, 576, dims.dtype)
    q = normal(rng, qsl[-1], H, 576, std=0.4, dtype=dims.dtype)
    o, lse = run_tree(dims, qsl, lens, mask, q, cache, table)
    check_tree(dims, od, qsl, lens, mask, q, cache, table, o, lse)


@pytest.mark.parametrize("shape,dtype,H,bs", [(LARGE, "bf16", 128, 64), (LARGE, "bf16", 128, 32), (LARGE, "bf16", 128, 8), (LARGE, "bf16", 40, 16),
                                              (LARGE, "bf16", 3, 64), (SMALL, "f32", 3, 16)])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
def test_rows_that_are_not_finite_reach_only_nodes_that_see_them(shape, dtype, H, bs, value):
    """New tokens' rows that are not finite, in one column or all: nodes that do
    not see them have what zeros in their place give.  (Nodes that see them are
    NaN, or weigh them nothing where a score is -inf.)"""
    rng = np.random.default_rng(5)
    dims, od = make_dims(shape, H, bs, dtype)
    L, P = shape[:2]
    lens, ql = [120, 70, 200], [9, 20, 70]
    qsl = loc(ql)
    mask, _ = TR.layout(sum((tree(rng, n) for n in ql), []), qsl, lens, 2)
    cache, table = make_cache(rng, lens, bs, L + P, dims.dtype)
    q = normal(rng, qsl[-1], H, L + P, std=0.4, dtype=dims.dtype)
    clean, bad = cache.clone(), [(0, 4), (1, 3), (1, 19), (2, 33), (2, 66)]
    for r, i in bad:
        p = lens[r] - ql[r] + i
        clean[table[r, p // bs], p % bs] = 0
        if i % 2:
            cache[table[r, p // bs], p % bs, (7 * i) % L] = value
        else:
            cache[table[r, p // bs], p % bs, :] = value
    o, lse = run_tree(dims, qsl, lens, mask, q, cache, table)
    o2, lse2 = run_tree(dims, qsl, lens, mask, q, clean, table)
    apart = [t for r in range(3) for t in range(qsl[r], qsl[r + 1])
             if not any(s == r and TR.bit(mask[t], i) for s, i in bad)]
    assert len(apart) > 20
    assert torch.equal(o[apart], o2[apart]) and torch.equal(lse[:, apart], lse2[:, apart])
    if math.isnan(value):
        for t in set(range(qsl[-1])) - set(apart):
            assert torch.isnan(o[t]).all() and torch.isnan(lse[:, t]).all()


@pytest.mark.parametrize("shape,dtype,H", [(LARGE, "bf16", 128), (LARGE, "bf16", 6), (SMALL, "f32", 3)])
def test_attention_bad_blocks_and_rows_of_no_sequence(shape, dtype, H):
    rng = np.random.default_rng(12)
    dims, od = make_dims(shape, H, 16, dtype)
    width = shape[0] + shape[1]
    lens, ql = [100, 50, 60], [20, 10, 6]
    qsl = [x + 2 for x in loc(ql)]
    T = qsl[-1] + 3
    mask = np.zeros((T, 1), dtype=np.int64)
    mask[2:-3] = masks(rng, "tree", ql)
    cache, table = make_cache(rng, lens, 16, width, dims.dtype)
    q = normal(rng, T, H, width, std=0.4, dtype=dims.dtype)
    status = status_word()
    o, lse = run_tree(dims, qsl, lens, mask, q, cache, table, status)
    assert status.item() == 0
    check_tree(dims, od, qsl, lens, mask, q, cache, table, o, lse)
    bad = table.clone()
    bad[0, 5] = cache.shape[0]                       # among the new tokens
    bad[1, 0] = -2
    o, lse = run_tree(dims, qsl, lens, mask, q, cache, bad, status)
    assert status.item() == M.MLA_STATUS_BAD_BLOCK
    zero = torch.cat([cache, torch.zeros_like(cache[:1])])
    ztab = bad.clone()
    ztab[(ztab < 0) | (ztab > len(cache))] = len(cache)
    check_tree(dims, od, qsl, lens, mask, q, zero, ztab, o, lse)


@pytest.mark.parametrize("H", [128, 40, 2])
def test_attention_of_chains_is_causal_attention(H):
    """Many requests, cut units, joins: as mla_latent_attn, within twice the
    roundings of an output and the weights' (each call's own)."""
    rng = np.random.default_rng(H)
    dims, od = make_dims(LARGE, H, 64, "bf16")
    ql = [int(x) for x in rng.integers(0, 6, size=60)]
    lens = [int(x) for x in rng.integers(6, 900, size=60)]
    qsl = loc(ql)
    mask, _ = TR.layout(sum((chain(n) for n in ql), []), qsl, lens, 1)
    cache, table = make_cache(rng, lens, 64, 576, dims.dtype)
    q = normal(rng, qsl[-1], H, 576, std=0.4, dtype=dims.dtype)
    o, lse = run_tree(dims, qsl, lens, mask, q, cache, table)
    o2, lse2 = run_attn(dims, True, qsl, lens, q, cache, table)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)   # the same tiles, cuts and order of sums
    check_tree(dims, od, qsl, lens, mask, q, cache, table, o, lse)


def test_attention_on_another_stream_and_far_offsets():
    dims, od = make_dims(LARGE, 16, 64, "bf16")
    blocks = 64000                                   # 64000*64*576 = 2.36e9 elements
    cache = torch.zeros(blocks, 64, 576, dtype=torch.bfloat16, device=DEV)
    rng = np.random.default_rng(3)
    small, table = make_cache(rng, [200], 64, 576, dims.dtype, spare=0)
    far = blocks - 1 - torch.arange(4)
    cache[far.to(DEV)] = small.to(DEV)
    q, mask = normal(rng, 7, 16, 576, std=0.4, dtype=dims.dtype), masks(rng, "tree", [7])
    ftab = table.clone()
    ftab[0, :4] = far[table[0, :4].long()].int()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        o, lse = run_tree(dims, [0, 7], [200], mask, q, cache, ftab)
    del cache
    check_tree(dims, od, [0, 7], [200], mask, q, small, table, o, lse)


# ----------------------------------------------------------------- verify --
def rows(rng, n, V, dtype, kind="peaked"):
    z = rng.normal(size=(n, V)) * (1.25 * math.sqrt(2 * math.log(V + 1)))
    e = np.exp(z - z.max(1, keepdims=True))
    return torch.from_numpy((e / e.sum(1, keepdims=True)).astype(np.float32)).to(dtype), z


def near(rng, z, dtype):
    y = z + 0.8 * rng.normal(size=z.shape)
    e = np.exp(y - y.max(1, keepdims=True))
    return torch.from_numpy((e / e.sum(1, keepdims=True)).astype(np.float32)).to(dtype)


def run_verify(p, q, tokens, parents, qsl, u, un, most, status=None):
    R = len(qsl) - 1
    path = torch.full((R, most), 99, dtype=torch.int32, device=DEV)
    kept, nxt = (torch.full((R,), 99, dtype=torch.int32, device=DEV) for _ in range(2))
    f = lambda x: None if x is None else torch.from_numpy(np.asarray(x, np.float32)).to(DEV)  # noqa: E731
    M.mla_verify_tree(p, q, i32(tokens), i32(parents), i32(qsl), f(u), f(un), path, kept, nxt, status)
    return path.cpu().numpy(), kept.cpu().numpy(), nxt.cpu().numpy()


# How near the next token's border decides otherwise than exact sums: a value p -
# t q is rounded to units of 2^-45, by at most 2^-46, and before that it is off by
# some 2^-47 (t has 48 bits, and t q at most the row's largest value, 1); sums of
# units are exact.  So cumulated values are off by at most 2^-45 V (before they
# are divided by their sum, which the oracle does).  The oracle's own sums are
# off by 2^-53 V.  (A row of equal shares whose border is exactly the end of one,
# as in test_verify_borders, is decided by the oracle's own rounding.)
def slack(V):
    return V * 2.0 ** -45


def check_verify(got, p, q, tokens, parents, qsl, u, un, most):
    path, kept, nxt = got
    p, q = p.cpu().double().numpy(), None if q is None else q.cpu().double().numpy()
    for r in range(len(qsl) - 1):
        lo, hi = qsl[r], qsl[r + 1]
        f = lambda x: None if x is None else np.asarray(x, np.float32)[lo:hi]  # noqa: E731
        rp, rn, near = TR.verify(p[lo:hi], None if q is None else q[lo:hi], tokens[lo:hi], parents[lo:hi], f(u),
                                 None if un is None else np.float32(un[r]), most, slack(p.shape[1]))
        assert kept[r] == len(rp) and nxt[r] in near, (r, kept[r], rp, nxt[r], rn)
        assert path[r].tolist() == rp + [-1] * (most - len(rp))


def drafted(rng, mode, sizes, V, dtype):
    """(p, q, tokens, parents, qsl, u, un) of trees drafted as `mode` says."""
    parents = sum((tree(rng, n) for n in sizes), [])
    qsl, T = loc(sizes), sum(sizes)
    up = np.array([qsl[r] + max(0, parents[qsl[r] + i]) for r, n in enumerate(sizes) for i in range(n)], dtype=int)
    q, z = rows(rng, T, V, dtype)
    p = near(rng, z, dtype)
    if mode == "draft":
        w = q.double().numpy()
        tokens = [int(rng.choice(V, p=w[x] / w[x].sum())) for x in up]
    elif mode == "point":
        order, seen, tokens = np.argsort(-z, axis=1), {}, []
        for x in up:
            tokens.append(int(order[x, seen.get(x, 0) % V]))
            seen[x] = seen.get(x, 0) + 1
    else:
        p = torch.from_numpy((z + rng.normal(size=z.shape)).astype(np.float32)).to(dtype)
        best = p.float().argmax(1).numpy()
        tokens = [int(best[x]) if rng.random() < 0.6 else int(rng.integers(V)) for x in up]
    u, un = (None, None) if mode == "greedy" else (rng.random(T).astype(np.float32), rng.random(len(sizes)).astype(np.float32))
    return p.to(DEV), q.to(DEV) if mode == "draft" else None, tokens, parents, qsl, u, un


@pytest.mark.parametrize("mode", ["draft", "point", "greedy"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("sizes,V", [([1], 1), ([5], 2), ([9, 1, 0, 4], 7), ([20] * 40, 63), ([16] * 9, 1000),
                                     ([12, 30], 32001), ([6] * 3, 131072), ([3] * 170, 513), ([40] * 6, 4)])
def test_verify(sizes, V, dtype, mode):
    rng = np.random.default_rng(sum(sizes) + V)
    status = status_word()
    args = drafted(rng, mode, sizes, V, dtype)
    got = run_verify(*args, 9, status)
    check_verify(got, *args, 9)
    assert status.item() == 0
    assert got[1].max() > 1 or V == 1 or len(sizes) < 5     # some are kept


@pytest.mark.parametrize("mode", ["draft", "point", "greedy"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("offset", [0, 1, 3])
def test_verify_rows_of_a_wider_tensor(offset, dtype, mode):
    """Rows that start at odd addresses, the draft's otherwise than the target's;
    what lies beside them is NaN."""
    rng = np.random.default_rng(offset)
    p, q, *rest = drafted(rng, mode, [7, 5], 1003, dtype)
    wide = torch.full((12, 1003 + 10), math.nan, dtype=dtype, device=DEV)
    wide[:, offset:offset + 1003] = p
    wide_q = torch.full((12, 1003 + 5), math.nan, dtype=dtype, device=DEV)
    if q is not None:
        wide_q[:, 2:2 + 1003] = q
        q = wide_q[:, 2:2 + 1003]
    p = wide[:, offset:offset + 1003]
    check_verify(run_verify(p, q, *rest, 6), p, q, *rest, 6)


@pytest.mark.parametrize("most", [1, 2, 3, 40])
def test_verify_stops_at_the_paths_room(most):
    rng = np.random.default_rng(most)
    p, _, _, _, _, _, _ = drafted(rng, "draft", [30], 50, torch.float32)
    args = (p, p, [0] + [int(p[i].argmax()) for i in range(29)], chain(30), [0, 30], np.full(30, 0.5, np.float32), [0.25])
    got = run_verify(*args, most)                    # p = q: every draft is kept
    assert got[1][0] == min(most, 30)
    check_verify(got, *args, most)


def test_verify_borders():
    """Random numbers at the ends of their range, rows with one token, rows with
    zeros first and last, children that are the same token, tokens without
    mass, target equal to draft, rows without mass, and one that is not
    normalised."""
    V, e = 300, np.zeros(300, np.float32)
    one = e.copy(); one[17] = 1
    ends = e.copy(); ends[5:290] = 1 / 285
    low = e.copy(); low[3] = 0.75; low[200] = 0.25
    big = np.full(V, 0.5, np.float32)
    last = np.float32(1 - 2.0 ** -24)
    P, Q, tok, par, qsl, u, un = [], [], [], [], [0], [], []
    for row_p, row_q in ((one, one), (one, low), (low, one), (ends, ends), (ends, low), (low, ends), (big, big),
                         (e, low), (low, e), (big, one), (one, big)):
        for ux in (0.0, last):
            for uy in (0.0, 0.5, last):
                for x in ([17, 17, 17], [3, 200, 3], [0, 5, 299]):
                    P += [row_p] * 4; Q += [row_q] * 4
                    tok += [0] + x; par += [-1, 0, 0, 0]; qsl.append(qsl[-1] + 4)
                    u += [0.0, ux, ux, ux]; un.append(uy)
    p, q = (torch.from_numpy(np.stack(x)).to(DEV) for x in (P, Q))
    for qq in (q, None):
        args = (p, qq, tok, par, qsl, np.array(u, np.float32), np.array(un, np.float32))
        check_verify(run_verify(*args, 3), *args, 3)


def test_verify_greedy_ties_and_rows_that_are_not_finite():
    V = 5000
    z = torch.zeros(6, V)
    z[0, [77, 4000]] = 3.0                           # the lowest of equals
    z[1] = -math.inf                                 # nothing: token 0
    z[2] = math.nan
    z[3] = math.nan; z[3, 4999] = -5.0
    z[4, 123] = math.inf
    z[5] = -1.0; z[5, 0] = -0.0; z[5, 9] = 0.0
    for dtype in (torch.float32, torch.bfloat16):
        p = z.to(dtype).to(DEV)
        got = run_verify(p, None, [0] * 6, [-1] * 6, list(range(7)), None, None, 2)
        assert got[2].tolist() == [77, 0, 0, 4999, 123, 0] and (got[1] == 1).all()


def test_verify_what_is_no_tree():
    """Tokens outside the vocabulary and parents that are no earlier node are
    passed over; more than 1024 nodes: the first ones; other roots are nobody's
    children; rows of no sequence are not looked at."""
    rng = np.random.default_rng(2)
    V, n = 40, 1500
    q, z = rows(rng, n + 2, V, torch.float32)
    p = near(rng, z, torch.float32).to(DEV)
    q = q.to(DEV)
    parents = [-1] + [max(0, i - 2) for i in range(1, n)]
    tokens = [int(x) for x in rng.integers(0, V, n)]
    u, un = rng.random(n + 2).astype(np.float32), [0.3]
    status = status_word()
    got = run_verify(p, q, [7] + tokens + [7], [0] + parents + [0], [1, n + 1], u, un, 5, status)
    assert status.item() == M.MLA_STATUS_BAD_TREE
    cut = (p[1:1025], q[1:1025], tokens[:1024], parents[:1024], [0, 1024], u[1:1025], un)
    check_verify(got, *cut, 5)
    for change in (dict(tokens=[0, V, 3]), dict(tokens=[0, -1, 3]), dict(parents=[-1, 5, 0]),
                   dict(parents=[-1, 1, 0]), dict(parents=[2, -7, 0])):
        status.zero_()
        a = dict(tokens=[0, 4, 3], parents=[-1, 0, 0])
        a.update(change)
        args = (p[:3], q[:3], a["tokens"], a["parents"], [0, 3], u[:3], [0.6])
        check_verify(run_verify(*args, 3, status), *args, 3)
        assert status.item() == M.MLA_STATUS_BAD_TREE
    status.zero_()
    args = (p[:3], q[:3], [0, 4, 3], [-1, -1, -1], [0, 3], u[:3], [0.6])
    got = run_verify(*args, 3, status)
    check_verify(got, *args, 3)
    assert got[1].tolist() == [1] and status.item() == 0


# ----------------------------------------------------------------- commit --
def run_commit(dims, path, kept, qsl, lens, caches, table, status=None):
    new = torch.full((len(lens),), -9, dtype=torch.int32, device=DEV)
    caches = [c.to(DEV) for c in caches]
    M.mla_commit_tree(dims, path.to(DEV), i32(kept), i32(qsl), i32(lens), caches, table.to(DEV), new, qsl[-1],
                      status)
    return [c.cpu() for c in caches], new.cpu().tolist()


def same(a, b):
    """Equal bit for bit (NaN among them)."""
    kind = torch.int16 if a.dtype == torch.bfloat16 else torch.int32
    return torch.equal(a.view(kind), b.view(kind))


@pytest.mark.parametrize("shape,dtype,bs,layers", [(LARGE, "bf16", 64, 1), (LARGE, "bf16", 5, 3), (SMALL, "f32", 16, 2),
                                                   (ODD, "bf16", 1, 4), (LARGE, "f32", 7, 2), (SMALL, "bf16", 16, 300)])
def test_commit(shape, dtype, bs, layers):
    """Paths whose rows move onto others that are still to move, long ones, none;
    everything else stays as it was."""
    rng = np.random.default_rng(layers)
    dims, od = make_dims(shape, 2, bs, dtype)
    ql = [1, 8, 8, 0, 5, 40, 700 if layers < 5 else 60]
    lens = [9, 8, 30, 12, 70, 41, 720]
    paths = [[0], [0, 2, 3, 4, 7], [0, 1, 2], [], [0, 4], list(range(0, 40, 1))[::3], None]
    n = ql[-1]
    paths[-1] = sorted(set([0] + [int(x) for x in rng.integers(1, n, n // 2)]))
    kept = [len(p) for p in paths]
    most = max(kept) + 2
    path = torch.tensor([p + [-1] * (most - len(p)) for p in paths], dtype=torch.int32)
    caches, table = [], None
    for _ in range(layers):
        c, table = make_cache(np.random.default_rng(4), lens, bs, shape[0] + shape[1], dims.dtype)
        caches.append((c.float() + float(rng.normal())).to(dims.dtype) if layers < 10 else c)
    status = status_word()
    got, new = run_commit(dims, path, kept, loc(ql), lens, caches, table, status)
    assert status.item() == 0
    for c, g in zip(caches, got):
        ref = f64(c)
        want = TR.commit(ref, table.numpy(), loc(ql), lens, path.numpy(), kept, bs)
        assert same(g, torch.from_numpy(ref).to(dims.dtype)) and new == want


def test_commit_of_what_is_no_path():
    rng = np.random.default_rng(1)
    dims, od = make_dims(SMALL, 2, 16, "f32")
    ql, lens = [6, 6, 6, 6, 4, 3], [20, 20, 20, 20, 2, 50]
    paths = [[0, 5, 1], [0, 6, 3], [-1, 3, 4], [0, 3, 5], [0, 3, 3], [0, 2, 2]]   # the fifth starts before 0
    kept = [3, 3, 3, 9, 3, 2]
    cache, table = make_cache(rng, lens, 16, 80, dims.dtype)
    path = torch.tensor(paths, dtype=torch.int32)
    for r, bad in enumerate([True, True, True, True, False, False]):
        status = status_word()
        got, new = run_commit(dims, path[r:r + 1], kept[r:r + 1], [0, ql[r]], lens[r:r + 1], [cache], table[r:r + 1],
                              status)
        ref = f64(cache)
        want = TR.commit(ref, table[r:r + 1].numpy(), [0, ql[r]], lens[r:r + 1], paths[r:r + 1], kept[r:r + 1], 16)
        assert same(got[0], torch.from_numpy(ref).float()) and new == want, r
        assert status.item() == (M.MLA_STATUS_BAD_TREE if bad else 0), r
    far = table[5:6].clone()                         # a bad block under the rows: nothing is touched
    far[0, 3] = cache.shape[0]
    status = status_word()
    got, _ = run_commit(dims, path[5:6], [2], [0, 3], [50], [cache], far, status)
    assert same(got[0], cache) and status.item() == M.MLA_STATUS_BAD_BLOCK
    status.zero_()                                   # and past the table's row
    got, _ = run_commit(dims, path[5:6], [2], [0, 3], [50], [cache], table[5:6, :3].contiguous(), status)
    assert same(got[0], cache) and status.item() == M.MLA_STATUS_BAD_BLOCK


def test_commit_far_offsets():
    dims, _ = make_dims(LARGE, 2, 64, "bf16")
    blocks = 64000
    cache = torch.zeros(blocks, 64, 576, dtype=torch.bfloat16, device=DEV)
    cache[blocks - 1] = torch.arange(64, device=DEV)[:, None].to(torch.bfloat16)
    M.mla_commit_tree(dims, i32([0, 5, 9]).view(1, 3), i32([3]), i32([0, 12]), i32([40]), cache,
                      i32([blocks - 1]).view(1, 1))
    assert cache[blocks - 1, 28:31, 3].tolist() == [28.0, 33.0, 37.0]
    assert cache[blocks - 1, 31:40, 575].tolist() == [float(x) for x in range(31, 40)]
    assert int(torch.count_nonzero(cache[:blocks - 1])) == 0


# ------------------------------------------------------------ whole steps --
def step_setup(rng, shape, dtype, H, lens, ql, layers, bs=16, spare_blocks=2):
    dims, od = make_dims(shape, H, bs, dtype)
    L, P, Dn, Dv = shape
    caches = []
    room = [n + 24 for n in lens]
    for _ in range(layers):
        c, table = make_cache(np.random.default_rng(9), room, bs, L + P, dims.dtype)
        caches.append(c.to(DEV))
    T = sum(ql)
    x = dict(rope=torch.from_numpy(O.rope_table(max(room) + 8, P).astype(np.float32)).to(DEV), table=table.to(DEV),
             w=[normal(rng, H * (Dn + Dv), L, std=0.1, dtype=dims.dtype).to(DEV) for _ in range(layers)],
             q=[normal(rng, T, H, Dn + P, dtype=dims.dtype).to(DEV) for _ in range(layers)],
             kv=[normal(rng, T, L + P, dtype=dims.dtype).to(DEV) for _ in range(layers)])
    return dims, od, caches, x


@pytest.mark.parametrize("shape,dtype,H", [(LARGE, "bf16", 128), (LARGE, "bf16", 8), (SMALL, "f32", 3)])
def test_a_step_of_trees_is_one_of_the_kept_tokens(shape, dtype, H):
    """A tree's step (plan, two layers, verify, commit) leaves in the cache, and
    computes for the nodes it keeps, what a step with only the kept tokens
    does.  The cache bit for bit (the same row at the same rope position); the
    outputs within the two calls' own attention errors, of which the weights'
    bf16 rounding (u sum p|c|, expanded) is far the largest: bounded by
    2 (2u + 2^-10) of the expanded sum p|c| |w| for bf16."""
    rng = np.random.default_rng(H)
    L, P, Dn, Dv = shape
    ql, lens = [11, 7, 1, 20], [95, 7, 40, 150]      # new ones included; the second has no context
    dims, od, caches, x = step_setup(rng, shape, dtype, H, lens, ql, 2)
    qsl, T, R = loc(ql), sum(ql), len(ql)
    parents = sum((tree(rng, n) for n in ql), [])
    V = 50
    qd, z = rows(rng, T, V, torch.float32)
    target = near(rng, z * 0.2, torch.float32).to(DEV)
    best = target.argmax(1).tolist()
    tokens = [best[qsl[r] + max(0, parents[qsl[r] + i])] for r, n in enumerate(ql) for i in range(n)]
    for i in range(T):                               # some drafts are wrong
        if rng.random() < 0.3:
            tokens[i] = (tokens[i] + 1) % V
    before = [c.clone() for c in caches]
    dec = M.TreeDecode(dims, T + 3, R + 1, max_path=8, device=DEV)
    out = [torch.empty(T, H, Dv, dtype=dims.dtype, device=DEV) for _ in range(2)]
    lse = [torch.empty(H, T, device=DEV) for _ in range(2)]
    new_lens, status = i32([0] * R), status_word()
    dec.plan(i32(parents), i32(qsl), i32(lens), status)
    for k in range(2):
        dec(x["q"][k], x["kv"][k], x["rope"], caches[k], x["table"], x["w"][k], out[k], lse[k], dev_status=status)
    path, kept, nxt = dec.verify(target, i32(tokens), dev_status=status)
    dec.commit(caches, x["table"], new_lens, status)
    path, kept, nxt = path.cpu().numpy(), kept.tolist(), nxt.tolist()
    assert status.item() == 0 and max(kept) > 2
    base = [n - m for n, m in zip(lens, ql)]
    assert new_lens.tolist() == [b + k for b, k in zip(base, kept)]
    rows_kept = [qsl[r] + int(i) for r in range(R) for i in path[r, :kept[r]]]
    for r in range(R):                               # greedy: kept drafts are the target's, then its next
        line = path[r, :kept[r]]
        assert [tokens[qsl[r] + i] for i in line[1:]] == [best[qsl[r] + i] for i in line[:-1]]
        assert nxt[r] == best[qsl[r] + line[-1]]
    plain = M.LatentDecode(dims, T, R, device=DEV)
    u = unit(dims.dtype)
    for k in range(2):
        c = before[k]
        o2 = torch.empty(len(rows_kept), H, Dv, dtype=dims.dtype, device=DEV)
        l2 = torch.empty(H, len(rows_kept), device=DEV)
        plain(x["q"][k][rows_kept], x["kv"][k][rows_kept], i32(loc(kept)), new_lens, x["rope"], c, x["table"],
              x["w"][k], o2, l2)
        for r in range(R):
            for j in range(base[r] + kept[r]):
                blk, at = int(x["table"][r, j // 16]), j % 16
                assert same(caches[k][blk, at].cpu(), c[blk, at].cpu()), (k, r, j)
        q_lat = plain.q_latent[:len(rows_kept)]
        _, _, mass, size = O.latent_attention(f64(q_lat), f64(c), x["table"].cpu().numpy(), loc(kept),
                                              new_lens.tolist(), od, True)
        E = (L + P + 8) * F * size + 2.0 ** -22
        within(f64(l2), f64(lse[k][:, rows_kept]), 2 * (E + (max(lens) / 8 + 16) * F + F * np.abs(f64(l2))), "lse")
        big = O.expand_output(mass, np.abs(f64(x["w"][k])), od)
        if dtype == "bf16":
            tol = 2 * (2 * u + 2.0 ** -10) * big + 2 * u * np.abs(f64(o2))
        else:
            tol = 2 * (2 * E.max() + (max(lens) / 8 + 64 + L) * F) * big + 4 * u * np.abs(f64(o2))
        within(f64(out[k][rows_kept]), f64(o2), tol, "out")


@pytest.mark.parametrize("shape,dtype", [(LARGE, "bf16"), (SMALL, "f32")])
def test_steps_captured_and_replayed_with_other_trees(shape, dtype):
    """Plan, layer, verify and commit in one graph, replayed while the trees, the
    tokens, the random numbers and the lengths change on the device; a second
    instance's graph in between."""
    rng = np.random.default_rng(6)
    H, V = 4, 700
    L, P, Dn, Dv = shape
    ql, lens = [9, 0, 14], [60, 0, 33]
    qsl, T, R = loc(ql), sum(ql), 3
    dims, od, caches, x = step_setup(rng, shape, dtype, H, lens, ql, 1)
    parents, lens_d, tokens = i32([-1] * T), i32(lens), i32([0] * T)
    p, q = torch.empty(T, V, device=DEV), torch.empty(T, V, device=DEV)
    u, un = torch.empty(T, device=DEV), torch.empty(R, device=DEV)

    class Side:
        def __init__(self):
            self.dec = M.TreeDecode(dims, T, R, device=DEV)
            self.cache = caches[0].clone()
            self.out, self.new = torch.zeros(T, H, Dv, dtype=dims.dtype, device=DEV), i32([0] * R)
            self.qsl = i32(qsl)

        def step(self):
            self.dec.plan(parents, self.qsl, lens_d)
            self.dec(x["q"][0], x["kv"][0], x["rope"], self.cache, x["table"], x["w"][0], self.out)
            self.dec.verify(p, tokens, u, un, draft=q)
            self.dec.commit(self.cache, x["table"], self.new)

        def results(self):
            d = self.dec
            return [t.clone() for t in (d.tree_mask, d.positions, d.path, d.num_kept, d.next_tokens, self.out,
                                        self.new, self.cache)]

    def fill(k):
        g = np.random.default_rng(100 + k)
        par = sum((tree(g, n) for n in ql), [])
        a = drafted(g, "draft", ql, V, torch.float32)
        p.copy_(a[0]); q.copy_(a[1]); tokens.copy_(i32(a[2])); parents.copy_(i32(a[3]))
        u.copy_(torch.from_numpy(a[5])); un.copy_(torch.from_numpy(a[6]))
        lens_d.copy_(i32([60 - k, 0, 33 + k]))

    a, b, eager = Side(), Side(), Side()
    fill(0)
    graphs = []
    for side in (a, b):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            side.step()
        torch.cuda.current_stream().wait_stream(s)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            side.step()
        graphs.append(graph)
    for side in (a, b, eager):
        side.cache.copy_(caches[0])
    for k in range(4):
        fill(k)
        eager.step()
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        for got in (a, b):
            for y, z in zip(got.results(), eager.results()):
                assert same(y, z) if y.is_floating_point() else torch.equal(y, z)


def test_bindings_refuse_on_the_device():
    d = M.Dims(2, 64, 16, 32, 32, 16, 0.1, torch.float32)
    z = lambda *s: torch.zeros(*s, device=DEV)  # noqa: E731
    n = lambda *s: torch.zeros(*s, dtype=torch.int32, device=DEV)  # noqa: E731
    m = torch.zeros(3, 1, dtype=torch.int64, device=DEV)
    for bad in (m.int(), m[:2], torch.zeros(3, 2, dtype=torch.int64, device=DEV)[:, :1]):
        with pytest.raises(ValueError, match="tree_mask"):
            M.mla_tree_layout(n(3), n(2), n(1), bad)
        with pytest.raises(ValueError, match="tree_mask"):
            M.mla_tree_attn(d, n(2), n(1), bad, z(3, 2, 80), z(4, 16, 80), n(1, 2), None, z(3, 2, 64))
    with pytest.raises(ValueError, match="positions"):
        M.mla_tree_layout(n(3), n(2), n(1), m, n(2))
    out = (n(1, 4), n(1), n(1))
    ok = (n(3), n(3), n(2), z(3), z(1))
    for name, call in (("draft", lambda: M.mla_verify_tree(z(3, 10), z(3, 9), *ok, *out)),
                       ("draft", lambda: M.mla_verify_tree(z(3, 10), z(3, 10).bfloat16(), *ok, *out)),
                       ("target", lambda: M.mla_verify_tree(z(10, 3).t(), None, *ok, *out)),
                       ("target", lambda: M.mla_verify_tree(z(1, 10).expand(3, 10), None, *ok, *out)),
                       ("tokens", lambda: M.mla_verify_tree(z(3, 10), None, n(2), *ok[1:], *out)),
                       ("uniform", lambda: M.mla_verify_tree(z(3, 10), None, *ok[:3], None, z(1), *out)),
                       ("uniform_next", lambda: M.mla_verify_tree(z(3, 10), None, *ok[:4], z(2), *out)),
                       ("num_kept", lambda: M.mla_verify_tree(z(3, 10), None, *ok, out[0], n(2), n(1)))):
        with pytest.raises(ValueError, match=name):
            call()
    for name, caches in (("kv_caches", [z(4, 16, 80), z(3, 16, 80)]), ("kv_caches", [z(4, 16, 80), None]),
                         ("kv_caches", z(4, 16, 79)), ("kv_caches", (z(4, 16, 80).bfloat16(),))):
        with pytest.raises(ValueError, match=name):
            M.mla_commit_tree(d, n(1, 4), n(1), n(2), n(1), caches, n(1, 2))
    lens = n(1)
    with pytest.raises(M.MlaError, match="invalid"):
        M.mla_commit_tree(d, n(1, 4), n(1), n(2), lens, [z(4, 16, 80)], n(1, 2), new_seq_lens=lens)
    new = n(1)
    M.mla_commit_tree(d, n(1, 4), n(1), n(2), i32([5]), [], n(1, 2), new_seq_lens=new)   # no layers: lengths
    assert new.item() == 5
