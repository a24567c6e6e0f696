"""Parity of the decode calls (paged append, query absorption, latent
attention, output expansion) with the float64 oracle.

Tolerances, derived from the roundings that the calls make (u = half a step of
the storage type relative to the value: bf16 2^-8, float32 2^-24; f = 2^-24):
  * append: one rounding of the result, u|ref|; before it float32 arithmetic,
    16 f times the size of the terms (for the norm, (L/32 + 16) f: 32 lanes sum
    L squares)
  * absorb, expand: u|ref| + (K + 4) f sum|a||b|
  * attention: with E = (L + P + 8) f max_j(scale sum|q||c_j|) + 2^-22 bounding
    the error of a scaled score and its exponential, and n keys:
    LSE: E + (n/8 + 16) f + f |LSE|
    O:   u|ref| + (2E + (n/8 + 64) f) sum p|c|, and for the tensor-core kernel
         u sum p|c| more (p is rounded to bf16 for the second product)
    (n/8: running sums are kept per thread or warp, at most n/8 terms each, and
    a handful of joins.)
The whole step composes them; its tolerance is written at its test."""

import math

import numpy as np
import pytest
import torch

import mla_chunked_context_gb300 as M
from oracle import mla as O

pytestmark = [pytest.mark.gpu,
              pytest.mark.filterwarnings("ignore::RuntimeWarning")]

DEV = "cuda:0"
F = 2.0 ** -24
LARGE = (512, 64, 128, 128)
SMALL = (64, 16, 32, 32)
ODD = (40, 24, 8, 16)
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("CUDA GPU required for -m gpu tests")
    M.lib()
    torch.cuda.set_device(0)


@pytest.fixture(autouse=True)
def _no_device_errors():
    yield
    assert M.mla_device_error_flags() == 0, "a tensor-core kernel gave up waiting"


def unit(dtype):
    return torch.finfo(dtype).eps / 2


def f64(t):
    return t.detach().to("cpu").double().numpy()


def make_dims(shape, H, bs, dtype):
    L, P, Dn, Dv = shape
    scale = 1.0 / math.sqrt(Dn + P)
    return (M.Dims(H, L, P, Dn, Dv, bs, scale, DTYPES[dtype]),
            O.MlaDims(H, L, P, Dn, Dv, bs, float(np.float32(scale))))


def normal(rng, *shape, std=1.0, dtype=torch.float32):
    return torch.from_numpy(rng.normal(0, std, shape).astype(np.float32)).to(dtype)


def make_cache(rng, lens, bs, width, dtype, spare=3):
    """A paged cache of the sequences' rows on shuffled blocks.  Everything
    no sequence owns is NaN: unused slots of the last blocks, unused blocks."""
    need = [-(-max(0, n) // bs) for n in lens]
    blocks = sum(need) + spare
    order = rng.permutation(blocks)
    cache = torch.full((blocks, bs, width), float("nan"), dtype=dtype)
    table = np.full((len(lens), max(1, max(need, default=1)) + 1), blocks - 1 - spare, dtype=np.int32)
    at = 0
    for r, n in enumerate(lens):
        table[r, :need[r]] = order[at:at + need[r]]
        at += need[r]
        for j in range(0, max(0, n), bs):
            k = min(bs, n - j)
            cache[table[r, j // bs], :k] = normal(rng, k, width, dtype=dtype)
    return cache, torch.from_numpy(table)


def i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device=DEV)


def loc(q_lens):
    return [0] + [int(x) for x in np.cumsum(q_lens)]


def within(got, ref, tol, what):
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    assert got.shape == ref.shape
    same = (got == ref)  # covers -inf
    bad = ~same & ~(np.abs(got - ref) <= tol)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        tol = np.broadcast_to(tol, ref.shape)
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} off; first {i}: {got[i]} for "
                             f"{ref[i]}, tolerance {tol[i]}")


# ------------------------------------------------------------------- attn --
def run_attn(dims, causal, qsl, lens, q, cache, table, T=None, status=None, stream=None):
    T = q.shape[0]
    o = torch.full((T, dims.num_heads, dims.kv_lora_rank), 7.0, dtype=dims.dtype, device=DEV)
    lse = torch.full((dims.num_heads, T), 7.0, device=DEV)
    ws = torch.full((M.mla_latent_attn_workspace_bytes(dims, T, len(lens)),), 0xFF,
                    dtype=torch.uint8, device=DEV)  # NaN wherever it is read before it is written
    M.mla_latent_attn(dims, causal, i32(qsl), i32(lens), q.to(DEV), cache.to(DEV), table.to(DEV),
                      ws, o, lse, status, stream)
    torch.cuda.synchronize()
    return o, lse


def check_attn(dims, od, causal, qsl, lens, q, cache, table, o, lse):
    ro, rl, mass, size = O.latent_attention(f64(q), f64(cache), table.numpy(), qsl, lens, od, causal)
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
    "one": ([1], [1]),
    "two keys": ([2], [1]),
    "short": ([70], [1]),
    "tile edges": ([63, 64, 65, 127, 128, 129, 191, 192], [1] * 8),
    "empty ones": ([0, 130, 0, 5, 0], [1, 1, 2, 1, 1]),
    "no new tokens": ([300, 17, 200], [0, 2, 0]),
    "drafts": ([33, 4, 3, 260], [4, 4, 7, 5]),   # one has more new tokens than tokens
    "ragged": ([700, 1, 64, 333, 129, 2, 1025], [1, 1, 3, 2, 1, 1, 1]),
    "long": ([3001], [1]),
}


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("bs", [64, 16])
@pytest.mark.parametrize("H", [128, 32, 5])
@pytest.mark.parametrize("case", list(CASES))
def test_latent_attention_large(case, H, bs, causal):
    lens, ql = CASES[case]
    rng = np.random.default_rng(len(case) * 1000 + H + bs)
    dims, od = make_dims(LARGE, H, bs, "bf16")
    qsl = loc(ql)
    cache, table = make_cache(rng, lens, bs, 576, dims.dtype)
    q = torch.cat([normal(rng, qsl[-1], H, 512, std=0.3), normal(rng, qsl[-1], H, 64)], 2).to(dims.dtype)
    o, lse = run_attn(dims, causal, qsl, lens, q, cache, table)
    check_attn(dims, od, causal, qsl, lens, q, cache, table, o, lse)


@pytest.mark.parametrize("bs", [1, 5, 8, 24, 100, 256])
@pytest.mark.parametrize("H", [128, 20])
def test_latent_attention_block_sizes(H, bs):
    """Pages that end inside a tile, of one row, of odd sizes, larger than a tile."""
    lens, ql = [301, 3, 130], [1, 2, 1]
    rng = np.random.default_rng(bs)
    dims, od = make_dims(LARGE, H, bs, "bf16")
    qsl = loc(ql)
    cache, table = make_cache(rng, lens, bs, 576, dims.dtype)
    q = normal(rng, qsl[-1], H, 576, std=0.4, dtype=dims.dtype)
    o, lse = run_attn(dims, True, qsl, lens, q, cache, table)
    check_attn(dims, od, True, qsl, lens, q, cache, table, o, lse)


@pytest.mark.parametrize("shape,dtype,bs", [(SMALL, "f32", 16), (ODD, "bf16", 7), (LARGE, "f32", 64),
                                            (SMALL, "bf16", 1), ((960, 64, 16, 8), "f32", 8)])
@pytest.mark.parametrize("case", ["one", "empty ones", "drafts", "ragged"])
def test_latent_attention_other_shapes(case, shape, dtype, bs):
    lens, ql = CASES[case]
    rng = np.random.default_rng(bs + len(case))
    dims, od = make_dims(shape, 3, bs, dtype)
    qsl = loc(ql)
    cache, table = make_cache(rng, lens, bs, shape[0] + shape[1], dims.dtype)
    q = normal(rng, qsl[-1], 3, shape[0] + shape[1], std=0.5, dtype=dims.dtype)
    o, lse = run_attn(dims, True, qsl, lens, q, cache, table)
    check_attn(dims, od, True, qsl, lens, q, cache, table, o, lse)


@pytest.mark.parametrize("H", [128, 64, 16])
def test_latent_attention_growing_scores(H):
    """Scores that rise steeply along the keys (the running maximum moves in
    every tile), fall, and reach hundreds: no overflow, the late keys win."""
    rng = np.random.default_rng(4)
    dims, od = make_dims(LARGE, H, 64, "bf16")
    lens, qsl = [900, 900, 900], [0, 1, 2, 3]
    cache, table = make_cache(rng, lens, 64, 576, dims.dtype)
    for r, ramp in enumerate((np.linspace(-40, 40, 900), np.linspace(40, -40, 900), np.full(900, -300.0))):
        for j in range(900):
            cache[table[r, j // 64], j % 64, 575] = float(ramp[j])
    q = normal(rng, 3, H, 576, std=0.2)
    q[:, :, 575] = 30.0
    q = q.to(dims.dtype)
    o, lse = run_attn(dims, True, qsl, lens, q, cache, table)
    check_attn(dims, od, True, qsl, lens, q, cache, table, o, lse)


def test_latent_attention_many_requests_and_rows_of_no_sequence():
    """Several units a cluster, several clusters a unit; rows before the first
    and after the last sequence stay as they were."""
    rng = np.random.default_rng(8)
    for H in (128, 8):
        dims, od = make_dims(LARGE, H, 16, "bf16")
        ql = [int(x) for x in rng.integers(0, 3, size=90)]
        lens = [int(x) for x in rng.integers(0, 200, size=90)]
        qsl = [x + 2 for x in loc(ql)]
        T = qsl[-1] + 3
        cache, table = make_cache(rng, lens, 16, 576, dims.dtype)
        q = normal(rng, T, H, 576, std=0.4, dtype=dims.dtype)
        o, lse = run_attn(dims, True, qsl, lens, q, cache, table)
        check_attn(dims, od, True, qsl, lens, q, cache, table, o, lse)


@pytest.mark.parametrize("shape,dtype", [(LARGE, "bf16"), (SMALL, "f32")])
def test_latent_attention_bad_blocks(shape, dtype):
    """Bad block ids: a status bit, the rows read as zeros; a length past the
    block table's row: the bit, and the keys end with the row."""
    rng = np.random.default_rng(12)
    dims, od = make_dims(shape, 4, 16, dtype)
    lens, qsl = [100, 50, 60], [0, 1, 2, 3]
    cache, table = make_cache(rng, lens, 16, shape[0] + shape[1], dims.dtype)
    q = normal(rng, 3, 4, shape[0] + shape[1], std=0.4, dtype=dims.dtype)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    o, lse = run_attn(dims, True, qsl, lens, q, cache, table, status=status)
    bad = table.clone()
    bad[0, 2] = cache.shape[0]
    bad[1, 0] = -1
    assert status.item() == 0
    bad[2] = table[2, 0]
    row = [100, 50, 16 * table.shape[1]]
    o, lse = run_attn(dims, True, qsl, row, q, cache, bad, status=status)
    assert status.item() == M.MLA_STATUS_BAD_BLOCK
    status.zero_()
    far = table.clone()
    far[2] = table[2, 0]  # (a full block of sequence 2, as often as the row is long)
    o2, lse2 = run_attn(dims, True, qsl, [100, 50, row[2] + 20], q, cache, far, status=status)
    assert status.item() == M.MLA_STATUS_BAD_BLOCK
    check_attn(dims, od, True, qsl, row, q, cache, far, o2, lse2)
    zero = torch.cat([cache, torch.zeros_like(cache[:1])])  # the same with zero blocks
    ztab = bad.clone()
    ztab[(ztab < 0) | (ztab > len(cache))] = len(cache)
    check_attn(dims, od, True, qsl, row, q, zero, ztab, o, lse)


def test_latent_attention_far_offsets():
    """A cache of more than 2^31 elements and 2^32 bytes: rows at its far end."""
    dims, od = make_dims(LARGE, 16, 64, "bf16")
    blocks = 64000                                   # 64000*64*576 = 2.36e9 elements
    cache = torch.zeros(blocks, 64, 576, dtype=torch.bfloat16, device=DEV)
    rng = np.random.default_rng(3)
    small, table = make_cache(rng, [200], 64, 576, dims.dtype, spare=0)
    far = blocks - 1 - torch.arange(4)
    cache[far.to(DEV)] = small.to(DEV)
    q = normal(rng, 1, 16, 576, std=0.4, dtype=dims.dtype)
    ftab = table.clone()
    ftab[0, :4] = far[table[0, :4].long()].int()
    o, lse = run_attn(dims, True, [0, 1], [200], q, cache, ftab)
    del cache
    check_attn(dims, od, True, [0, 1], [200], q, small, table, o, lse)


# ----------------------------------------------------------- absorb/expand --
@pytest.mark.parametrize("shape,dtype,H", [(LARGE, "bf16", 128), (LARGE, "bf16", 3), (SMALL, "f32", 16),
                                           (ODD, "bf16", 5), (LARGE, "f32", 2)])
@pytest.mark.parametrize("T", [1, 3, 64, 129, 200])
def test_absorb_and_expand(shape, dtype, H, T):
    rng = np.random.default_rng(T + H)
    dims, od = make_dims(shape, H, 16, dtype)
    L, P, Dn, Dv = shape
    q = normal(rng, T, H, Dn + P, dtype=dims.dtype)
    w = normal(rng, H * (Dn + Dv), L, std=0.1, dtype=dims.dtype)
    ol = normal(rng, T, H, L, dtype=dims.dtype)
    u = unit(dims.dtype)
    for rope in (True, False):
        got = torch.full((T, H, L + P), 7.0, dtype=dims.dtype, device=DEV)
        M.mla_absorb_query(dims, q.to(DEV), w.to(DEV), got, rope_columns=rope)
        ref = O.absorb_query(f64(q), f64(w), od)
        mass = O.absorb_query(np.abs(f64(q)), np.abs(f64(w)), od)
        mass[..., L:] = 0
        if not rope:
            ref[..., L:] = 7.0
        within(f64(got), ref, u * np.abs(ref) + (Dn + 4) * F * mass, "absorb")
        assert (f64(got)[..., L:] == ref[..., L:]).all()
    out = torch.full((T, H, Dv), 7.0, dtype=dims.dtype, device=DEV)
    M.mla_expand_output(dims, ol.to(DEV), w.to(DEV), out)
    ref = O.expand_output(f64(ol), f64(w), od)
    mass = O.expand_output(np.abs(f64(ol)), np.abs(f64(w)), od)
    within(f64(out), ref, u * np.abs(ref) + (L + 4) * F * mass, "expand")


# ----------------------------------------------------------------- append --
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shape,dtype,bs,norm,wide,dense,queries", [
    (LARGE, "bf16", 64, True, 0, True, "own"),
    (LARGE, "bf16", 16, True, 64, False, "place"),
    (LARGE, "bf16", 1, False, 3, True, "latent"),
    (SMALL, "f32", 16, True, 1, True, "own"),
    (ODD, "bf16", 5, True, 0, True, "place"),
    ((64, 4, 6, 8), "f32", 3, False, 0, False, "latent"),
    (LARGE, "f32", 64, True, 0, True, None),
])
def test_append(shape, dtype, bs, norm, wide, dense, queries, interleaved):
    rng = np.random.default_rng(bs + wide)
    H = 5
    dims, od = make_dims(shape, H, bs, dtype)
    L, P, Dn, Dv = shape
    lens, ql = [70, 1, 0, 6, 2, 64, 33], [3, 1, 0, 6, 5, 1, 0]   # one has more new tokens than tokens
    qsl = [x + 1 for x in loc(ql)]
    T = qsl[-1] + 2
    cache, table = make_cache(rng, lens, bs, L + P, dims.dtype)
    before = cache.clone()
    store = normal(rng, T, L + P + wide, dtype=dims.dtype)
    kv_a = store[:, wide:]
    gw = (1 + 0.2 * normal(rng, L)).to(dims.dtype) if norm else None
    tab = torch.from_numpy(O.rope_table(80, P).astype(np.float32))
    q = normal(rng, T, H, Dn + P, dtype=dims.dtype)
    g_store, g_q, g_cache = store.to(DEV), q.to(DEV), cache.to(DEV)
    lat = torch.full((T, L + P), 7.0, dtype=dims.dtype, device=DEV) if dense else None
    ql_buf = torch.full((T, H, L + P), 7.0, dtype=dims.dtype, device=DEV)
    own = torch.full((T, H, P), 7.0, dtype=dims.dtype, device=DEV)
    pe = {"own": own, "place": g_q[..., Dn:], "latent": ql_buf[..., L:], None: None}[queries]
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    M.mla_append_latent(dims, g_store[:, wide:], i32(qsl), i32(lens), tab.to(DEV), g_cache,
                        table.to(DEV), norm_weight=None if gw is None else gw.to(DEV), norm_eps=1e-5,
                        interleaved=interleaved, new_latent=lat, q=g_q if queries else None,
                        q_pe_out=pe, dev_status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    u = unit(dims.dtype)
    eps = float(np.float32(1e-5))
    want = f64(before)
    ftab, touched = f64(tab), set()
    for t, r, pos in O.token_positions(qsl, lens):
        if pos < 0:
            continue
        touched.add(t)
        ref = O.latent_row(f64(kv_a[t]), od, None if gw is None else f64(gw), eps, ftab[pos], interleaved)
        size = np.abs(ref) * (L / 32 + 16)
        pair = np.abs(f64(kv_a[t]))[L:]
        size[L:] = 16 * 2 * pair.max()
        tol = u * np.abs(ref) + F * size
        blk, slot = int(table[r, pos // bs]), pos % bs
        within(f64(g_cache[blk, slot]), ref, tol, "cache row")
        want[blk, slot] = f64(g_cache[blk, slot])
        if dense:
            assert torch.equal(lat[t], g_cache[blk, slot])
        if queries:
            ref = O.rotate(f64(q[t, :, Dn:]), ftab[pos], interleaved)
            tol = u * np.abs(ref) + F * 32 * np.abs(f64(q[t, :, Dn:])).max()
            within(f64(pe[t]), ref, tol, "q_pe")
    assert np.array_equal(f64(g_cache), want, equal_nan=True)  # no other slot written
    for t in set(range(T)) - touched:
        assert lat is None or (lat[t] == 7.0).all()
        if queries == "place":
            assert torch.equal(g_q[t].cpu(), q[t])
        elif queries:
            assert (pe[t] == 7.0).all()
    if queries == "place":
        assert torch.equal(g_q[..., :Dn].cpu(), q[..., :Dn])
    if queries == "latent":
        assert (ql_buf[..., :L] == 7.0).all()


def test_append_positions_and_bad_ones():
    """Own rope positions; one outside the table and bad blocks set their bits
    and leave the cache alone."""
    rng = np.random.default_rng(1)
    dims, od = make_dims(SMALL, 2, 4, "f32")
    qsl, lens = [0, 3, 5], [3, 30]
    cache, table = make_cache(rng, lens, 4, 80, dims.dtype)
    kv_a = normal(rng, 5, 80)
    tab = torch.from_numpy(O.rope_table(10, 16).astype(np.float32))
    pos = [9, 0, 4, 10, -1]                   # the last two: outside
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    g, lat = cache.to(DEV), torch.full((5, 80), 7.0, device=DEV)
    M.mla_append_latent(dims, kv_a.to(DEV), i32(qsl), i32(lens), tab.to(DEV), g, table.to(DEV),
                        positions=i32(pos), new_latent=lat, dev_status=status)
    assert status.item() == M.MLA_STATUS_BAD_POSITION
    for t in range(3):
        ref = O.latent_row(f64(kv_a[t]), od, None, 0.0, f64(tab)[pos[t]], False)
        within(f64(lat[t]), ref, F * np.abs(ref) + F * 32 * np.abs(f64(kv_a[t])).max(), "row")
        assert torch.equal(g[table[0, 0], t], lat[t])
    assert (lat[3:] == 7.0).all()
    status.zero_()
    bad = table.clone()
    bad[0, 0] = cache.shape[0]
    g = cache.to(DEV)
    M.mla_append_latent(dims, kv_a.to(DEV), i32(qsl), i32([3, 4 * table.shape[1] + 2]), None, g,
                        bad.to(DEV), new_latent=lat, dev_status=status)
    assert status.item() == M.MLA_STATUS_BAD_BLOCK
    assert torch.equal(torch.nan_to_num(g.cpu(), 5.0), torch.nan_to_num(cache, 5.0))
    assert torch.equal(lat.cpu(), kv_a)       # no norm, no rotation: copied


# ------------------------------------------------------------- whole step --
@pytest.mark.parametrize("shape,dtype,H", [(LARGE, "bf16", 128), (LARGE, "bf16", 16), (SMALL, "f32", 16)])
def test_decode_steps_match_the_expanded_form(shape, dtype, H):
    """Prefill the cache with appended rows, then decode steps of one and two
    tokens, against the expanded attention (per-head keys and values) on the
    rows that the cache holds.  Tolerance: the framework's for attention output
    (O: 2e-2 + 2e-2 |ref|, LSE 1e-3 for float32); in bf16 the absorbed query is
    rounded once more, u |q_lat| |c| summed over L in quadrature would do, the
    linear bound u scale sum|q_lat||c| is taken."""
    rng = np.random.default_rng(H)
    dims, od = make_dims(shape, H, 16, dtype)
    L, P, Dn, Dv = shape
    R, start = 3, [37, 0, 90]
    total = [s + 4 for s in start]
    cache, table = make_cache(rng, total, 16, L + P, dims.dtype)
    g_cache, g_table = cache.to(DEV), table.to(DEV)
    tab = torch.from_numpy(O.rope_table(200, P).astype(np.float32)).to(DEV)
    w = normal(rng, H * (Dn + Dv), L, std=0.5 / math.sqrt(L), dtype=dims.dtype)
    gw = (1 + 0.1 * normal(rng, L)).to(dims.dtype).to(DEV)
    dec = M.LatentDecode(dims, 8, 4, device=DEV)
    have = list(start)
    for n in (1, 2, 1):
        have = [h + n for h in have]
        T = R * n
        q = normal(rng, T, H, Dn + P, dtype=dims.dtype)
        kv_a = normal(rng, T, L + P, dtype=dims.dtype)
        out = torch.empty(T, H, Dv, dtype=dims.dtype, device=DEV)
        lse = torch.empty(H, T, device=DEV)
        dec(q.to(DEV), kv_a.to(DEV), i32(range(0, T + 1, n)), i32(have), tab, g_cache, g_table,
            w.to(DEV), out, lse, norm_weight=gw)
        torch.cuda.synchronize()
        c, wn = f64(g_cache), f64(w)
        for r in range(R):
            rows = np.stack([O.context_row(c, table.numpy(), r, j, 16) for j in range(have[r])])
            assert np.isfinite(rows).all()
            kn, v = O.up_project(rows, wn, od)
            qr = f64(q[r * n:(r + 1) * n])
            for i in range(n):
                qr[i, :, Dn:] = O.rotate(qr[i, :, Dn:], f64(tab)[have[r] - n + i], False)
            vis = np.arange(have[r])[None, :] <= (have[r] - n + np.arange(n))[:, None]
            ro, rl = O.attention_with_lse(qr, kn, rows[:, L:], v, od.softmax_scale, vis)
            slack = 0.0
            if dtype == "bf16":
                ql = np.abs(O.absorb_query(qr, wn, od))
                slack = unit(dims.dtype) * od.softmax_scale * np.einsum(
                    "thl,nl->thn", ql, np.abs(rows), optimize=True).max()
            sl = slice(r * n, (r + 1) * n)
            within(f64(lse)[:, sl], rl, 1e-3 + slack, "lse")
            within(f64(out)[sl], ro, 2e-2 + 2e-2 * np.abs(ro), "out")


@pytest.mark.parametrize("shape,dtype", [(LARGE, "bf16"), (SMALL, "f32")])
def test_decode_step_captured_and_replayed(shape, dtype):
    """One step captured into a graph and replayed while the lengths on the
    device grow gives what eager calls give."""
    rng = np.random.default_rng(77)
    H, R = 32, 4
    dims, od = make_dims(shape, H, 16, dtype)
    L, P, Dn, Dv = shape
    start, steps = [100, 1, 511, 37], 3
    cache, table = make_cache(rng, [s + steps + 1 for s in start], 16, L + P, dims.dtype)
    tab = torch.from_numpy(O.rope_table(600, P).astype(np.float32)).to(DEV)
    w = normal(rng, H * (Dn + Dv), L, std=0.1, dtype=dims.dtype).to(DEV)
    qs = [normal(rng, R, H, Dn + P, dtype=dims.dtype).to(DEV) for _ in range(steps)]
    ks = [normal(rng, R, L + P, dtype=dims.dtype).to(DEV) for _ in range(steps)]
    qsl, table = i32(range(R + 1)), table.to(DEV)

    def step(dec, q, k, lens, c, out, lse):
        dec(q, k, qsl, lens, tab, c, table, w, out, lse)

    eager, c, lens = [], cache.to(DEV), i32(start)
    dec = M.LatentDecode(dims, R, R, device=DEV)
    for q, k in zip(qs, ks):
        lens += 1
        out, lse = torch.empty(R, H, Dv, dtype=dims.dtype, device=DEV), torch.empty(H, R, device=DEV)
        step(dec, q, k, lens, c, out, lse)
        eager.append((out, lse))
    torch.cuda.synchronize()
    c2, lens2 = cache.to(DEV), i32([s + 1 for s in start])
    q, k = qs[0].clone(), ks[0].clone()
    out, lse = torch.empty(R, H, Dv, dtype=dims.dtype, device=DEV), torch.empty(H, R, device=DEV)
    dec2 = M.LatentDecode(dims, R, R, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(dec2, q, k, lens2, c2, out, lse)
    for i in range(steps):
        q.copy_(qs[i])
        k.copy_(ks[i])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager[i][0]) and torch.equal(lse, eager[i][1])
        lens2 += 1
    assert torch.equal(torch.nan_to_num(c.float(), 5.0), torch.nan_to_num(c2.float(), 5.0))


def test_latent_attention_same_result_on_another_stream_and_again():
    """Bit for bit the same, on a side stream and with a used workspace."""
    rng = np.random.default_rng(5)
    dims, od = make_dims(LARGE, 128, 64, "bf16")
    lens, qsl = [2000, 300, 5], [0, 1, 3, 4]
    cache, table = make_cache(rng, lens, 64, 576, dims.dtype)
    q = normal(rng, 4, 128, 576, std=0.4, dtype=dims.dtype)
    o, lse = run_attn(dims, True, qsl, lens, q, cache, table)
    s = torch.cuda.Stream()
    gq, gc, gt, a, b = q.to(DEV), cache.to(DEV), table.to(DEV), i32(qsl), i32(lens)
    ws = torch.empty(M.mla_latent_attn_workspace_bytes(dims, 4, 3), dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    for _ in range(3):
        o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
        s.wait_stream(torch.cuda.current_stream())
        M.mla_latent_attn(dims, True, a, b, gq, gc, gt, ws, o2, lse2, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


# -------------------------------------------------- cut units and their joins --
@pytest.mark.parametrize("H,lens,ql", [
    (128, [20011], [1]),                            # dozens of pieces
    (20, [20011], [1]),                             # the same, 44 of 64 rows dead
    (33, [5000, 64, 7001], [4, 1, 3]),              # units of 128 and of a few rows
    (128, [1500 - 17 * i for i in range(60)], [1] * 60),   # a few pieces each
    (128, [900, 30, 901, 29], [9, 1, 2, 40]),
    (16, [700 + i for i in range(200)], [1] * 200),
    (64, [4000, 4000, 0, 4000], [1, 1, 1, 1]),
])
def test_latent_attention_cut_units(H, lens, ql):
    rng = np.random.default_rng(H + len(lens))
    dims, od = make_dims(LARGE, H, 64, "bf16")
    qsl = loc(ql)
    cache, table = make_cache(rng, lens, 64, 576, dims.dtype)
    q = normal(rng, qsl[-1], H, 576, std=0.4, dtype=dims.dtype)
    for causal in (True, False):
        o, lse = run_attn(dims, causal, qsl, lens, q, cache, table)
        check_attn(dims, od, causal, qsl, lens, q, cache, table, o, lse)


@pytest.mark.parametrize("H", [16, 128])
def test_latent_attention_thousand_requests(H):
    """More sequences than a block has threads; sequences that share pages."""
    rng = np.random.default_rng(H)
    dims, od = make_dims(LARGE, H, 16, "bf16")
    R = 1000
    lens = [int(x) for x in rng.integers(0, 90, size=R)]
    qsl = loc([int(x) for x in rng.integers(0, 3, size=R)])
    cache, table = make_cache(rng, lens[:50], 16, 576, dims.dtype)
    table = table[torch.arange(R) % 50]
    lens = [min(n, lens[r % 50]) for r, n in enumerate(lens)]
    q = normal(rng, qsl[-1], H, 576, std=0.4, dtype=dims.dtype)
    o, lse = run_attn(dims, True, qsl, lens, q, cache, table)
    check_attn(dims, od, True, qsl, lens, q, cache, table, o, lse)


@pytest.mark.parametrize("blocks", [6, 7, 8, 9])
@pytest.mark.parametrize("H", [64, 128])
def test_latent_attention_short_tables(H, blocks):
    """Block tables at and around the length up to which no unit is cut."""
    rng = np.random.default_rng(blocks)
    dims, od = make_dims(LARGE, H, 64, "bf16")
    R = 170
    lens = [int(x) for x in rng.integers(1, blocks * 64 + 1, size=R)]
    lens[0] = blocks * 64
    cache, table = make_cache(rng, lens, 64, 576, dims.dtype)
    table = table[:, :blocks].contiguous()
    q = normal(rng, R, H, 576, std=0.4, dtype=dims.dtype)
    o, lse = run_attn(dims, True, list(range(R + 1)), lens, q, cache, table)
    check_attn(dims, od, True, list(range(R + 1)), lens, q, cache, table, o, lse)


def test_latent_attention_without_blocks():
    """A cache of no blocks: every position is bad and read as zeros, so the
    scores are 0, the output 0 and the log-sum ln n."""
    import ctypes as C
    dims, _ = make_dims(LARGE, 8, 16, "bf16")
    d = dims.c()
    cache = torch.ones(2, 16, 576, dtype=dims.dtype, device=DEV)
    q = torch.ones(1, 8, 576, dtype=dims.dtype, device=DEV)
    o = torch.full((1, 8, 512), 7.0, dtype=dims.dtype, device=DEV)
    lse, table = torch.zeros(8, 1, device=DEV), torch.zeros(1, 8, dtype=torch.int32, device=DEV)
    ws = torch.empty(M.mla_latent_attn_workspace_bytes(dims, 1, 1), dtype=torch.uint8, device=DEV)
    status, qsl, lens = i32([0]), i32([0, 1]), i32([100])
    rc = M.lib().mla_latent_attn(
        C.byref(d), 1, 1, qsl.data_ptr(), lens.data_ptr(), 1, q.data_ptr(), cache.data_ptr(), 0,
        table.data_ptr(), 8, ws.data_ptr(), ws.numel(), o.data_ptr(), lse.data_ptr(),
        status.data_ptr(), None)
    torch.cuda.synchronize()
    assert rc == 0 and status.item() == M.MLA_STATUS_BAD_BLOCK and (o == 0).all()
    # the sum 100 is exact; log2f of it (6.6) is within its last place 2^-21,
    # times ln 2; the rounding of ln 2 (2^-25) times 6.6 and the product's 2^-22
    within(f64(lse), np.full((8, 1), math.log(100)), 2.0 ** -21 * 0.7 + 6.7 * 2.0 ** -25 + 2.0 ** -22,
           "lse")


def test_append_and_attention_far_offsets_elsewhere():
    """The append, and the CUDA-core attention, past 2^31 elements of a cache."""
    dims, od = make_dims(SMALL, 2, 64, "f32")
    blocks = 2 ** 31 // (64 * 80) + 100
    cache = torch.empty(blocks, 64, 80, device=DEV)
    rng = np.random.default_rng(9)
    kv_a = normal(rng, 70, 80)
    table = torch.tensor([[blocks - 1, blocks - 7]], dtype=torch.int32)
    M.mla_append_latent(dims, kv_a.to(DEV), i32([0, 70]), i32([70]), None, cache, table.to(DEV))
    assert torch.equal(cache[blocks - 1].cpu(), kv_a[:64])
    assert torch.equal(cache[blocks - 7, :6].cpu(), kv_a[64:])
    q = normal(rng, 1, 2, 80)
    o, lse = run_attn(dims, True, [0, 1], [70], q, cache, table)
    small = torch.full((2, 64, 80), float("nan"))
    small[0], small[1, :6] = kv_a[:64], kv_a[64:]
    del cache
    check_attn(dims, od, True, [0, 1], [70], q, small, torch.tensor([[0, 1]], dtype=torch.int32), o, lse)


# ------------------------------------------------- memory, streams, refusals --
@pytest.mark.parametrize("shape,dtype,H", [(LARGE, "bf16", 128), (LARGE, "bf16", 20), (SMALL, "f32", 3),
                                           (ODD, "bf16", 5)])
def test_nothing_is_written_beside_the_outputs(shape, dtype, H):
    """Outputs and workspace lie between guard bytes, which stay as they were."""
    rng = np.random.default_rng(H)
    dims, od = make_dims(shape, H, 16, dtype)
    L, P, Dn, Dv = shape
    T, lens, qsl = 5, [1200, 40], [0, 3, 4]                 # the last row: of no sequence
    cache, table = make_cache(rng, lens, 16, L + P, dims.dtype)
    guards = []

    def guarded(*size, dtype):
        n = math.prod(size) * dtype.itemsize
        raw = torch.full((n + 512,), 0x5A, dtype=torch.uint8, device=DEV)
        guards.append((raw, n))
        return raw[256:256 + n].view(dtype).view(*size)

    q = normal(rng, T, H, Dn + P, dtype=dims.dtype).to(DEV)
    w = normal(rng, H * (Dn + Dv), L, std=0.1, dtype=dims.dtype).to(DEV)
    q_lat = guarded(T, H, L + P, dtype=dims.dtype)
    o_lat = guarded(T, H, L, dtype=dims.dtype)
    out = guarded(T, H, Dv, dtype=dims.dtype)
    lse = guarded(H, T, dtype=torch.float32)
    g_cache = guarded(*cache.shape, dtype=dims.dtype)
    lat = guarded(T, L + P, dtype=dims.dtype)
    ws = guarded(M.mla_latent_attn_workspace_bytes(dims, T, 2), dtype=torch.uint8)
    g_cache.copy_(cache)
    tab = torch.from_numpy(O.rope_table(1300, P).astype(np.float32)).to(DEV)
    kv_a = normal(rng, T, L + P, dtype=dims.dtype).to(DEV)
    a, b, t = i32(qsl), i32(lens), table.to(DEV)
    M.mla_append_latent(dims, kv_a, a, b, tab, g_cache, t, new_latent=lat, q=q, q_pe_out=q_lat[..., L:])
    M.mla_absorb_query(dims, q, w, q_lat, rope_columns=False)
    M.mla_latent_attn(dims, True, a, b, q_lat, g_cache, t, ws, o_lat, lse)
    M.mla_expand_output(dims, o_lat, w, out)
    torch.cuda.synchronize()
    for raw, n in guards:
        assert (raw[:256] == 0x5A).all() and (raw[256 + n:] == 0x5A).all()
    assert (lat[4].view(torch.uint8) == 0x5A).all() and (o_lat[4].view(torch.uint8) == 0x5A).all()
    q_lat_ref = q_lat.clone()
    q_lat_ref[4] = 0
    _, rl, _, size = O.latent_attention(f64(q_lat_ref), f64(g_cache), table.numpy(), qsl, lens, od, True)
    tol = (L + P + 8) * F * size + 2.0 ** -22 + (1200 / 8 + 16) * F + F * np.abs(rl)
    within(f64(lse)[:, :4], rl[:, :4], tol[:, :4], "lse")


def test_two_streams_at_once():
    """Two attentions on two streams, a workspace each, give what each gives
    alone; a side stream's inputs are made on it."""
    rng = np.random.default_rng(21)
    dims, od = make_dims(LARGE, 128, 64, "bf16")
    sets = []
    for lens in ([3000, 1200, 700], [64, 2500]):
        cache, table = make_cache(rng, lens, 64, 576, dims.dtype)
        q = normal(rng, len(lens), 128, 576, std=0.4, dtype=dims.dtype)
        o, lse = run_attn(dims, True, list(range(len(lens) + 1)), lens, q, cache, table)
        ws = torch.empty(M.mla_latent_attn_workspace_bytes(dims, len(lens), len(lens)),
                         dtype=torch.uint8, device=DEV)
        sets.append((i32(range(len(lens) + 1)), i32(lens), q.to(DEV), cache.to(DEV), table.to(DEV), ws,
                     o, lse, torch.empty_like(o), torch.empty_like(lse), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        for a, b, q, c, t, ws, _, _, o2, lse2, s in sets:
            with torch.cuda.stream(s):
                q2 = q * 1
                M.mla_latent_attn(dims, True, a, b, q2, c, t, ws, o2, lse2)
        torch.cuda.synchronize()
        for *_, o, lse, o2, lse2, _ in sets:
            assert torch.equal(o, o2) and torch.equal(lse, lse2)
            o2.fill_(0)
            lse2.fill_(0)
        torch.cuda.synchronize()


@pytest.mark.parametrize("shape,dtype", [(LARGE, "bf16"), (SMALL, "f32")])
def test_two_graphs_and_a_padded_batch(shape, dtype):
    """Two captured steps that share an instance (its workspace too), replayed
    in turn, the second for fewer tokens than its arrays have rows: what eager
    calls of the tokens alone give, and the cache of the others untouched."""
    rng = np.random.default_rng(6)
    H = 16
    dims, od = make_dims(shape, H, 16, dtype)
    L, P, Dn, Dv = shape
    lens = [600, 33, 1, 250]
    cache, table = make_cache(rng, lens, 16, L + P, dims.dtype)
    tab = torch.from_numpy(O.rope_table(700, P).astype(np.float32)).to(DEV)
    w = normal(rng, H * (Dn + Dv), L, std=0.1, dtype=dims.dtype).to(DEV)
    q = normal(rng, 8, H, Dn + P, dtype=dims.dtype).to(DEV)
    kv_a = normal(rng, 8, L + P, dtype=dims.dtype).to(DEV)
    table, dec = table.to(DEV), M.LatentDecode(dims, 8, 4, device=DEV)
    eager = []
    for n in (4, 2):
        c, out = cache.to(DEV), torch.empty(n, H, Dv, dtype=dims.dtype, device=DEV)
        dec(q[:n].contiguous(), kv_a[:n], i32(range(n + 1)), i32(lens[:n]), tab, c,
            table[:n].contiguous(), w, out)
        eager.append((c, out))
    torch.cuda.synchronize()
    graphs = []
    for n, qsl in ((4, i32(range(5))), (2, i32([0, 1, 2, 2, 2]))):
        c, ls = cache.to(DEV), i32(lens)
        out = torch.empty(8, H, Dv, dtype=dims.dtype, device=DEV)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            dec(q, kv_a, qsl, ls, tab, c, table, w, out)
        graphs.append((g, c, out, n, qsl, ls))
    for _ in range(2):
        for (g, c, out, n, _, _), (rc, ro) in zip(graphs, eager):
            out.fill_(0)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out[:n], ro)
            assert torch.equal(torch.nan_to_num(c.float(), 5.0), torch.nan_to_num(rc.float(), 5.0))


def test_bindings_refuse():
    """Wrong types, shapes and strides raise before anything is enqueued."""
    dims, _ = make_dims(SMALL, 3, 16, "f32")
    q = torch.zeros(2, 3, 48, device=DEV)
    kv_a, ql, ol = torch.zeros(2, 80, device=DEV), torch.zeros(2, 3, 80, device=DEV), torch.zeros(2, 3, 64, device=DEV)
    w, out = torch.zeros(3 * 64, 64, device=DEV), torch.zeros(2, 3, 32, device=DEV)
    cache, table = torch.zeros(4, 16, 80, device=DEV), torch.zeros(2, 2, dtype=torch.int32, device=DEV)
    a, b, tab = i32([0, 1, 2]), i32([5, 6]), torch.zeros(9, 16, device=DEV)
    before = M.mla_kernel_launches()

    def refuses(f, *args, **kw):
        with pytest.raises((ValueError, M.MlaError)):
            f(dims, *args, **kw)

    wide = torch.zeros(2, 3, 160, device=DEV)
    refuses(M.mla_absorb_query, q.bfloat16(), w, ql)
    refuses(M.mla_absorb_query, q[:, :2], w, ql)
    refuses(M.mla_absorb_query, q, w.t(), ql)
    refuses(M.mla_absorb_query, q, w, wide[..., :80])
    refuses(M.mla_absorb_query, q, w[:-1], ql)
    refuses(M.mla_expand_output, ol, w, out[:1])
    refuses(M.mla_expand_output, ol, w.cpu(), out)
    refuses(M.mla_expand_output, ol[0], w, out)
    refuses(M.mla_append_latent, kv_a[:, :79], a, b, tab, cache, table)
    refuses(M.mla_append_latent, kv_a.t().contiguous().t(), a, b, tab, cache, table)
    refuses(M.mla_append_latent, kv_a[:1].expand(2, 80), a, b, tab, cache, table)
    refuses(M.mla_append_latent, kv_a, a.long(), b, tab, cache, table)
    refuses(M.mla_append_latent, kv_a, a[:2], b, tab, cache, table)
    refuses(M.mla_append_latent, kv_a, a, b, tab.double(), cache, table)
    refuses(M.mla_append_latent, kv_a, a, b, tab, cache[:, :8], table)
    refuses(M.mla_append_latent, kv_a, a, b, tab, cache, table, q=q)
    refuses(M.mla_append_latent, kv_a, a, b, tab, cache, table, q=q, q_pe_out=ql[:, :2, 64:])
    refuses(M.mla_append_latent, kv_a, a, b, tab, cache, table, q=q, q_pe_out=ql[..., ::5])
    refuses(M.mla_append_latent, kv_a, a, b, tab, cache, table, q=q, q_pe_out=ql[..., 64:].flip(0)[:1])
    refuses(M.mla_latent_attn, True, a, b, ql, cache.transpose(0, 1), table, None, ol)
    refuses(M.mla_latent_attn, True, a, b, ql, cache, table[:1], None, ol)
    refuses(M.mla_latent_attn, True, a, b, ql, cache, table, None, ol, torch.zeros(2, 3, device=DEV))
    refuses(M.mla_latent_attn, True, a, b, ql[..., :64], cache, table, None, ol)
    torch.cuda.synchronize()
    assert M.mla_kernel_launches() == before
    large, _ = make_dims(LARGE, 3, 16, "bf16")
    need = M.mla_latent_attn_workspace_bytes(large, 2, 2)
    h = {"dtype": torch.bfloat16, "device": DEV}
    qb, cb, ob = torch.zeros(2, 3, 576, **h), torch.zeros(4, 16, 576, **h), torch.zeros(2, 3, 512, **h)
    for ws in (None, torch.empty(need - 1, dtype=torch.uint8, device=DEV),
               torch.empty(need + 16, dtype=torch.uint8, device=DEV)[1:]):
        with pytest.raises((ValueError, M.MlaError)):
            M.mla_latent_attn(large, True, a, b, qb, cb, table, ws, ob)
    assert M.mla_kernel_launches() == before


@pytest.mark.parametrize("shape,dtype,H,bs", [
    (LARGE, "bf16", 128, 64), (LARGE, "bf16", 32, 64), (LARGE, "bf16", 48, 16), (LARGE, "bf16", 32, 1),
    (LARGE, "bf16", 16, 64), (LARGE, "bf16", 5, 4), (LARGE, "bf16", 40, 5), (SMALL, "f32", 4, 16)])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
def test_rows_that_are_not_finite_reach_only_tokens_that_see_them(shape, dtype, H, bs, value):
    """Of four new tokens' cache rows the third's is not finite: the first two
    tokens' results are bit for bit what they are without it, the others NaN
    (but for heads that score the row -inf: it may weigh nothing there)."""
    rng = np.random.default_rng(H + bs)
    dims, od = make_dims(shape, H, bs, dtype)
    L, LP = shape[0], shape[0] + shape[1]
    lens, qsl = [700, 4, 66, 130], [0, 4, 8, 12, 13]
    cache, table = make_cache(rng, lens, bs, LP, dims.dtype)
    q = normal(rng, 13, H, LP, std=0.4, dtype=dims.dtype)
    o, lse = run_attn(dims, True, qsl, lens, q, cache, table)
    check_attn(dims, od, True, qsl, lens, q, cache, table, o, lse)
    bad = cache.clone()
    for r in range(3):
        j = lens[r] - 2
        for col in (L - 1, 0, L // 2, L + 1):
            if r == 0 or col % 2:
                bad[table[r, j // bs], j % bs, col] = value
    o2, lse2 = run_attn(dims, True, qsl, lens, q, bad, table)
    for t in range(13):
        sees = t < 12 and t % 4 >= 2
        if sees:
            r = t // 4
            row = f64(bad[table[r, (lens[r] - 2) // bs], (lens[r] - 2) % bs])
            score = f64(q[t]) @ row
            nan = torch.isnan(o2[t]).any(-1).cpu().numpy()
            assert (nan | (score == -np.inf)).all() and nan.any()
        else:
            assert torch.equal(o2[t], o[t]) and torch.equal(lse2[:, t], lse[:, t]), t


def test_decode_step_without_rope_columns_and_without_tokens():
    rng = np.random.default_rng(2)
    dims, od = make_dims((64, 0, 32, 32), 3, 16, "f32")
    lens, qsl = [40, 7], [0, 1, 3]
    cache, table = make_cache(rng, lens, 16, 64, dims.dtype)
    q, kv_a = normal(rng, 3, 3, 32), normal(rng, 3, 64)
    w = normal(rng, 3 * 64, 64, std=0.1)
    g_cache, out, lse = cache.to(DEV), torch.empty(3, 3, 32, device=DEV), torch.empty(3, 3, device=DEV)
    dec = M.LatentDecode(dims, 4, 2, device=DEV)
    dec(q.to(DEV), kv_a.to(DEV), i32(qsl), i32(lens), None, g_cache, table.to(DEV), w.to(DEV), out, lse)
    torch.cuda.synchronize()
    for t, r, pos in O.token_positions(qsl, lens):
        assert torch.equal(g_cache[table[r, pos // 16], pos % 16].cpu(), kv_a[t])
    q_lat = f64(dec.q_latent[:3])
    within(q_lat, O.absorb_query(f64(q), f64(w), od),
           36 * F * O.absorb_query(np.abs(f64(q)), np.abs(f64(w)), od), "absorb")
    _, rl, _, size = O.latent_attention(q_lat, f64(g_cache), table.numpy(), qsl, lens, od, True)
    within(f64(lse), rl, 72 * F * size + 2.0 ** -22 + 21 * F + F * np.abs(rl), "lse")
    o_lat = f64(dec.o_latent[:3])
    within(f64(out), O.expand_output(o_lat, f64(w), od),
           68 * F * O.expand_output(np.abs(o_lat), np.abs(f64(w)), od) + F * np.abs(f64(out)), "out")
    before, n = out.clone(), M.mla_kernel_launches()
    dec(q[:0].to(DEV), kv_a[:0].to(DEV), i32([0, 0, 0]), i32(lens), None, g_cache, table.to(DEV),
        w.to(DEV), out[:0])
    dec(q[:0].to(DEV), kv_a[:0].to(DEV), i32([0]), i32([]), None, g_cache, table[:0].to(DEV),
        w.to(DEV), out[:0])
    torch.cuda.synchronize()
    assert torch.equal(out, before) and M.mla_kernel_launches() == n


@pytest.mark.parametrize("H", [128, 40])
def test_latent_attention_outputs_at_16_bytes(H):
    """An output that starts 16 bytes into a sector gives the same bits."""
    rng = np.random.default_rng(H)
    dims, od = make_dims(LARGE, H, 64, "bf16")
    lens, qsl = [70, 900, 2600], [0, 1, 3, 4]
    cache, table = make_cache(rng, lens, 64, 576, dims.dtype)
    q = normal(rng, 4, H, 576, std=0.4, dtype=dims.dtype)
    o, lse = run_attn(dims, True, qsl, lens, q, cache, table)
    raw = torch.full((4 * H * 512 + 24,), 7.0, dtype=dims.dtype, device=DEV)
    o2 = raw[8:8 + 4 * H * 512].view(4, H, 512)
    assert o2.data_ptr() % 32 == 16
    ws = torch.empty(M.mla_latent_attn_workspace_bytes(dims, 4, 3), dtype=torch.uint8, device=DEV)
    M.mla_latent_attn(dims, True, i32(qsl), i32(lens), q.to(DEV), cache.to(DEV), table.to(DEV), ws, o2)
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and (raw[:8] == 7).all() and (raw[-16:] == 7).all()


@pytest.mark.parametrize("T,H", [(8, 128), (33, 80), (40, 128), (97, 128), (120, 9), (121, 128), (128, 40),
                                 (500, 12), (257, 160)])
def test_absorb_and_expand_tile_edges(T, H):
    """Token counts at the edges of boxes, tiles, stages and of columns a CTA."""
    rng = np.random.default_rng(T)
    dims, od = make_dims(LARGE, H, 16, "bf16")
    q = normal(rng, T, H, 192, dtype=dims.dtype)
    w = normal(rng, H * 256, 512, std=0.1, dtype=dims.dtype)
    ol = normal(rng, T, H, 512, dtype=dims.dtype)
    got = torch.full((T, H, 576), 7.0, dtype=dims.dtype, device=DEV)
    out = torch.full((T, H, 128), 7.0, dtype=dims.dtype, device=DEV)
    M.mla_absorb_query(dims, q.to(DEV), w.to(DEV), got)
    M.mla_expand_output(dims, ol.to(DEV), w.to(DEV), out)
    for h in sorted({0, H // 2, H - 1}):
        wh = f64(w[h * 256:(h + 1) * 256])
        for a, b, g, K in ((f64(q[:, h, :128]), wh[:128], got[:, h, :512], 128),
                           (f64(ol[:, h]), wh[128:].T, out[:, h], 512)):
            ref = a @ b
            within(f64(g), ref, unit(dims.dtype) * np.abs(ref) + (K + 4) * F * (np.abs(a) @ np.abs(b)),
                   f"head {h}")
    assert torch.equal(got[..., 512:].cpu(), q[..., 128:])


@pytest.mark.parametrize("T", [1, 16, 300, 500])
def test_chained_calls_back_to_back(T):
    """Absorptions, expansions and attentions enqueued one after another, whose
    blocks may be resident beside each other's, give what each gives alone."""
    rng = np.random.default_rng(T)
    H = 128
    dims, od = make_dims(LARGE, H, 64, "bf16")
    q = normal(rng, T, H, 192, dtype=dims.dtype).to(DEV)
    w = normal(rng, H * 256, 512, std=0.1, dtype=dims.dtype).to(DEV)
    q_small = q[:1].contiguous()
    cache, table = make_cache(rng, [200] * T if T < 20 else [64] * T, 64, 576, dims.dtype)
    cache, table = torch.nan_to_num(cache).to(DEV), table.to(DEV)
    lens, qsl = i32([200] * T if T < 20 else [64] * T), i32(range(T + 1))
    ws = torch.empty(M.mla_latent_attn_workspace_bytes(dims, T, T), dtype=torch.uint8, device=DEV)

    def step(sync):
        ql, small = torch.zeros(T, H, 576, dtype=dims.dtype, device=DEV), torch.zeros(1, H, 576, dtype=dims.dtype, device=DEV)
        ol, out = torch.zeros(T, H, 512, dtype=dims.dtype, device=DEV), torch.zeros(T, H, 128, dtype=dims.dtype, device=DEV)
        torch.cuda.synchronize()
        for _ in range(1 if sync else 5):
            for f in (lambda: M.mla_absorb_query(dims, q, w, ql),
                      lambda: M.mla_latent_attn(dims, True, qsl, lens, ql, cache, table, ws, ol),
                      lambda: M.mla_expand_output(dims, ol, w, out),
                      lambda: M.mla_absorb_query(dims, q_small, w, small)):
                f()
                if sync:
                    torch.cuda.synchronize()
        torch.cuda.synchronize()
        return ql, ol, out, small

    alone = step(True)
    for _ in range(4):
        for x, y in zip(step(False), alone):
            assert torch.equal(x, y)
