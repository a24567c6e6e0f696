"""Calls at the edges of what the decode calls' documentation allows: tokens
that are not appended, invalid blocks and far offsets in both forms of the
attention.  Tolerances as in test_gpu_decode.py, whose helpers these are."""

import math

import numpy as np
import pytest
import torch

import mla_chunked_context_gb300 as M
from oracle import mla as O

from test_gpu_decode import (DEV, F, LARGE, SMALL, _cuda, _no_device_errors, check_attn,  # noqa: F401
                             f64, i32, loc, make_cache, make_dims, normal, run_attn, within)

pytestmark = [pytest.mark.gpu,
              pytest.mark.filterwarnings("ignore::RuntimeWarning")]


# --------------------------------------------- tokens that are not appended --
@pytest.mark.parametrize("shape,dtype,H", [(LARGE, "bf16", 128), (LARGE, "bf16", 16), (SMALL, "f32", 3)])
def test_step_with_tokens_that_are_not_appended(shape, dtype, H):
    """Tokens with rope positions outside the table, and more new tokens than
    tokens: nothing of an earlier step, or of what the instance's buffers held
    at first, reaches the results; these tokens' queries count as they are
    given, unrotated."""
    rng = np.random.default_rng(H)
    dims, od = make_dims(shape, H, 16, dtype)
    L, P, Dn, Dv = shape
    lens, ql = [70, 2, 33], [2, 4, 1]         # of the second's four two are before its start
    qsl = loc(ql)
    T = qsl[-1]
    pos = [68, 99, 0, 0, 0, 1, -1]            # the table has 80: two outside
    lost = [1, 2, 3, 6]
    cache, table = make_cache(rng, lens, 16, L + P, dims.dtype)
    tab = torch.from_numpy(O.rope_table(80, P).astype(np.float32)).to(DEV)
    w = normal(rng, H * (Dn + Dv), L, std=0.1, dtype=dims.dtype).to(DEV)
    q = normal(rng, T, H, Dn + P, dtype=dims.dtype).to(DEV)
    kv_a = normal(rng, T, L + P, dtype=dims.dtype).to(DEV)
    results = []
    for held in (math.nan, 3.0, None):
        dec = M.LatentDecode(dims, T, 3, device=DEV)
        c, status = cache.to(DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
        out, lse = torch.empty(T, H, Dv, dtype=dims.dtype, device=DEV), torch.empty(H, T, device=DEV)
        if held is None:                      # an earlier step of other tokens
            c2 = cache.to(DEV)
            dec(q.flip(0), kv_a, i32(qsl), i32([70, 40, 33]), tab, c2, table.to(DEV), w, out, lse)
        else:
            dec.q_latent.fill_(held)
            dec.o_latent.fill_(held)
        dec(q, kv_a, i32(qsl), i32(lens), tab, c, table.to(DEV), w, out, lse, positions=i32(pos),
            causal=False, dev_status=status)
        torch.cuda.synchronize()
        assert status.item() == M.MLA_STATUS_BAD_POSITION
        for t in lost:
            assert torch.equal(dec.q_latent[t, :, L:], q[t, :, Dn:])
        for t, r, p in O.token_positions(qsl, lens):
            if t in lost and p >= 0:          # not appended: the slot is as it was
                assert torch.equal(c[table[r, p // 16], p % 16].cpu(), cache[table[r, p // 16], p % 16])
        results.append((out, lse, c, dec.q_latent.clone()))
    out, lse, c, q_lat = results[0]
    assert torch.isfinite(out.float()).all() and torch.isfinite(lse).all()
    for other in results[1:]:
        assert torch.equal(out, other[0]) and torch.equal(lse, other[1])
    _, rl, _, size = O.latent_attention(f64(q_lat), f64(c), table.numpy(), qsl, lens, od, False)
    within(f64(lse), rl, (L + P + 8) * F * size + 2.0 ** -22 + (70 / 8 + 16) * F + F * np.abs(rl), "lse")


# ------------------------------------------ invalid blocks, in both forms --
@pytest.mark.parametrize("bs", [1, 8, 16, 32, 64])
@pytest.mark.parametrize("H", [128, 40, 8])
def test_bad_blocks_beside_rows_that_are_not_finite(H, bs):
    """Bad block ids in the middle of sequences, in a tile of which the new
    tokens see different parts, and among those parts; in the same tiles rows
    that are not finite and that only some tokens see.  (128 and 40 heads of
    these tokens are more than 64 rows a sequence, the form of two blocks.)"""
    rng = np.random.default_rng(H + bs)
    dims, od = make_dims(LARGE, H, bs, "bf16")
    lens, ql = [300, 130, 700, 90], [4, 4, 1, 2]
    qsl = loc(ql)
    cache, table = make_cache(rng, lens, bs, 576, dims.dtype)
    q = normal(rng, qsl[-1], H, 576, std=0.4, dtype=dims.dtype)
    bad = table.clone()
    bad[0, (272 if bs <= 16 else 192) // bs] = cache.shape[0]      # beside the first's new tokens
    bad[1, 128 // bs] = -1                                         # two of the second's are in it
    for j in (130, 131, 400):
        bad[2, j // bs] = 2 ** 31 - 1
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    o, lse = run_attn(dims, True, qsl, lens, q, cache, bad, status=status)
    assert status.item() == M.MLA_STATUS_BAD_BLOCK
    zero = torch.cat([cache, torch.zeros_like(cache[:1])])
    ztab = bad.clone()
    ztab[(ztab < 0) | (ztab > len(cache))] = len(cache)
    check_attn(dims, od, True, qsl, lens, q, zero, ztab, o, lse)
    wild = cache.clone()
    for r, j in ((0, 298), (1, 127), (3, 89)):                     # the third or the last new token's
        wild[table[r, j // bs], j % bs] = math.nan
    o2, lse2 = run_attn(dims, True, qsl, lens, q, wild, bad, status=status)
    for t in range(qsl[-1]):
        if t in (0, 1, 4, 8, 9):                                   # those that do not see them
            assert torch.equal(o2[t], o[t]) and torch.equal(lse2[:, t], lse[:, t]), t
        else:
            assert torch.isnan(o2[t]).all() and torch.isnan(lse2[:, t]).all(), t


@pytest.mark.parametrize("H,T", [(128, 1), (128, 3), (40, 2)])
def test_no_blocks_in_the_form_of_two_blocks(H, T):
    """A cache of no blocks: scores 0, output 0, the log-sum ln n."""
    import ctypes as C
    dims, _ = make_dims(LARGE, H, 16, "bf16")
    d = dims.c()
    cache = torch.ones(2, 16, 576, dtype=dims.dtype, device=DEV)
    q = torch.ones(T, H, 576, dtype=dims.dtype, device=DEV)
    o = torch.full((T, H, 512), 7.0, dtype=dims.dtype, device=DEV)
    lse, table = torch.zeros(H, T, device=DEV), torch.zeros(1, 8, dtype=torch.int32, device=DEV)
    ws = torch.empty(M.mla_latent_attn_workspace_bytes(dims, T, 1), dtype=torch.uint8, device=DEV)
    status, qsl, lens = i32([0]), i32([0, T]), i32([100])
    rc = M.lib().mla_latent_attn(
        C.byref(d), 0, 1, qsl.data_ptr(), lens.data_ptr(), T, q.data_ptr(), cache.data_ptr(), 0,
        table.data_ptr(), 8, ws.data_ptr(), ws.numel(), o.data_ptr(), lse.data_ptr(),
        status.data_ptr(), None)
    torch.cuda.synchronize()
    assert rc == 0 and status.item() == M.MLA_STATUS_BAD_BLOCK and (o == 0).all()
    # as in test_gpu_decode.py: the sum is exact, log2f and ln 2 are rounded
    within(f64(lse), np.full((H, T), math.log(100)), 2.0 ** -21 * 0.7 + 6.7 * 2.0 ** -25 + 2.0 ** -22,
           "lse")


@pytest.mark.parametrize("bs", [64, 8])
def test_far_offsets_in_the_form_of_two_blocks(bs):
    """Cache rows beyond 2^31 elements and 2^32 bytes, of two new tokens, the
    second's not finite."""
    dims, od = make_dims(LARGE, 128, bs, "bf16")
    blocks = 64000 * 64 // bs
    cache = torch.zeros(blocks, bs, 576, dtype=torch.bfloat16, device=DEV)
    rng = np.random.default_rng(bs)
    lens, qsl = [200], [0, 2]
    small, table = make_cache(rng, lens, bs, 576, dims.dtype, spare=0)
    far = blocks - 1 - torch.arange(len(small))
    cache[far.to(DEV)] = small.to(DEV)
    q = normal(rng, 2, 128, 576, std=0.4, dtype=dims.dtype)
    need = -(-200 // bs)
    ftab = table.clone()
    ftab[0, :need] = far[table[0, :need].long()].int()
    o, lse = run_attn(dims, True, qsl, lens, q, cache, ftab)
    cache[int(ftab[0, 199 // bs]), 199 % bs] = math.inf
    o2, lse2 = run_attn(dims, True, qsl, lens, q, cache, ftab)
    del cache
    check_attn(dims, od, True, qsl, lens, q, small, table, o, lse)
    assert torch.equal(o2[0], o[0]) and torch.equal(lse2[:, 0], lse[:, 0])
    score = f64(q[1]) @ np.full(576, np.inf)                       # inf - inf: NaN
    assert np.isnan(score).all() and torch.isnan(o2[1]).all()


# ------------------------------------------------------------ long calls --
def test_seconds_of_work_are_no_timeout():
    """A call of some three seconds (4096 tokens over 3.2 million keys, a few
    pages again and again) is right, and no wait of it counts as given up: what
    a barrier's wait is limited by is one step of the pipeline, not the call."""
    rng = np.random.default_rng(31)
    H, T, blocks, times = 128, 4096, 5, 10000
    dims, od = make_dims(LARGE, H, 64, "bf16")
    n = 64 * blocks * times
    cache = normal(rng, blocks, 64, 576, dtype=dims.dtype)
    table = torch.arange(blocks, dtype=torch.int32).repeat(times)[None]
    q = (0.4 * torch.randn(T, H, 576, device=DEV)).to(dims.dtype)
    o, lse = run_attn(dims, False, [0, T], [n], q, cache, table)
    assert M.mla_device_error_flags() == 0
    for t in (0, 1777, T - 1):
        ro, rl, mass, size = O.latent_attention(f64(q[t:t + 1]), f64(cache), np.arange(blocks)[None],
                                                [0, 1], [64 * blocks], od, False)
        E = (512 + 64 + 8) * F * size + 2.0 ** -22
        rl = rl + math.log(times)
        within(f64(lse[:, t:t + 1]), rl, E + (n / 8 + 16) * F + F * np.abs(rl), "lse")
        u = torch.finfo(dims.dtype).eps / 2
        within(f64(o[t:t + 1]), ro, u * np.abs(ro) + (2 * E.T[:, :, None] + (n / 8 + 64) * F + u) * mass, "o")


# ------------------------------------------------- batches, streams, graphs --
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("bs", [64, 16])
def test_more_slots_than_tokens(bs, causal):
    """Many sequence slots of which few have new tokens: the form of one block
    with several units a sequence, whose rows see different keys; lengths below
    zero count as none."""
    rng = np.random.default_rng(bs)
    H, R = 128, 60
    dims, od = make_dims(LARGE, H, bs, "bf16")
    ql, lens = [0] * R, [5] * R
    for r, (n, k) in {3: (3, 300), 17: (1, 1000), 40: (5, 129), 41: (2, 0), 59: (4, 66)}.items():
        ql[r], lens[r] = n, k
    qsl = loc(ql)
    cache, table = make_cache(rng, lens, bs, 576, dims.dtype)
    q = normal(rng, qsl[-1] + 2, H, 576, std=0.4, dtype=dims.dtype)
    assert (qsl[-1] + 2) * H <= 64 * R
    device_lens = [-7 if r == 41 else n for r, n in enumerate(lens)]
    o, lse = run_attn(dims, causal, qsl, device_lens, q, cache, table)
    check_attn(dims, od, causal, qsl, lens, q, cache, table, o, lse)
    wild = cache.clone()                      # seen by two of the third's three, one of the last's four
    for r, j in ((3, 298), (59, 65)):
        wild[table[r, j // bs], j % bs] = math.inf
    o2, lse2 = run_attn(dims, causal, qsl, device_lens, q, wild, table)
    for t in range(qsl[-1]):
        sees = t in ((1, 2, qsl[-1] - 1) if causal else (0, 1, 2, *range(qsl[-1] - 4, qsl[-1])))
        if not sees:
            assert torch.equal(o2[t], o[t]) and torch.equal(lse2[:, t], lse[:, t]), t
        else:
            assert torch.isnan(o2[t]).all(), t


def step_inputs(rng, shape, dtype, H, lens, bs=16):
    dims, od = make_dims(shape, H, bs, dtype)
    L, P, Dn, Dv = shape
    R = len(lens)
    cache, table = make_cache(rng, [n + 4 for n in lens], bs, L + P, dims.dtype)
    return dims, od, dict(
        q=normal(rng, R, H, Dn + P, dtype=dims.dtype).to(DEV), kv_a=normal(rng, R, L + P, dtype=dims.dtype).to(DEV),
        qsl=i32(range(R + 1)), lens=i32(lens), cache=cache.to(DEV), table=table.to(DEV),
        tab=torch.from_numpy(O.rope_table(max(lens) + 8, P).astype(np.float32)).to(DEV),
        w=normal(rng, H * (Dn + Dv), L, std=0.1, dtype=dims.dtype).to(DEV),
        out=torch.empty(R, H, Dv, dtype=dims.dtype, device=DEV), lse=torch.empty(H, R, device=DEV))


def run_step(dec, x, **kw):
    return dec(x["q"], x["kv_a"], x["qsl"], x["lens"], x["tab"], x["cache"], x["table"], x["w"], x["out"],
               x["lse"], **kw)


@pytest.mark.parametrize("shape,dtype", [(LARGE, "bf16"), (SMALL, "f32")])
def test_captured_between_other_work(shape, dtype):
    """Steps captured between memory sets, copies, other kernels and work of a
    second stream that forks and joins give what eager calls give."""
    rng = np.random.default_rng(50)
    H = 32
    dims, od, x = step_inputs(rng, shape, dtype, H, [100, 40, 700])
    start = x["cache"].clone()
    dec = M.LatentDecode(dims, 3, 3, device=DEV)
    run_step(dec, x)
    torch.cuda.synchronize()
    want = [t.clone() for t in (x["out"], x["lse"], x["cache"])]
    src = {k: x[k].clone() for k in ("q", "kv_a", "cache", "w")}
    src["cache"].copy_(start)
    other, side = torch.zeros_like(x["out"]), torch.cuda.Stream()
    host = torch.zeros_like(x["lens"]).cpu().pin_memory()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        main = torch.cuda.current_stream()
        x["lse"].zero_()                              # a memory set before the first call
        x["cache"].copy_(src["cache"])
        x["q"].copy_(src["q"])                        # a copy
        side.wait_stream(main)
        with torch.cuda.stream(side):
            x["w"].copy_(src["w"])                    # on the second stream, joined before the first call
            x["kv_a"].copy_(src["kv_a"] * 1)
        main.wait_stream(side)
        run_step(dec, x)
        side.wait_stream(main)
        with torch.cuda.stream(side):                 # the expansion once more, behind the join
            M.mla_expand_output(dims, dec.o_latent[:3], x["w"], other)
        host.copy_(x["lens"], non_blocking=True)
        main.wait_stream(side)
    for _ in range(3):
        for t in (x["out"], x["lse"], x["q"], x["kv_a"], x["w"], other):
            t.fill_(5.0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(x["out"], want[0]) and torch.equal(x["lse"], want[1]) and torch.equal(other, want[0])
        assert torch.equal(torch.nan_to_num(x["cache"].float(), 5.0), torch.nan_to_num(want[2].float(), 5.0))


def test_two_threads_a_stream_and_an_instance_each():
    import threading
    rng = np.random.default_rng(51)
    sets = []
    for lens in ([900, 30], [64, 2000, 5]):
        dims, od, x = step_inputs(rng, LARGE, "bf16", 128, lens, bs=64)
        dec = M.LatentDecode(dims, len(lens), len(lens), device=DEV)
        run_step(dec, x)
        torch.cuda.synchronize()
        sets.append((dec, x, x["out"].clone(), x["lse"].clone(), torch.cuda.Stream()))
    failed = []

    def work(dec, x, out, lse, stream):
        try:
            torch.cuda.set_device(0)
            for _ in range(40):
                with torch.cuda.stream(stream):
                    x["out"].fill_(0)
                    run_step(dec, x)
                    stream.synchronize()
                    if not (torch.equal(x["out"], out) and torch.equal(x["lse"], lse)):
                        failed.append("result")
        except Exception as e:  # noqa: BLE001
            failed.append(repr(e))

    threads = [threading.Thread(target=work, args=s) for s in sets]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed


@pytest.mark.parametrize("shape,dtype,H", [(LARGE, "bf16", 16), (SMALL, "f32", 4)])
def test_append_prepares_a_prefill(shape, dtype, H):
    """The append's dense rows and rotated queries are a prefill's inputs; its
    cache rows then serve a decode step.  Tolerance: the framework's for
    attention output (O: 2e-2 + 2e-2 |ref|, LSE 1e-3), in bf16 with the step's
    rounding of the absorbed query as in test_gpu_decode.py."""
    rng = np.random.default_rng(H)
    bs, ctx, new = 16, [200, 0, 37], [70, 33, 1]
    dims, od = make_dims(shape, H, bs, dtype)
    L, P, Dn, Dv = shape
    R, T = len(ctx), sum(new)
    total = [c + n for c, n in zip(ctx, new)]
    cache, table = make_cache(rng, [n + 1 for n in total], bs, L + P, dims.dtype)
    g_cache, g_table = cache.to(DEV), table.to(DEV)
    tab = torch.from_numpy(O.rope_table(400, P).astype(np.float32)).to(DEV)
    gw = (1 + 0.1 * normal(rng, L)).to(dims.dtype).to(DEV)
    w = normal(rng, H * (Dn + Dv), L, std=0.5 / math.sqrt(L), dtype=dims.dtype).to(DEV)
    q, kv_a = normal(rng, T, H, Dn + P, dtype=dims.dtype), normal(rng, T, L + P, dtype=dims.dtype)
    g_q, lat = q.to(DEV), torch.empty(T, L + P, dtype=dims.dtype, device=DEV)
    M.mla_append_latent(dims, kv_a.to(DEV), i32(loc(new)), i32(total), tab, g_cache, g_table,
                        norm_weight=gw, new_latent=lat, q=g_q, q_pe_out=g_q[..., Dn:])
    out, lse = torch.empty(T, H, Dv, dtype=dims.dtype, device=DEV), torch.empty(H, T, device=DEV)
    pf = M.ChunkedPrefill(dims, ctx, new, 128, 128, 16, device=DEV)
    pf(g_q, lat, g_cache, g_table, w, out, lse)
    # the same tokens as one decode step of many new tokens, on a cache of its own
    c2 = cache.to(DEV)
    out2, lse2 = torch.empty_like(out), torch.empty_like(lse)
    M.LatentDecode(dims, T, R, device=DEV)(q.to(DEV), kv_a.to(DEV), i32(loc(new)), i32(total), tab, c2,
                                           g_table, w, out2, lse2, norm_weight=gw)
    torch.cuda.synchronize()
    assert torch.equal(torch.nan_to_num(g_cache.float(), 5.0), torch.nan_to_num(c2.float(), 5.0))
    c, wn = f64(g_cache), f64(w)
    for r in range(R):
        sl = slice(loc(new)[r], loc(new)[r + 1])
        rows = np.stack([O.context_row(c, table.numpy(), r, j, bs) for j in range(total[r])])
        kn, v = O.up_project(rows, wn, od)
        qr = f64(q[sl])
        for i in range(new[r]):
            qr[i, :, Dn:] = O.rotate(qr[i, :, Dn:], f64(tab)[ctx[r] + i], False)
        vis = np.arange(total[r])[None, :] <= (ctx[r] + np.arange(new[r]))[:, None]
        ro, rl = O.attention_with_lse(qr, kn, rows[:, L:], v, od.softmax_scale, vis)
        slack, turned = 0.0, 0.0
        if dtype == "bf16":
            u = torch.finfo(dims.dtype).eps / 2
            ql = np.abs(O.absorb_query(qr, wn, od))
            slack = u * od.softmax_scale * np.einsum("thl,nl->thn", ql, np.abs(rows), optimize=True).max()
            # the prefill's rotated query is rounded to bf16 before its scores
            turned = u * od.softmax_scale * np.einsum("thp,np->thn", np.abs(qr[..., Dn:]),
                                                      np.abs(rows[:, L:]), optimize=True).max()
        within(f64(lse)[:, sl], rl, 1e-3 + turned, "prefill lse")
        within(f64(lse2)[:, sl], rl, 1e-3 + slack, "step lse")
        within(f64(out)[sl], ro, 2e-2 + 2e-2 * np.abs(ro), "prefill out")
        within(f64(out2)[sl], ro, 2e-2 + 2e-2 * np.abs(ro), "step out")
