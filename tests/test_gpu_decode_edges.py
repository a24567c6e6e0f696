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
