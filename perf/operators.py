"""Cases of the single-token (decode) side of MLA and of the step that fills the
paged latent cache: what the operators compute, on which sizes, and what they
cannot do without.

Operators
  append   RMS norm of the latent part of new tokens' rows, rotation of their
           rope part, both written to the token's slot of the paged cache (and
           as dense rows where asked); rotation of the queries' rope part
  absorb   q_latent[t, h] = [q_nope[t, h] . W_uk[h] | q_pe[t, h]]
  attn     softmax attention of absorbed queries over the paged latent cache,
           keys = whole rows, values = the rows' latent part; (o_latent, LSE)
  expand   out[t, h] = W_uv[h] . o_latent[t, h]

W_kv_b is [H*(Dn+Dv), L]: rows h*(Dn+Dv) + [0, Dn) are W_uk[h], the next Dv
rows W_uv[h].  The last query_lens[r] of a request's seq_lens[r] tokens are its
new ones.
"""

import math
import random

import numpy as np
import torch

own = False

# the DeepSeek-V3 layer shape of the prefill workloads, and the small float32 one
LARGE = dict(L=512, P=64, Dn=128, Dv=128, dtype="bf16")
SMALL = dict(L=64, P=16, Dn=32, Dv=32, dtype="f32")


def listed():
    attn = dict(LARGE, op="attn", bs=64, H=128, nq=1, causal=True)
    app = dict(LARGE, op="append", bs=64, H=128, norm=True, dense=True, queries=True)
    return [
        # one short conversation, one token: launch latency
        dict(attn, name="attn 1x70", R=1, lens="fixed", top=70),
        # the uniform prefill batch, decoding: 16 requests of 4096 tokens
        dict(attn, name="attn 16x4096", R=16, lens="fixed", top=4096),
        # the hetero prefill batch, decoding: one context of 131072 among short and empty ones
        dict(attn, name="attn hetero 32", R=32, lens="hetero", top=131072),
        # a quarter of the heads (tensor parallel shard), many ragged requests
        dict(attn, name="attn 128 ragged, 32 heads", R=128, H=32, lens="uniform", top=8192),
        # four drafted tokens a request, verified causally; pages of 16
        dict(attn, name="attn 24 ragged, 4 tokens", R=24, nq=4, bs=16, lens="uniform", top=8192),
        # float32 storage and small heads
        dict(SMALL, name="attn small f32", op="attn", bs=16, H=16, nq=3, causal=True, R=4, lens="uniform", top=700),
        # one decode step of 16 requests
        dict(app, name="append 16x1", R=16, nq=1, lens="uniform", top=8192, interleaved=True),
        # the uniform prefill batch's new tokens: 16 x 512 rows behind 4096 cached ones
        dict(app, name="append 16x512", R=16, nq=512, lens="fixed", top=4608, interleaved=False),
        dict(LARGE, name="absorb 1", op="absorb", T=1, H=128),
        dict(LARGE, name="absorb 500", op="absorb", T=500, H=128),
        dict(LARGE, name="expand 16", op="expand", T=16, H=128),
        dict(LARGE, name="expand 500", op="expand", T=500, H=128),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["attn"] * 5 + ["append"] * 2 + ["absorb", "expand"])
    small = rng.random() < 0.15
    shape = dict(SMALL if small else LARGE)
    H = rng.choice([1, 4, 16, 40] if small else [8, 20, 32, 64, 96, 128])
    seed = rng.randrange(1 << 30)
    if kind in ("absorb", "expand"):
        return dict(shape, op=kind, H=H, T=_log_int(rng, 1, 500))
    if kind == "append":
        nq = rng.choice([1, 1, 2, _log_int(rng, 3, 500)])
        R = _log_int(rng, 1, max(1, min(256, 8000 // nq)))
        return dict(shape, op="append", H=H, R=R, nq=nq, bs=rng.choice([16, 32, 64, 128]), lens="uniform",
                    top=max(nq, _log_int(rng, 1, min(16384, (1 << 19) // R))), lens_seed=seed, norm=rng.random() < 0.8,
                    dense=rng.random() < 0.5, queries=rng.random() < 0.7, interleaved=rng.random() < 0.5)
    nq = rng.choice([1, 1, 1, 2, 3, 4, 7])
    if small:
        R, top = _log_int(rng, 1, 8), _log_int(rng, 1, 700)
    else:
        R = _log_int(rng, 1, 256)
        top = _log_int(rng, 1, min(131072, (1 << 19) // R, max(1, 36_000_000 // (R * H * nq))))
    return dict(shape, op="attn", H=H, R=R, nq=nq, bs=rng.choice([16, 32, 64, 128]), causal=rng.random() < 0.8,
                lens=rng.choice(["uniform", "uniform", "log", "fixed"]), top=max(top, nq), lens_seed=seed)


def _lens(c):
    """Tokens of each request, new ones included: a matter of the case, not of its seed."""
    r = random.Random(c.get("lens_seed", 7))
    R, top, nq = c["R"], c["top"], c["nq"]
    if c["lens"] == "fixed":
        return [top] * R
    if c["lens"] == "hetero":
        v = [top] + [int(round(math.exp(r.uniform(0, math.log(2048))))) for _ in range(R - 8)] + [0] * 7
        r.shuffle(v)
        return v
    if c["lens"] == "log":
        return [max(nq, int(round(math.exp(r.uniform(0, math.log(max(2, top))))))) for _ in range(R)]
    return [r.randint(min(nq, top), top) for _ in range(R)]


def _type(c):
    return torch.bfloat16 if c["dtype"] == "bf16" else torch.float32


def _rope_table(n, P, dev):
    """[n, P] float32, cos then sin of position * 10000^(-2i/P); the angles in 64 bits."""
    inv = 10000.0 ** (-torch.arange(0, P, 2, dtype=torch.float64, device=dev) / P)
    a = torch.arange(n, dtype=torch.float64, device=dev)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float()


def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(device=dev).manual_seed(int(seed))
    dt = _type(c)
    L, P, Dn, Dv, H = c["L"], c["P"], c["Dn"], c["Dv"], c["H"]

    def normal(*shape, std=1.0, dtype=dt):
        return (torch.randn(shape, generator=g, device=dev, dtype=torch.float32) * std).to(dtype)

    s = {"case": dict(c)}
    if c["op"] in ("absorb", "expand"):
        s["w"] = normal(H * (Dn + Dv), L, std=0.02 if L > 64 else 0.1)
        s["x"] = normal(c["T"], H, Dn + P) if c["op"] == "absorb" else normal(c["T"], H, L, std=0.2)
        s["out"] = torch.empty(c["T"], H, L + P if c["op"] == "absorb" else Dv, device=dev, dtype=dt)
        return s
    lens, R, nq, bs = _lens(c), c["R"], c["nq"], c["bs"]
    T = R * nq
    need = [-(-n // bs) for n in lens]
    blocks = sum(need) + 2
    order = torch.randperm(blocks, generator=g, device=dev).cpu().numpy().astype(np.int32)
    table = np.zeros((R, max(1, max(need))), np.int32)  # unused entries: block 0, as an engine leaves them
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = order[at:at + n]
        at += n
    s.update(block_table=torch.from_numpy(table).to(dev), seq_lens=torch.tensor(lens, dtype=torch.int32, device=dev),
             qsl=torch.arange(0, T + 1, nq, dtype=torch.int32, device=dev),
             kv_cache=torch.empty(blocks, bs, L + P, device=dev, dtype=dt).normal_(generator=g), longest=max(lens))
    if c["op"] == "attn":
        # absorbed queries: W_uk draws of 0.02 make the latent part 0.23 wide, the rope part is 1 wide
        s["q"] = torch.cat([normal(T, H, L, std=0.23 if L > 64 else 1.0), normal(T, H, P)], 2)
        s["o"] = torch.empty(T, H, L, device=dev, dtype=dt)
        s["lse"] = torch.empty(H, T, device=dev)
        return s
    wide = normal(T, L + P + 64)  # the rows come as columns of a wider projection
    s["kv_a"] = wide[:, 64:]
    s["norm_weight"] = (1 + 0.1 * normal(L, dtype=torch.float32)).to(dt) if c["norm"] else None
    s["rope"] = _rope_table(max(lens) + 1, P, dev)
    s["new_latent"] = torch.empty(T, L + P, device=dev, dtype=dt) if c["dense"] else None
    s["q"] = normal(T, H, Dn + P) if c["queries"] else None
    s["q_pe"] = torch.empty(T, H, P, device=dev, dtype=dt) if c["queries"] else None
    return s


def _scale(c):
    return 1.0 / math.sqrt(c["Dn"] + c["P"])


def _rotate(x, cos, sin, interleaved):
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    a, b = x.chunk(2, -1)
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _plain(s):
    c = s["case"]
    dt, L, P, Dn, Dv, H = _type(c), c["L"], c["P"], c["Dn"], c["Dv"], c["H"]
    if c["op"] == "absorb":
        w = s["w"].float().view(H, Dn + Dv, L)[:, :Dn]
        q = s["x"].float()
        lat = torch.bmm(q[..., :Dn].transpose(0, 1), w).transpose(0, 1)
        return torch.cat([lat, q[..., Dn:]], 2).to(dt)
    if c["op"] == "expand":
        w = s["w"].float().view(H, Dn + Dv, L)[:, Dn:]
        return torch.bmm(s["x"].float().transpose(0, 1), w.transpose(1, 2)).transpose(0, 1).to(dt)
    nq, bs, R = c["nq"], c["bs"], c["R"]
    lens = s["seq_lens"].long()
    if c["op"] == "append":
        x = s["kv_a"].float()
        pos = (lens[:, None] - nq + torch.arange(nq, device=x.device)).flatten()
        lat, pe = x[:, :L], x[:, L:]
        if c["norm"]:
            lat = lat * torch.rsqrt(lat.square().mean(1, keepdim=True) + 1e-6) * s["norm_weight"].float()
        cos, sin = s["rope"][pos].chunk(2, 1)
        row = torch.cat([lat, _rotate(pe, cos, sin, c["interleaved"])], 1).to(dt)
        block = s["block_table"].gather(1, (pos // bs).view(R, nq)).flatten().long()
        s["kv_cache"].view(-1, L + P)[block * bs + pos % bs] = row
        out = {"kv_cache": s["kv_cache"]}
        if c["dense"]:
            out["new_latent"] = row
        if c["queries"]:
            out["q_pe"] = _rotate(s["q"][..., Dn:].float(), cos[:, None], sin[:, None], c["interleaved"]).to(dt)
        return out
    n = max(1, s["longest"])
    col = torch.arange(n, device=lens.device)
    page = s["block_table"][:, col // bs].long()
    k = s["kv_cache"][page, col % bs].float()                                   # [R, n, L+P]
    q = s["q"].float().view(R, nq, H, L + P)
    score = torch.bmm(q.reshape(R, nq * H, L + P), k.transpose(1, 2)).view(R, nq, H, n) * _scale(c)
    last = lens[:, None] - nq + torch.arange(nq, device=lens.device) if c["causal"] else (lens[:, None] - 1).expand(R, nq)
    seen = col <= last[:, :, None]                                              # [R, nq, n]
    score = score.masked_fill(~seen[:, :, None], -math.inf)
    top = score.amax(3, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(score - top)
    total = p.sum(3, keepdim=True)
    o = torch.bmm(p.view(R, nq * H, n), k[..., :L]).view(R, nq, H, L) / torch.where(total == 0, torch.ones_like(total), total)
    lse = (top + torch.log(total)).view(R * nq, H).t()
    return {"o": o.reshape(R * nq, H, L).to(dt), "lse": lse.contiguous()}


def run(state):
    if not own:
        return _plain(state)
    import mla_chunked_context_gb300 as M
    s, c = state, state["case"]
    if "dims" not in s:
        s["dims"] = M.Dims(c["H"], c["L"], c["P"], c["Dn"], c["Dv"], c.get("bs", 64), _scale(c), _type(c))
    d = s["dims"]
    if c["op"] == "absorb":
        M.mla_absorb_query(d, s["x"], s["w"], s["out"])
        return s["out"]
    if c["op"] == "expand":
        M.mla_expand_output(d, s["x"], s["w"], s["out"])
        return s["out"]
    if c["op"] == "append":
        M.mla_append_latent(d, s["kv_a"], s["qsl"], s["seq_lens"], s["rope"], s["kv_cache"], s["block_table"],
                            norm_weight=s["norm_weight"], norm_eps=1e-6, interleaved=c["interleaved"],
                            new_latent=s["new_latent"], q=s["q"], q_pe_out=s["q_pe"])
        return {k: s[k] for k in ("kv_cache", "new_latent", "q_pe") if s[k] is not None}
    if "workspace" not in s:
        s["workspace"] = torch.empty(M.mla_latent_attn_workspace_bytes(d, s["q"].shape[0], c["R"]), dtype=torch.uint8,
                                     device=s["q"].device)
    M.mla_latent_attn(d, c["causal"], s["qsl"], s["seq_lens"], s["q"], s["kv_cache"], s["block_table"], s["workspace"],
                      s["o"], s["lse"])
    return {"o": s["o"], "lse": s["lse"]}


def work(case):
    c = case
    es = 2 if c["dtype"] == "bf16" else 4
    L, P, Dn, Dv, H = c["L"], c["P"], c["Dn"], c["Dv"], c["H"]
    if c["op"] == "absorb":
        return {"bytes": es * (c["T"] * H * (Dn + P + L + P) + H * Dn * L), "flops": 2.0 * c["T"] * H * Dn * L}
    if c["op"] == "expand":
        return {"bytes": es * (c["T"] * H * (L + Dv) + H * Dv * L), "flops": 2.0 * c["T"] * H * Dv * L}
    lens, T = _lens(c), c["R"] * c["nq"]
    if c["op"] == "append":
        rows = 2 + (1 if c["dense"] else 0)
        b = es * T * (rows * (L + P) + (2 * H * P if c["queries"] else 0)) + 4 * T * P + (es * L if c["norm"] else 0)
        return {"bytes": b, "flops": T * (4.0 * L + 3.0 * P * (1 + (H if c["queries"] else 0)))}
    pairs = sum(max(0, n - c["nq"] + 1 + i) if c["causal"] else n for n in lens for i in range(c["nq"]))
    b = es * (sum(lens) * (L + P) + T * H * (2 * L + P)) + 4 * T * H
    return {"bytes": b, "flops": 2.0 * pairs * H * (2 * L + P)}


def exact(case, seed):
    """The definitions in 64 bits: one request (or head) at a time, on gathered rows."""
    s, c = prepare(case, seed), case
    L, P, Dn, Dv, H = c["L"], c["P"], c["Dn"], c["Dv"], c["H"]
    f = torch.float64
    if c["op"] in ("absorb", "expand"):
        parts = []
        for h in range(H):
            w = s["w"][h * (Dn + Dv):(h + 1) * (Dn + Dv)].to(f)
            x = s["x"][:, h].to(f)
            parts.append(torch.cat([x[:, :Dn] @ w[:Dn], x[:, Dn:]], 1) if c["op"] == "absorb" else x @ w[Dn:].T)
        return torch.stack(parts, 1)
    lens, nq, bs = _lens(c), c["nq"], c["bs"]
    table = s["block_table"].cpu().numpy()
    if c["op"] == "append":
        inv = 10000.0 ** (-2.0 * np.arange(P // 2) / P)
        cache, rows, rotated = s["kv_cache"].to(f), [], []

        def turn(z, ang):
            """Rotation by complex numbers; z [n, ..., P] numpy float64."""
            pair = z.reshape(*z.shape[:-1], P // 2, 2) if c["interleaved"] else np.stack([z[..., :P // 2], z[..., P // 2:]], -1)
            # the table holds cos and sin as float32 inputs
            e = np.cos(ang).astype(np.float32).astype(np.float64) + 1j * np.sin(ang).astype(np.float32).astype(np.float64)
            v = (pair[..., 0] + 1j * pair[..., 1]) * e
            return np.stack([v.real, v.imag], -1).reshape(z.shape) if c["interleaved"] else np.concatenate([v.real, v.imag], -1)

        x = s["kv_a"].to(f).cpu().numpy()
        w = s["norm_weight"].to(f).cpu().numpy() if c["norm"] else None
        q = s["q"][..., Dn:].to(f).cpu().numpy() if c["queries"] else None
        slots = []
        for r, n in enumerate(lens):
            pos = np.arange(n - nq, n)
            ang = pos[:, None] * inv
            a = x[r * nq:(r + 1) * nq]
            lat = a[:, :L]
            if w is not None:
                lat = lat / np.sqrt((lat ** 2).mean(1, keepdims=True) + 1e-6) * w
            rows.append(np.concatenate([lat, turn(a[:, L:], ang)], 1))
            slots.append(table[r, pos // bs].astype(np.int64) * bs + pos % bs)
            if q is not None:
                rotated.append(turn(q[r * nq:(r + 1) * nq], ang[:, None]))
        rows = torch.from_numpy(np.concatenate(rows)).to(cache.device)
        cache.view(-1, L + P)[torch.from_numpy(np.concatenate(slots)).to(cache.device)] = rows
        out = {"kv_cache": cache}
        if c["dense"]:
            out["new_latent"] = rows
        if q is not None:
            out["q_pe"] = torch.from_numpy(np.concatenate(rotated))
        return out
    T = c["R"] * nq
    o = torch.zeros(T, H, L, dtype=f, device=s["q"].device)
    lse = torch.full((H, T), -math.inf, dtype=f, device=s["q"].device)
    for r, n in enumerate(lens):
        pages = torch.from_numpy(table[r, :-(-n // bs)].astype(np.int64)).to(s["q"].device)
        k = s["kv_cache"][pages].reshape(-1, L + P)[:n].to(f)
        for i in range(nq):
            m = n - nq + 1 + i if c["causal"] else n
            if m < 1:
                continue
            t = r * nq + i
            z = (s["q"][t].to(f) @ k[:m].T) * _scale(c)
            lse[:, t] = torch.logsumexp(z, 1)
            o[t] = torch.softmax(z, 1) @ k[:m, :L]
    return {"o": o, "lse": lse}
