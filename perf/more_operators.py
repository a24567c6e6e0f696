"""Cases of speculative decoding with trees of drafted tokens on the paged latent
cache: what the operators compute, on which sizes, and what they cannot do
without.

Operators, in the order of a step.  A sequence's new tokens are the nodes of a
tree: the last sampled token (the root) and drafts; parents[t] is a node's
parent as an index within its sequence, smaller than its own, -1 for a root.
  layout  tree_mask[t]: bit j set when node j of the sequence is t or an ancestor
          of t (64 bits a word); positions[t] = cached tokens + depth of t
  attn    latent attention of absorbed queries: a node sees the cached tokens and
          the new tokens in its mask
  verify  which nodes the target keeps, walking from the root, children in index
          order, and the token that follows them.  With draft probabilities q,
          a child drawn from its parent's q: accepted when u q(x) < r(x), r the
          parent's target row p; else r <- max(r - q, 0) / sum and the next
          child.  Without: accepted when u S < p(x), S = 1 first and then the
          mass that is left; else x is taken out.  Without random numbers
          (greedy): the first child that is the row's largest value.
          The next token: the first v whose cumulated r exceeds u_next sum(r).
  commit  cache rows of the kept nodes moved behind the cached tokens, in all
          layers, and the new lengths
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
    attn = dict(LARGE, op="attn", bs=64, H=128, mask="tree", nodes="fixed")
    ver = dict(op="verify", dtype="f32", nodes="fixed", mask="tree")
    com = dict(LARGE, op="commit", bs=64, mask="tree", nodes="fixed", lens="uniform")
    return [
        # one short conversation, a small tree: launch latency
        dict(attn, name="attn 1x70, 8 nodes", R=1, n=8, lens="fixed", top=70),
        # the uniform batch of 16 requests x 4096 tokens, full trees
        dict(attn, name="attn 16x4096, 32 nodes", R=16, n=32, lens="fixed", top=4096),
        # ragged requests and trees, pages of 16, a quarter of the heads (tensor parallel shard)
        dict(attn, name="attn 24 ragged, up to 24 nodes, 32 heads", R=24, n=24, H=32, bs=16, nodes="uniform", lens="uniform",
             top=8192),
        # one long document
        dict(attn, name="attn 1x131072, 16 nodes, 32 heads", R=1, n=16, H=32, lens="fixed", top=131072),
        # float32 storage and small heads
        dict(SMALL, name="attn small f32, 7 nodes", op="attn", bs=16, H=16, n=7, R=4, nodes="uniform", mask="tree",
             lens="uniform", top=700),
        # a step's tree of a few requests, and of a full batch with large trees
        dict(op="layout", name="layout 16x32", R=16, n=32, nodes="fixed", mask="tree", lens="fixed", top=4096),
        dict(op="layout", name="layout 256 ragged, up to 100 nodes", R=256, n=100, nodes="uniform", mask="tree",
             lens="uniform", top=8192),
        # one conversation, a chain of 4 drafts from a small model
        dict(ver, name="verify 1 chain of 5, V 32000", R=1, n=5, V=32000, mask="chain", mode="draft"),
        # a batch with trees drawn from the draft model, a large vocabulary
        dict(ver, name="verify 64 trees of 16, V 131072", R=64, n=16, V=131072, mode="draft"),
        # drafts without probabilities (the most likely continuations), bfloat16 rows of an odd length
        dict(ver, name="verify 24 trees of up to 21, V 100003, bf16", R=24, n=21, V=100003, mode="point", dtype="bf16",
             nodes="uniform"),
        # one conversation's layer, and a batch's cache of many layers at once
        dict(com, name="commit 1, 1 layer", R=1, n=16, layers=1, top=300),
        dict(com, name="commit 64, 32 layers", R=64, n=32, layers=32, top=200, nodes="uniform"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["attn"] * 4 + ["verify"] * 4 + ["commit"] * 2 + ["layout"])
    c = dict(op=op, shape_seed=rng.randrange(1 << 30), nodes=rng.choice(["fixed", "uniform"]),
             mask=rng.choice(["tree", "tree", "tree", "chain"]))
    lens = rng.choice(["uniform", "uniform", "fixed"])
    if op == "layout":
        n = _log_int(rng, 1, 130)
        return dict(c, n=n, R=_log_int(rng, 1, max(1, 20000 // n)) if n > 78 else _log_int(rng, 1, 256), lens=lens,
                    top=_log_int(rng, n, 16384))
    if op == "verify":
        V = _log_int(rng, 1000, 131072)
        n = _log_int(rng, 1, 24)
        return dict(c, V=V, n=n, R=_log_int(rng, 1, max(1, min(128, (1 << 27) // (n * V)))),
                    mode=rng.choice(["draft", "draft", "point", "greedy"]), dtype=rng.choice(["f32", "f32", "bf16"]))
    shape = dict(SMALL if rng.random() < 0.15 else LARGE)
    if op == "commit":
        R = _log_int(rng, 1, 64)
        top = _log_int(rng, 1, max(2, min(1000, 12800 // R)))
        return dict(c, **shape, n=_log_int(rng, 1, 64), R=R, lens=lens, bs=rng.choice([16, 32, 64, 128]), top=top,
                    layers=_log_int(rng, 1, max(1, min(48, 300_000 // (R * (top + 128))))))
    if rng.random() < 0.3:
        c["mask"] = "any"
    if shape["dtype"] == "f32":
        return dict(c, **shape, H=rng.choice([1, 4, 16]), R=_log_int(rng, 1, 8), n=_log_int(rng, 1, 20), lens=lens,
                    bs=rng.choice([16, 32]), top=_log_int(rng, 1, 700))
    H, n = rng.choice([8, 16, 32, 64, 96, 128]), _log_int(rng, 1, 80)
    R = _log_int(rng, 1, max(1, min(128, 65536 // (n * H))))
    return dict(c, **shape, H=H, n=n, R=R, lens=lens, bs=rng.choice([16, 32, 64, 128]),
                top=_log_int(rng, 1, max(1, min(131072, (1 << 18) // R, 250_000_000 // (R * n * H)))))


def _shape(c):
    """(parents of each sequence's nodes, tokens of each, new ones included): a matter of the case, not of its seed."""
    r = random.Random(c.get("shape_seed", 11))
    trees, lens = [], []
    for _ in range(c["R"]):
        n = c["n"] if c["nodes"] == "fixed" else r.randint(1, c["n"])
        if c["mask"] == "chain":
            p = list(range(-1, n - 1))
        else:  # breadth first; the first nodes have the most children
            p = [-1] + sorted(int(r.random() ** 2 * i) for i in range(1, n))
        trees.append(p)
        top = c.get("top", n)
        lens.append(max(n, top if c.get("lens") == "fixed" else r.randint(1, top)))
    return trees, lens


def _bits(trees, words):
    """[T, words] int64: a node's ancestors and itself."""
    out = []
    for p in trees:
        m = []
        for i, up in enumerate(p):
            m.append((m[up] if up >= 0 else 0) | 1 << i)
        out += m
    v = [(m >> 64 * w) & (1 << 64) - 1 for m in out for w in range(words)]
    return torch.tensor([x - (1 << 64) if x >> 63 else x for x in v], dtype=torch.int64).view(len(out), words)


def _type(c):
    return torch.bfloat16 if c["dtype"] == "bf16" else torch.float32


def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(device=dev).manual_seed(int(seed))
    trees, lens = _shape(c)
    R, T, big = c["R"], sum(map(len, trees)), max(map(len, trees))
    qsl = np.concatenate([[0], np.cumsum([len(p) for p in trees])])
    words = -(-big // 64)

    def i32(x):
        return torch.tensor(np.asarray(x), dtype=torch.int32, device=dev)

    # slot[r, i]: row of node i of sequence r; beyond its nodes: its last one
    slot = np.minimum(qsl[:-1, None] + np.arange(big), qsl[1:, None] - 1)
    s = {"case": dict(c), "T": T, "big": big, "qsl": i32(qsl), "seq_lens": i32(lens), "parents": i32(sum(trees, [])),
         "slot": torch.from_numpy(slot).to(dev), "real": torch.from_numpy(np.arange(big) < np.diff(qsl)[:, None]).to(dev),
         "row": torch.from_numpy(np.concatenate([r * big + np.arange(len(p)) for r, p in enumerate(trees)])).to(dev)}
    if c["op"] == "layout":
        # other trees of the same sizes for other seeds
        r = random.Random(int(seed))
        s["parents"] = i32(sum(([-1] + sorted(int(r.random() ** 2 * i) for i in range(1, len(p))) for p in trees), []))
        s.update(mask=torch.zeros(T, words, dtype=torch.int64, device=dev),
                 positions=torch.zeros(T, dtype=torch.int32, device=dev))
        return s
    if c["op"] == "verify":
        V, dt = c["V"], _type(c)
        # logits so wide that the likeliest tokens have probabilities of some ten percent
        z = torch.randn(T, V, generator=g, device=dev) * (1.25 * math.sqrt(2 * math.log(V)))
        near = torch.randn(T, V, generator=g, device=dev).mul_(0.8).add_(z)
        up = (s["parents"].long() + torch.repeat_interleave(s["qsl"][:-1].long(), s["qsl"][1:] - s["qsl"][:-1])).clamp_(min=0)
        if c["mode"] == "draft":
            q = torch.softmax(z, 1).to(dt)
            tokens = torch.cat([torch.multinomial(q[x].float(), 1, generator=g)[:, 0] for x in up.split(256)])
            s["q"] = q
        elif c["mode"] == "point":  # a node's children: the draft's likeliest tokens in order
            rank = torch.tensor([p[:i].count(x) for p in trees for i, x in enumerate(p)], device=dev)
            tokens = z.topk(int(rank.max()) + 1, 1).indices[up, rank]
        else:
            wrong = torch.randint(0, V, (T,), generator=g, device=dev)
            tokens = torch.where(torch.rand(T, generator=g, device=dev) < 0.75, near.to(dt).float().argmax(1)[up], wrong)
        s["p"] = (near if c["mode"] == "greedy" else torch.softmax(near, 1)).to(dt)
        s["tokens"] = tokens.int()
        if c["mode"] != "greedy":
            s["u"], s["u_next"] = torch.rand(T, generator=g, device=dev), torch.rand(R, generator=g, device=dev)
        s["depth"] = max(_depths(trees)) + 1                       # nodes of the longest path
        s["most"] = max(max(p.count(x) for x in p) for p in trees)  # children of a node
        s.update(path=torch.zeros(R, s["depth"], dtype=torch.int32, device=dev),
                 kept=torch.zeros(R, dtype=torch.int32, device=dev), next=torch.zeros(R, dtype=torch.int32, device=dev))
        return s
    dt, L, P, bs = _type(c), c["L"], c["P"], c["bs"]
    need = [-(-n // bs) for n in lens]
    blocks = sum(need) + 2
    order = torch.randperm(blocks, generator=g, device=dev).cpu().numpy().astype(np.int32)
    table = np.zeros((R, max(need)), np.int32)  # unused entries: block 0, as an engine leaves them
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = order[at:at + n]
        at += n
    s["table"] = torch.from_numpy(table).to(dev)
    if c["op"] == "commit":
        s["cache"] = torch.empty(c["layers"], blocks, bs, L + P, device=dev, dtype=dt).normal_(generator=g)
        s["layers"] = list(s["cache"].unbind(0))
        paths = [_path(random.Random(int(seed) * 1000 + r), p) for r, p in enumerate(trees)]
        deep = max(map(len, paths))
        s["path"] = i32([p + [-1] * (deep - len(p)) for p in paths])
        s["kept"] = i32([len(p) for p in paths])
        s["new_lens"] = torch.zeros(R, dtype=torch.int32, device=dev)
        return s
    H = c["H"]
    s["cache"] = torch.empty(blocks, bs, L + P, device=dev, dtype=dt).normal_(generator=g)
    s["mask"] = _bits(trees, words).to(dev)
    if c["mask"] == "any":  # bits of no tree; some rows see none of the new tokens
        lo = torch.randint(-(1 << 62), 1 << 62, (T, words), generator=g, device=dev)
        s["mask"] = torch.where(torch.rand(T, 1, generator=g, device=dev) < 0.2, torch.zeros_like(lo), lo)
    # absorbed queries: W_uk draws of 0.02 make the latent part 0.23 wide, the rope part is 1 wide
    q = torch.randn(T, H, L + P, generator=g, device=dev)
    q[..., :L] *= 0.23 if L > 64 else 1.0
    s.update(q=q.to(dt), o=torch.empty(T, H, L, device=dev, dtype=dt), lse=torch.empty(H, T, device=dev), longest=max(lens))
    return s


def _depths(trees):
    out = []
    for p in trees:
        d = []
        for x in p:
            d.append(d[x] + 1 if x >= 0 else 0)
        out += d
    return out


def _path(r, parents):
    """A path from the root that can be committed again and again: no row that it moves from is one that it moves to."""
    for _ in range(30):
        p, at = [], r.randrange(len(parents))
        while at >= 0:
            p.insert(0, at)
            at = parents[at]
        if all(x == d or x >= len(p) for d, x in enumerate(p)):
            return p
    return [0]


def _scale(c):
    return 1.0 / math.sqrt(c["Dn"] + c["P"])


def _children(s):
    """[R, big, big]: node i of sequence r has parent j; and the rank of i among its parent's children."""
    par = torch.where(s["real"], s["parents"][s["slot"]], -2)
    node = torch.arange(s["big"], device=par.device)
    child = par[:, :, None] == node
    rank = ((par[:, :, None] == par[:, None, :]) & (node[None, :] < node[:, None])).sum(2)
    return par, child, rank


def _plain(s):
    c = s["case"]
    R, big = c["R"], s["big"]
    if c["op"] == "layout":
        par, up, _ = _children(s)
        reach = up.float() + torch.eye(big, device=up.device)
        for _ in range(max(1, (big - 1).bit_length())):
            reach = (reach @ reach > 0).float()
        words = s["mask"].shape[1]
        bit = torch.ones((), dtype=torch.int64, device=up.device) << (torch.arange(big, device=up.device) % 64)
        word = torch.arange(big, device=up.device) // 64 == torch.arange(words, device=up.device)[:, None]
        mask = (reach.bool()[:, :, None, :] & word) * bit
        base = s["seq_lens"].long() - s["real"].sum(1)
        pos = base[:, None] + reach.sum(2).long() - 1
        return {"mask": mask.sum(3).view(-1, words)[s["row"]], "positions": pos.flatten()[s["row"]].int()}
    if c["op"] == "verify":
        return _plain_greedy(s) if c["mode"] == "greedy" else _plain_verify(s)
    lens, bs, L, P = s["seq_lens"].long(), c["bs"], c["L"], c["P"]
    base = lens - s["real"].sum(1)
    if c["op"] == "commit":
        path, d = s["path"].long(), torch.arange(s["path"].shape[1], device=lens.device)
        keep = d < s["kept"][:, None]
        src, dst = base[:, None] + torch.where(keep, path, 0), base[:, None] + torch.where(keep, d, 0)
        rows = s["cache"].view(c["layers"], -1, L + P)
        at = lambda x: (s["table"].gather(1, x // bs).long() * bs + x % bs).flatten()  # noqa: E731
        rows[:, at(dst)] = rows[:, at(src)]
        return {"cache": s["cache"], "new_lens": (base + s["kept"]).int()}
    dt, H, n = _type(c), c["H"], s["longest"]
    col = torch.arange(n, device=lens.device)
    page = s["table"][:, col // bs].long()
    k = s["cache"][page, col % bs].float()                                       # [R, n, L+P]
    q = s["q"][s["slot"]].float()                                                # [R, big, H, L+P]
    score = torch.bmm(q.reshape(R, big * H, L + P), k.transpose(1, 2)).view(R, big, H, n) * _scale(c)
    new = col - base[:, None]                                                    # [R, n], index among the new tokens
    word = s["mask"][s["slot"]]                                                  # [R, big, words]
    j = new.clamp(0, 64 * word.shape[2] - 1)[:, None].expand(R, big, n)
    seen = (word.gather(2, j // 64) >> (j % 64)) & 1 == 1
    seen = torch.where(new[:, None] < 0, True, seen) & (col < lens[:, None])[:, None]
    score = score.masked_fill(~seen[:, :, None], -math.inf)
    top = score.amax(3, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(score - top)
    total = p.sum(3, keepdim=True)
    o = torch.bmm(p.view(R, big * H, n), k[..., :L]).view(R, big, H, L) / torch.where(total == 0, torch.ones_like(total), total)
    lse = (top + torch.log(total)).view(R * big, H)
    return {"o": o.view(R * big, H, L)[s["row"]].to(dt), "lse": lse[s["row"]].t().contiguous()}


def _plain_verify(s):
    """All sequences at once, level by level and child by child; sums and borders in 64 bits."""
    R, V, f = s["case"]["R"], s["case"]["V"], torch.float64
    par, child, rank = _children(s)
    seq = torch.arange(R, device=par.device)
    qsl = s["qsl"][:-1].long()
    cur = torch.zeros(R, dtype=torch.int64, device=par.device)
    alive = torch.ones(R, dtype=torch.bool, device=par.device)
    path = torch.full((R, s["depth"]), -1, dtype=torch.int64, device=par.device)
    path[:, 0] = 0
    kept = torch.ones(R, dtype=torch.int64, device=par.device)
    draft = s["case"]["mode"] == "draft"
    w = torch.empty(R, V, dtype=f, device=par.device)                            # what is left of the row, not normalised
    mass = torch.ones(R, dtype=f, device=par.device)
    for level in range(s["depth"]):
        w = torch.where(alive[:, None], s["p"][qsl + cur].to(f), w)
        mass = torch.where(alive, torch.ones_like(mass), mass)
        moved = torch.zeros_like(alive)
        for k in range(s["most"] if level + 1 < s["depth"] else 0):
            here = child[seq, :, cur] & (rank == k)                              # [R, big], at most one
            node = here.int().argmax(1)
            asked = alive & ~moved & here.any(1)
            x = s["tokens"][qsl + node].long()
            u = s["u"][qsl + node].to(f)
            if draft:
                q = s["q"][qsl + cur].to(f)
                good = asked & (u * q[seq, x] * mass < w[seq, x])
                left = (w / torch.where(mass > 0, mass, torch.ones_like(mass))[:, None] - q).clamp(min=0)
            else:
                good = asked & (u * mass < w[seq, x])
                left = w.scatter(1, x[:, None], 0.0)
            bad = asked & ~good
            w = torch.where(bad[:, None], left, w)
            mass = torch.where(bad, w.sum(1), mass)
            path[:, level + 1] = torch.where(good, node, path[:, level + 1])
            kept, moved, cur = kept + good, moved | good, torch.where(good, node, cur)
        alive = alive & moved
    w = torch.where((w.sum(1) > 0)[:, None], w, s["p"][qsl + cur].to(f))
    total = w.cumsum(1)
    border = s["u_next"].to(f) * total[:, -1]
    return {"path": path.int(), "kept": kept.int(), "next": (total <= border[:, None]).sum(1).int()}


def _plain_greedy(s):
    """Every row's largest value first, then the walk over whole numbers."""
    R = s["case"]["R"]
    best = s["p"].float().argmax(1)
    par, child, _ = _children(s)
    seq, qsl = torch.arange(R, device=par.device), s["qsl"][:-1].long()
    token = torch.where(s["real"], s["tokens"][s["slot"]].long(), -1)
    cur = torch.zeros(R, dtype=torch.int64, device=par.device)
    alive, path, kept = torch.ones_like(cur).bool(), torch.full((R, s["depth"]), -1, dtype=torch.int64, device=par.device), 1
    path[:, 0] = 0
    for level in range(1, s["depth"]):
        hit = child[seq, :, cur] & (token == best[qsl + cur][:, None]) & alive[:, None]
        alive = hit.any(1)
        cur = torch.where(alive, hit.int().argmax(1), cur)
        path[:, level] = torch.where(alive, cur, -1)
        kept = kept + alive.int()
    return {"path": path.int(), "kept": (torch.zeros_like(qsl) + kept).int(), "next": best[qsl + cur].int()}


def run(state):
    if not own:
        return _plain(state)
    import mla_chunked_context_gb300 as M
    s, c = state, state["case"]
    if c["op"] == "layout":
        M.mla_tree_layout(s["parents"], s["qsl"], s["seq_lens"], s["mask"], s["positions"])
        return {"mask": s["mask"], "positions": s["positions"]}
    if c["op"] == "verify":
        M.mla_verify_tree(s["p"], s.get("q"), s["tokens"], s["parents"], s["qsl"], s.get("u"), s.get("u_next"),
                          s["path"], s["kept"], s["next"])
        return {"path": s["path"], "kept": s["kept"], "next": s["next"]}
    if "dims" not in s:
        s["dims"] = M.Dims(c.get("H", 1), c["L"], c["P"], c["Dn"], c["Dv"], c["bs"], _scale(c), _type(c))
    d = s["dims"]
    if c["op"] == "commit":
        M.mla_commit_tree(d, s["path"], s["kept"], s["qsl"], s["seq_lens"], s["layers"], s["table"],
                          new_seq_lens=s["new_lens"])
        return {"cache": s["cache"], "new_lens": s["new_lens"]}
    if "workspace" not in s:
        s["workspace"] = torch.empty(M.mla_latent_attn_workspace_bytes(d, s["T"], c["R"]), dtype=torch.uint8,
                                     device=s["q"].device)
    M.mla_tree_attn(d, s["qsl"], s["seq_lens"], s["mask"], s["q"], s["cache"], s["table"], s["workspace"], s["o"], s["lse"])
    return {"o": s["o"], "lse": s["lse"]}


def work(case):
    c = case
    trees, lens = _shape(c)
    sizes = [len(p) for p in trees]
    T, R = sum(sizes), c["R"]
    if c["op"] == "layout":
        return {"bytes": 4 * T + 8 * T * -(-max(sizes) // 64) + 4 * T + 8 * R, "flops": 2.0 * T}
    es = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "verify":
        # the rows that the next token is drawn from, and a value of each child
        rows = 2 if c["mode"] == "draft" else 1
        return {"bytes": es * rows * (R * c["V"] + T) + 12 * T + 12 * R, "flops": 4.0 * R * c["V"]}
    L, P = c["L"], c["P"]
    if c["op"] == "commit":
        moved = sum(sum(x != d for d, x in enumerate(_path(random.Random(r), p))) for r, p in enumerate(trees))
        return {"bytes": 2 * es * c["layers"] * moved * (L + P) + 16 * R, "flops": 1.0 * R}
    # a node's own and its ancestors' keys, besides the cached ones
    new = len(_depths(trees)) + sum(_depths(trees)) if c["mask"] != "any" else 0.4 * sum(n * n for n in sizes)
    pairs = sum((m - n) * n for m, n in zip(lens, sizes)) + new
    return {"bytes": es * (sum(lens) * (L + P) + T * c["H"] * (2 * L + P)) + 4 * T * c["H"] + 8 * T,
            "flops": 2.0 * pairs * c["H"] * (2 * L + P)}


def exact(case, seed):
    """The definitions in 64 bits, one sequence at a time, walked in Python."""
    s, c = prepare(case, seed), case
    trees, lens = _shape(c)
    f = torch.float64
    if c["op"] == "verify":
        out, at = [], 0
        for r, p in enumerate(trees):
            out.append(_exact_walk(s, c, p, at, r))
            at += len(p)
        deep = s["depth"]
        return {"path": torch.tensor([x + [-1] * (deep - len(x)) for x, _ in out], dtype=torch.int32),
                "kept": torch.tensor([len(x) for x, _ in out], dtype=torch.int32),
                "next": torch.tensor([v for _, v in out], dtype=torch.int32)}
    if c["op"] == "layout":
        par, at, trees = s["parents"].tolist(), 0, [list(p) for p in trees]
        for p in trees:
            p[:] = par[at:at + len(p)]
            at += len(p)
        base = [m - len(p) for m, p in zip(lens, trees) for _ in p]
        return {"mask": _bits(trees, s["mask"].shape[1]),
                "positions": torch.tensor([b + d for b, d in zip(base, _depths(trees))], dtype=torch.int32)}
    table, bs = s["table"].cpu().numpy(), c["bs"]
    if c["op"] == "commit":
        cache, path, kept = s["cache"], s["path"].tolist(), s["kept"].tolist()
        for r, p in enumerate(trees):
            base = lens[r] - len(p)
            slot = lambda j: (int(table[r, j // bs]), j % bs)  # noqa: E731
            rows = [cache[(slice(None),) + slot(base + path[r][d])].clone() for d in range(kept[r])]
            for d, row in enumerate(rows):
                cache[(slice(None),) + slot(base + d)] = row
        return {"cache": cache.to(f), "new_lens": torch.tensor([n - len(p) + k for n, p, k in zip(lens, trees, kept)],
                                                               dtype=torch.int32)}
    L, H = c["L"], c["H"]
    o = torch.zeros(s["T"], H, L, dtype=f, device="cuda")
    lse = torch.full((H, s["T"]), -math.inf, dtype=f, device="cuda")
    words, t = s["mask"].tolist(), 0
    for r, p in enumerate(trees):
        pages = torch.from_numpy(table[r, :-(-lens[r] // bs)].astype(np.int64)).cuda()
        k = s["cache"][pages].flatten(0, 1)[:lens[r]].to(f)
        for _ in p:
            base = lens[r] - len(p)
            see = list(range(base)) + [base + j for j in range(len(p)) if words[t][j // 64] >> j % 64 & 1]
            if see:
                # (the cached rows as they are, without a copy of them for every node)
                z = (s["q"][t].to(f) @ k.T) * _scale(c)
                z = torch.cat([z[:, :base], z[:, see[base:]]], 1)
                e = torch.softmax(z, 1)
                lse[:, t] = torch.logsumexp(z, 1)
                o[t] = e[:, :base] @ k[:base, :L] + e[:, base:] @ k[see[base:], :L]
            t += 1
    return {"o": o, "lse": lse}


def _exact_walk(s, c, parents, at, r):
    """(path, next token) of the sequence whose first node is row `at`."""
    tokens, cur, path = s["tokens"][at:at + len(parents)].tolist(), 0, [0]
    while True:
        p = s["p"][at + cur].double().cpu().numpy()
        kids = [i for i, x in enumerate(parents) if x == cur]
        if c["mode"] == "greedy":
            best = int(np.flatnonzero(p == p.max())[0])
            hit = [i for i in kids if tokens[i] == best]
            if not hit:
                return path, best
            cur = hit[0]
            path.append(cur)
            continue
        left, nxt = p, None  # what the next token may still be, normalised from the first rejection on
        q = s["q"][at + cur].double().cpu().numpy() if c["mode"] == "draft" else None
        for i in kids:
            u, x = float(s["u"][at + i]), tokens[i]
            if u * (1.0 if q is None else q[x]) < left[x]:
                nxt = i
                break
            if q is None:
                left = left.copy()
                left[x] = 0.0
            else:
                left = np.maximum(left - q, 0.0)
            total = left.sum()
            left = left / total if total > 0 else left
        if nxt is None:
            total = np.cumsum(left if left.sum() > 0 else p)
            return path, int(np.searchsorted(total, float(s["u_next"][r]) * total[-1], side="right"))
        cur = nxt
        path.append(cur)
