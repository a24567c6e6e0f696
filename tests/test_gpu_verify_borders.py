"""Verification at its borders: more sequences than fit the device at once; siblings
rejected one after the other and random numbers right beside each border, against
the rule in exact fractions."""

from fractions import Fraction

import numpy as np
import pytest
import torch

from test_gpu_decode import DEV, _cuda, _no_device_errors  # noqa: F401
from test_gpu_tree import check_verify, drafted, run_verify

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("R", [304, 305, 1000, 5000])
@pytest.mark.parametrize("mode", ["draft", "point", "greedy"])
def test_more_sequences_than_fit_at_once(mode, R):
    """Four CTAs on each of 152 SMs, a cluster of two CTAs for each sequence: 304 of
    them fit."""
    rng = np.random.default_rng(R)
    sizes = [int(x) for x in rng.integers(0, 6, R)]
    for dtype, V in ((torch.float32, 97), (torch.bfloat16, 40)):
        args = drafted(rng, mode, sizes, V, dtype)
        check_verify(run_verify(*args, 4), *args, 4)


def walk(p, q, tokens, parents, u, u_next, most):
    """The rule in fractions, of one sequence with draft rows: (kept nodes, next
    token)."""
    cur, path = 0, [0]
    while True:
        left = [Fraction(float(x)) for x in p[cur]]
        draft = [Fraction(float(x)) for x in q[cur]]
        kids = [i for i, x in enumerate(parents) if x == cur] if len(path) < most else []
        for i in kids:
            x = tokens[i]
            if Fraction(float(u[i])) * draft[x] < left[x]:
                break
            left = [max(a - b, Fraction(0)) for a, b in zip(left, draft)]
            total = sum(left)
            left = [a / total for a in left] if total else left
        else:
            if not any(left):
                left = [Fraction(float(x)) for x in p[cur]]
            border, run = Fraction(float(u_next)) * sum(left), Fraction(0)
            for v, a in enumerate(left):
                run += a
                if run > border:
                    return path, v
            return path, len(left) - 1
        cur = i
        path.append(cur)


def check(p, q, tokens, parents, qsl, u, un, most, dtype=torch.float32):
    """Lists of rows and so on, one after the other: exactly the rule's results."""
    p, q = (torch.tensor(np.asarray(x, np.float32)).to(dtype) for x in (p, q))
    path, kept, nxt = run_verify(p.to(DEV), q.to(DEV), tokens, parents, qsl, u, un, most)
    p, q, u, un = p.float().numpy(), q.float().numpy(), np.float32(u), np.float32(un)
    for r in range(len(qsl) - 1):
        lo, hi = qsl[r], qsl[r + 1]
        line, v = walk(p[lo:hi], q[lo:hi], tokens[lo:hi], parents[lo:hi], u[lo:hi], un[r], most)
        assert path[r].tolist() == line + [-1] * (most - len(line)) and kept[r] == len(line) and nxt[r] == v, \
            (r, path[r], line, nxt[r], v)


def test_two_rejected_siblings_of_four_tokens():
    """t = 1 + 0.0111: token 0 has 0.999 of what is left, its border is far from
    0.97 and from 0.9985."""
    p, q = [0.001, 0.919, 0.0, 0.080], [0.0, 0.909, 0.0, 0.091]
    un = [0.5, 0.97, 0.9985, 0.9995]
    R = len(un)
    check([p] * 3 * R, [q] * 3 * R, [0, 3, 3] * R, [-1, 0, 0] * R, list(range(0, 3 * R + 1, 3)), [0.95] * 3 * R, un, 3)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kids", [1, 4, 6, 40, 1023])
def test_many_rejected_siblings_of_heavy_rows(kids, dtype):
    """Rows that sum to 300 with a draft whose mass lies elsewhere: t grows by 300
    with each sibling, to 306600, while r stays p.  The last sibling of the second
    sequence has mass in p alone and is kept whatever its random number."""
    V = 400
    p, q = np.zeros(V, np.float32), np.zeros(V, np.float32)
    p[::2], q[1::2] = 1.5, 1 / 256
    n = kids + 1
    tokens = [0] + [2 * (i % 200) + 1 for i in range(kids)]
    check([p] * 2 * n, [q] * 2 * n, tokens + tokens[:-1] + [46], [-1] + [0] * kids + [-1] + [0] * kids, [0, n, 2 * n],
          [0.5] * 2 * n, [0.1234, 0.9876], 2, dtype)


def neighbours(x):
    """The float32 values on either side of a fraction in [0, 1)."""
    a = np.float32(float(x))
    if Fraction(float(a)) > x:
        a = np.nextafter(a, np.float32(-1))
    return [v for v in (a, np.nextafter(a, np.float32(2))) if 0 <= v < 1]


def rounded(x, dtype):
    return torch.from_numpy(np.float32(x)).to(dtype).float().numpy()


def beside_borders(rng, V, kids, dtype):
    """A root with `kids` children: rows, tokens drawn from the draft, and random
    numbers that are the float32 next to the border of each test (mostly on the side
    of a rejection) and of the next token; and how many children are rejected.  None
    where one is nearer to its border than what the call promises: 1.1 units of 2^-45
    a value and rejection, of what is left before it is divided by its sum."""
    n = kids + 1
    z = rng.normal(size=(n, V)) * rng.uniform(0.5, 4)
    soft = lambda x: np.exp(x) / np.exp(x).sum(1, keepdims=True)  # noqa: E731
    p = rounded(soft(z + rng.uniform(0.05, 0.8) * rng.normal(size=(n, V))), dtype)
    q = rounded(np.minimum(soft(z), 0.95), dtype)
    weight = q[0].astype(np.float64) / q[0].astype(np.float64).sum()
    tokens = [0] + [int(x) for x in rng.choice(V, kids, p=weight)]
    u = np.full(n, 0.5, np.float32)
    left, draft = ([Fraction(float(x)) for x in row[0]] for row in (p, q))
    scale, last, rejected = Fraction(1), 0, 0
    for i in range(1, n):
        x, room = tokens[i], Fraction(11, 10) * (rejected + 1) * V / 2 ** 45
        if left[x] and draft[x]:
            near = neighbours(left[x] / draft[x])
            u[i] = near[-1 if rng.random() < 0.8 else 0] if near else 0.999
            if abs(Fraction(float(u[i])) * draft[x] - left[x]) * scale <= room:
                return None
        if Fraction(float(u[i])) * draft[x] < left[x]:
            last, left, scale = i, [Fraction(float(v)) for v in p[i]], Fraction(1)
            break
        left = [max(a - b, Fraction(0)) for a, b in zip(left, draft)]
        total = sum(left)
        if not total:
            return None
        left, scale, rejected = [a / total for a in left], scale * total, rejected + 1
    ends, run = [], Fraction(0)
    for a in left:
        run += a
        if a:
            ends.append(run)
    near = neighbours(ends[rng.integers(len(ends))] / run) or [np.float32(0.5)]
    un = near[rng.integers(len(near))]
    room = Fraction(11, 10) * (rejected + 1) * V / 2 ** 45
    if min(abs(Fraction(float(un)) * run - e) for e in ends) * scale <= room:
        return None
    return p, q, tokens, [-1] + [0] * kids, u, un, rejected if not last else 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V,count", [(2, 2400), (5, 2400), (12, 2400), (40, 2400), (3001, 100)])
def test_random_numbers_beside_the_borders(V, count, dtype):
    rng = np.random.default_rng(V)
    P, Q, tok, par, qsl, u, un, deep = [], [], [], [], [0], [], [], []
    for k in range(count):
        made = beside_borders(rng, V, 1 + k % 6, dtype)
        if made:
            P += list(made[0]); Q += list(made[1]); tok += made[2]; par += made[3]; u += list(made[4]); un.append(made[5])
            qsl.append(len(tok))
            deep.append(made[6])
    if 2 < V < 100:                                  # (of two tokens one rejection leaves one)
        assert len(deep) > 0.8 * count and max(deep) >= 5 and sum(d >= 2 for d in deep) > 0.1 * count
    check(P, Q, tok, par, qsl, u, un, 3, dtype)


def test_products_from_one_on():
    """Draft values above 1.  The first sibling leaves token 0 alone, r(0) = 1: the
    second one is rejected where u q is 1 or more, even by less than float32 sees,
    and kept where it is less by that little."""
    step = 2.0 ** -23
    rows = [([1.5, 0.1], [1.25, 0.5], 0.95), ([1.5, 0.1], [1 + 1000 * step, 0.5], 1 - 1000 * step),
            ([1.5, 0.1], [1 + 1001 * step, 0.5], 1 - 1000.5 * step), ([1.75, 0.1], [1.5, 0.5], 0.5)]
    P, Q, u = [], [], []
    for p, q, x in rows:
        P += [p] * 3
        Q += [q] * 3
        u += [0.5, 0.9, x]
    R = len(rows)
    check(P, Q, [0, 1, 0] * R, [-1, 0, 0] * R, list(range(0, 3 * R + 1, 3)), u, [0.5] * R, 3)
    kept = [walk(P[3 * r:3 * r + 3], Q[3 * r:3 * r + 3], [0, 1, 0], [-1, 0, 0], np.float32(u[3 * r:3 * r + 3]), 0.5, 3)[0]
            for r in range(R)]
    assert kept == [[0], [0, 2], [0], [0, 2]]
