"""Verification at its borders: more sequences than fit the device at once; siblings
rejected one after the other, against the rule in exact fractions."""

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
