"""Which views of one buffer the norm and rotation of heads takes as inputs and outputs (no GPU needed): views
whose rows meet are refused, whatever their strides; views of one layout whose rows do not meet are taken."""
import itertools
import random

import pytest
import torch

import fp8_kv_cache_exp_b200 as sz
from test_paged_ops_refusals import A, NONE, heads, norm_rope

# a call that is taken would be launched where there is a GPU, and its addresses are nobody's
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="needs a machine without a GPU")

DIM = 16


def rows(at, ts, hs, n, tokens):
    return [at + t * ts + h * hs for t in range(tokens) for h in range(n)]


def meet(a, b):
    return any(abs(x - y) < DIM for x in a for y in b)


def taken(tokens, q, q_out, k, k_out):
    """Whether the call passes the checks; views are (first element, token stride, head stride, heads)."""
    v = [NONE if x is None else heads(A + 2 * x[0], x[1], x[2], x[3]) for x in (q, q_out, k, k_out)]
    status = norm_rope(tokens=tokens, q=v[0], q_out=v[1], k=v[2], k_out=v[3], dim=DIM)
    assert status in (sz.SZ_ERR_INVALID_ARG, sz.SZ_ERR_CUDA)
    return status == sz.SZ_ERR_CUDA


def sound(tokens, q, q_out, k, k_out):
    r = [None if x is None else rows(*x, tokens) for x in (q, q_out, k, k_out)]
    for out in (r[1], r[3]):
        if out and any(abs(x - y) < DIM for x, y in itertools.combinations(out, 2)):
            return False
    if r[1] and r[3] and meet(r[1], r[3]):
        return False
    for i, j in ((0, 1), (2, 1), (0, 3), (2, 3)):
        if r[i] and r[j] and meet(r[i], r[j]) and not (j == i + 1 and r[i] == r[j]):
            return False
    return True


def test_heads_of_one_projection_in_place():
    """Queries, keys and values one behind the other in a token, side by side for each head, and tokens inside
    a head."""
    for t in (1, 2, 5):
        for q, k in (((0, 12 * DIM, DIM, 4), (4 * DIM, 12 * DIM, DIM, 4)),
                     ((0, 12 * DIM, 3 * DIM, 4), (DIM, 12 * DIM, 3 * DIM, 4)),
                     ((0, DIM, t * DIM, 4), (4 * t * DIM, DIM, t * DIM, 2)),
                     ((0, 2 * DIM, 2 * t * DIM, 4), (DIM, 2 * DIM, 2 * t * DIM, 4))):
            assert sound(t, q, q, k, k) and taken(t, q, q, k, k)
    # one head, whose stride is nothing
    assert taken(3, (0, 6 * DIM, 0, 1), (0, 6 * DIM, 0, 1), (DIM, 6 * DIM, 2 * DIM, 2), (DIM, 6 * DIM, 2 * DIM, 2))


@pytest.mark.parametrize("shift", [8, DIM, 4 * DIM - 8])
def test_columns_that_meet_are_refused(shift):
    """Keys that begin inside the queries' columns."""
    q, k = (0, 12 * DIM, DIM, 4), (4 * DIM - shift, 12 * DIM, DIM, 4)
    assert not sound(2, q, q, k, k) and not taken(2, q, q, k, k)


def test_views_of_any_strides():
    rng = random.Random(5)
    took = 0
    for _ in range(20000):
        t = rng.randint(1, 4)

        def view(like=None):
            at = 8 * rng.randint(0, 40)
            if like and rng.random() < 0.7:
                return at, like[1], like[2], rng.randint(1, 3)
            return at, 8 * rng.randint(0, 16), 8 * rng.randint(0, 16), rng.randint(1, 3)

        q = view()
        q_out = q if rng.random() < 0.5 else view(q)[:3] + q[3:]
        k = view(q) if rng.random() < 0.7 else None
        k_out = None if k is None else k if rng.random() < 0.6 else view(q)[:3] + k[3:]
        ok = taken(t, q, q_out, k, k_out)
        took += ok
        good = sound(t, q, q_out, k, k_out)
        assert good or not ok, (t, q, q_out, k, k_out)
        one = all(x is None or x[1:3] == q[1:3] for x in (q_out, k, k_out))
        nested = min(q[1], q[2]) * (q[3] if q[2] <= q[1] else t) <= max(q[1], q[2])  # heads inside a token, or the other way
        if good and one and nested and (k is None or k[3] == q[3]):
            assert ok, (t, q, q_out, k, k_out)
    assert took > 1000
