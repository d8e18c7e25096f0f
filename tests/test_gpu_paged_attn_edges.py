"""sz_attn_paged at its numerical edges, on the GPU, against the plain forms in 64 bits (paged_ops): values
that are not finite at places that some rows of a tile see and others do not, and scores that vanish."""
import math

import pytest
import torch

import paged_ops as P
from gpu_helpers import sz
from test_gpu_paged_ops import BF16, E5M2, check_attention, close, gen, run_attention

pytestmark = pytest.mark.gpu


def put(c, seq, place, x, dtype):
    """x [kv_heads, dim] as the value of a place, in the pool and in its copy."""
    page = c.v_pool.shape[1]
    c.v_pool[int(c.table[seq, place // page]), place % page] = x.to(dtype).cuda()
    c.v[seq][place] = x.to(dtype)


def with_infinities(q, k, v, causal, window):
    """P.attention's values, and where a row sees infinities or NaN what those add up to."""
    ref, rl, mag, reach = P.attention(q, k, torch.where(torch.isfinite(v.float()), v.float(), 0.0), causal, window)
    m, n, group = q.shape[0], k.shape[0], q.shape[1] // k.shape[1]
    j, place = torch.arange(n)[None], torch.arange(n - m, n)[:, None]
    seen = (j <= place) if causal else torch.ones(m, n, dtype=torch.bool)
    if window:
        seen = seen & (j > place - window)
    hit = [torch.einsum("mn,nhd->mhd", seen.double(), (v.double() == x).double()) > 0 for x in (math.inf, -math.inf)]
    nan = torch.einsum("mn,nhd->mhd", seen.double(), torch.isnan(v.double()).double()) > 0
    up, down, nan = (x.repeat_interleave(group, 1) for x in (*hit, nan))
    ref = torch.where(up, math.inf, ref)
    ref = torch.where(down, -math.inf, ref)
    return torch.where(nan | (up & down), math.nan, ref), rl, mag, reach


def check(dtype, q_len, kv, heads, kv_heads, dim, page, places, causal=True, window=0, seed=41):
    """places: {place: value, or None for one of each kind along the elements}."""
    m, g = sz(), gen(seed)
    c = P.build_cache(g, dtype, [kv], page, kv_heads, dim)
    for at, x in places.items():
        row = c.v[0][at].float().clone()
        if x is None:
            row[:, 1::5], row[:, 2::5], row[:, 3::5] = math.inf, -math.inf, math.nan
        else:
            row[:, ::3] = x
        put(c, 0, at, row, dtype)
    q = torch.randn(q_len, heads, dim, generator=g).bfloat16()
    out, lse = run_attention(m, c, q.cuda(), [q_len], [kv], causal, window)
    ref, rl, mag, reach = with_infinities(q, c.k[0], c.v[0], causal, window)
    close(out, ref, P.attention_bound(ref, mag, reach, dtype == E5M2), "out")
    close(lse, rl, 2.0 ** -18 * (reach + rl.abs().nan_to_num(0, 0, 0)) + 2.0 ** -16, "lse")


@pytest.mark.parametrize("dtype", [BF16, E5M2])
@pytest.mark.parametrize("heads,kv_heads,dim,page", [(8, 2, 64, 16), (4, 1, 128, 13), (3, 3, 80, 64), (2, 1, 192, 16)])
@pytest.mark.parametrize("q_len,kv", [(3, 40), (7, 700), (60, 60), (100, 900), (300, 300)])
def test_infinities_and_nan_at_the_edges(dtype, heads, kv_heads, dim, page, q_len, kv):
    """At the last place, in the middle of the new tokens, and at the first of them."""
    first = kv - q_len
    check(dtype, q_len, kv, heads, kv_heads, dim, page, {kv - 1: None, kv - 1 - q_len // 2: math.inf, first + 1: -math.inf})
    check(dtype, q_len, kv, heads, kv_heads, dim, page, {kv - 1 - q_len // 3: math.nan})
    check(dtype, q_len, kv, heads, kv_heads, dim, page, {kv - 2: None, kv - q_len: math.inf}, causal=False)


@pytest.mark.parametrize("dtype", [BF16, E5M2])
@pytest.mark.parametrize("heads,kv_heads,dim,page", [(8, 2, 64, 16), (4, 1, 128, 13), (3, 3, 80, 64)])
@pytest.mark.parametrize("q_len,kv,window", [(5, 90, 17), (6, 300, 1), (90, 700, 128), (200, 500, 50), (40, 40, 7)])
def test_infinities_and_nan_at_both_ends_of_a_window(dtype, heads, kv_heads, dim, page, q_len, kv, window):
    behind = max(0, kv - q_len - window + 1)
    for causal in (True, False):
        check(dtype, q_len, kv, heads, kv_heads, dim, page, {behind + 1: math.inf, behind: None, kv - 2: -math.inf},
              causal, window)


@pytest.mark.parametrize("dtype", [BF16, E5M2])
@pytest.mark.parametrize("q_len,heads", [(4, 4), (60, 8)])
def test_infinities_and_nan_in_parts_of_many_ctas(dtype, q_len, heads):
    check(dtype, q_len, 15000, heads, 1, 64, 16, {14999: None, 15000 - q_len: math.inf, 14998: math.nan})


def test_rows_that_see_nothing_beside_values_that_are_not_finite():
    for dtype in (BF16, E5M2):
        check(dtype, 90, 40, 4, 2, 64, 16, {0: None, 39: math.inf})
        check(dtype, 7, 3, 4, 2, 64, 16, {0: None, 2: math.inf})


@pytest.mark.parametrize("dtype", [BF16, E5M2])
@pytest.mark.parametrize("q_len", [6, 512])
@pytest.mark.parametrize("all_tokens", [False, True])
def test_values_that_are_not_finite_cost_no_more_than_others(dtype, q_len, all_tokens):
    """One NaN, or a whole chunk of them, behind 16,384 places: no row is done again from its first place."""
    m, g = sz(), gen(43)
    kv, page = 16384, 16
    c = P.build_cache(g, dtype, [kv], page, 2, 64)
    cache = m.KVCache(c.k_pool, c.v_pool, c.table)
    ws = m.new_ops_workspace(cache)
    q = torch.randn(q_len, 8, 64, generator=g).bfloat16().cuda()
    out = torch.empty_like(q)
    cu, kl = P.lengths([q_len], [kv])

    def fastest():
        times = []
        for _ in range(7):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            m.sz_attn_paged(cache, q, cu, kl, out, ws)
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b))
        return min(times)

    clean = fastest()
    pos = torch.arange(kv - q_len, kv) if all_tokens else torch.tensor([kv - 2])
    c.v_pool[c.table[0].long().cpu()[pos // page].cuda(), (pos % page).cuda()] = torch.tensor(math.nan, device="cuda").to(dtype)
    spoiled = fastest()
    assert torch.isnan(out[-1]).all() and torch.isnan(out[0]).all() == all_tokens
    print("%.3f ms, and %.3f without NaN" % (spoiled, clean))
    assert spoiled < 4 * clean + 0.2, "%.3f ms, and %.3f without NaN" % (spoiled, clean)


@pytest.mark.parametrize("dtype", [BF16, E5M2])
@pytest.mark.parametrize("q_lens,kv_lens,window", [([100, 70], [300, 70], 0), ([90], [500], 33), ([2, 1], [90, 30], 0)])
def test_scores_that_vanish(dtype, q_lens, kv_lens, window):
    """Queries near the smallest numbers and a small scale: every place that a row sees weighs the same."""
    check_attention(sz(), dtype, q_lens, kv_lens, 4, 2, 64, 16, window=window, scale=2.0 ** -40, spread=2.0 ** -115, seed=44)
