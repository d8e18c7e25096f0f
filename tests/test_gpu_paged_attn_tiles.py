"""sz_attn_paged over many rows (tiles of 256 rows, blocks of 128 places, shared out over the SMs) and the
operators beyond 4 GB of pool, on the GPU, against the plain forms in 64 bits (paged_ops)."""
import math

import pytest
import torch

import paged_ops as P
from gpu_helpers import sz
from test_gpu_paged_ops import BF16, E5M2, check_attention, close, gen, run_attention

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF16, E5M2])
@pytest.mark.parametrize("heads,kv_heads,dim,page", [
    (4, 2, 16, 16), (4, 2, 48, 8), (8, 1, 64, 128), (2, 2, 80, 32), (3, 1, 96, 64), (14, 2, 112, 16), (8, 2, 128, 256),
    (5, 5, 128, 24), (256, 2, 64, 16), (10, 1, 128, 100), (2, 1, 128, 1)])
def test_head_layouts_and_pages(dtype, heads, kv_heads, dim, page):
    """Groups that divide 128 and others, pages that a box fits and others, tiles of one and of two halves."""
    check_attention(sz(), dtype, [70, 34], [333, 34], heads, kv_heads, dim, page, seed=dim + page, tail=2)


@pytest.mark.parametrize("dtype", [BF16, E5M2])
@pytest.mark.parametrize("q_lens,kv_lens", [
    ([33], [33]), ([64], [127]), ([64], [128]), ([64], [129]), ([128], [128]), ([129], [129]), ([256], [257]),
    ([1, 200, 0, 40], [1, 200, 0, 40]), ([50] * 40, [50 + i for i in range(40)]), ([300, 1, 1], [300, 4000, 1]),
    ([40] * 3, [0, 10, 40])])
def test_lengths_around_a_block(dtype, q_lens, kv_lens):
    check_attention(sz(), dtype, q_lens, kv_lens, 4, 2, 64, 16, seed=sum(kv_lens))
    check_attention(sz(), dtype, q_lens, kv_lens, 4, 2, 64, 16, causal=False, seed=1)
    check_attention(sz(), dtype, q_lens, kv_lens, 4, 2, 64, 16, window=30, seed=2)


@pytest.mark.parametrize("dtype", [BF16, E5M2])
@pytest.mark.parametrize("page", [16, 13])
def test_a_long_context_of_few_tiles(dtype, page):
    """More parts to a tile than the last of them joins."""
    check_attention(sz(), dtype, [60], [20000], 8, 2, 128, page, seed=3)
    check_attention(sz(), dtype, [50, 40], [15000, 90], 4, 2, 80, page, window=9000, seed=4)


def grow(c, kv_heads, dim, dtype):
    """Scores that grow along the context: the running maximum moves at nearly every place."""
    n = c.k[0].shape[0]
    ramp = torch.linspace(0.1, 6.0, n)[:, None, None].expand(n, kv_heads, dim)
    x = ramp.to(dtype)
    c.k[0] = x
    pos = torch.arange(n)
    page = c.k_pool.shape[1]
    c.k_pool[c.table[0].long().cpu()[pos // page], pos % page] = x.to("cuda")


@pytest.mark.parametrize("dtype", [BF16, E5M2])
@pytest.mark.parametrize("q_len", [1, 8, 100])
def test_maxima_that_keep_growing(dtype, q_len):
    m, g = sz(), gen(21)
    c = P.build_cache(g, dtype, [1500], 16, 2, 64)
    grow(c, 2, 64, dtype)
    q = (1 + torch.rand(q_len, 4, 64, generator=g)).bfloat16()
    out, lse = run_attention(m, c, q.cuda(), [q_len], [1500])
    ref, rl, mag, reach = P.attention(q, c.k[0], c.v[0])
    close(out, ref, P.attention_bound(ref, mag, reach, dtype == E5M2), "out")
    close(lse, rl, 2.0 ** -18 * (reach + rl.abs()) + 2.0 ** -16, "lse")


@pytest.mark.parametrize("dtype", [BF16, E5M2])
@pytest.mark.parametrize("heads,q_len,kv", [(4, 100, 12000), (4, 300, 700)])
def test_values_that_are_not_finite_in_places_that_some_rows_do_not_see(dtype, heads, q_len, kv):
    """In tiles that many parts are joined to, and in those of one CTA."""
    m, g = sz(), gen(22)
    c = P.build_cache(g, dtype, [kv], 16, 1, 64)
    at = kv - q_len // 3
    page, off = int(c.table[0, at // 16]), at % 16
    c.v_pool[page, off] = torch.tensor(math.inf, device="cuda").to(dtype)
    q = torch.randn(q_len, heads, 64, generator=g).bfloat16()
    out, lse = run_attention(m, c, q.cuda(), [q_len], [kv])
    clean = q_len - q_len // 3
    ref, rl, mag, reach = P.attention(q[:clean], c.k[0][: kv - q_len + clean], c.v[0][: kv - q_len + clean])
    close(out[:clean], ref, P.attention_bound(ref, mag, reach, dtype == E5M2), "rows that do not see it")
    close(lse[:clean], rl, 2.0 ** -18 * (reach + rl.abs()) + 2.0 ** -16, "their lse")
    assert not torch.isfinite(out[clean:]).any()


@pytest.mark.parametrize("dtype", [BF16, E5M2])
def test_queries_and_keys_that_are_not_finite(dtype):
    """NaN in one query row, or in one key that some rows see, stays with the rows that see it."""
    m, g = sz(), gen(23)
    n = 200
    c = P.build_cache(g, dtype, [n], 16, 1, 64)
    q = torch.randn(n, 2, 64, generator=g).bfloat16()
    q[70, 1, 5] = math.nan
    at = 150
    c.k_pool[int(c.table[0, at // 16]), at % 16, 0, 3] = torch.tensor(math.nan, device="cuda").to(dtype)
    out, lse = run_attention(m, c, q.cuda(), [n], [n])
    ref, rl, mag, reach = P.attention(q[:at], c.k[0][:at], c.v[0][:at])
    good = torch.ones(at, 2, dtype=torch.bool)
    good[70, 1] = False
    close(out[:at][good], ref[good], P.attention_bound(ref, mag, reach, dtype == E5M2)[good], "rows without NaN")
    assert torch.isnan(out[70, 1]).all() and torch.isnan(out[at:]).all()
    assert torch.isnan(lse[70, 1]) and torch.isnan(lse[at:]).all()


@pytest.mark.parametrize("dtype", [BF16, E5M2])
def test_queries_that_repeat(dtype):
    """A query view with stride 0 over the heads: the same as its copy."""
    m, g = sz(), gen(24)
    c = P.build_cache(g, dtype, [300], 16, 2, 128)
    q = torch.randn(90, 1, 128, generator=g).bfloat16().cuda().expand(90, 8, 128)
    out, lse = run_attention(m, c, q, [90], [300])
    again, l2 = run_attention(m, c, q.contiguous(), [90], [300])
    assert torch.equal(out, again) and torch.equal(lse, l2)


def test_two_calls_at_once():
    """Two streams, each with its own workspace and outputs, over one cache: the bits of one call alone."""
    m, g = sz(), gen(25)
    c = P.build_cache(g, BF16, [2000, 2000], 16, 2, 128)
    cache = m.KVCache(c.k_pool, c.v_pool, c.table)
    lens = [300, 120], [2000, 1100]
    q = torch.randn(420, 8, 128, generator=g).bfloat16().cuda()
    want, _ = run_attention(m, c, q, *lens)
    cu, kl = P.lengths(*lens)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs, wss = [torch.empty_like(q) for _ in streams], [m.new_ops_workspace(cache) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, o, w in zip(streams, outs, wss):
            m.sz_attn_paged(cache, q, cu, kl, o, w, stream=s)
    torch.cuda.synchronize()
    for o, w in zip(outs, wss):
        assert m.sz_last_device_status(w) == 0 and torch.equal(o, want)


def test_decoding_and_prompts_take_turns_on_one_workspace():
    """Calls of both kinds of rows, long and short, leave the workspace as the next one needs it."""
    m, g = sz(), gen(26)
    c = P.build_cache(g, BF16, [9000, 700], 16, 1, 128)
    cache = m.KVCache(c.k_pool, c.v_pool, c.table)
    ws = m.new_ops_workspace(cache)
    shapes = [([1, 1], [9000, 700]), ([60, 60], [9000, 700]), ([3, 0], [5000, 0]), ([700, 100], [800, 100])]
    qs = [torch.randn(sum(a), 4, 128, generator=g).bfloat16().cuda() for a, _ in shapes]
    want = [run_attention(m, c, q, *s)[0] for q, s in zip(qs, shapes)]
    for _ in range(3):
        for q, s, w in zip(qs, shapes, want):
            out, _ = run_attention(m, c, q, *s, cache=cache, ws=ws)
            assert torch.equal(out, w)


@pytest.mark.parametrize("dtype", [BF16, E5M2])
def test_pools_beyond_4_gb(dtype):
    """Pages whose byte offsets pass 32 bits: written by the append, read by both attention kernels."""
    m, g = sz(), gen(27)
    page, kv_heads, dim, heads = 64, 4, 128, 16
    es = 2 if dtype == BF16 else 1
    pages = (1 << 32) // (page * kv_heads * dim * es) + 200
    pools = [torch.empty(pages, page, kv_heads, dim, dtype=dtype, device="cuda") for _ in range(2)]
    ids = pages - 1 - 2 * torch.arange(8)
    cache = m.KVCache(pools[0], pools[1], ids.int().view(1, 8).cuda())
    ws = m.new_ops_workspace(cache)
    n = 500
    kv = torch.randn(2, n, kv_heads, dim, generator=g).bfloat16()
    cu, kl = P.lengths([n], [n])
    m.sz_kv_append_paged(cache, kv[0].cuda(), kv[1].cuda(), cu, kl, ws)
    assert m.sz_last_device_status(ws) == 0
    pos = torch.arange(n)
    held = [p[ids[pos // page].cuda(), (pos % page).cuda()].cpu() for p in pools]
    for h, x in zip(held, kv):
        assert torch.equal(h.float(), x.to(dtype).float())
    for q_len in (1, 60):
        q = torch.randn(q_len, heads, dim, generator=g).bfloat16()
        cu, kl = P.lengths([q_len], [n])
        out = torch.empty_like(q, device="cuda")
        m.sz_attn_paged(cache, q.cuda(), cu, kl, out, ws)
        ref, _, mag, reach = P.attention(q, held[0], held[1])
        close(out, ref, P.attention_bound(ref, mag, reach, dtype == E5M2), "out")
    assert m.sz_last_device_status(ws) == 0


def test_the_binding_refuses_what_does_not_fit():
    m = sz()
    c = P.build_cache(gen(28), BF16, [40], 16, 2, 64)
    cache = m.KVCache(c.k_pool, c.v_pool, c.table)
    ws = m.new_ops_workspace(cache)
    q = torch.zeros(3, 4, 64, dtype=BF16, device="cuda")
    kv = q[:, :2]
    cu, kl = P.lengths([3], [40])
    ok = dict(q=q, cu_q=cu, kv_len=kl, out=torch.empty_like(q), ws=ws)
    for bad in (dict(q=q.float()), dict(out=q.half()), dict(cu_q=cu.long()), dict(kv_len=kl.float())):
        with pytest.raises(TypeError):
            m.sz_attn_paged(cache, **dict(ok, **bad))
    for bad in (dict(q=q[0]), dict(q=q[:, :, :32]), dict(q=q.transpose(1, 2)), dict(out=q[:2]), dict(cu_q=cu[:1]),
                dict(kv_len=kl.repeat(2)), dict(window=-1), dict(window=1 << 31), dict(lse=torch.zeros(3, device="cuda")),
                dict(q=q.cpu()), dict(ws=ws.cpu())):
        with pytest.raises(ValueError):
            m.sz_attn_paged(cache, **dict(ok, **bad))
    for bad in (dict(out=q), dict(ws=ws[:1024]), dict(scale=0.0), dict(q=q[:, :3], out=torch.empty(3, 3, 64, dtype=BF16, device="cuda"))):
        with pytest.raises(m.SplitZipError):
            m.sz_attn_paged(cache, **dict(ok, **bad))
    with pytest.raises(ValueError):
        m.sz_kv_append_paged(cache, kv, kv[:2], cu, kl, ws)
    with pytest.raises(ValueError):
        m.sz_kv_append_paged(cache, kv, kv, cu, kl, ws, q_out=q)
    with pytest.raises(ValueError):
        m.sz_kv_append_paged(cache, kv, kv, cu, kl, ws, rope=torch.zeros(10, 64, device="cuda"), positions=cu)
    with pytest.raises(ValueError):
        m.sz_qk_norm_rope(q, None, None, None, ws)
    with pytest.raises(m.SplitZipError):
        m.sz_qk_norm_rope(q, None, torch.empty_like(q), None, ws, rope=torch.zeros(10, 64, device="cuda"))
    assert m.sz_last_device_status(ws) == 0


@pytest.mark.parametrize("dtype", [BF16, E5M2])
@pytest.mark.parametrize("q_lens,kv_lens,heads,kv_heads,dim,window", [
    ([140, 200, 33], [140, 300, 900], 64, 64, 64, 0), ([300], [300], 160, 160, 16, 0), ([1024, 700], [1024, 700], 32, 32, 80, 0),
    ([70, 0, 1, 500], [1000, 3, 1, 1024], 160, 40, 32, 0), ([600], [600], 64, 64, 48, 100), ([100] * 32, [100 + i for i in range(32)], 8, 8, 64, 0)])
def test_tiles_that_are_not_cut(dtype, q_lens, kv_lens, heads, kv_heads, dim, window):
    """Short tiles, at least as many as the SMs: each by one CTA, the longest first."""
    check_attention(sz(), dtype, q_lens, kv_lens, heads, kv_heads, dim, 16, window=window, seed=dim, tail=1)


def test_values_that_are_not_finite_in_tiles_that_are_not_cut():
    m, g = sz(), gen(29)
    n, heads = 300, 160
    c = P.build_cache(g, BF16, [n], 16, heads, 16)
    at = 150
    c.v_pool[int(c.table[0, at // 16]), at % 16] = math.nan
    q = torch.randn(n, heads, 16, generator=g).bfloat16()
    out, lse = run_attention(m, c, q.cuda(), [n], [n])
    ref, rl, mag, reach = P.attention(q[:at], c.k[0][:at], c.v[0][:at])
    close(out[:at], ref, P.attention_bound(ref, mag, reach, False), "rows that do not see it")
    close(lse[:at], rl, 2.0 ** -18 * (reach + rl.abs()) + 2.0 ** -16, "their lse")
    assert torch.isnan(out[at:]).all()
