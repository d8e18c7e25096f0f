"""The operators on a paged cache on the GPU, against their plain forms in 64 bits."""
import math

import pytest
import torch

import paged_ops as P
from gpu_helpers import sz

pytestmark = pytest.mark.gpu

BF16, E5M2 = torch.bfloat16, torch.float8_e5m2


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def close(got, ref, bound, what):
    got, ref = got.double().cpu(), ref.cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), what + ": NaN in other places"
    inf = torch.isinf(ref)
    assert torch.equal(got[inf], ref[inf]), what + ": infinities"
    far = (got - ref).abs() > bound.cpu()
    far &= torch.isfinite(ref)
    assert not far.any(), "%s: %d of %d off, worst %g beyond %g" % (
        what, int(far.sum()), far.numel(), float((got - ref).abs()[far].max()), float(bound.cpu()[far].max()))


# ------------------------------------------------------------------ attention

def run_attention(m, c, q, q_lens, kv_lens, causal=True, window=0, scale=None, lse=True, ws=None, cache=None,
                  out=None, stream=None):
    cu, kl = P.lengths(q_lens, kv_lens)
    cache = cache or m.KVCache(c.k_pool, c.v_pool, c.table)
    ws = m.new_ops_workspace(cache) if ws is None else ws
    out = torch.full(q.shape, 7.0, dtype=BF16, device="cuda") if out is None else out
    ls = torch.full(q.shape[:2], 7.0, device="cuda") if lse else None
    m.sz_attn_paged(cache, q, cu, kl, out, ws, scale=scale, causal=causal, window=window, lse=ls, stream=stream)
    assert m.sz_last_device_status(ws) == 0
    return out, ls


def check_attention(m, dtype, q_lens, kv_lens, heads, kv_heads, dim, page, causal=True, window=0, scale=None, gap=0,
                    seed=0, spread=1.0, tail=0):
    g = gen(seed)
    c = P.build_cache(g, dtype, kv_lens, page, kv_heads, dim, gap=gap)
    total = sum(q_lens)
    q = (torch.randn(total + tail, heads, dim, generator=g) * spread).bfloat16()
    out, lse = run_attention(m, c, q.cuda(), q_lens, kv_lens, causal, window, scale)
    at = 0
    for b, (ql, kl) in enumerate(zip(q_lens, kv_lens)):
        ref, rl, mag, reach = P.attention(q[at: at + ql], c.k[b], c.v[b], causal, window, scale)
        close(out[at: at + ql], ref, P.attention_bound(ref, mag, reach, dtype == E5M2), "out of sequence %d" % b)
        close(lse[at: at + ql], rl, 2.0 ** -18 * (reach + rl.abs().nan_to_num(0, 0, 0)) + 2.0 ** -16, "lse of sequence %d" % b)
        at += ql
    assert (out[total:] == 7.0).all() and (lse[total:] == 7.0).all(), "rows behind the last sequence"


@pytest.mark.parametrize("dtype", [BF16, E5M2])
@pytest.mark.parametrize("q_lens,kv_lens,heads,kv_heads,dim,page", [
    ([1], [1], 1, 1, 16, 1),
    ([1], [777], 32, 8, 128, 16),
    ([1, 1, 1], [0, 1, 64], 4, 2, 64, 16),
    ([1, 1, 1, 1], [63, 65, 16, 15], 8, 1, 128, 13),
    ([1, 0, 2, 1], [100, 50, 2, 200], 6, 2, 80, 3),
    ([5, 3], [5, 200], 14, 2, 128, 100),
    ([7], [3], 4, 4, 96, 8),                         # four rows see nothing
    ([1, 1], [1000, 3], 16, 1, 48, 7),
    ([1, 2], [130, 70], 20, 1, 112, 5),              # more rows than one 16-row tile
    ([1, 1, 4], [300, 257, 9], 3, 1, 256, 4),
    ([2, 1], [90, 33], 8, 8, 192, 16),
    ([40, 1, 17], [40, 500, 130], 8, 2, 128, 16),    # mixed prompt and decode
    ([33], [290], 7, 7, 32, 9),
    ([129, 64], [129, 300], 2, 1, 64, 24),
    ([300], [300], 4, 1, 80, 13),
    ([200, 3], [900, 3], 8, 2, 128, 40),
    ([150], [1200], 16, 2, 128, 11),
])
def test_attention(dtype, q_lens, kv_lens, heads, kv_heads, dim, page):
    check_attention(sz(), dtype, q_lens, kv_lens, heads, kv_heads, dim, page)


@pytest.mark.parametrize("dtype", [BF16, E5M2])
@pytest.mark.parametrize("q_lens,kv_lens,causal,window", [
    ([1, 1], [300, 40], True, 1),
    ([1, 1, 1], [300, 40, 64], True, 17),
    ([9, 30], [100, 30], True, 16),
    ([9, 30], [100, 30], False, 0),
    ([4, 12], [100, 6], False, 20),
    ([140, 20], [700, 20], True, 100),
    ([140, 20], [300, 5], False, 0),
    ([260], [1000], True, 129),
    ([260], [1000], False, 300),
    ([2], [500], True, 2 ** 31 - 1),
])
def test_attention_masks(dtype, q_lens, kv_lens, causal, window):
    check_attention(sz(), dtype, q_lens, kv_lens, 8, 2, 128, 16, causal, window, seed=3)


@pytest.mark.parametrize("dtype", [BF16, E5M2])
@pytest.mark.parametrize("q", [1, 150])
def test_attention_page_gaps_scale_and_peaks(dtype, q):
    """Pages apart in the pool, a scale of one's own, and scores that one place dominates."""
    check_attention(sz(), dtype, [q, q], [400, 333], 8, 2, 128, 16, scale=0.5, gap=64, seed=4, tail=3)


@pytest.mark.parametrize("dtype", [BF16, E5M2])
def test_attention_long_context_split_over_ctas(dtype):
    """One sequence of one KV head: every CTA has a piece, and the last joins them."""
    check_attention(sz(), dtype, [1], [20011], 4, 1, 128, 16, seed=5)
    check_attention(sz(), dtype, [30], [9001], 8, 1, 128, 32, seed=6)


def test_attention_many_sequences():
    """More sequences than a CTA has threads, some of them empty."""
    g = gen(7)
    q_lens = [int(x) for x in torch.randint(0, 3, (700,), generator=g)]
    kv_lens = [a + int(x) for a, x in zip(q_lens, torch.randint(0, 40, (700,), generator=g))]
    check_attention(sz(), BF16, q_lens, kv_lens, 2, 1, 32, 8, seed=7)


def test_attention_large_queries_on_e5m2():
    """Queries beyond fp16's range keep their bits (a power of two is taken out of each row)."""
    check_attention(sz(), E5M2, [2, 1], [90, 30], 4, 2, 64, 16, seed=8, spread=2.0 ** 20, scale=2.0 ** -24)
    check_attention(sz(), E5M2, [140], [200], 4, 2, 64, 16, seed=8, spread=2.0 ** -30, scale=2.0 ** 28)


@pytest.mark.parametrize("dtype", [BF16, E5M2])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("q_len", [6, 200])
def test_attention_unseen_places_have_no_say(dtype, bad, q_len):
    """Keys and values that are not finite at places that some rows of a tile see and others do not."""
    m = sz()
    g = gen(9)
    n = q_len + 50
    c = P.build_cache(g, dtype, [n], 16, 2, 64)
    at = n - q_len // 2
    page, off = int(c.table[0, at // 16]), at % 16
    c.v_pool[page, off] = torch.tensor(bad, device="cuda").to(dtype)
    c.v[0][at] = torch.tensor(bad).to(dtype)
    q = torch.randn(q_len, 4, 64, generator=g).bfloat16()
    out, lse = run_attention(m, c, q.cuda(), [q_len], [n])
    ref, rl, mag, reach = P.attention(q, c.k[0], c.v[0])
    clean = q_len - q_len // 2                       # rows before the place
    close(out[:clean], ref[:clean], P.attention_bound(ref, mag, reach, dtype == E5M2)[:clean], "rows that do not see it")
    assert not torch.isfinite(out[clean:]).any()
    # a key, behind the window of the last rows
    c.v_pool[page, off] = 1.0
    c.v[0][at] = 1.0
    c.k_pool[page, off] = torch.tensor(bad, device="cuda").to(dtype)
    out, lse = run_attention(m, c, q.cuda(), [q_len], [n])
    ref, rl, mag, reach = P.attention(q[:clean], c.k[0][: n - q_len + clean], c.v[0][: n - q_len + clean])
    close(out[:clean], ref, P.attention_bound(ref, mag, reach, dtype == E5M2), "rows that do not see the key")
    close(lse[:clean], rl, 2.0 ** -18 * (reach + rl.abs()) + 2.0 ** -16, "their lse")


@pytest.mark.parametrize("q_len", [1, 150])
def test_attention_strides_and_streams(q_len):
    """Queries as columns of a wider buffer, outputs with gaps, another stream, repeated calls with one
    workspace: the same bits."""
    m = sz()
    g = gen(11)
    c = P.build_cache(g, BF16, [q_len + 600, q_len + 77], 16, 2, 128)
    qkv = torch.randn(2 * q_len, 12, 128, generator=g).bfloat16().cuda()
    q = qkv[:, :8]
    cache = m.KVCache(c.k_pool, c.v_pool, c.table)
    ws = m.new_ops_workspace(cache)
    lens = [q_len] * 2, [q_len + 600, q_len + 77]
    first, l1 = run_attention(m, c, q, *lens, cache=cache, ws=ws)
    wide = torch.zeros(2 * q_len, 10, 136, dtype=BF16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        again, l2 = run_attention(m, c, q, *lens, cache=cache, ws=ws, out=wide[:, 1:9, :128])
    torch.cuda.current_stream().wait_stream(s)
    heads_first = torch.empty(8, 2 * q_len, 128, dtype=BF16, device="cuda").transpose(0, 1)
    third, l3 = run_attention(m, c, q.contiguous(), *lens, cache=cache, ws=ws, out=heads_first)
    assert torch.equal(first, again) and torch.equal(first, third)
    assert torch.equal(l1, l2) and torch.equal(l1, l3)
    assert (wide[:, 0] == 0).all() and (wide[:, 9] == 0).all() and (wide[:, :, 128:] == 0).all()


@pytest.mark.parametrize("q_len", [1, 40])
def test_attention_in_graphs_that_share_a_workspace(q_len):
    """Two captured graphs, replayed in turn with new contents and lengths, on one workspace."""
    m = sz()
    g = gen(12)
    c = P.build_cache(g, BF16, [900, 900], 16, 2, 128)
    cache = m.KVCache(c.k_pool, c.v_pool, c.table)
    ws = m.new_ops_workspace(cache)
    q = torch.randn(2 * q_len, 8, 128, generator=g).bfloat16().cuda()
    cu, kl = P.lengths([q_len] * 2, [900, 40])
    outs = [torch.zeros_like(q) for _ in range(2)]
    m.sz_attn_paged(cache, q, cu, kl, outs[0], ws)   # the first call sets the kernel up
    graphs = []
    for o in outs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            m.sz_attn_paged(cache, q, cu, kl, o, ws)
        graphs.append(graph)
    for lens in ([900, 40], [500, 900], [41, 850]):
        kl.copy_(torch.tensor(lens, dtype=torch.int32))
        for graph in graphs:
            graph.replay()
        ref, _ = run_attention(m, c, q, [q_len] * 2, lens)
        assert torch.equal(outs[0], ref) and torch.equal(outs[1], ref)
    assert m.sz_last_device_status(ws) == 0


def test_attention_errors_on_the_device():
    m = sz()
    g = gen(13)
    c = P.build_cache(g, BF16, [100, 60], 16, 2, 64)
    cache = m.KVCache(c.k_pool, c.v_pool, c.table)
    ws = m.new_ops_workspace(cache)
    for q_len in (1, 90):
        q = torch.randn(2 * q_len, 4, 64, generator=g).bfloat16().cuda()
        out = torch.zeros_like(q)
        cu, kl = P.lengths([q_len] * 2, [100, 60])
        m.sz_attn_paged(cache, q, cu, kl, out, ws)
        assert m.sz_last_device_status(ws) == 0
        good = out.clone()
        kl[1] = 10 ** 6                              # beyond the table
        m.sz_attn_paged(cache, q, cu, kl, out, ws)
        assert m.sz_last_device_status(ws) == m.SZ_ERR_INVALID_ARG
        kl[1] = 60
        for bad in (c.k_pool.shape[0], -1):
            keep = int(c.table[1, 1])
            c.table[1, 1] = bad
            m.sz_attn_paged(cache, q, cu, kl, out, ws)
            assert m.sz_last_device_status(ws) == m.SZ_ERR_INVALID_ARG
            assert torch.equal(out[:q_len], good[:q_len])
            c.table[1, 1] = keep
        m.sz_workspace_init(ws)
        m.sz_attn_paged(cache, q, cu, kl, out, ws)
        assert m.sz_last_device_status(ws) == 0 and torch.equal(out, good)


def test_attention_no_tokens_and_all_empty():
    m = sz()
    c = P.build_cache(gen(14), BF16, [20, 20], 16, 2, 64)
    q = torch.zeros(0, 4, 64, dtype=BF16, device="cuda")
    run_attention(m, c, q, [0, 0], [20, 20])
    q = torch.zeros(3, 4, 64, dtype=BF16, device="cuda")
    out, lse = run_attention(m, c, q, [0, 0], [20, 20])  # three padded rows
    assert (out == 7.0).all() and (lse == 7.0).all()


# ------------------------------------------------------------------ norm and rotation

@pytest.mark.parametrize("dim,rot,heads,kv_heads,tokens", [
    (16, 8, 1, 1, 1), (64, 64, 6, 2, 5), (80, 32, 32, 32, 3), (80, 40, 4, 4, 700), (128, 128, 64, 8, 33),
    (128, 0, 3, 1, 9), (112, 112, 5, 1, 4), (256, 64, 2, 1, 17), (192, 192, 3, 3, 900), (128, 128, 32, 8, 4000)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("normed", ["both", "k", "none"])
def test_norm_rope(dim, rot, heads, kv_heads, tokens, interleaved, normed):
    m = sz()
    g = gen(dim + rot + tokens)
    qkv = torch.randn(tokens, heads + kv_heads + 1, dim, generator=g).bfloat16()
    qkv[tokens // 2, 0] = 0                          # a head of zeros
    w = [(1 + 0.3 * torch.randn(dim, generator=g)).bfloat16() for _ in range(2)]
    qw, kw = (w[0] if normed == "both" else None), (None if normed == "none" else w[1])
    table = m.rope_table(131072, rot, device="cpu") if rot else None
    pos = torch.randint(0, 131072, (tokens,), generator=g)
    dev = qkv.cuda()
    q, k = dev[:, :heads], dev[:, heads: heads + kv_heads]
    q_out, k_out = torch.empty(tokens, heads, dim, dtype=BF16, device="cuda"), torch.empty_like(k)
    ws = m.new_ops_workspace()
    kw_ = dict(q_norm=None if qw is None else qw.cuda(), k_norm=None if kw is None else kw.cuda(), eps=1e-5,
               rope=None if table is None else table.cuda(), positions=pos.int().cuda() if rot else None,
               interleaved=interleaved)
    m.sz_qk_norm_rope(q, k, q_out, k_out, ws, **kw_)
    assert m.sz_last_device_status(ws) == 0
    for x, wt, out in ((qkv[:, :heads], qw, q_out), (qkv[:, heads: heads + kv_heads], kw, k_out)):
        n = P.norm(x, wt, 1e-5)
        ref = P.rotate(n, table, pos, interleaved)
        close(out, ref, P.rope_bound(ref, n, BF16), "rotated heads")
    # in place, and one of the two alone
    m.sz_qk_norm_rope(q, None, q, None, ws, **kw_)
    m.sz_qk_norm_rope(None, k, None, k, ws, **kw_)
    assert m.sz_last_device_status(ws) == 0
    assert torch.equal(q, q_out) and torch.equal(k, k_out)
    assert torch.equal(dev[:, -1].cpu(), qkv[:, -1])


def test_norm_rope_positions_outside_the_table():
    m = sz()
    q = torch.ones(4, 2, 64, dtype=BF16, device="cuda")
    out = torch.full_like(q, 7.0)
    ws = m.new_ops_workspace()
    pos = torch.tensor([0, 100, -1, 99], dtype=torch.int32, device="cuda")
    m.sz_qk_norm_rope(q, None, out, None, ws, rope=m.rope_table(100, 64), positions=pos)
    assert m.sz_last_device_status(ws) == m.SZ_ERR_INVALID_ARG
    assert (out[1:3] == 7.0).all() and (out[0] == 1.0).all() and (out[3] != 7.0).all()


# ------------------------------------------------------------------ append

@pytest.mark.parametrize("dtype", [BF16, E5M2])
@pytest.mark.parametrize("q_lens,before,heads,kv_heads,dim,rot,page,interleaved,normed,gap", [
    ([1], [0], 1, 1, 16, 16, 1, False, False, 0),
    ([1], [776], 32, 8, 128, 128, 16, False, False, 0),
    ([3, 0, 1, 20], [5, 7, 0, 13], 64, 8, 128, 128, 16, False, True, 64),
    ([1] * 70, list(range(70)), 4, 4, 80, 32, 13, False, False, 0),
    ([700, 40], [0, 300], 8, 2, 64, 64, 7, True, True, 0),
    ([500], [3], 32, 32, 80, 40, 13, True, False, 0),
    ([900, 300], [0, 4], 32, 8, 128, 128, 16, False, True, 0),
    ([11], [2], 2, 1, 256, 256, 100, False, True, 0),
])
def test_append(dtype, q_lens, before, heads, kv_heads, dim, rot, page, interleaved, normed, gap):
    m = sz()
    g = gen(len(q_lens) + dim + page)
    kv_lens = [a + b for a, b in zip(q_lens, before)]
    c = P.build_cache(g, dtype, before, page, kv_heads, dim, gap=gap, room=max(q_lens))
    tokens, tail = sum(q_lens), 2                    # two padded rows
    qkv = torch.randn(tokens + tail, heads + 2 * kv_heads, dim, generator=g).bfloat16() * 3
    w = [(1 + 0.3 * torch.randn(dim, generator=g)).bfloat16() if normed else None for _ in range(2)]
    table = m.rope_table(max(kv_lens), rot)
    cu, kl = P.lengths(q_lens, kv_lens)
    dev = qkv.cuda()
    q, k, v = dev[:, :heads], dev[:, heads: heads + kv_heads], dev[:, heads + kv_heads:]
    q_out = torch.full((tokens + tail, heads, dim), 7.0, dtype=BF16, device="cuda")
    cache = m.KVCache(c.k_pool, c.v_pool, c.table)
    ws = m.new_ops_workspace(cache)
    old = [x.clone() for x in (c.k_pool, c.v_pool)]
    kw = dict(q_norm=None if w[0] is None else w[0].cuda(), k_norm=None if w[1] is None else w[1].cuda(), rope=table,
              interleaved=interleaved)
    m.sz_kv_append_paged(cache, k, v, cu, kl, ws, q=q, q_out=q_out, **kw)
    assert m.sz_last_device_status(ws) == 0
    pos = torch.cat([torch.arange(b, n) for b, n in zip(before, kv_lens)])
    cols = (slice(0, heads), slice(heads, heads + kv_heads), slice(heads + kv_heads, None))
    nq, nk = P.norm(qkv[:tokens, cols[0]], w[0], 1e-6), P.norm(qkv[:tokens, cols[1]], w[1], 1e-6)
    rq, rk = (P.rotate(x, table.cpu(), pos, interleaved) for x in (nq, nk))
    close(q_out[:tokens], rq, P.rope_bound(rq, nq, BF16), "queries")
    assert (q_out[tokens:] == 7.0).all()
    # the tokens' places hold them, and nothing else changed
    seq = torch.cat([torch.full((n,), b) for b, n in enumerate(q_lens)]).long()
    pg, off = c.table.cpu()[seq, pos // page].long(), pos % page
    close(c.k_pool[pg, off], rk, P.rope_bound(rk, nk, dtype), "keys")
    assert torch.equal(c.v_pool[pg, off].cpu().float(), qkv[:tokens, cols[2]].to(dtype).float())
    for pool, was in zip((c.k_pool, c.v_pool), old):
        same = torch.ones(pool.shape[:2], dtype=torch.bool)
        same[pg, off] = False
        assert torch.equal(pool.view(torch.uint8).cpu()[same], was.view(torch.uint8).cpu()[same])
    # in place, without queries, with positions of one's own
    again = [torch.zeros_like(x) for x in old]
    cache2 = m.KVCache(again[0], again[1], c.table)
    m.sz_kv_append_paged(cache2, k, v, cu, kl, ws, positions=torch.cat([pos, pos[:1], pos[:1]]).int().cuda(), **kw)
    assert torch.equal(again[0][pg, off].view(torch.uint8), c.k_pool[pg, off].view(torch.uint8))
    m.sz_kv_append_paged(cache2, k, v, cu, kl, ws, q=q, **kw)
    assert torch.equal(q[:tokens], q_out[:tokens]) and torch.equal(q[tokens:].cpu(), qkv[tokens:, :heads])
    assert m.sz_last_device_status(ws) == 0


def test_append_e5m2_rounds_like_the_cast():
    """All bf16 values as values of V: ties to even, subnormals, infinity beyond the range, NaN."""
    m = sz()
    x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(BF16).view(512, 1, 128)
    pool = torch.zeros(2, 512, 1, 128, dtype=E5M2, device="cuda")
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    cache = m.KVCache(pool[:1], pool[1:], table)
    ws = m.new_ops_workspace(cache)
    cu, kl = P.lengths([512], [512])
    d = x.cuda()
    m.sz_kv_append_paged(cache, torch.zeros_like(d), d, cu, kl, ws)
    assert m.sz_last_device_status(ws) == 0
    got, ref = pool[1].cpu().float(), x.float().to(E5M2).float()
    assert torch.equal(torch.isnan(got), torch.isnan(ref))
    assert torch.equal(got.nan_to_num(0, 1e9, -1e9), ref.nan_to_num(0, 1e9, -1e9))


def test_append_leaves_out_what_has_no_place():
    m = sz()
    c = P.build_cache(gen(20), BF16, [32, 32], 16, 1, 64)
    c.k_pool.zero_(), c.v_pool.zero_()
    cache = m.KVCache(c.k_pool, c.v_pool, c.table)
    ws = m.new_ops_workspace(cache)
    k = torch.ones(4, 1, 64, dtype=BF16, device="cuda")
    # sequence 0 is shorter than its new tokens, sequence 1 longer than its table
    cu, kl = P.lengths([2, 2], [1, 33])
    m.sz_kv_append_paged(cache, k, k, cu, kl, ws)
    assert m.sz_last_device_status(ws) == m.SZ_ERR_INVALID_ARG
    want = torch.zeros(c.k_pool.shape[:2])
    want[int(c.table[0, 0]), 0] = 1
    want[int(c.table[1, 1]), 15] = 1
    assert torch.equal(c.k_pool[:, :, 0, 0].cpu().float(), want)
    # a page outside the pool
    c.k_pool.zero_()
    for bad in (c.k_pool.shape[0], -5):
        c.table[1, 1] = bad
        cu, kl = P.lengths([2, 2], [2, 32])
        m.sz_kv_append_paged(cache, k, k, cu, kl, ws)
        assert m.sz_last_device_status(ws) == m.SZ_ERR_INVALID_ARG
        want.zero_()
        want[int(c.table[0, 0]), :2] = 1
        assert torch.equal(c.k_pool[:, :, 0, 0].cpu().float(), want)


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("dtype", [BF16, E5M2])
def test_serving_run(dtype):
    """Prompts, then decoding steps: append and attend, with the cache coded, sent to another pool's pages
    and decoded there half-way; attention there gives the same bits."""
    m = sz()
    g = gen(30)
    heads, kv_heads, dim, page, steps = 8, 2, 64, 16, 4   # 16 * 2 * 64 elements to a page, as the codec wants
    prompts = [37, 5, 64]
    width = -(-(max(prompts) + steps) // page)
    pages = width * 3 + 1

    def pool():
        p = torch.zeros(2, pages, page, kv_heads, dim, dtype=dtype, device="cuda")
        t = torch.randperm(pages, generator=g)[: width * 3].int().view(3, width).cuda()
        return m.KVCache(p[0], p[1], t)

    a, b = pool(), pool()
    ws = m.new_ops_workspace(a)
    rope = m.rope_table(width * page, dim)
    w = (1 + 0.2 * torch.randn(dim, generator=g)).bfloat16()
    hist = [[] for _ in prompts]                     # every token's q, k, v as the layer made them
    kv = [0, 0, 0]
    cache = a
    for step in range(steps + 1):
        q_lens = prompts if step == 0 else [1, 1, 1]
        kv = [x + y for x, y in zip(kv, q_lens)]
        qkv = torch.randn(sum(q_lens), heads + 2 * kv_heads, dim, generator=g).bfloat16()
        at = 0
        for s, n in enumerate(q_lens):
            hist[s].append(qkv[at: at + n])
            at += n
        dev = qkv.cuda()
        cu, kl = P.lengths(q_lens, kv)
        q = torch.empty(sum(q_lens), heads, dim, dtype=BF16, device="cuda")
        m.sz_kv_append_paged(cache, dev[:, heads: heads + kv_heads], dev[:, heads + kv_heads:], cu, kl, ws,
                             q=dev[:, :heads], q_out=q, q_norm=w.cuda(), k_norm=w.cuda(), rope=rope)
        out = torch.empty_like(q)
        m.sz_attn_paged(cache, q, cu, kl, out, ws)
        if step == 2:                                # send the cache over, coded where it lies
            descs = [a.pages(s, kv[s]) for s in range(3)]
            dst = [b.pages(s, kv[s]) for s in range(3)]
            srcs = [d for pair, _ in descs for d in pair]
            dsts = [d for pair, _ in dst for d in pair]
            ns = [n for _, n in descs for _ in range(2)]
            cws = m.new_workspace(a.dtype, ns)
            plans = m.new_plans(6)
            bufs = [torch.empty(m.sz_max_compressed_size(a.dtype, n), dtype=torch.uint8, device="cuda") for n in ns]
            bat = m.Batch(a.dtype, None, bufs, cws, plans, src_pages=srcs, dst_pages=dsts, n=ns)
            bat.plan()
            bat.encode()
            bat.decode()
            assert m.sz_last_device_status(cws) == 0
            there = torch.empty_like(q)
            m.sz_attn_paged(b, q, cu, kl, there, ws)
            assert torch.equal(out, there)
            cache = b
        assert m.sz_last_device_status(ws) == 0
        at = 0
        for s, n in enumerate(q_lens):
            full = torch.cat(hist[s])
            pos = torch.arange(full.shape[0])
            k = P.rotate(P.norm(full[:, heads: heads + kv_heads], w, 1e-6), rope.cpu(), pos, False)
            qq = q[at: at + n].cpu()
            # the keys as the cache holds them: the attention's own bounds apply
            pg = cache.table.cpu()[s, pos // page].long()
            kk = cache.k_pool[pg, pos % page].cpu()
            close(kk, k, P.rope_bound(k, k, dtype) + 2.0 ** -17 * k.abs().amax(-1, keepdim=True), "keys in the cache")
            vv = cache.v_pool[pg, pos % page].cpu()
            ref, _, mag, reach = P.attention(qq, kk, vv)
            close(out[at: at + n], ref, P.attention_bound(ref, mag, reach, dtype == E5M2), "step %d" % step)
            at += n
