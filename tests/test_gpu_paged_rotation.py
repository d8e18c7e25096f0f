"""Norm and rotation where inputs and outputs are views of one buffer, and to the last bit, on the GPU."""
import pytest
import torch

import paged_ops as P
from gpu_helpers import sz
from test_gpu_paged_ops import BF16, E5M2, gen

pytestmark = pytest.mark.gpu


def split(layout, tokens, heads, dim, g):
    """A projection's output and its queries, keys and values: behind one another in a token, side by side for
    each head, or a matrix for each head."""
    if layout == "columns":
        x = torch.randn(tokens, 3 * heads, dim, generator=g).bfloat16().cuda()
        return x, x[:, :heads], x[:, heads: 2 * heads], x[:, 2 * heads:]
    if layout == "each head":
        x = torch.randn(tokens, heads, 3, dim, generator=g).bfloat16().cuda()
        return x, x[:, :, 0], x[:, :, 1], x[:, :, 2]
    x = torch.randn(3 * heads, tokens, dim, generator=g).bfloat16().cuda()
    y = x.transpose(0, 1)
    return x, y[:, :heads], y[:, heads: 2 * heads], y[:, 2 * heads:]


@pytest.mark.parametrize("layout", ["columns", "each head", "heads first"])
@pytest.mark.parametrize("tokens,heads,dim,rot", [(1, 4, 64, 64), (37, 3, 80, 40), (600, 8, 128, 128)])
def test_queries_and_keys_in_place_together(layout, tokens, heads, dim, rot):
    """One call, both in place: the bits of a call that writes elsewhere, and the values left alone."""
    m, g = sz(), gen(61)
    x, q, k, v = split(layout, tokens, heads, dim, g)
    v0 = v.clone()
    w = (1 + 0.2 * torch.randn(dim, generator=g)).bfloat16().cuda()
    ws = m.new_ops_workspace()
    kw = dict(q_norm=w, k_norm=w, rope=m.rope_table(1000, rot),
              positions=torch.randint(0, 1000, (tokens,), generator=g).int().cuda())
    q_out, k_out = (torch.empty(tokens, heads, dim, dtype=BF16, device="cuda") for _ in range(2))
    m.sz_qk_norm_rope(q, k, q_out, k_out, ws, **kw)
    m.sz_qk_norm_rope(q, k, q, k, ws, **kw)
    assert m.sz_last_device_status(ws) == 0
    assert torch.equal(q, q_out) and torch.equal(k, k_out) and torch.equal(v, v0)


@pytest.mark.parametrize("layout", ["columns", "each head", "heads first"])
def test_appending_beside_queries_in_place(layout):
    m, g = sz(), gen(62)
    tokens, heads, dim = 50, 4, 64
    x, q, k, v = split(layout, tokens, heads, dim, g)
    c = P.build_cache(g, BF16, [0], 16, heads, dim, room=64)
    cache = m.KVCache(c.k_pool, c.v_pool, c.table)
    ws = m.new_ops_workspace(cache)
    cu, kl = P.lengths([tokens], [tokens])
    kw = dict(rope=m.rope_table(64, dim))
    q_out = torch.empty(tokens, heads, dim, dtype=BF16, device="cuda")
    m.sz_kv_append_paged(cache, k, v, cu, kl, ws, q=q, q_out=q_out, **kw)
    keys = c.k_pool.clone()
    m.sz_kv_append_paged(cache, k, v, cu, kl, ws, q=q, **kw)
    assert m.sz_last_device_status(ws) == 0
    assert torch.equal(q, q_out) and torch.equal(c.k_pool.view(torch.int16), keys.view(torch.int16))


def test_columns_that_meet_are_refused():
    m = sz()
    x = torch.zeros(5, 12, 64, dtype=BF16, device="cuda")
    ws = m.new_ops_workspace()
    m.sz_qk_norm_rope(x[:, :4], x[:, 4:6], x[:, :4], x[:, 4:6], ws)
    for a, b in ((x[:, :4], x[:, 3:5]), (x[:, 2:4], x[:, :3])):
        with pytest.raises(m.SplitZipError):
            m.sz_qk_norm_rope(a, b, a, b, ws)
    each = x.view(5, 4, 3, 64)
    with pytest.raises(m.SplitZipError):
        m.sz_qk_norm_rope(each[:, :, 0], each[:, 1:, 0], each[:, :, 0], each[:, 1:, 0], ws)


def at_borders(tokens, dim, rot, interleaved, dtype, g):
    """Keys [tokens, 1, dim] and a table such that a cos - b sin of every pair is as near as 32 bits allow to the
    middle between two neighbours of the output's type."""
    bits = {BF16: 7, E5M2: 2}[dtype]
    x = (torch.randn(tokens, dim, generator=g) + 0.01).bfloat16()
    half = rot // 2
    a, b = ((x[:, 0:rot:2], x[:, 1:rot:2]) if interleaved else (x[:, :half], x[:, half:rot]))
    a, b = a.float(), b.float()
    odd = 2 * torch.randint(0, 1 << bits, (tokens, half), generator=g) + 1
    middle = (1 + odd / 2.0 ** (bits + 1)) * 2.0 ** torch.randint(-3, 4, (tokens, half), generator=g)
    sin = torch.rand(tokens, half, generator=g) * 2 - 1
    cos = ((middle.double() + b.double() * sin.double()) / a.double()).float()
    return x.view(tokens, 1, dim), torch.cat([cos, sin], 1)


def turned(x, table, rot, interleaved, fused=False):
    """The rotation in 32 bits, each product and sum rounded by itself, or the products of cosines not."""
    x = x[:, 0].float()
    half = rot // 2
    a, b = (x[:, 0:rot:2], x[:, 1:rot:2]) if interleaved else (x[:, :half], x[:, half:rot])
    cos, sin = table[:, :half], table[:, half:]
    if fused:
        u = (a.double() * cos.double() - (b * sin).double()).float()
        v = (b.double() * cos.double() + (a * sin).double()).float()
    else:
        u, v = a * cos - b * sin, b * cos + a * sin
    out = x.clone()
    if interleaved:
        out[:, 0:rot:2], out[:, 1:rot:2] = u, v
    else:
        out[:, :half], out[:, half:rot] = u, v
    return out


@pytest.mark.parametrize("dtype", [BF16, E5M2])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens,dim,rot", [(40, 128, 128), (700, 64, 32), (33, 80, 40), (3000, 128, 120)])
def test_the_rotation_rounds_each_step_by_itself(dtype, interleaved, tokens, dim, rot):
    """Keys at the borders of the cache's type: the bits of the formula in 32 bits, which products that are not
    rounded before they are added would miss."""
    m, g = sz(), gen(63)
    x, table = at_borders(tokens, dim, rot, interleaved, dtype, g)
    want = turned(x, table, rot, interleaved).to(dtype)
    raw = torch.int16 if dtype == BF16 else torch.uint8
    other = turned(x, table, rot, interleaved, fused=True).to(dtype)
    assert (want.view(raw) != other.view(raw)).sum() > tokens * rot // 100
    c = P.build_cache(g, dtype, [0], 16, 1, dim, room=tokens)
    cache = m.KVCache(c.k_pool, c.v_pool, c.table)
    ws = m.new_ops_workspace(cache)
    cu, kl = P.lengths([tokens], [tokens])
    k = x.cuda()
    m.sz_kv_append_paged(cache, k, k, cu, kl, ws, rope=table.cuda(), interleaved=interleaved)
    assert m.sz_last_device_status(ws) == 0
    pos = torch.arange(tokens)
    got = c.k_pool.cpu()[c.table.cpu()[0, pos // 16].long(), pos % 16][:, 0]
    assert torch.equal(got.contiguous().view(raw), want.view(raw))
