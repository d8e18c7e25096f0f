"""What the operators on a paged cache refuse on the host, before anything is launched: through the C ABI
with addresses that nothing reads, and through the binding (no GPU needed)."""
import ctypes
import struct

import pytest
import torch

import fp8_kv_cache_exp_b200 as sz

A = 1 << 20                       # an aligned address; a refused call touches none
CACHE = struct.Struct("@3Q2Q8I")
HEADS = struct.Struct("@3Q2I")
NORM = struct.Struct("@2QfI")
ROPE = struct.Struct("@2Q4I")


def cache(k=A, v=A, table=A, pages=10, page_bytes=16 * 2 * 64 * 2, stride=4, width=4, seqs=2, tokens=16, heads=2, dim=64,
          dtype=sz.SZ_BF16):
    return CACHE.pack(k, v, table, pages, page_bytes, stride, width, seqs, tokens, heads, dim, dtype, 0)


def heads(data=A, ts=4 * 64, hs=64, n=4):
    return HEADS.pack(data, ts, hs, n, 0)


def norm(q=0, k=0, eps=1e-6):
    return NORM.pack(q, k, eps, 0)


def rope(table=0, positions=0, n=100, rot=64, interleaved=0):
    return ROPE.pack(table, positions, n, rot, interleaved, 0)


Q, OUT = heads(), heads(data=A + (1 << 24))
KV = heads(ts=2 * 64, n=2)
NONE = HEADS.pack(0, 0, 0, 0, 0)
WS = 1 << 30


def attn(c=None, tokens=3, q=Q, out=OUT, cu_q=A, kv_len=A, lse=0, scale=0.125, window=0, ws=A, ws_bytes=WS):
    args = struct.pack("@Q", tokens) + q + out + struct.pack("@3Qf3I", cu_q, kv_len, lse, scale, 1, window, 0)
    return sz.lib.sz_attn_paged(cache() if c is None else c, args, ws, ws_bytes, None)


def append(c=None, tokens=3, k=KV, v=KV, q=NONE, q_out=NONE, cu_q=A, kv_len=A, n=norm(), r=rope(), ws=A, ws_bytes=WS):
    args = struct.pack("@Q", tokens) + k + v + q + q_out + struct.pack("@2Q", cu_q, kv_len) + n + r
    return sz.lib.sz_kv_append_paged(cache() if c is None else c, args, ws, ws_bytes, None)


def norm_rope(tokens=3, q=Q, q_out=OUT, k=NONE, k_out=NONE, n=norm(), r=rope(), dim=64, ws=A, ws_bytes=WS):
    args = struct.pack("@Q", tokens) + q + q_out + k + k_out + n + r + struct.pack("@2I", dim, 0)
    return sz.lib.sz_qk_norm_rope(args, ws, ws_bytes, None)


BAD_CACHES = [dict(k=0), dict(v=0), dict(table=0), dict(k=A + 8), dict(v=A + 2), dict(table=A + 2), dict(pages=0),
              dict(page_bytes=16 * 2 * 64 * 2 - 16), dict(page_bytes=16 * 2 * 64 * 2 + 8), dict(page_bytes=1 << 41),
              dict(stride=3), dict(width=0), dict(width=1 << 27, stride=1 << 27), dict(seqs=0), dict(seqs=65537),
              dict(tokens=0), dict(tokens=(1 << 20) + 1), dict(heads=0), dict(heads=4097), dict(dim=0), dict(dim=24),
              dict(dim=272)]


@pytest.mark.parametrize("bad", BAD_CACHES)
def test_caches(bad):
    c = cache(**bad)
    assert attn(c) == append(c) == sz.SZ_ERR_INVALID_ARG
    assert sz.lib.sz_ops_workspace_bytes(c) == 0


def test_cache_dtype_and_no_cache():
    assert attn(cache(dtype=7)) == append(cache(dtype=7)) == sz.SZ_ERR_UNSUPPORTED_DTYPE
    assert sz.lib.sz_attn_paged(None, None, A, WS, None) == sz.SZ_ERR_INVALID_ARG
    assert sz.lib.sz_attn_paged(cache(), None, A, WS, None) == sz.SZ_ERR_INVALID_ARG
    assert sz.lib.sz_kv_append_paged(cache(), None, A, WS, None) == sz.SZ_ERR_INVALID_ARG
    assert sz.lib.sz_qk_norm_rope(None, A, WS, None) == sz.SZ_ERR_INVALID_ARG


def test_workspaces():
    need = sz.lib.sz_ops_workspace_bytes(cache())
    assert need > 0 and attn(ws_bytes=need - 1) == sz.SZ_ERR_BUFFER_TOO_SMALL
    assert append(ws_bytes=255) == norm_rope(ws_bytes=255) == sz.SZ_ERR_BUFFER_TOO_SMALL
    for call in (attn, append, norm_rope):
        assert call(ws=0) == call(ws=A + 4) == sz.SZ_ERR_INVALID_ARG
    assert sz.lib.sz_ops_workspace_bytes(None) == 256


def test_no_tokens_is_no_work():
    assert attn(tokens=0) == append(tokens=0) == norm_rope(tokens=0) == sz.SZ_OK


@pytest.mark.parametrize("bad", [
    dict(tokens=1 << 31), dict(tokens=1 << 30), dict(q=heads(data=0)), dict(q=heads(data=A + 8)), dict(q=heads(ts=4)),
    dict(q=heads(hs=65)), dict(q=heads(n=0)), dict(q=heads(n=3), out=heads(data=A + (1 << 24), n=3)),
    dict(out=heads(data=A + (1 << 24), n=2)), dict(out=heads(data=A + (1 << 24), ts=64)),
    dict(out=heads(data=A + (1 << 24), ts=0)), dict(out=heads(data=A + (1 << 24), hs=32)), dict(out=Q),
    dict(out=heads(data=A + 2 * 64)), dict(cu_q=0), dict(cu_q=A + 2), dict(kv_len=0), dict(kv_len=A + 1), dict(lse=A + 2),
    dict(scale=0.0), dict(scale=-1.0), dict(scale=float("inf")), dict(scale=float("nan")), dict(window=1 << 31)])
def test_attention(bad):
    assert attn(**bad) == sz.SZ_ERR_INVALID_ARG


WIDE = dict(q=heads(data=A + (1 << 25)), q_out=OUT)


@pytest.mark.parametrize("bad", [
    dict(tokens=1 << 31), dict(k=heads(n=4)), dict(v=heads(n=1)), dict(k=heads(data=0, n=2)), dict(v=heads(data=A + 4, n=2)),
    dict(q=Q), dict(q_out=OUT), dict(WIDE, q_out=heads(data=A + (1 << 24), n=3)),
    dict(WIDE, q_out=heads(data=A + (1 << 24), ts=8)), dict(WIDE, q_out=heads(data=A + (1 << 25) + 16)),
    dict(WIDE, q_out=heads(data=A)), dict(cu_q=0), dict(kv_len=0), dict(kv_len=A + 3), dict(n=norm(q=A + 8)),
    dict(n=norm(k=A + 2)), dict(n=norm(k=A, eps=-1.0)), dict(n=norm(k=A, eps=float("nan"))),
    dict(n=norm(k=A, eps=float("inf"))), dict(r=rope(table=A + 4)), dict(r=rope(table=A, positions=A + 2)),
    dict(r=rope(table=A, rot=0)), dict(r=rope(table=A, rot=12)), dict(r=rope(table=A, rot=72)), dict(r=rope(table=A, n=0)),
    dict(r=rope(table=A, n=1 << 31))])
def test_append(bad):
    assert append(**bad) == sz.SZ_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [
    dict(tokens=1 << 31), dict(dim=8), dict(dim=40), dict(dim=512), dict(q=NONE, q_out=NONE), dict(q_out=NONE),
    dict(k=KV), dict(k_out=KV), dict(q_out=heads(data=A + (1 << 24), n=2)), dict(q_out=heads(data=A + 16)),
    dict(k=heads(data=A + (1 << 26)), k_out=OUT), dict(k=OUT, k_out=heads(data=A + (1 << 26))),
    dict(r=rope(table=A)), dict(r=rope(table=A, positions=A, rot=128)), dict(n=norm(q=A + 4))])
def test_norm_rope(bad):
    assert norm_rope(**bad) == sz.SZ_ERR_INVALID_ARG


def test_the_columns_of_one_buffer_do_not_overlap():
    """Queries and keys in place, as columns of the projection's output: accepted up to the check that follows."""
    q, k = heads(ts=8 * 64, n=4), heads(data=A + 2 * 4 * 64, ts=8 * 64, n=2)
    assert norm_rope(q=q, q_out=q, k=k, k_out=k, r=rope(table=A)) == sz.SZ_ERR_INVALID_ARG     # (no positions)
    assert norm_rope(tokens=0, q=q, q_out=q, k=k, k_out=k) == sz.SZ_OK


# ------------------------------------------------------------------ the binding

def small(dtype=torch.bfloat16, pages=4):
    k = torch.zeros(pages, 16, 2, 64).to(dtype)
    return sz.KVCache(k, k.clone(), torch.zeros(1, 4, dtype=torch.int32))


def test_cache_tensors():
    k, t = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16), torch.zeros(1, 4, dtype=torch.int32)
    for bad in (lambda: sz.KVCache(k, k[:2], t), lambda: sz.KVCache(k[0], k[0], t), lambda: sz.KVCache(k, k, t[0]),
                lambda: sz.KVCache(k.transpose(1, 2), k.transpose(1, 2), t), lambda: sz.KVCache(k[:0], k[:0], t),
                lambda: sz.KVCache(k, torch.zeros(8, 16, 2, 64, dtype=torch.bfloat16)[::2], t),
                lambda: sz.KVCache(k, k, torch.zeros(4, 2, dtype=torch.int32).t())):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: sz.KVCache(k.float(), k.float(), t), lambda: sz.KVCache(k, k, t.long())):
        with pytest.raises(TypeError):
            bad()


def test_tensors_of_another_device_and_of_none():
    """Host tensors are refused before their addresses go anywhere; so is what is not a tensor."""
    c = small()
    q, i, ws = torch.zeros(1, 4, 64, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32), torch.zeros(1 << 20, dtype=torch.uint8)
    kv = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    calls = [lambda x: sz.sz_attn_paged(c, x, i, i, q, ws), lambda x: sz.sz_kv_append_paged(c, x, kv, i, i, ws),
             lambda x: sz.sz_qk_norm_rope(x, None, q, None, ws)]
    for call in calls:
        with pytest.raises(ValueError):
            call(q)
        for junk in (3, "q", [1.0]):
            with pytest.raises(TypeError):
                call(junk)
    with pytest.raises(ValueError):
        sz.sz_qk_norm_rope(None, None, None, None, ws)
    with pytest.raises(AttributeError):
        sz.sz_attn_paged(None, q, i, i, q, ws)
    with pytest.raises(sz.SplitZipError):
        bad = small()
        bad._c = cache(dim=24)
        sz.new_ops_workspace(bad)


def test_workspace_grows_with_the_head():
    sizes = [sz.lib.sz_ops_workspace_bytes(cache(dim=d, page_bytes=16 * 2 * d * 2)) for d in (16, 64, 128, 256)]
    assert sizes == sorted(sizes) and sizes[0] > 256
    assert isinstance(ctypes.c_size_t(sizes[-1]).value, int)
