"""Giving up in sz_attn_paged's tensor-memory kernel: a copy of the library whose waits run out after as
little as nothing, on calls that are in order.  A CTA that gives up reports SZ_ERR_TIMEOUT, waits for its
copies and products under way, gives its tensor memory back and returns; nothing faults or hangs."""
import ctypes
import os

import pytest
import torch

import __graft_entry__
import paged_ops as P
from gpu_helpers import sz
from test_gpu_paged_ops import BF16, E5M2, gen, run_attention

pytestmark = pytest.mark.gpu

ENTRIES = ("sz_kv_append_paged", "sz_qk_norm_rope", "sz_attn_paged")


def addresses(lib):
    return [ctypes.cast(getattr(lib, f), ctypes.c_void_p).value for f in ENTRIES]


@pytest.fixture(scope="module")
def copy(tmp_path_factory):
    """The operators with a limit that the environment gives, a look at the clock at every poll, and polls
    that do not suspend the thread."""
    folder = tmp_path_factory.mktemp("lib")
    limits = folder / "limits.h"
    limits.write_text('#include <cstdlib>\n#define SZ_ATTN_POLLS 1\n'
                      '#define SZ_ATTN_WAIT_NS strtoull(getenv("SZ_ATTN_WAIT_NS"), nullptr, 10)\n')
    out = str(folder / "limits.so")
    __graft_entry__._build_module().build(force=True, out=out, extra_flags=["-include", str(limits)],
                                          files=["sz_ops.cu", "sz_rope.cu", "sz_attn.cu", "sz_attn_tc.cu"])
    return ctypes.CDLL(out)


@pytest.fixture
def limited(copy, monkeypatch):
    """Attention calls go to the copy; returns what sets its limit in ns."""
    m = sz()
    assert m._host.bind(*addresses(copy)) == 0
    yield lambda ns: monkeypatch.setitem(os.environ, "SZ_ATTN_WAIT_NS", str(ns))
    torch.cuda.synchronize()
    assert m._host.bind(*addresses(m.lib)) == 0


@pytest.mark.parametrize("dtype", [BF16, E5M2])
@pytest.mark.parametrize("heads,kv_heads,dim,page", [
    (8, 2, 128, 16),      # keys, values and queries by tensor copies
    (8, 2, 128, 13),      # keys and values row by row
    (6, 2, 64, 64),       # queries row by row
])
def test_waits_that_run_out(limited, dtype, heads, kv_heads, dim, page):
    m, g = sz(), gen(31)
    lens = [300, 70, 45], [3000, 70, 2000]
    c = P.build_cache(g, dtype, lens[1], page, kv_heads, dim)
    cache = m.KVCache(c.k_pool, c.v_pool, c.table)
    q = torch.randn(sum(lens[0]), heads, dim, generator=g).bfloat16().cuda()
    cu, kl = P.lengths(*lens)
    ws = m.new_ops_workspace(cache)
    limited(2 * 10 ** 9)
    want, want_lse = run_attention(m, c, q, *lens, cache=cache, ws=ws)
    seen = set()
    for ns in (0, 200, 500, 1000, 1500, 2000, 3000, 5000, 10000):
        for _ in range(3):
            limited(ns)
            out = torch.empty_like(q)
            m.sz_attn_paged(cache, q, cu, kl, out, ws)
            status = m.sz_last_device_status(ws)
            assert status in (0, m.SZ_ERR_TIMEOUT)
            assert status == m.SZ_ERR_TIMEOUT or torch.equal(out, want)
            if ns == 0:
                assert status == m.SZ_ERR_TIMEOUT
            seen.add(status)
            # the workspace anew, and the same call gives the bits that it gave
            m.sz_workspace_init(ws)
            limited(2 * 10 ** 9)
            out, lse = run_attention(m, c, q, *lens, cache=cache, ws=ws)
            assert torch.equal(out, want) and torch.equal(lse, want_lse)
    assert m.SZ_ERR_TIMEOUT in seen
