"""The Python binding of the operators on a paged cache: what it loads, and when (no GPU needed)."""
import os
import subprocess
import sys

import pytest
import torch

import __graft_entry__
import fp8_kv_cache_exp_b200 as sz

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

OTHER_TORCH = """
import torch
torch.__version__ = "0.0.other"
import fp8_kv_cache_exp_b200 as sz
assert sz.sz_max_compressed_size(0, 4096) > 0
k = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
cache = sz.KVCache(k, k.clone(), torch.zeros(1, 4, dtype=torch.int32))
q, i, ws = k[0, :1, :2], torch.zeros(2, dtype=torch.int32), torch.zeros(1 << 20, dtype=torch.uint8)
for _ in range(2):
    try:
        sz.sz_attn_paged(cache, q, i, i, q, ws)
    except ImportError as e:
        assert "build.py" in str(e)
    else:
        raise AssertionError("loaded")
"""


def test_a_module_built_for_another_torch_is_not_loaded():
    """The codec works without it; an operator's call says what is missing."""
    subprocess.run([sys.executable, "-c", OTHER_TORCH], cwd=ROOT, check=True)


def test_a_module_for_another_torch_is_not_up_to_date(monkeypatch):
    b = __graft_entry__._build_module()
    b.build()
    assert b.host_up_to_date()
    monkeypatch.setattr(torch, "__version__", "0.0.other")
    assert not b.host_up_to_date()


def test_the_library_comes_before_the_module(monkeypatch):
    """Where the module cannot be built the library is there all the same."""
    b = __graft_entry__._build_module()
    done = []
    monkeypatch.setattr(b, "up_to_date", lambda: False)
    monkeypatch.setattr(b, "build_library", lambda *a: done.append("library"))

    def fails(*a):
        raise RuntimeError("no headers")

    monkeypatch.setattr(b, "build_host", fails)
    with pytest.raises(RuntimeError):
        b.build()
    assert done == ["library"]


def test_the_module_is_loaded_once():
    assert sz._host.append is sz._host.append
    assert type(sz._host).__name__ == "module"


def cache(page, heads, dim, seqs=2, width=4):
    k = torch.zeros(6, page, heads, dim, dtype=torch.bfloat16)
    return sz.KVCache(k, k.clone(), torch.zeros(seqs, width, dtype=torch.int32))


@pytest.mark.parametrize("page,heads,dim", [(13, 4, 128), (13, 32, 80), (1, 1, 16), (1 << 12, 1, 128)])
def test_pages_that_the_codec_does_not_take_are_refused(page, heads, dim):
    c = cache(page, heads, dim)
    assert sz.sz_ops_workspace_bytes(c) > 0          # (the operators do)
    with pytest.raises(ValueError, match="1024"):
        c.pages(0, 1)


def test_descriptors_of_a_sequences_pages():
    c = cache(16, 2, 64)
    (k, v), n = c.pages(1, 50)
    assert n == 50 * 128 and k.page_elems == v.page_elems == 2048 and k.pool_pages == 6
    assert k.pages == c.table[1].data_ptr() and k.pool == c.k_pool.data_ptr() and v.pool == c.v_pool.data_ptr()
    assert c.pages(0, 64)[1] == 64 * 128 and c.pages(0, 0)[1] == 0
    for tokens in (65, -1):
        with pytest.raises(ValueError):
            c.pages(0, tokens)


def test_a_timeout_is_not_only_the_codecs():
    assert "look-back" not in sz.sz_status_string(sz.SZ_ERR_TIMEOUT) and "limit" in sz.sz_status_string(sz.SZ_ERR_TIMEOUT)
