"""The Python binding of the operators on a paged cache on the GPU: threads and streams."""
import ctypes
import gc
import threading
import time

import pytest
import torch

import paged_ops as P
from gpu_helpers import sz
from test_gpu_paged_ops import BF16, gen

pytestmark = pytest.mark.gpu


def test_other_threads_run_during_a_call():
    """In place of the library's entry point libc's nanosleep: the argument struct begins with the number of
    tokens (its seconds) and the absent queries' address (its nanoseconds)."""
    m = sz()
    k = torch.zeros(1, 2, 64, dtype=BF16, device="cuda")
    ws = m.new_ops_workspace()
    m.sz_qk_norm_rope(None, k, None, k, ws)
    entries = [ctypes.cast(f, ctypes.c_void_p).value for f in (
        m.lib.sz_kv_append_paged, m.lib.sz_qk_norm_rope, m.lib.sz_attn_paged)]
    sleeps = ctypes.cast(ctypes.CDLL(None).nanosleep, ctypes.c_void_p).value
    ticks, stop = [], threading.Event()

    def run():
        while not stop.is_set():
            ticks.append(time.monotonic())
            time.sleep(0.01)

    other = threading.Thread(target=run)
    other.start()
    try:
        assert m._host.bind(entries[0], sleeps, entries[2]) == 0
        begin = time.monotonic()
        m.sz_qk_norm_rope(None, k, None, k, ws)
        end = time.monotonic()
    finally:
        assert m._host.bind(*entries) == 0
        stop.set()
        other.join()
    assert end - begin > 0.9
    assert sum(begin + 0.1 < t < end - 0.1 for t in ticks) > 20


@pytest.mark.parametrize("operators", [True, False])
def test_a_workspace_zeroed_on_another_stream(operators):
    """Memory that work of the current stream still writes to is zeroed behind that work."""
    m = sz()
    c = P.build_cache(gen(51), BF16, [40], 16, 2, 64)
    cache = m.KVCache(c.k_pool, c.v_pool, c.table)
    ns = [1 << 24] * 4
    s = torch.cuda.Stream()
    n = m.sz_ops_workspace_bytes(cache) if operators else m.sz_workspace_bytes_batched(m.SZ_BF16, ns)
    gc.collect()
    torch.cuda.empty_cache()                         # (no other block of this size to hand out)
    old = torch.empty(n, dtype=torch.uint8, device="cuda")
    address = old.data_ptr()
    old.fill_(1), m.new_ops_workspace(stream=s)      # (first calls wait for the device)
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)                   # some 50 ms
    old.fill_(255)
    del old
    ws = m.new_ops_workspace(cache, stream=s) if operators else m.new_workspace(m.SZ_BF16, ns, stream=s)
    assert ws.data_ptr() == address
    torch.cuda.synchronize()
    assert not ws.any()
