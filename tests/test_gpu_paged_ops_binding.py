"""The Python binding of the operators on a paged cache on the GPU: threads and streams."""
import ctypes
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
