"""Other threads of the interpreter go on while a call of the binding is in the
library, as they do for every call through ctypes: a launch waits where a
stream's queue is full.  The library's place is taken by a function that waits
for another thread, for two seconds at most; nothing reaches the GPU."""
import ctypes
import subprocess
import threading
import time

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda"
SOURCE = r"""
#include <unistd.h>
volatile int go;
int entered(void) {
  for (int i = 0; i < 2000; ++i) {
    if (go) return 0;
    usleep(1000);
  }
  return 4;
}
"""


@pytest.mark.parametrize("name", ["rope", "store", "load", "attn"])
def test_other_threads_go_on_during_a_call(tmp_path, name):
    assert torch.cuda.is_available(), "needs the MI355X"
    from ternary_packed_weight_amd import _tq2call, tq2
    (tmp_path / "w.c").write_text(SOURCE)
    subprocess.run(["gcc", "-O1", "-shared", "-fPIC", str(tmp_path / "w.c"), "-o", str(tmp_path / "w.so")], check=True)
    lib = ctypes.CDLL(str(tmp_path / "w.so"))
    wait = ctypes.cast(lib.entered, ctypes.c_void_p).value
    real = [ctypes.cast(getattr(tq2.lib(), f), ctypes.c_void_p).value for f in (
        "tq2_qk_norm_rope", "tq2_kv4_store", "tq2_kv4_load", "tq2_kv4_attn", "tq2_kv4_attn_workspace_bytes")]
    h = torch.zeros((2, 2, 64), device=DEV, dtype=torch.float16)
    o = [torch.empty_like(h) for _ in range(2)]
    pos, inv = torch.zeros(2, dtype=torch.int32, device=DEV), torch.zeros(32, device=DEV)
    slots, table = torch.zeros(2, dtype=torch.int64, device=DEV), torch.zeros((2, 1), dtype=torch.int32, device=DEV)
    cache = torch.zeros((1, 2, 32 * 72), dtype=torch.uint8, device=DEV)
    calls = {"rope": lambda: tq2.tq2_qk_norm_rope(h, h, pos, inv, q_out=o[0], k_out=o[1]),
             "store": lambda: tq2.tq2_kv4_store(cache, h, h, slots),
             "load": lambda: tq2.tq2_kv4_load(cache, slots, 64, k_out=o[0], v_out=o[1]),
             "attn": lambda: tq2.tq2_kv4_attn(h, cache, table, pos, out=o[0])}
    started = threading.Event()

    def other():
        started.wait()
        time.sleep(0.2)          # the call is in the library by then
        ctypes.c_int.in_dll(lib, "go").value = 1

    thread = threading.Thread(target=other)
    thread.start()
    _tq2call.bind(wait, wait, wait, wait, real[4])
    try:
        started.set()
        calls[name]()            # raises on the status of a wait that nobody ended
    finally:
        _tq2call.bind(*real)
        thread.join()
