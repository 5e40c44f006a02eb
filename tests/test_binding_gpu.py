"""The extension that calls the large products: what it does around the library's functions."""
import ctypes
import subprocess
import threading

import pytest
import torch

import segmented_gather_gemm_expand_b200 as sg
from segmented_gather_gemm_expand_b200 import _abi

pytestmark = pytest.mark.gpu

STAND_IN = r"""
#include <time.h>
static volatile int entered, go;
/* in the place of an entry point: returns 0 once another thread has called let_go, -99 after five seconds */
int stand_in(void) {
    entered = 1;
    for (int i = 0; i < 5000 && !go; ++i) { struct timespec t = {0, 1000000}; nanosleep(&t, 0); }
    return go ? 0 : -99;
}
int has_entered(void) { return entered; }
void let_go(void) { go = 1; }
"""


@pytest.mark.parametrize("entry", ["lora_linear", "grouped_gemm", "grouped_wgrad"])
def test_other_python_threads_run_during_a_call(entry, tmp_path):
    """A call that waits inside the library (a full launch queue) does not hold Python's lock."""
    (tmp_path / "s.c").write_text(STAND_IN)
    subprocess.run(["gcc", "-O1", "-shared", "-fPIC", "-o", str(tmp_path / "s.so"), str(tmp_path / "s.c")], check=True)
    c = ctypes.CDLL(str(tmp_path / "s.so"))
    lib = _abi.load()
    binding = _abi.load_binding(lib)
    x, w = torch.zeros(4, 8, device="cuda").bfloat16(), torch.zeros(2, 8, 8, device="cuda").bfloat16()
    m = [torch.zeros(2, dtype=torch.int32, device="cuda")] * 3
    args = {"lora_linear": (x, w[0], None, w, w, x, *m, 2, 4, None), "grouped_gemm": (x, w, x, *m, 2, 4, False),
            "grouped_wgrad": (x, x, w, *m, 2, 4, False)}[entry]
    got = []
    address = ctypes.cast(c.stand_in, ctypes.c_void_p).value
    binding.init(address, address, address)
    try:
        t = threading.Thread(target=lambda: got.append(getattr(binding, entry)(*args)))
        t.start()
        while t.is_alive() and not c.has_entered():
            pass
        c.let_go()
        t.join()
    finally:
        _abi.load_binding(lib)
    assert got == [0]
    sg.sgmv_grouped_gemm(x, w, x.clone(), *m, 2, 4)
