"""The compiled calls run without the interpreter's lock: another Python thread goes on while a launch waits."""
import ctypes
import shutil
import subprocess
import threading
import time

import pytest
import torch

pytestmark = pytest.mark.gpu

# Stands in for an entry point: its arguments are left alone, it takes 0.3 s and says that all is well.
SOURCE = r"""
#include <time.h>
int slow(void) {
    struct timespec t = {0, 300000000};
    nanosleep(&t, 0);
    return 0;
}
"""


@pytest.fixture(scope="module")
def vh():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import verify_head_gb300 as vh
    vh.build()
    return vh


def test_another_thread_goes_on(vh, tmp_path):
    cc = shutil.which("gcc")
    m = vh._compiled_calls()
    if not cc or not m:
        pytest.skip("no C compiler or no compiled calls")
    (tmp_path / "s.c").write_text(SOURCE)
    subprocess.run([cc, "-shared", "-fPIC", str(tmp_path / "s.c"), "-o", str(tmp_path / "s.so")], check=True)
    slow = ctypes.cast(ctypes.CDLL(str(tmp_path / "s.so")).slow, ctypes.c_void_p).value

    R, V, H = 2, 64, 64
    x = torch.zeros(R, H, dtype=torch.bfloat16, device="cuda")
    W = torch.zeros(V, H, dtype=torch.bfloat16, device="cuda")
    t = torch.zeros(R, dtype=torch.int32, device="cuda")
    f = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
    o = [f(R), f(R), f(R), torch.empty(R, 0, dtype=torch.int32, device="cuda"), f(R, 0)]
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    calls = {"vh_add_rmsnorm": lambda: m.add_rmsnorm(x, None, None, 1e-6, 0.0, x, None, None),
             "vh_add_rmsnorm_grad": lambda: m.add_rmsnorm_grad(x, x, None, 1e-6, 0.0, None, x, None, None),
             "vh_logits_logprobs": lambda: m.logits_logprobs(x, t, 0, *o, ws),
             "vh_logits_logprobs_grad": lambda: m.logits_logprobs_grad(x, t, o[2], o[1], o[0], None, x),
             "vh_head_logprobs": lambda: m.head_logprobs(x, W, t, 0, *o, ws)}
    for name, call in calls.items():
        stop, ticks = threading.Event(), []

        def tick():
            while not stop.is_set():
                ticks.append(time.monotonic())
                time.sleep(0.005)

        m.bind(name, slow)
        try:
            other = threading.Thread(target=tick)
            other.start()
            t0 = time.monotonic()
            assert call() == 0, name
            t1 = time.monotonic()
        finally:
            m.bind(name, ctypes.cast(getattr(vh.lib(), name), ctypes.c_void_p).value)
            stop.set()
            other.join()
        assert t1 - t0 > 0.29, name
        assert sum(t0 + 0.05 < k < t1 - 0.05 for k in ticks) > 3, name
