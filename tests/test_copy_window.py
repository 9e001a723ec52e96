"""Which granules of a row are copied and which elements read one by one (csrc/vh_window.h, compiled for the host): the
copies stay within the tensor, and the two parts hold every element of the row once."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SOURCE = r"""
#include <cstdio>
#include "vh_window.h"

int main() {
    long cases = 0;
    for (int size = 2; size <= 4; size += 2)
        for (int H = 1; H <= 40; ++H)
            for (int pitch = H; pitch <= H + 9; ++pitch)
                for (int T = 1; T <= 20; ++T)
                    for (int offset = 0; offset < 16 / size; ++offset) {
                        const uintptr_t start = 4096 + offset * size;
                        const uint32_t bytes = H * size;
                        const uintptr_t end = start + (uintptr_t)(T - 1) * pitch * size + bytes;
                        for (int t = 0; t < T; ++t, ++cases) {
                            const uintptr_t b = start + (uintptr_t)t * pitch * size;
                            uintptr_t lo, hi;
                            int head, tail;
                            vh::copy_window(b, bytes, start, end, lo, hi);
                            vh::outside_window(b, bytes, size, lo, hi, head, tail);
                            bool ok = lo % 16 == 0 && hi % 16 == 0 && lo <= hi && head >= 0 && head <= tail && tail <= H;
                            if (hi > lo) ok = ok && lo >= start && hi <= end;
                            // its place holds them from the row's first granule on
                            ok = ok && lo >= (b & ~(uintptr_t)15) && hi - (b & ~(uintptr_t)15) <= ((uintptr_t)bytes + 30) / 16 * 16;
                            for (int i = 0; i < H; ++i) {
                                const uintptr_t at = b + (uintptr_t)i * size;
                                const bool copied = at >= lo && at + size <= hi, single = i < head || i >= tail;
                                ok = ok && copied != single;
                            }
                            if (!ok) {
                                std::printf("size %d H %d pitch %d T %d offset %d token %d\n", size, H, pitch, T, offset, t);
                                return 1;
                            }
                        }
                    }
    std::printf("%ld\n", cases);
    return 0;
}
"""


def test_every_short_row(tmp_path):
    cxx = shutil.which("g++")
    if not cxx:
        pytest.skip("no C++ compiler")
    (tmp_path / "w.cpp").write_text(SOURCE)
    subprocess.run([cxx, "-O2", "-std=c++17", "-I" + os.path.join(ROOT, "verify_head_gb300", "csrc"), str(tmp_path / "w.cpp"),
                    "-o", str(tmp_path / "w")], check=True)
    r = subprocess.run([str(tmp_path / "w")], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
    assert int(r.stdout) > 10 ** 6
