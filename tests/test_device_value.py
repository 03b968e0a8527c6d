"""What the library keeps for a device is that device's: with a stand-in for the
CUDA calls that name the device and count its SMs (no GPU needed)."""
import os
import shutil
import subprocess
import sys

import pytest

from tests.util import build_lib

ROOT = os.path.join(os.path.dirname(__file__), "..")
CSRC = os.path.join(ROOT, "bit_quantized_expert_moe_gb300", "csrc")

SHIM = r"""
static int current = 0;
extern "C" {
void stand_on(int device) { current = device; }
int cudaGetDevice(int* d) { *d = current; return 0; }
int cudaDeviceGetAttribute(int* v, int, int device) { *v = device == 0 ? 152 : 20; return 0; }
}
"""

PROGRAM = r"""
import ctypes, sys
shim, lib = ctypes.CDLL(sys.argv[1]), ctypes.CDLL(sys.argv[2])
size = lib.moe_grouped_mm_workspace_size
size.restype = ctypes.c_size_t
got = []
for device in (0, 1, 0):
    shim.stand_on(device)
    got.append(size(512, 1, 256, 7168))
print(*got)
"""

VALUES = r"""
#include "device_value.h"
#include <cstdio>
#include <thread>
#include <vector>
int main() {
    static moe::DeviceValue v;
    int bad = 0, found = 0;
    bad += v.get(3, [] { return 0; }) != 0;                   // not to be had: asked again
    bad += v.get(3, [&] { ++found; return 152; }) != 152;
    bad += v.get(3, [&] { ++found; return 1; }) != 152;       // kept
    bad += v.get(4, [&] { ++found; return 20; }) != 20;
    bad += v.get(1000, [] { return 7; }) != 7;                // beyond what is kept
    bad += found != 2;
    std::vector<std::thread> ts;
    static moe::DeviceValue w;
    std::atomic<int> wrong{0};
    for (int t = 0; t < 8; ++t)
        ts.emplace_back([&] { for (int d = 0; d < 64; ++d) wrong += w.get(d, [d] { return d + 1; }) != d + 1; });
    for (auto& t : ts) t.join();
    std::printf("%d\n", bad + wrong.load());
    return 0;
}
"""


def compiled(tmp_path, name, source, *flags):
    src, out = tmp_path / f"{name}.cpp", tmp_path / name
    src.write_text(source)
    subprocess.run(["g++", "-O1", "-std=c++17", "-I", CSRC, str(src), "-o", str(out), *flags], check=True)
    return str(out)


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_sizes_are_those_of_the_current_device(tmp_path):
    """Shares of a sum depend on the SMs: 152 on one device and 20 on the other."""
    try:
        lib = build_lib()
    except RuntimeError as e:  # pragma: no cover
        pytest.skip(f"cannot build: {e}")
    shim = compiled(tmp_path, "shim.so", SHIM, "-shared", "-fPIC")
    r = subprocess.run([sys.executable, "-c", PROGRAM, shim, lib], env={**os.environ, "LD_PRELOAD": shim},
                       capture_output=True, text=True, check=True)
    large, small, again = map(int, r.stdout.split())
    assert large > small and large == again


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_values_are_kept_by_device_and_found_by_any_thread(tmp_path):
    exe = compiled(tmp_path, "values", VALUES, "-pthread")
    assert subprocess.run([exe], capture_output=True, text=True, check=True).stdout == "0\n"


SIZES = r"""
import ctypes, sys
shim, lib = ctypes.CDLL(sys.argv[1]), ctypes.CDLL(sys.argv[2])
size = lib.moe_grouped_mm_workspace_size
size.restype = ctypes.c_size_t
shim.stand_on(0)
for E, N, K in ((1, 256, 7168), (2, 1024, 4096), (4, 88, 2072), (8, 1536, 2048), (256, 4096, 7168), (3, 232, 5608), (1, 96, 80)):
    last = 0
    for R in sorted({r + d for r in (0, 1, 8, 32, 64, 128, 300, 512, 1000, 2048, 4096, 6000, 20000, 10 ** 6) for d in (0, 1, 3)}):
        n = size(R, E, N, K)
        assert last <= n <= 256 + max(4 * 76 * 65536, 8 * 4 * E * N * K), (E, N, K, R, last, n)
        last = n
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_grouped_workspace_for_many_rows_does_for_fewer(tmp_path):
    """On a device of 152 SMs: the size never falls with the rows."""
    try:
        lib = build_lib()
    except RuntimeError as e:  # pragma: no cover
        pytest.skip(f"cannot build: {e}")
    shim = compiled(tmp_path, "shim.so", SHIM, "-shared", "-fPIC")
    subprocess.run([sys.executable, "-c", SIZES, shim, lib], env={**os.environ, "LD_PRELOAD": shim}, check=True)


NORM_SIZES = r"""
import ctypes, sys
shim, lib = ctypes.CDLL(sys.argv[1]), ctypes.CDLL(sys.argv[2])
size = lib.moe_block_norm_backward_workspace_size
size.restype = ctypes.c_size_t
shim.stand_on(0)
for D in (64, 1288, 2048, 4104, 8192, 16384):
    for several in (False, True):
        last = 0
        for T in sorted({r + d for r in (2, 150, 152, 304, 456, 700, 1000, 4096, 20000) for d in (0, 1, 2)}):
            n = size(T, D, T if several else 1)
            assert last <= n, (D, several, T, last, n)
            last = n
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_norm_gradients_workspace_for_many_rows_does_for_fewer(tmp_path):
    try:
        lib = build_lib()
    except RuntimeError as e:  # pragma: no cover
        pytest.skip(f"cannot build: {e}")
    shim = compiled(tmp_path, "shim.so", SHIM, "-shared", "-fPIC")
    subprocess.run([sys.executable, "-c", NORM_SIZES, shim, lib], env={**os.environ, "LD_PRELOAD": shim}, check=True)
