"""Host-side pieces of the training operators, compiled by themselves on the CPU."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "zero_sharded_optimizer_flat_gb300", "csrc")


def cuda_include():
    from zero_sharded_optimizer_flat_gb300 import build_lib
    return os.path.join(os.path.dirname(os.path.dirname(build_lib._nvcc())), "include")


def run(tmp_path, source):
    """The lines that a C++ program prints."""
    src, exe = tmp_path / "a.cpp", tmp_path / "a"
    src.write_text(source)
    subprocess.run(["g++", "-std=c++17", f"-I{CSRC}", f"-I{cuda_include()}", f"-I{os.path.join(ROOT, 'include')}", str(src), "-o",
                    str(exe)], check=True)
    return subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split("\n")[:-1]


@pytest.mark.parametrize("size", [1, 2, 4])
def test_row_bytes_of_long_rows(tmp_path, size):
    """Rows of up to 2^30 columns, results of 1, 2 and 4 bytes: a whole row passes 31 bits."""
    cases = [(n, col) for n in (1, 7, 127, 128, 129, 1 << 20, 1 << 29, (1 << 30) - 1, 1 << 30)
             for col in {0, 64, 128, max(n - 130, 0), max(n - 128, 0), max(n - 64, 0), n - 1, n + 1, n + 255}]
    rows = "".join(f'std::printf("%d\\n", zopt::lm::row_bytes({n}, {col}, {size}));\n' for n, col in cases)
    got = run(tmp_path, f'#include <cstdio>\n#include "row_bytes.h"\nint main() {{\n{rows}}}\n')
    for (n, col), g in zip(cases, got):
        want = (n - col) * size  # in Python's integers
        # a warp's part is 128 columns at most: how many of its bytes lie in the row
        assert min(max(int(g), 0), 128 * size) == min(max(want, 0), 128 * size), (n, col, g)


def test_set_up_once_on_every_device(tmp_path):
    """A kernel's shared-memory attribute is set on each device's first call, and again after a failure:
    against a fake of the runtime's current device."""
    got = run(tmp_path, r"""
#include <cstdio>
#include "per_device.h"
static int device = 0, calls = 0;
static cudaError_t answer = cudaSuccess, device_answer = cudaSuccess;
extern "C" cudaError_t CUDARTAPI cudaGetDevice(int* d) { *d = device; return device_answer; }
template <int kSite> static int call() { return zopt::once_per_device([] { ++calls; return answer; }); }
#define SAY(site) do { const int e = call<site>(); std::printf("%d %d\n", e, calls); } while (0)
int main() {
  SAY(0);                                            // set up on device 0
  SAY(0);                                            // done already
  device = 1; SAY(0);                                // a second device
  device = 0; SAY(0);
  SAY(1);                                            // another kernel
  device = 2; answer = cudaErrorInvalidValue; SAY(0);  // fails,
  answer = cudaSuccess; SAY(0);                      // is tried again,
  SAY(0);                                            // and then is done
  device = 70; SAY(0); SAY(0);
  device_answer = cudaErrorNoDevice; SAY(0);
}
""")
    bad, none = 1, 100  # cudaErrorInvalidValue, cudaErrorNoDevice
    assert [tuple(map(int, g.split())) for g in got] == [(0, 1), (0, 1), (0, 2), (0, 2), (0, 3), (bad, 4), (0, 5), (0, 5),
                                                         (0, 6), (0, 7), (none, 7)]
