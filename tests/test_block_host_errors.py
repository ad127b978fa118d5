"""What the host side of the residual join does when the CUDA runtime fails:
norm_api.cu compiled against a runtime that the test makes fail."""
import ctypes
import subprocess
from pathlib import Path

import pytest

ROOT = Path(__file__).resolve().parents[1]
CSRC = ROOT / "bit_error_compensated_gb300" / "csrc"

API = r"""
#include "norm_common.h"

namespace echo {
int note_cuda_error(cudaError_t) { return ECHO_ERR_CUDA; }
#define STUB(T)                                                                                          \
  template <> cudaError_t launch_norm<T>(const NormArgs&, int, bool, int, cudaStream_t) {                 \
    return cudaSuccess;                                                                                   \
  }                                                                                                       \
  template <> cudaError_t launch_norm_grad<T>(NormGradArgs, int, bool, int, cudaStream_t) { return cudaSuccess; }
STUB(float)
STUB(__nv_bfloat16)
STUB(__half)
}

#include "norm_api.cu"
"""

RUNTIME = r"""
#include <stddef.h>
static int g_last = 0, g_live = 0, g_fail = 0;
static size_t g_allocated = 0;
extern "C" {
int cudaGetDevice(int* d) { *d = 0; return 0; }
int cudaDeviceGetAttribute(int* v, int, int) { *v = 152; return 0; }
int cudaMalloc(void** p, size_t n) {
  if (g_fail) return g_last = 2;
  g_allocated = n;
  ++g_live;
  *p = reinterpret_cast<void*>(0x1000);
  return 0;
}
int cudaFree(void*) { --g_live; return 0; }
int cudaGetLastError(void) { const int e = g_last; g_last = 0; return e; }
void fake_fail(int on) { g_fail = on; }
int fake_last(void) { return g_last; }
int fake_live(void) { return g_live; }
size_t fake_allocated(void) { return g_allocated; }
}
"""


@pytest.fixture(scope="module")
def fake(tmp_path_factory):
    from bit_error_compensated_gb300.build import ARCH, nvcc
    where = tmp_path_factory.mktemp("fake_runtime")
    (where / "api.cu").write_text(API)
    (where / "runtime.cpp").write_text(RUNTIME)
    subprocess.check_call([nvcc(), *ARCH, "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr", "-I", str(CSRC),
                           "-I", str(ROOT / "include"), "-shared", "-cudart", "shared",
                           "-Xlinker", "-Bsymbolic", "-o", str(where / "fake.so"),
                           str(where / "api.cu"), str(where / "runtime.cpp")])
    lib = ctypes.CDLL(str(where / "fake.so"))
    lib.echo_norm_plan.argtypes = [ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_float,
                                   ctypes.c_float, ctypes.POINTER(ctypes.c_void_p)]
    lib.echo_norm_plan_destroy.argtypes = [ctypes.c_void_p]
    lib.fake_allocated.restype = ctypes.c_size_t
    return lib


def plan(lib, width):
    h = ctypes.c_void_p()
    return lib.echo_norm_plan(width, 1, 1, 0, 1, 1e-6, 1.0, ctypes.byref(h)), h


def test_a_plan_without_memory_leaves_no_error_behind(fake):
    """The call reports the failure; the runtime's last error, which the next
    check of someone else's launch would find, is cleared."""
    fake.fake_fail(1)
    try:
        status, h = plan(fake, 4096)
        assert status == 5 and h.value is None
        assert fake.fake_last() == 0 and fake.fake_live() == 0
    finally:
        fake.fake_fail(0)
        fake.cudaGetLastError()


@pytest.mark.parametrize("width", [1, 31, 512, 513, 1000, 4096, 4097, 8192, 8193, 12288, 16383, 16384])
def test_a_plan_allocates_for_the_threads_that_there_are(fake, width):
    """Six fp32 sums for each column of 152 SMs' 512 threads of 16 columns at
    most, and a whole row's at least; freed with the plan."""
    status, h = plan(fake, width)
    assert status == 0 and fake.fake_live() == 1
    assert 6 * 4 * width <= fake.fake_allocated() <= 6 * 4 * 152 * 512 * 16
    fake.echo_norm_plan_destroy(h)
    assert fake.fake_live() == 0
