"""What the block operators' entry points hand to their launchers, on the CPU: csrc/api_block.cpp built
with launchers that only write down their arguments."""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "fp8_delayed_scaling_amd", "csrc")
A16 = 1 << 20        # a fake 16-byte aligned address: never dereferenced

STUB = r"""
#include <hip/hip_runtime.h>
#include "launch.h"
extern "C" { int64_t seen[16]; int calls; }
namespace fp8ds {
static hipError_t note(const Grouped &g) {
    const int64_t v[] = {(int64_t)g.A, (int64_t)g.B, g.lda, g.ldb, g.stride_b, g.ldd, g.stride_d, g.cap, g.E, g.N, g.K};
    for (int i = 0; i < 11; ++i) seen[i] = v[i];
    ++calls;
    return hipSuccess;
}
hipError_t launch_grouped_gemm(const Grouped &g, int, int, int, hipStream_t) { return note(g); }
hipError_t launch_grouped_wgrad(const Grouped &g, int, int, int, hipStream_t) { return note(g); }
bool grouped_gemm_fits(int64_t, int64_t, int64_t) { return true; }
bool grouped_wgrad_fits(int64_t, int64_t, int64_t) { return true; }
size_t norm_workspace_bytes(int64_t, int64_t, int64_t) { return 0; }
hipError_t launch_norm_fwd(const NormFwd &, int, int, hipStream_t) { return hipSuccess; }
hipError_t launch_norm_bwd(NormBwd, int, int64_t, void *, hipStream_t) { return hipSuccess; }
size_t moe_workspace_bytes(int64_t, int64_t) { return 0; }
hipError_t launch_moe_plan(const int32_t *, int64_t, int64_t, int64_t, int64_t, int32_t *, int32_t *, int32_t *, void *,
                           hipStream_t) { return hipSuccess; }
hipError_t launch_moe_sort(const MoeSort &, int, hipStream_t) { return hipSuccess; }
hipError_t launch_moe_combine(const uint16_t *, const int32_t *, const float *, uint16_t *, int64_t, int64_t, int64_t, int64_t,
                              hipStream_t) { return hipSuccess; }
hipError_t launch_moe_weight_grad(const uint16_t *, const uint16_t *, const int32_t *, float *, int64_t, int64_t, int64_t,
                                  int64_t, hipStream_t) { return hipSuccess; }
}
"""
NAMES = ("A", "B", "lda", "ldb", "stride_b", "ldd", "stride_d", "cap", "E", "N", "K")


@pytest.fixture(scope="module")
def api(tmp_path_factory):
    d = tmp_path_factory.mktemp("api")
    (d / "stub.cpp").write_text(STUB)
    out = str(d / "api.so")
    cmd = ["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-w", "-D__HIP_PLATFORM_AMD__", "-I", CSRC, "-isystem", "/opt/rocm/include",
           os.path.join(CSRC, "api_block.cpp"), str(d / "stub.cpp"), "-o", out]
    subprocess.run(cmd, check=True)
    return ctypes.CDLL(out)


def _call(api, name, types, args):
    f = getattr(api, name)
    f.argtypes, f.restype = types, ctypes.c_int
    before = ctypes.c_int.in_dll(api, "calls").value
    status = f(*args)
    assert ctypes.c_int.in_dll(api, "calls").value - before == (status == 0)
    return status, dict(zip(NAMES, (ctypes.c_int64 * 16).in_dll(api, "seen")))


P, I64, INT = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
GEMM = [P, INT, P, I64, P, INT, P, I64, I64, P, I64, P, I64, INT, I64, I64, I64, P]
WGRAD = [P, INT, P, I64, P, INT, P, I64, P, I64, P, INT, I64, I64, I64, P]


def test_operands_and_strides_reach_the_launcher(api):
    st, g = _call(api, "fp8_grouped_gemm", GEMM, (A16, 0, A16, 80, 2 * A16, 0, A16, 96, 4096, A16, 3, A16, 40, 0, 128, 32, 64, None))
    assert st == 0 and g == dict(A=A16, B=2 * A16, lda=80, ldb=96, stride_b=4096, ldd=40, stride_d=0, cap=128, E=3, N=32, K=64)
    st, g = _call(api, "fp8_grouped_wgrad", WGRAD, (A16, 0, A16, 144, 2 * A16, 0, A16, 160, A16, 3, A16, 0, 128, 32, 64, None))
    assert st == 0 and g == dict(A=A16, B=2 * A16, lda=144, ldb=160, stride_b=0, ldd=64, stride_d=32 * 64, cap=128, E=3, N=32, K=64)


# Strides are unchecked without a contraction; the kernels form 32-bit offsets of up to 255 rows' strides,
# which from 2^23 on wrap back into the operand's bound.
@pytest.mark.parametrize("ld", [0, 1 << 23, 1 << 26, (1 << 24) + 16, 1 << 40])
def test_an_empty_contraction_has_no_strides(api, ld):
    for A in (None, A16):
        st, g = _call(api, "fp8_grouped_gemm", GEMM, (A, 0, A16, ld, A, 0, A16, ld, ld, A16, 3, A16, 40, 0, 128, 32, 0, None))
        assert st == 0 and (g["lda"], g["ldb"], g["stride_b"], g["ldd"]) == (0, 0, 0, 40)
        st, g = _call(api, "fp8_grouped_wgrad", WGRAD, (A, 0, A16, ld, A, 0, A16, ld, A16, 3, A16, 0, 0, 32, 64, None))
        assert st == 0 and (g["lda"], g["ldb"], g["ldd"], g["stride_d"]) == (0, 0, 64, 32 * 64)
