"""Without query heads (or key heads) their norm weights are not looked at: kvc_norm_rotate and kvpage_append check no such
pointer, so none may reach a kernel, which loads weights wherever it has their address. kvattend_abi.cpp is built here for
the host, with launches that keep the arguments they get."""

import ctypes
import os
import subprocess

import numpy as np
import pytest

from agent_handoff_amd import build
from agent_handoff_amd import kvattend as ka

A = 1 << 40
D, N = 64, 5

LAUNCHES = r"""
#include "attend.h"
#include "kvattend.h"
extern "C" { const void* got[2]; }
namespace kvc {
template <class T> hipError_t keep(const T& a) { got[0] = a.q_weight; got[1] = a.k_weight; return hipSuccess; }
hipError_t launch_norm_rotate(const RotateArgs& a, hipStream_t) { return keep(a); }
hipError_t launch_append(const AppendArgs& a, hipStream_t) { return keep(a); }
hipError_t launch_page_write(const PageLayout&, void*, uint32_t, const RowsDev&, const RowsDev&, const int64_t*, int32_t*,
                             hipStream_t) { return hipErrorUnknown; }
hipError_t launch_page_read(const PageLayout&, const void*, uint32_t, const int64_t*, const RowsDev&, const RowsDev&, int32_t*,
                            hipStream_t) { return hipErrorUnknown; }
hipError_t launch_attend(const AttendArgs&, hipStream_t) { return hipErrorUnknown; }
hipError_t launch_attend_prompt(const PromptArgs&, const PromptPlan&, hipStream_t) { return hipErrorUnknown; }
AttendPlan page_attend_plan(uint32_t, uint32_t, uint32_t, uint32_t, uint64_t, bool) { return {}; }
AttendPlan pool_attend_plan(uint32_t, uint32_t, uint32_t, uint32_t, uint32_t, bool) { return {}; }
PromptPlan prompt_plan(uint32_t, uint32_t, uint32_t, uint32_t, uint32_t, uint64_t, uint32_t, uint32_t) { return {}; }
}
extern "C" size_t kvpool_bytes(const kvc_shape*) { return 0; }
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    at = tmp_path_factory.mktemp("abi")
    (at / "launches.cpp").write_text(LAUNCHES)
    out = str(at / "libabi.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-fPIC", "-shared", "-D__HIP_PLATFORM_AMD__", "-I", "/opt/rocm/include",
                    "-I", build.INCLUDE, "-I", build.CSRC, os.path.join(build.CSRC, "kvattend_abi.cpp"),
                    str(at / "launches.cpp"), "-o", out], check=True)
    return ka._declare(ctypes.CDLL(out))


def weights(lib):
    return list((ctypes.c_void_p * 2).in_dll(lib, "got"))


def rows(base, heads):
    return ka.kvc_rows(base, heads * D, D)


# q_weight and k_weight: an address, none, or what no load could take
@pytest.mark.parametrize("q_heads, kv_heads, given, kept", [
    (4, 2, (5 * A, 6 * A), [5 * A, 6 * A]), (4, 2, (None, 6 * A), [None, 6 * A]), (4, 2, (5 * A, None), [5 * A, None]),
    (0, 2, (3, 6 * A), [None, 6 * A]), (4, 0, (5 * A, 3), [5 * A, None]), (0, 2, (3, None), [None, None])])
def test_weights_that_reach_the_kernels(lib, q_heads, kv_heads, given, kept):
    f = np.ones(D // 2, np.float32)
    q, k, qo, ko = rows(2 * A, q_heads), rows(3 * A, kv_heads), rows(10 * A, q_heads), rows(11 * A, kv_heads)
    assert lib.kvc_norm_rotate(N, q_heads, kv_heads, D, q, k, *given, 1e-6, 7 * A, f.ctypes.data, D // 2, 0, qo, ko, None) == 0
    assert weights(lib) == kept
    if kv_heads:
        spec = ka.kvc_pages(6, kv_heads, 16, D, ka.KVC_PAGE_FP4)
        assert lib.kvpage_append(spec, A, ka.kvpage_bytes(spec), N, q_heads, q, k, rows(4 * A, kv_heads), *given, 1e-6, 7 * A,
                                 f.ctypes.data, D // 2, 0, 8 * A, qo, None, None) == 0
        assert weights(lib) == kept
