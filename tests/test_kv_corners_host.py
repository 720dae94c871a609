"""The attention block's host code against a CUDA runtime that only records: what the launchers get, and which
stream and device a call works on."""
import ctypes
import os
import subprocess

import pytest

from quantized_moe_expert_gemv_gb300 import binding, build
from test_kv_host import Call, host_plan

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "quantized_moe_expert_gemv_gb300", "csrc")

RECORD = """
#include "si_kv.h"
#include <cstring>
static int g_max_new = -1, g_word = 0, g_cleared_elsewhere = 0;
static void *g_cleared_in = nullptr;
extern "C" {
int last_max_new() { return g_max_new; }
void report(int word) { g_word = word; g_cleared_in = nullptr; g_cleared_elsewhere = 0; }
void *cleared_in() { return g_cleared_in; }
int cleared_elsewhere() { return g_cleared_elsewhere; }
cudaError_t cudaDeviceGetAttribute(int *v, cudaDeviceAttr a, int) {
    *v = a == cudaDevAttrMultiProcessorCount ? 152 : a == cudaDevAttrClockRate ? 2000000 : 232448;
    return cudaSuccess;
}
cudaError_t cudaMemsetAsync(void *, int, size_t, cudaStream_t s) { g_cleared_in = s; g_word = 0; return cudaSuccess; }
cudaError_t cudaMemset(void *, int, size_t) { g_cleared_elsewhere = 1; g_word = 0; return cudaSuccess; }
cudaError_t cudaMemcpy(void *to, const void *, size_t, cudaMemcpyKind) { std::memcpy(to, &g_word, 4); return cudaSuccess; }
cudaError_t cudaStreamSynchronize(cudaStream_t) { return cudaSuccess; }
cudaError_t cudaGetLastError() { return cudaSuccess; }
}
namespace si { namespace kv {
size_t scratch_bytes(const Plan &, int, int, int, int) { return kCtrlBytes; }
static cudaError_t seen(const Ctx &c) { g_max_new = c.max_new; return cudaSuccess; }
cudaError_t launch_append(const Plan &, const Ctx &c, Rows, Rows, int32_t *, cudaStream_t) { return seen(c); }
cudaError_t launch_read(const Plan &, const Ctx &c, const int32_t *, int, uint16_t *, uint16_t *, cudaStream_t) { return seen(c); }
cudaError_t launch_attend(const Plan &, const Ctx &c, Rows, Rows, float *, float, void *, cudaStream_t) { return seen(c); }
cudaError_t launch_weigh(const Plan &, const Ctx &c, Rows, const float *, const float *, float *, int64_t, float, float, cudaStream_t) { return seen(c); }
cudaError_t launch_evict(const Plan &, const Ctx &c, const float *, float *, int64_t, int, int, int, const int32_t *, const int32_t *, int32_t *, int32_t *, cudaStream_t) { return seen(c); }
}}
"""


@pytest.fixture(scope="module")
def recorder(tmp_path_factory):
    """csrc/si_kv_api.cu (host code) linked with launchers and runtime calls that record."""
    d = tmp_path_factory.mktemp("kv_record")
    (d / "record.cc").write_text(RECORD)
    cuda = os.path.dirname(os.path.dirname(build._nvcc()))
    so = str(d / "libkvrecord.so")
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-Wl,-Bsymbolic", "-I", CSRC, "-I", os.path.join(cuda, "include"), "-o", so,
                    str(d / "record.cc"), "-x", "c++", os.path.join(CSRC, "si_kv_api.cu")], check=True)
    lib = ctypes.CDLL(so)
    binding._declare_kv(lib)
    return lib


@pytest.mark.parametrize("name", ["append", "attend", "weigh"])
def test_the_row_bound_is_what_the_others_leave(recorder, name):
    """max_new, or total_new where that is less, and never more rows than a kv head's can be numbered in 32 bits."""
    plan = host_plan(recorder, 64, 1, 128, 64)
    for total, most, want in ((6, 4, 4), (6, 2 ** 31 - 1, 6), (2 ** 31 - 1, 2 ** 31 - 1, 2 ** 30 // 64), (2 ** 25, 5, 5)):
        call = Call(plan)
        call.batch.total_new, call.batch.max_new = total, most
        call.out = binding.si_kv_rows(0x90000, 64 * 128, 128)
        assert call(recorder, name) == binding.SI_OK
        assert recorder.last_max_new() == want
    recorder.si_kv_plan_destroy(plan.handle)


ATTRIBUTES = """
#include "si_kv.h"
static int g_device = 0, g_set[2] = {0, 0}, g_fail = 0;
extern "C" {
cudaError_t cudaGetDevice(int *d) { *d = g_device; return cudaSuccess; }
cudaError_t cudaFuncSetAttribute(const void *, cudaFuncAttribute, int) {
    if (g_fail) return cudaErrorInvalidValue;
    ++g_set[g_device];
    return cudaSuccess;
}
void kernel() {}
int call(int device, int fail) { g_device = device; g_fail = fail; return (int)si::kv::allow_smem<&kernel>(100000); }
int sets(int device) { return g_set[device]; }
}
"""


def test_shared_memory_is_allowed_once_on_each_device_that_launches(tmp_path):
    """The attribute belongs to the current device: a call on one device settles nothing for another."""
    (tmp_path / "attributes.cc").write_text(ATTRIBUTES)
    cuda = os.path.dirname(os.path.dirname(build._nvcc()))
    so = str(tmp_path / "libattributes.so")
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-Wl,-Bsymbolic", "-I", CSRC, "-I", os.path.join(cuda, "include"), "-o", so,
                    str(tmp_path / "attributes.cc")], check=True)
    lib = ctypes.CDLL(so)
    assert lib.call(1, 1) != 0 and lib.sets(1) == 0  # a failure is not remembered
    for _ in range(3):
        assert lib.call(0, 0) == 0
        assert lib.call(1, 0) == 0
    assert lib.sets(0) == lib.sets(1) == 1


def test_outputs_that_overlap_are_refused(recorder):
    """8 heads of 128 in 6 rows: strides that put two rows or heads in one place, and outputs in q's place."""
    plan = host_plan(recorder, 8, 2, 128, 64)

    def attend(q, out, rows=6):
        call = Call(plan)
        call.batch.total_new = rows
        call.rows, call.out = binding.si_kv_rows(*q), binding.si_kv_rows(*out)
        return call(recorder, "attend")

    far, q = 0x900000, (0x80000, 1024, 128)
    for strides in ((128, 128), (512, 128), (128, 640), (1016, 128), (136, 136), (256, 128), (640, 256)):
        assert attend(q, (far, *strides)) == binding.SI_ERR_INVALID_ARG, strides
    for strides in ((1024, 128), (1032, 128), (128, 768), (4096, 384), (136, 816), (256, 1536 + 128), (1024 + 128, 144)):
        assert attend(q, (far, *strides)) == binding.SI_OK, strides
    # neither stride spans the other dimension, and no two places meet: rows at 2 x 128, heads at odd multiples
    assert attend(q, (far, 256, 128 * 13)) == binding.SI_OK
    assert attend(q, (far, 128, 128), rows=1) == binding.SI_OK   # one row
    # q's place, one row on, half a head on; q's own buffer where the parts of a projection lie side by side
    assert attend(q, q) == attend(q, (0x80000 + 2048, 1024, 128)) == attend(q, (0x80000 + 128, 1024, 128)) == binding.SI_ERR_INVALID_ARG
    wide = (0x80000, 4096, 128)
    assert attend(wide, (0x80000 + 2048, 4096, 128)) == binding.SI_OK
    assert attend(wide, (0x80000 - 2048, 4096, 128)) == binding.SI_OK
    assert attend(wide, (0x80000 + 4096 * 2 - 2048 + 256, 4096, 128)) == binding.SI_ERR_INVALID_ARG  # its last head is the next row's first
    assert attend((0x80000, 0, 128), (0x80000, 1024, 128)) == binding.SI_ERR_INVALID_ARG
    recorder.si_kv_plan_destroy(plan.handle)


def brute(places, D):
    at = sorted(places)
    return any(b - a < D for a, b in zip(at, at[1:]))


def test_overlap_of_any_strides(recorder):
    """Against every pair of places, for small rows and heads."""
    import random
    rng = random.Random(3)
    plan = host_plan(recorder, 6, 2, 64, 64)
    seen = set()
    for _ in range(3000):
        rows, row, head = rng.randrange(1, 9), 8 * rng.randrange(8, 80), 8 * rng.randrange(8, 80)
        call = Call(plan)
        call.batch.total_new = rows
        call.out = binding.si_kv_rows(0x900000, row, head)
        call.rows = binding.si_kv_rows(0x900000 + 16 * rng.randrange(-600, 600), row, head)
        out = [r * row + h * head for r in range(rows) for h in range(6)]
        apart = (call.rows.data - 0x900000) // 2
        meets = any(abs(x - y - apart) < 64 for x in out for y in out)
        want = binding.SI_ERR_INVALID_ARG if brute(out, 64) or meets else binding.SI_OK
        assert call(recorder, "attend") == want, (rows, row, head, apart)
        seen.add((brute(out, 64), meets))
    assert len(seen) == 4
    recorder.si_kv_plan_destroy(plan.handle)


def test_the_status_is_cleared_in_the_callers_stream(recorder):
    """A clear in another stream could come after what the stream's next call reports."""
    recorder.cleared_in.restype = ctypes.c_void_p
    plan = host_plan(recorder, 8, 2, 128, 64)
    recorder.report(binding.SI_ERR_DEVICE)
    assert recorder.si_kv_read_status(plan.handle, 0x10000, 0x5000) == binding.SI_ERR_DEVICE
    assert recorder.cleared_in() == 0x5000 and not recorder.cleared_elsewhere()
    assert recorder.si_kv_read_status(plan.handle, 0x10000, 0x5000) == binding.SI_OK
    recorder.si_kv_plan_destroy(plan.handle)


@pytest.mark.parametrize("name", ["append", "attend", "weigh"])
def test_calls_without_rows_need_no_data(recorder, name):
    """An empty tensor has no address."""
    plan = host_plan(recorder, 8, 2, 128, 64)
    for total, want in ((0, binding.SI_OK), (1, binding.SI_ERR_INVALID_ARG)):
        call = Call(plan)
        call.batch.total_new = total
        call.rows.data = call.out.data = None
        if name == "weigh":
            call.a["lse"] = None
        assert call(recorder, name) == want
    if name == "weigh":
        call.rows.data = 0x80000
        assert call(recorder, name) == binding.SI_ERR_INVALID_ARG
    recorder.si_kv_plan_destroy(plan.handle)
