"""The attention block's C ABI on the host: layouts, exported names and the refusal of every bad argument
before anything touches a device (the pointers here are numbers that nothing may follow)."""
import ctypes
import os
import re
import subprocess

import pytest

from quantized_moe_expert_gemv_gb300 import binding, build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
STRUCTS = {"si_kv_desc": binding.si_kv_desc, "si_kv_cache": binding.si_kv_cache, "si_kv_batch": binding.si_kv_batch,
           "si_kv_rows": binding.si_kv_rows}
BAD, NO, ODD, SMALL = (binding.SI_ERR_INVALID_ARG, binding.SI_ERR_UNSUPPORTED, binding.SI_ERR_MISALIGNED,
                       binding.SI_ERR_SCRATCH_TOO_SMALL)


@pytest.fixture(scope="module")
def lib():
    return binding.load_library(build.build())


def _c_program(tmp_path, lines):
    src, exe = tmp_path / "probe.c", tmp_path / "probe"
    src.write_text("\n".join(['#include <stdio.h>', '#include <stddef.h>', '#include "si_kv.h"', "int main(void) {"] +
                             lines + ["return 0;", "}"]) + "\n")
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), "-o", str(exe), str(src)], check=True)
    return subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split("\n")


def test_structs_and_constants_match_the_header(tmp_path):
    lines, want = [], []
    for name, cls in STRUCTS.items():
        lines.append(f'printf("%zu\\n", sizeof({name}));')
        want.append(ctypes.sizeof(cls))
        for f, _ in cls._fields_:
            lines.append(f'printf("%zu\\n", offsetof({name}, {f}));')
            want.append(getattr(cls, f).offset)
    with open(binding.KV_HEADER_PATH) as f:
        consts = re.findall(r"^#define (SI_KV_[A-Z0-9_]+) ", f.read(), flags=re.M)
    assert len(consts) >= 8
    for n in consts:
        lines.append(f'printf("%d\\n", (int)({n}));')
        want.append(getattr(binding, n))
    assert [int(v) for v in _c_program(tmp_path, lines) if v] == want


def test_header_is_declared_and_exported(lib):
    names = binding.declared_symbols()
    for n in ("si_kv_plan", "si_kv_append", "si_kv_read", "si_kv_attend", "si_kv_weigh", "si_kv_evict",
              "si_kv_read_status"):
        assert n in names and getattr(lib, n) is not None


def test_plan_refuses_bad_shapes(lib):
    D = binding.make_kv_desc
    for desc, want in [(D(32, 5, 128, 64), BAD), (D(0, 1, 128, 64), BAD), (D(8, 0, 128, 64), BAD),
                       (D(512, 8, 128, 64), NO), (D(8, 8, 96, 64), NO), (D(8, 8, 128, 48), NO),
                       (D(8, 8, 128, 64, code=3), NO), (D(8, 8, 128, 64, dtype=0), NO)]:
        assert binding.si_kv_plan_status(desc) == want, (desc.n_heads, desc.n_kv_heads, desc.head_dim)
    assert lib.si_kv_plan(None, 0, ctypes.byref(ctypes.c_void_p())) == BAD
    assert lib.si_kv_plan(ctypes.byref(D(8, 8, 128, 64)), 0, None) == BAD


def test_null_plans_are_refused(lib):
    n = ctypes.c_size_t()
    assert lib.si_kv_scratch_bytes(None, 1, 1, 1, 1, ctypes.byref(n)) == BAD
    assert lib.si_kv_scratch_init(None, 16, 1 << 20, None) == BAD
    assert lib.si_kv_append(None, None, None, None, None, None, None, 0, None) == BAD
    assert lib.si_kv_read(None, None, None, 0, None, None, None, 0, None) == BAD
    assert lib.si_kv_attend(None, None, None, None, None, None, 1.0, None, 0, None) == BAD
    assert lib.si_kv_weigh(None, None, None, None, None, None, None, 0, 1.0, 1.0, None, 0, None) == BAD
    assert lib.si_kv_evict(None, None, None, None, None, 0, 1, 0, 0, None, None, None, None, None, 0, None) == BAD
    assert lib.si_kv_read_status(None, None, None) == BAD


class Call:
    """One call with good arguments (addresses that are never followed) of which a test changes one."""

    def __init__(self, plan):
        self.plan = plan
        self.cache = binding.si_kv_cache(0x10000, 0x20000, 0x30000, 0x40000, 0x50000, 0x60000, 100, 4)
        self.batch = binding.si_kv_batch(2, 6, 4, 1000, 0x70000, 0x71000, 0x72000, None, 40)
        self.rows = binding.si_kv_rows(0x80000, 1024, 128)
        self.out = binding.si_kv_rows(0x90000, 1024, 128)
        self.a = dict(lens_out=0xA0000, lse=0xB0000, acc_in=0xC0000, acc_out=0xE0000, stride=1024, scratch=0x100000,
                      size=1 << 30, sm=0.1, decay=1.0, budget=8, sink=1, recent=2, new_table=0xF0000, new_slots=0,
                      keep=0xF1000, n=3, pages=0xF2000, k_out=0x110000, v_out=0x120000)

    def __call__(self, lib, name):
        a, h = self.a, self.plan.handle
        c = ctypes.byref(self.cache) if self.cache else None
        b = ctypes.byref(self.batch) if self.batch else None
        r = ctypes.byref(self.rows) if self.rows else None
        o = ctypes.byref(self.out) if self.out else None
        tail = (a["scratch"], a["size"], None)
        if name == "append":
            return lib.si_kv_append(h, c, b, r, r, a["lens_out"], *tail)
        if name == "read":
            return lib.si_kv_read(h, c, a["pages"], a["n"], a["k_out"], a["v_out"], *tail)
        if name == "attend":
            return lib.si_kv_attend(h, c, b, r, o, a["lse"], a["sm"], *tail)
        if name == "weigh":
            return lib.si_kv_weigh(h, c, b, r, a["lse"], a["acc_in"], a["acc_out"], a["stride"], a["decay"], a["sm"],
                                   *tail)
        return lib.si_kv_evict(h, c, b, a["acc_in"], a["acc_out"], a["stride"], a["budget"], a["sink"], a["recent"],
                               a["new_table"], a["new_slots"], a["keep"], a["lens_out"], *tail)


def refusals():
    def cache(**kw):
        return lambda x: [setattr(x.cache, k, v) for k, v in kw.items()]

    def batch(**kw):
        return lambda x: [setattr(x.batch, k, v) for k, v in kw.items()]

    def rows(**kw):
        return lambda x: [setattr(x.rows, k, v) for k, v in kw.items()]

    def out(**kw):
        return lambda x: [setattr(x.out, k, v) for k, v in kw.items()]

    def arg(**kw):
        return lambda x: x.a.update(kw)

    def gone(name):
        return lambda x: setattr(x, name, None)

    every, batched, rowed = ("append", "read", "attend", "weigh", "evict"), ("append", "attend", "weigh", "evict"), \
        ("append", "attend", "weigh")
    table = []
    for f in ("k_codes", "v_codes", "k_scale", "v_scale", "k_tail", "v_tail"):
        table += [(every, cache(**{f: None}), BAD), (every, cache(**{f: 0x10008}), ODD)]
    table += [(every, gone("cache"), BAD), (every, cache(n_pages=0), BAD), (every, cache(n_pages=1 << 31), BAD),
              (every, cache(n_slots=0), BAD), (every, arg(scratch=None), BAD), (every, arg(scratch=0x100008), ODD),
              (every, arg(size=64), SMALL), (batched, gone("batch"), BAD), (batched, batch(n_seqs=0), BAD),
              (batched, batch(n_seqs=1025), NO), (batched, batch(max_len=-1), BAD), (batched, batch(max_len=(1 << 22) + 1), NO),
              (rowed, batch(total_new=-1), BAD), (rowed, batch(max_new=-1), BAD), (rowed, batch(q_start=None), BAD),
              (batched, batch(lens=None), BAD), (batched, batch(lens=0x71002), ODD), (batched, batch(page_table=None), BAD),
              (batched, batch(table_stride=1000 // 64 - 1), BAD), (batched, batch(slots=0x73001), ODD),
              (rowed, gone("rows"), BAD), (rowed, rows(data=None), BAD), (rowed, rows(data=0x80008), ODD),
              (rowed, rows(row_stride=1028), ODD), (rowed, rows(head_stride=-128), BAD),
              (("attend",), gone("out"), BAD), (("attend",), out(head_stride=64), BAD), (("attend",), out(row_stride=0), BAD),
              (("attend",), out(data=0x90002), ODD), (("attend",), arg(lse=0xB0002), ODD),
              (("attend", "weigh"), arg(sm=-1.0), BAD), (("attend", "weigh"), arg(sm=float("nan")), BAD),
              (("attend", "weigh"), arg(sm=float("inf")), BAD),
              (("append", "evict"), arg(lens_out=None), BAD), (("append", "evict"), arg(lens_out=0x71004), BAD),
              (("weigh",), arg(lse=None), BAD), (("weigh",), arg(decay=float("nan")), BAD),
              (("weigh", "evict"), arg(acc_out=None), BAD), (("evict",), arg(acc_in=None), BAD),
              (("weigh", "evict"), arg(stride=999), BAD), (("weigh", "evict"), arg(acc_out=0xC0004), BAD),
              (("evict",), arg(acc_out=0xC0000), BAD), (("evict",), arg(budget=0), BAD), (("evict",), arg(sink=-1), BAD),
              (("evict",), arg(recent=8), BAD), (("evict",), arg(new_table=None), BAD), (("evict",), arg(keep=None), BAD),
              (("evict",), batch(max_len=1 << 22, table_stride=1 << 18), NO),
              (("read",), arg(n=-1), BAD), (("read",), arg(pages=None), BAD), (("read",), arg(k_out=0x110008), ODD)]
    return table


STUBS = """
#include <cstring>
#include "si_kv.h"
static int g_launches = 0;
extern "C" {
int launches() { return g_launches; }
cudaError_t cudaDeviceGetAttribute(int *v, cudaDeviceAttr a, int) {
    *v = a == cudaDevAttrMultiProcessorCount ? 152 : a == cudaDevAttrClockRate ? 2000000 : 232448;
    return cudaSuccess;
}
cudaError_t cudaMemsetAsync(void *, int, size_t, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaMemset(void *, int, size_t) { return cudaSuccess; }
cudaError_t cudaMemcpy(void *, const void *, size_t, cudaMemcpyKind) { return cudaSuccess; }
cudaError_t cudaStreamSynchronize(cudaStream_t) { return cudaSuccess; }
cudaError_t cudaGetLastError() { return cudaSuccess; }
}
namespace si { namespace kv {
size_t scratch_bytes(const Plan &, int, int, int, int) { return kCtrlBytes; }
#define LAUNCH(name, ...) cudaError_t name(__VA_ARGS__) { ++g_launches; return cudaSuccess; }
LAUNCH(launch_append, const Plan &, const Ctx &, Rows, Rows, int32_t *, cudaStream_t)
LAUNCH(launch_read, const Plan &, const Ctx &, const int32_t *, int, uint16_t *, uint16_t *, cudaStream_t)
LAUNCH(launch_attend, const Plan &, const Ctx &, Rows, Rows, float *, float, void *, cudaStream_t)
LAUNCH(launch_weigh, const Plan &, const Ctx &, Rows, const float *, const float *, float *, int64_t, float, float, cudaStream_t)
LAUNCH(launch_evict, const Plan &, const Ctx &, const float *, float *, int64_t, int, int, int, const int32_t *, const int32_t *, int32_t *, int32_t *, cudaStream_t)
}}
"""


@pytest.fixture(scope="module")
def host_lib(tmp_path_factory):
    """The argument checks (csrc/si_kv_api.cu is host code) linked with launchers that only count: no device."""
    d = tmp_path_factory.mktemp("kv_host")
    (d / "stubs.cc").write_text(STUBS)
    csrc = os.path.join(ROOT, "quantized_moe_expert_gemv_gb300", "csrc")
    cuda = os.path.dirname(os.path.dirname(build._nvcc()))
    so = str(d / "libkvhost.so")
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-Wl,-Bsymbolic", "-I", csrc, "-I", os.path.join(cuda, "include"), "-o", so,
                    str(d / "stubs.cc"), "-x", "c++", os.path.join(csrc, "si_kv_api.cu")], check=True)
    lib = ctypes.CDLL(so)
    binding._declare_kv(lib)
    return lib


def host_plan(lib, *args, **kw):
    h = ctypes.c_void_p()
    assert lib.si_kv_plan(ctypes.byref(binding.make_kv_desc(*args, **kw)), 0, ctypes.byref(h)) == binding.SI_OK

    class P:
        handle = h.value
    return P


def test_refusals(host_lib):
    plan = host_plan(host_lib, 8, 2, 128, 64)
    for names, change, want in refusals():
        for name in names:
            call, before = Call(plan), host_lib.launches()
            change(call)
            assert call(host_lib, name) == want, (name, want)
            assert host_lib.launches() == before
    for name in ("append", "read", "attend", "weigh", "evict"):
        before = host_lib.launches()
        assert Call(plan)(host_lib, name) == binding.SI_OK
        assert host_lib.launches() == before + 1, name
    host_lib.si_kv_plan_destroy(plan.handle)


def test_calls_with_nothing_to_do_launch_nothing(host_lib):
    plan = host_plan(host_lib, 8, 2, 128, 64)
    before = host_lib.launches()
    call = Call(plan)
    call.a["n"] = 0
    assert call(host_lib, "read") == binding.SI_OK
    call = Call(plan)
    call.batch.total_new = call.batch.max_new = 0
    assert call(host_lib, "attend") == binding.SI_OK
    call = Call(plan)
    call.batch.max_len = call.batch.table_stride = 0
    call.batch.page_table = None
    assert call(host_lib, "weigh") == binding.SI_OK
    assert host_lib.launches() == before
    assert call(host_lib, "append") == binding.SI_OK  # lens_out is still written
    assert host_lib.launches() == before + 1
    host_lib.si_kv_plan_destroy(plan.handle)


def test_scratch_calls(host_lib):
    plan = host_plan(host_lib, 8, 2, 128, 64)
    n = ctypes.c_size_t()
    assert host_lib.si_kv_scratch_bytes(plan.handle, 0, 1, 1, 1, ctypes.byref(n)) == BAD
    assert host_lib.si_kv_scratch_bytes(plan.handle, 1, 1, 1, 1, None) == BAD
    assert host_lib.si_kv_scratch_bytes(plan.handle, 1025, 1, 1, 1, ctypes.byref(n)) == NO
    assert host_lib.si_kv_scratch_init(plan.handle, None, 1 << 20, None) == BAD
    assert host_lib.si_kv_scratch_init(plan.handle, 0x10008, 1 << 20, None) == ODD
    assert host_lib.si_kv_scratch_init(plan.handle, 0x10000, 256, None) == SMALL
    host_lib.si_kv_plan_destroy(plan.handle)
