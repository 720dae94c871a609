// si_kv_device.cuh -- device functions shared by the cache's kernels.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "si_device.cuh"
#include "si_kv.h"

namespace si {
namespace kv {

// The start of every kernel: the next one may be launched, and this one goes on once the one before it
// in the stream has ended.  What it reads may thus be written while it is already there, so no load of the cache,
// the tables or the lse may be one of memory that stays as it is for the kernel's life (ld.global.nc, __ldg).
__device__ __forceinline__ void start_after() {
    pdl_launch_dependents();
    pdl_wait();
}

// One sequence of the call, checked against the host's bounds: a sequence
// that breaks one has no rows and no tokens here, and the status says so.
struct Seq {
    int row0, n, len, slot;  // first row, rows, tokens, ring slot (-1: outside the cache)
};
__device__ __forceinline__ Seq load_seq(const Ctx &c, int b, bool rows = true) {
    Seq s;
    const int r0 = rows ? c.q_start[b] : 0, r1 = rows ? c.q_start[b + 1] : 0;
    s.len = c.lens[b];
    s.slot = c.slots ? c.slots[b] : b;
    const bool rows_ok = r0 >= 0 && r1 >= r0 && r1 <= c.T && r1 - r0 <= c.max_new;
    if (!rows_ok || s.len < 0 || s.len > c.max_len) {
        set_status(c.status, SI_ERR_DEVICE);
        s.row0 = s.n = s.len = 0;
    } else {
        s.row0 = r0;
        s.n = r1 - r0;
    }
    if (s.slot < 0 || s.slot >= c.n_slots) {
        set_status(c.status, SI_ERR_DEVICE);
        s.slot = -1;
    }
    return s;
}
// Page j of sequence b; -1 (and the status) where the table names none of the cache's.
__device__ __forceinline__ int64_t load_page(const Ctx &c, int b, int j) {
    const int p = c.table[(int64_t)b * c.table_stride + j];
    if (p < 0 || p >= c.n_pages) {
        set_status(c.status, SI_ERR_DEVICE);
        return -1;
    }
    return p;
}
// Element offsets: of a page's head in the codes, of ring row t of a slot's head.
__device__ __forceinline__ int64_t page_at(const Ctx &c, int64_t page, int h) {
    return (page * c.Hk + h) * ((int64_t)c.P * c.D);
}
__device__ __forceinline__ int64_t ring_at(const Ctx &c, int slot, int h, int t) {
    return (((int64_t)slot * c.Hk + h) * (2 * c.P) + (t & (2 * c.P - 1))) * c.D;
}

// ------------------------------------------------------------------ 16-bit values
// Two values, the first in the low half.
template <int DT>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    if constexpr (DT == SI_KV_BF16) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&v);
    } else {
        const __half2 v = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
}

// ------------------------------------------------------------------ codes
constexpr float kQInt8 = 127.0f, kQE4m3 = 448.0f;

template <int CODE>
__device__ __forceinline__ float code_value(uint8_t c) {
    if constexpr (CODE == SI_KV_INT8) return (float)(int8_t)c;
    __nv_fp8_e4m3 v;
    v.__x = c;
    return (float)v;
}
// Four 16-bit values (a pair a word) times inv, each product rounded to 32 bits, to four codes, the first in
// the low byte.  (An amax whose reciprocal rounds up gives at most Q(1 + 2^-23), which rounds to Q.)
template <int CODE, int DT>
__device__ __forceinline__ uint32_t to_codes(uint32_t ab, uint32_t cd, float inv) {
    float f[4];
    if constexpr (DT == SI_KV_BF16) {
        f[0] = __uint_as_float(ab << 16);
        f[1] = __uint_as_float(ab & 0xffff0000u);
        f[2] = __uint_as_float(cd << 16);
        f[3] = __uint_as_float(cd & 0xffff0000u);
    } else {
        const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&ab)), y = __half22float2(*reinterpret_cast<const __half2 *>(&cd));
        f[0] = x.x;
        f[1] = x.y;
        f[2] = y.x;
        f[3] = y.y;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = __fmul_rn(f[e], inv);
    if constexpr (CODE == SI_KV_INT8) {
        // 1.5 * 2^23 + x, rounded half to even, has round(x) in its low bits, in two's complement
        uint32_t r[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) r[e] = __float_as_uint(__fadd_rn(f[e], 12582912.0f));
        return __byte_perm(__byte_perm(r[0], r[1], 0x0040), __byte_perm(r[2], r[3], 0x0040), 0x5410);
    } else {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(f[0], f[1]), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(f[2], f[3]), __NV_SATFINITE, __NV_E4M3);
        return lo | (hi << 16);
    }
}

}  // namespace kv
}  // namespace si
