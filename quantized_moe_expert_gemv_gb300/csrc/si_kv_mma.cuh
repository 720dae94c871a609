// si_kv_mma.cuh -- pieces of the cache's warp-level matrix kernels: the fp16
// m16n8k16 product, codes to fp16 operands, and rows to scaled fp16 operands.
//
// All products run on fp16 operands with fp32 sums: an int8 or E4M3 code is
// exact in fp16.  A row of 16-bit values (q, or an unfinished page's K or V) is
// multiplied by a power of two that brings its largest value below 128, so
// bf16's range fits and what is lost lies 2^-31 below the row's largest value;
// the power of two goes into the row's fp32 factor.  A row with a value that
// is not finite has zero operands and the factor NaN.
#pragma once
#include "si_kv_device.cuh"

namespace si {
namespace kv {

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t half2_bits(float a, float b) {  // a in the low half
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// An 8 x 8 tile of 16-bit values, in the layout of a product's result, transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// Codes of a word to fp16 pairs: (byte 0, byte 1) and (byte 2, byte 3).  int8: the
// byte with its sign bit flipped is code + 128; as the low byte of 0x6400 it reads 1024 + code + 128.
// bias() is done once for a word before its bytes may be interleaved.
template <int CODE>
__device__ __forceinline__ uint32_t code_bias(uint32_t w) {
    return CODE == SI_KV_INT8 ? w ^ 0x80808080u : w;
}
template <int CODE>
__device__ __forceinline__ void codes_to_half(uint32_t w, uint32_t &lo, uint32_t &hi) {
    if constexpr (CODE == SI_KV_INT8) {
        const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));  // 1152
        uint32_t a = __byte_perm(w, 0x64646464u, 0x4140), b = __byte_perm(w, 0x64646464u, 0x4342);
        const __half2 x = __hsub2(*reinterpret_cast<__half2 *>(&a), off);
        const __half2 y = __hsub2(*reinterpret_cast<__half2 *>(&b), off);
        lo = *reinterpret_cast<const uint32_t *>(&x);
        hi = *reinterpret_cast<const uint32_t *>(&y);
    } else {
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
            : "=r"(lo), "=r"(hi)
            : "r"(w));
    }
}

template <int CODE>
__device__ __forceinline__ void codes4(const uint4 &v, uint32_t (&to)[4]) {
    to[0] = code_bias<CODE>(v.x);
    to[1] = code_bias<CODE>(v.y);
    to[2] = code_bias<CODE>(v.z);
    to[3] = code_bias<CODE>(v.w);
}
template <int CODE>
__device__ __forceinline__ void codes2(const uint2 &v, uint32_t (&to)[2]) {
    to[0] = code_bias<CODE>(v.x);
    to[1] = code_bias<CODE>(v.y);
}

// The power-of-two scaling of a row whose largest magnitude is amax: values
// are multiplied by `mul`, and `factor` undoes it.  mul is zero, and factor NaN,
// for a row that is not finite.
__device__ __forceinline__ void row_scale(float amax, float &mul, float &factor) {
    int e = (int)((__float_as_uint(amax) >> 23) & 255) - 127 - 6;  // amax / 2^e in [64, 128)
    e = max(e, -100);
    mul = __uint_as_float((uint32_t)(127 - e) << 23);
    factor = __uint_as_float((uint32_t)(127 + e) << 23);
    if (!(amax <= 3.4e38f)) {
        mul = 0.0f;
        factor = __int_as_float(0x7fc00000);
    }
}
// max|x| over 8 packed 16-bit values (NaN becomes infinity).
template <typename T4>
__device__ __forceinline__ float amax8(const T4 &x, bool bf16) {
    // Magnitudes of either type order as their 15 low bits, and those above the infinity are NaN.
    const uint32_t w[4] = {x.x & 0x7fff7fffu, x.y & 0x7fff7fffu, x.z & 0x7fff7fffu, x.w & 0x7fff7fffu};
    const uint32_t m = __vmaxu2(__vmaxu2(w[0], w[1]), __vmaxu2(w[2], w[3]));
    const uint32_t top = max(m & 0xffffu, m >> 16);
    if (bf16) return top >= 0x7f80u ? __int_as_float(0x7f800000) : __uint_as_float(top << 16);
    return top >= 0x7c00u ? __int_as_float(0x7f800000) : __half2float(__ushort_as_half((unsigned short)top));
}
// Two packed 16-bit values times mul, as fp16.  mul = 0 gives zeros, whatever the values.
__device__ __forceinline__ uint32_t scale2(uint32_t w, float mul, bool bf16) {
    float a, b;
    if (bf16) {
        a = __uint_as_float(w << 16);
        b = __uint_as_float(w & 0xffff0000u);
    } else {
        const float2 f = __half22float2(*reinterpret_cast<__half2 *>(&w));
        a = f.x;
        b = f.y;
    }
    return mul == 0.0f ? 0u : half2_bits(a * mul, b * mul);
}

// Where 16-byte chunk c of row r lies in a tile of D-byte rows, so that the
// loads of either product's operand (rows 2m, 2m+1 with chunks of one parity;
// rows of one parity with two chunks) touch every bank once.
template <int D>
__device__ __forceinline__ uint32_t tile_at(int r, int c) {
    if constexpr (D == 64) {
        const int p = r ^ ((r >> 1) & 1);
        return (uint32_t)(p * 64 + ((c ^ (((r >> 2) & 1) << 1)) << 4));
    }
    return (uint32_t)(r * D + (((c & ~7) | ((c ^ r) & 7)) << 4));
}

// 16 bytes at src + SRC to dst + DST.
template <int DST, int SRC>
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0 + %2], [%1 + %3], 16;" ::"r"(dst), "l"(src), "n"(DST), "n"(SRC) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
template <int OFF = 0>
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4 + %5];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a), "n"(OFF));
    return v;
}
template <int OFF = 0>
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0,%1}, [%2 + %3];" : "=r"(v.x), "=r"(v.y) : "r"(a), "n"(OFF));
    return v;
}

// A warp's copy of a piece, 16 rows of D bytes that follow each other at src,
// into a tile: lane's chunks are lane + 32 k.  Rows eight apart have the same
// place but for their distance, so a lane needs few addresses.
template <int D>
struct PieceCopy {
    static constexpr int CH = D / 16, STEP = 32 / CH, DISTINCT = 8 / STEP;  // rows between a lane's chunks; addresses
    uint32_t at[DISTINCT];
    __device__ __forceinline__ void init(int lane) {
#pragma unroll
        for (int k = 0; k < DISTINCT; ++k) at[k] = tile_at<D>(lane / CH + STEP * k, lane % CH);
    }
    // chunks of `src` (already at the lane's first) to the tile at `to`, OFF bytes on
    template <int OFF>
    __device__ __forceinline__ void run(uint32_t to, const uint8_t *src) const {
        if constexpr (D == 64) {
            cp_async16<OFF, 0>(to + at[0], src);
            cp_async16<OFF + 8 * 64, 1 * 512>(to + at[0], src);
        } else if constexpr (D == 128) {
            cp_async16<OFF, 0>(to + at[0], src);
            cp_async16<OFF, 1 * 512>(to + at[1], src);
            cp_async16<OFF + 8 * 128, 2 * 512>(to + at[0], src);
            cp_async16<OFF + 8 * 128, 3 * 512>(to + at[1], src);
        } else {
            cp_async16<OFF, 0>(to + at[0], src);
            cp_async16<OFF, 1 * 512>(to + at[1], src);
            cp_async16<OFF, 2 * 512>(to + at[2], src);
            cp_async16<OFF, 3 * 512>(to + at[3], src);
            cp_async16<OFF + 8 * 256, 4 * 512>(to + at[0], src);
            cp_async16<OFF + 8 * 256, 5 * 512>(to + at[1], src);
            cp_async16<OFF + 8 * 256, 6 * 512>(to + at[2], src);
            cp_async16<OFF + 8 * 256, 7 * 512>(to + at[3], src);
        }
    }
};

// Which d's a lane's bytes of a key hold.  Lane (g, j) = (lane / 4, lane % 4).  In
// the first product its bytes of a key are D/4 values in D/64 chunks of 16: chunk
// i starts at d = k_dim(j, i), and step s of the product (k = 16) takes 4 of
// them, two for k = 2j, 2j+1 and two for k = 2j+8, 2j+9.  (The order of d is free
// as long as q has the same one.)
template <int D>
__device__ __forceinline__ constexpr int k_dim(int j, int i) {
    return D == 64 ? j * 16 : 128 * (i >> 1) + j * 32 + 16 * (i & 1);
}

// The first product's operand of one 16-bit row, this lane's D/4 values of it: op[s] of step s is
// (two values for k = 2j, 2j+1; two for k = 2j+8, 2j+9).  The four lanes of a g hold a row
// together.  The loads are apart, so that others can be under way with them; all 32 lanes call operand(), which
// returns the factor that undoes the scaling.
template <int D>
struct RowPart {
    uint4 x[D / 32];
    __device__ __forceinline__ void load(const uint16_t *src, bool live, int j) {
#pragma unroll
        for (int k = 0; k < D / 64; ++k)
#pragma unroll
            for (int z = 0; z < 2; ++z)
                x[2 * k + z] = live ? *reinterpret_cast<const uint4 *>(src + k_dim<D>(j, k) + 8 * z) : make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ float operand(bool bf16, uint2 (&op)[D / 16]) const {
        float amax = 0.0f;
#pragma unroll
        for (int k = 0; k < D / 32; ++k) amax = fmaxf(amax, amax8(x[k], bf16));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        float mul, f;
        row_scale(amax, mul, f);
#pragma unroll
        for (int st = 0; st < D / 16; ++st) {  // chunk st / 4, four values at 4 * (st % 4)
            const uint4 &v = x[2 * (st >> 2) + ((st >> 1) & 1)];
            op[st] = make_uint2(scale2(st & 1 ? v.z : v.x, mul, bf16), scale2(st & 1 ? v.w : v.y, mul, bf16));
        }
        return f;
    }
};

// The keys' operand of every step, from a tile of codes: keys g (ka[.][0], [2]) and g + 8 ([1], [3]).
// at[q]: tile_at<D>(g, k_dim(j, q) / 16) for q < 2.
template <int D>
struct KeyLoad {
    uint32_t at[D == 64 ? 1 : 2];
    __device__ __forceinline__ void init(int g, int j) {
        at[0] = tile_at<D>(g, k_dim<D>(j, 0) / 16);
        if constexpr (D > 64) at[1] = tile_at<D>(g, k_dim<D>(j, 1) / 16);
    }
    // chunk Q of key g (HI 0) or g + 8 (HI 1)
    template <int Q, int HI>
    __device__ __forceinline__ uint4 load(uint32_t tile) const {
        return lds128<128 * (Q >> 1) + 8 * D * HI>(tile + at[D == 64 ? 0 : Q & 1]);
    }
};

}  // namespace kv
}  // namespace si
