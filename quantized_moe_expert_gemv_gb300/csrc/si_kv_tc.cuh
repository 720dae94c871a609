// si_kv_tc.cuh -- pieces of the cache's tcgen05 kernels: tensor-memory stores,
// the product with its first operand in tensor memory, fp16 operand tiles in
// shared memory and their making from codes and 16-bit rows, packed fp32 pairs.
#pragma once
#include "si_kv_mma.cuh"
#include "si_tc.cuh"

namespace si {
namespace kv {

constexpr int kTileRows = 128;  // rows of an operand tile

// Tensor-memory stores and the product with its first operand in tensor memory.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
        "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
        "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// The products (M = 128, k = 16) are issued by one elected lane of a warp whose
// 32 lanes all run the issuing code: descriptors and tensor-memory addresses
// then stay in the warp's uniform registers.  Issued from a branch that one lane
// takes, each product cost 150 to 180 cycles of moving them there; so, 64, which
// is what the product itself takes at N = 128.
// D[tmem] (+)= A[smem] B[smem]; the same with A in tensor memory.
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Arrive on an mbarrier once the products that the elected lane issued so far are done.
__device__ __forceinline__ void mma_done(uint32_t mbar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(mbar)
        : "memory");
}
// Descriptor of an operand whose 64 innermost values (128 swizzled bytes) run
// along M or N: 8-row groups of K follow each other at 1024 bytes (stride
// offset), the next 64 values along M or N lie `next` bytes on (leading offset).
__device__ __forceinline__ uint64_t sdesc_sw128_mn(uint32_t smem_addr, uint32_t next) {
    return (uint64_t)((smem_addr & 0x3FFFFu) >> 4) | ((uint64_t)(next >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           (1ull << 46) | (2ull << 61);
}

// Byte offset of 16-byte unit u (8 values of d) of row r in an fp16 tile of 128
// rows: 64 values of d (128 bytes) a row and half, halves 16 KB apart.
__device__ __forceinline__ uint32_t f16_tile_at(int r, int u) {
    return (uint32_t)((u >> 3) * 16384 + r * 128 + (((u ^ r) & 7) << 4));
}
template <int OFF = 0>
__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.b32 [%0 + %5], {%1,%2,%3,%4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w), "n"(OFF) : "memory");
}

typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pk2(float a, float b) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void up2(f32x2 v, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// One row of 16-bit values into an fp16 tile, by the four neighbouring threads
// ch = 0..3 of its quad (each D/4 values): the loads, then the scaled tile.
template <int D>
struct RowLoad {
    uint4 y[D / 64][2];
    __device__ __forceinline__ void load(const uint16_t *src, bool live, int ch) {
#pragma unroll
        for (int q = 0; q < D / 64; ++q)
#pragma unroll
            for (int e = 0; e < 2; ++e)
                y[q][e] = live ? *reinterpret_cast<const uint4 *>(src + ch * 16 + 64 * q + 8 * e) : make_uint4(0, 0, 0, 0);
    }
    // Returns the factor that undoes the scaling.
    __device__ __forceinline__ float store(uint32_t tile, int row, int ch, bool bf16) const {
        float amax = 0.0f;
#pragma unroll
        for (int q = 0; q < D / 64; ++q) amax = fmaxf(amax, fmaxf(amax8(y[q][0], bf16), amax8(y[q][1], bf16)));
        const unsigned quad = 0xfu << (threadIdx.x & 28);  // (the quad may be apart from the rest of its warp)
        amax = fmaxf(amax, __shfl_xor_sync(quad, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(quad, amax, 2));
        float mul, f;
        row_scale(amax, mul, f);
#pragma unroll
        for (int q = 0; q < D / 64; ++q)
#pragma unroll
            for (int e = 0; e < 2; ++e)
                sts128(tile + f16_tile_at(row, 2 * (ch + 4 * q) + e), scale2(y[q][e].x, mul, bf16), scale2(y[q][e].y, mul, bf16),
                       scale2(y[q][e].z, mul, bf16), scale2(y[q][e].w, mul, bf16));
        return f;
    }
};

// 16 codes as two 16-byte units of an fp16 tile, OFF bytes after a0 and a1.
template <int CODE, int OFF>
__device__ __forceinline__ void codes_to_tile(const uint4 &y, uint32_t a0, uint32_t a1) {
    uint32_t o[8];
    codes_to_half<CODE>(code_bias<CODE>(y.x), o[0], o[1]);
    codes_to_half<CODE>(code_bias<CODE>(y.y), o[2], o[3]);
    codes_to_half<CODE>(code_bias<CODE>(y.z), o[4], o[5]);
    codes_to_half<CODE>(code_bias<CODE>(y.w), o[6], o[7]);
    sts128<OFF>(a0, o[0], o[1], o[2], o[3]);
    sts128<OFF>(a1, o[4], o[5], o[6], o[7]);
}

// The K (or V) rows of tokens key0 .. key0 + 127 of one kv head into an fp16
// tile, and a factor for each, by 128 threads (pt): page rows, the unfinished page's
// rows, zeros past the length.
template <int CODE, int D>
__device__ __forceinline__ void key_rows(const Ctx &c, const Seq &s, int b, int h, bool v, int key0, int log_page, bool bf16,
                                         uint32_t tile, float *factor, int pt) {
    constexpr int CC = D / 64;
    const int ch = pt & 3, r0 = pt >> 2, paged = s.len & ~(c.P - 1);
    const float nan = __int_as_float(0x7fc00000);
    for (int k = 0; k < 4; ++k) {
        const int row = r0 + 32 * k, t = key0 + row;
        float f;
        if (t < paged) {
            const int64_t p = load_page(c, b, t >> log_page);
            const uint8_t *at = (v ? c.vc : c.kc) + page_at(c, p < 0 ? 0 : p, h) + (int64_t)(t & (c.P - 1)) * D + ch * 16;
            uint4 y[CC];
#pragma unroll
            for (int q = 0; q < CC; ++q) y[q] = *reinterpret_cast<const uint4 *>(at + 64 * q);
#pragma unroll
            for (int q = 0; q < CC; ++q)
                codes_to_tile<CODE, 0>(y[q], tile + f16_tile_at(row, 2 * (ch + 4 * q)), tile + f16_tile_at(row, 2 * (ch + 4 * q) + 1));
            f = p < 0 ? nan : (v ? c.vs : c.ks)[p * c.Hk + h];
        } else {
            const bool in = t < s.len && s.slot >= 0;
            RowLoad<D> x;
            x.load((v ? c.vt : c.kt) + ring_at(c, in ? s.slot : 0, h, t), in, ch);
            f = x.store(tile, row, ch, bf16);
            if (t < s.len && s.slot < 0) f = nan;
            if (t >= s.len) f = 0.0f;
        }
        if (ch == 0) factor[row] = f;
    }
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// One row's scores of a tile of full pages (kf, vf: a factor for every 16 tokens): z raw, the first `see` of them
// visible (MASK; else all).
// The largest score: z times the factors, rounded.
template <bool MASK>
__device__ __forceinline__ float row_top(const uint32_t (&z)[4][32], const float *kf, float qf, int see) {
    float top = -INFINITY;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        auto at = [&](int k) {
            const float x = __uint_as_float(z[q >> 1][16 * (q & 1) + k]);
            return MASK && 16 * q + k >= see ? -INFINITY : x;
        };
        float a = max3(at(0), at(1), at(2)), b = max3(at(3), at(4), at(5));
        a = max3(a, at(6), at(7));
        b = max3(b, at(8), at(9));
        a = max3(a, at(10), at(11));
        b = max3(b, at(12), at(13));
        top = fmaxf(top, __fmul_rn(max3(a, b, fmaxf(at(14), at(15))), kf[q] * qf));
    }
    return top;
}
// Their weights 2^(score - m), with their sum, and in tensor memory at ts (two a column) the weights
// times V's factors and v_inv, as fp16.  m is taken from the product of z and the factors before that is rounded: off by
// up to 2^-24 m from the score that became m, nothing where m is small, but 2^30 would leave no weight or an infinite
// one.  So rows past kFar (`far`: the warp has one) take the form with MASK, which rounds the product first.  (A packed
// product and a packed sum in turn were measured to be joined into one step, hence the zero.  A third form for such
// rows costs all others registers: the prompts of si_kv_prompt.cuh took 255 to 290 us, with the sum in this form 249,
// without either 243.)
constexpr float kFar = 1048576.0f;
template <bool MASK>
__device__ __forceinline__ void row_weights(const uint32_t (&z)[4][32], const float *kf, const float *vf, float qf, float v_inv,
                                            float m, bool far, int see, uint32_t ts, f32x2 &sum) {
    const float now = MASK && far ? 0.0f : -m, then = MASK && far ? -m : 0.0f;
    const f32x2 now2 = pk2(now, now), then2 = pk2(then, then);
    f32x2 s0 = pk2(0.0f, 0.0f), s1 = s0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        float y[32];  // one step for all 32 values before the next: each step's are independent
#pragma unroll
        for (int k = 0; k < 32; k += 2) {
            const float f = kf[2 * q + k / 16] * qf;
            f32x2 s = fma2(pk2(__uint_as_float(z[q][k]), __uint_as_float(z[q][k + 1])), pk2(f, f), now2);
            if (MASK) s = add2(s, then2);
            up2(s, y[k], y[k + 1]);
        }
#pragma unroll
        for (int k = 0; k < 32; ++k) {
            y[k] = ex2(y[k]);
            if (MASK && 32 * q + k >= see) y[k] = 0.0f;
        }
        uint32_t p[16];
#pragma unroll
        for (int k = 0; k < 32; k += 2) {
            const f32x2 pp = pk2(y[k], y[k + 1]);
            if (k & 2)
                s1 = add2(s1, pp);
            else
                s0 = add2(s0, pp);
            const float w = vf[2 * q + k / 16] * v_inv;
            float w0, w1;
            up2(mul2(pp, pk2(w, w)), w0, w1);
            if (MASK && 32 * q + k >= see) w0 = 0.0f;  // (whatever V's factor is)
            if (MASK && 32 * q + k + 1 >= see) w1 = 0.0f;
            p[k / 2] = half2_bits(w0, w1);
        }
        tmem_st16(ts + 16 * q, p);
    }
    sum = add2(s0, s1);
}

}  // namespace kv
}  // namespace si
