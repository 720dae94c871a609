// si_fp8_matmul.cu -- the matrix product of quantised rows and weights.
//
//   out[t][n] = add[t][n] + sum_kb (sa[kb][t] * sw[n/128][kb]) * dot_kb(t, n)
//
// dot_kb, the sum over one block of 128 columns, comes from the tensor cores
// (kind::f8f6f4: E4M3 operands, products exact, 32-bit sums in tensor memory).
// The scales are general 32-bit numbers, so a block's sums leave tensor memory
// once they are complete and are added, scaled, to 32-bit sums in registers
// while the tensor cores work on the next block in another part of tensor
// memory.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>

#include "si_fp8_device.cuh"
#include "si_tc.cuh"

namespace si {
namespace fp8 {
namespace {

constexpr long long kDrain = 4000000000LL;  // cycles: the longest wait for what is in flight, after another ran out
constexpr long long kLinger = 1000000LL;

// Instruction descriptor of kind::f8f6f4 with E4M3 operands (type fields 0), both K-major, and fp32 sums.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(int M, int N) {
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// D[tmem] = A[smem] B[smem]^T over 128 columns: four products of 32 (a row of 128 swizzled bytes), by one elected
// lane of a warp whose 32 lanes all run the code.
__device__ __forceinline__ void mma_k128(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc) {
    asm volatile(
        "{\n\t.reg .pred e, p, q;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.u32 p, %10, %10;\n\t"
        "setp.eq.u32 q, %10, %10;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %5, %9, p;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %2, %6, %9, q;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %3, %7, %9, q;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %4, %8, %9, q;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(a + 2), "l"(a + 4), "l"(a + 6), "l"(b), "l"(b + 2), "l"(b + 4), "l"(b + 6), "r"(idesc), "r"(0u)
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

__device__ __forceinline__ float load_value(const Mat &m, int64_t at) {
    if (m.dtype == SI_FP8_F32) return static_cast<const float *>(m.p)[at];
    const uint32_t w = static_cast<const uint16_t *>(m.p)[at];
    return unpack16(w, m.dtype == SI_FP8_BF16).x;
}
__device__ __forceinline__ void store_value(const Mat &m, int64_t at, float v) {
    if (m.dtype == SI_FP8_F32) static_cast<float *>(m.p)[at] = v;
    else static_cast<uint16_t *>(m.p)[at] = (uint16_t)pack16(v, 0.0f, m.dtype == SI_FP8_BF16);
}

constexpr int kTile = 128 * 128;  // bytes of an operand tile: 128 rows x 128 columns

// Wait for phase `parity` of an mbarrier for at most `budget` cycles.  A phase that is complete costs one poll: the clock
// is not read before.
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity, long long budget) {
    if (mbar_try_wait(bar, parity)) return true;
    return mbar_wait_spin(bar, parity, budget);
}
// The last phases of a ring of N barriers of which `n` were used in all: nobody else waits for them, and they complete before
// the CTA gives the barriers' memory back.  After a wait that ran out they may never.
template <int N>
__device__ __forceinline__ void drain(uint32_t bars, int n, long long budget, volatile int *err) {
    for (int q = n > N ? n - N : 0; q < n && !*err; ++q)
        if (!mbar_wait_bounded(bars + 8 * (q % N), (q / N) & 1, budget)) break;
}
// A place in a ring of N barriers, and the parity of its next phase.
template <int N>
struct Ring {
    uint32_t at = 0, phase = 0;
    __device__ __forceinline__ void next() {
        if (++at == N) {
            at = 0;
            phase ^= 1;
        }
    }
};

// Four neighbouring values of a matrix whose row stride is a multiple of four.
__device__ __forceinline__ void add4(const Mat &m, int64_t at, float (&v)[4]) {
    if (m.dtype == SI_FP8_F32) {
        const float4 x = *reinterpret_cast<const float4 *>(static_cast<const float *>(m.p) + at);
        v[0] += x.x;
        v[1] += x.y;
        v[2] += x.z;
        v[3] += x.w;
        return;
    }
    const uint2 w = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(m.p) + at);
    const float2 x = unpack16(w.x, m.dtype == SI_FP8_BF16), y = unpack16(w.y, m.dtype == SI_FP8_BF16);
    v[0] += x.x;
    v[1] += x.y;
    v[2] += y.x;
    v[3] += y.y;
}
__device__ __forceinline__ void store4(const Mat &m, int64_t at, const float (&v)[4]) {
    if (m.dtype == SI_FP8_F32)
        *reinterpret_cast<float4 *>(static_cast<float *>(m.p) + at) = make_float4(v[0], v[1], v[2], v[3]);
    else
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(m.p) + at) =
            make_uint2(pack16(v[0], v[1], m.dtype == SI_FP8_BF16), pack16(v[2], v[3], m.dtype == SI_FP8_BF16));
}

// ---------------------------------------------------------------- few rows
template <int TN>
struct Few {
    static constexpr int kScales = kTile + TN * 128;                  // of a stage: weights, rows, the rows' scales
    static constexpr int kStage = (kScales + TN * 4 + 1023) & ~1023;  // (operand tiles begin at multiples of 1024 bytes)
    static constexpr int kStages = 3;
    static constexpr int kCtas = TN == 64 ? 2 : 3;                    // of an SM, where no CTA shares its tile
    static constexpr int kBufs = 4;                                   // sums of a block in tensor memory
    static constexpr int kParts = kStages * kStage;                   // the CTAs' sums: [CTA][row][128 weights' rows]
    static constexpr int kSmemOne = kParts + 1024;                    // (of one CTA alone: where its stages were)
    static constexpr int kSmem = kSmemOne + TN * 512;
    static_assert(TN * 512 <= kParts && kCtas * (kSmemOne + 1536) <= 233472 && 2 * (kSmem + 1536) <= 233472, "shared memory of an SM");
    static_assert(kCtas * TN * kBufs <= 512, "tensor memory of an SM");
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
                 "r"(bytes), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t *v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(taddr)
        : "memory");
}

// Store v at shared-memory address `to` (as it is in this CTA) of CTA `rank` of the cluster, its four bytes counted by that
// CTA's mbarrier at `bar`.
__device__ __forceinline__ void send(uint32_t to, uint32_t bar, uint32_t rank, float v) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(mapa_shared(to, rank)),
                 "r"(__float_as_uint(v)), "r"(mapa_shared(bar, rank))
                 : "memory");
}

// Few rows: the weights' bytes are what it costs.  The weights are the first operand (128 of their rows are the products'
// M) and the rows the second (N = TN, of which the tile may hold fewer), so that no product works on rows that are not
// there.  A cluster of S CTAs shares a tile, each with its part of the blocks of columns: that brings enough loads into
// flight where there are few tiles.  Row t's sums are added up by CTA t mod S, which the others send theirs, in the CTAs'
// order.  1 x 5120 x 2048: 3.6 us in a graph (start, copy, four blocks, join); 1 x 100003 x 2048: 34.6 us, 5.9 TB/s.
// Warp 0 loads, warp 1 issues the products, and warps 2 to 5 add the blocks' sums up, one row of the weights a thread.
template <int TN>
__global__ void __launch_bounds__(192, Few<TN>::kCtas) k_matmul_few(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_w,
                                                    const MatmulArgs a, int t_tiles, int S) {
    using C = Few<TN>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ __align__(8) uint64_t s_bar[2 * C::kStages + 2 * C::kBufs + 3];
    __shared__ uint32_t s_taddr;
    __shared__ int s_err;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int rank = (int)cluster_ctarank(), tile = blockIdx.x / S;
    const int nt = tile / t_tiles, t0 = tile % t_tiles * TN, rows = min(TN, a.T - t0);
    const int kb0 = (int)((int64_t)a.KB * rank / S), nk = (int)((int64_t)a.KB * (rank + 1) / S) - kb0;
    const uint32_t full = smem_addr(s_bar), empty = full + 8 * C::kStages, d_full = empty + 8 * C::kStages, d_empty = d_full + 8 * C::kBufs,
                   fin = d_empty + 8 * C::kBufs, never = fin + 8, parts = never + 8;
    const int mine = (rows - rank + S - 1) / S;  // rows that this CTA adds up and stores
    volatile int *err = &s_err;
    if (threadIdx.x == 0) {
        s_err = 0;
        prefetch_tensormap(&tm_a);
        prefetch_tensormap(&tm_w);
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(full + 8 * s, 1);
            mbar_init(empty + 8 * s, 5);  // the products, and the four warps that read the scales
        }
        for (int b = 0; b < C::kBufs; ++b) {
            mbar_init(d_full + 8 * b, 1);
            mbar_init(d_empty + 8 * b, 4);
        }
        mbar_init(fin, 1);
        mbar_init(never, 1);
        mbar_init(parts, 1);
        fence_mbar_init();
        mbar_arrive_expect_tx(parts, (uint32_t)(S == 1 ? 0 : mine * S) * 512);
    }
    if (warp == 1) {
        tc::tmem_alloc(smem_addr(&s_taddr), TN * C::kBufs);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");  // this CTA's barriers are there
    tc::fence_after_sync();
    start_after();
    const uint32_t taddr = __shfl_sync(0xffffffffu, s_taddr, 0);
    auto fail = [&]() {
        set_status(a.status, SI_ERR_TIMEOUT);
        *err = 1;
    };

    if (warp == 0) {
        if (lane == 0) {
            Ring<C::kStages> st;
            int k = 0;
            const uint32_t scale_bytes = (uint32_t)((rows + 3) & ~3) * 4;
            if (a.fault_wait && !mbar_wait_spin(never, 0, a.wait_budget)) fail();
            for (; k < nk && !*err; ++k, st.next()) {
                const uint32_t bar = full + 8 * st.at;
                if (k >= C::kStages && !wait_phase(empty + 8 * st.at, st.phase ^ 1, a.wait_budget)) {
                    fail();
                    break;
                }
                const uint32_t dst = smem_addr(sm) + st.at * C::kStage;
                mbar_arrive_expect_tx(bar, kTile + TN * 128 + scale_bytes);
                tma_load_2d_plain(dst, &tm_w, (kb0 + k) * 128, nt * 128, bar);
                tma_load_2d_plain(dst + kTile, &tm_a, (kb0 + k) * 128, t0, bar);
                bulk_load(dst + C::kScales, a.a_scale + (kb0 + k) * a.a_stride + t0, scale_bytes, bar);
            }
            for (int q = k > C::kStages ? k - C::kStages : 0; q < k; ++q)  // what was issued has landed
                mbar_wait_bounded(full + 8 * (q % C::kStages), (q / C::kStages) & 1, kDrain);
            drain<C::kStages>(empty, k, a.wait_budget, err);
        }
        __syncwarp();
    } else if (warp == 1) {
        const uint64_t desc = tc::sdesc_sw128(smem_addr(sm));
        Ring<C::kStages> st;
        Ring<C::kBufs> buf;
        for (int k = 0; k < nk; ++k) {
            const bool ok = wait_phase(full + 8 * st.at, st.phase, a.wait_budget) &&
                            (k < C::kBufs || wait_phase(d_empty + 8 * buf.at, buf.phase ^ 1, a.wait_budget));
            if (!__all_sync(0xffffffffu, ok)) {
                if (lane == 0) fail();
                break;
            }
            tc::fence_after_sync();
            const uint64_t wd = desc + (uint64_t)(st.at * (C::kStage >> 4));
            mma_k128(taddr + TN * buf.at, wd, wd + (kTile >> 4), idesc_e4m3_f32(128, TN));
            mma_done(d_full + 8 * buf.at);
            mma_done(empty + 8 * st.at);
            st.next();
            buf.next();
        }
        mma_done(fin);  // every product is done before the CTA gives its memory back
        mbar_wait_spin(fin, 0, kDrain);
        __syncwarp();
    } else {
        const int quad = warp & 3;  // the tensor-memory lanes that this warp reaches
        const int r = quad * 32 + lane;
        const float *const w_scale = a.w_scale + (int64_t)nt * a.KB + kb0;
        f32x2 acc[TN / 2];
#pragma unroll
        for (int i = 0; i < TN / 2; ++i) acc[i] = 0ull;
        Ring<C::kStages> st;
        Ring<C::kBufs> buf;
        float sw = nk > 0 ? w_scale[0] : 0.0f;
        // (a wait that runs out does not end the loop: no later one waits, and what is stored is as good as any)
        auto wait = [&](uint32_t bar, uint32_t phase) {
            if (!mbar_try_wait(bar, phase) && !*err && !mbar_wait_spin(bar, phase, a.wait_budget)) fail();
        };
        for (int k = 0; k < nk; ++k) {
            const float ahead = k + 1 < nk ? w_scale[k + 1] : 0.0f;
            const f32x2 sw2 = pack2(sw, sw);
            wait(full + 8 * st.at, st.phase);  // (the rows' scales)
            wait(d_full + 8 * buf.at, buf.phase);
            __syncwarp();
            tc::fence_after_sync();
            const uint32_t from = taddr + ((uint32_t)(32 * quad) << 16) + TN * buf.at;
            const uint32_t scales = smem_addr(sm) + st.at * C::kStage + C::kScales;
#pragma unroll
            for (int q = 0; q < TN / 16; ++q) {
                uint32_t v[16];
                tmem_ld16(from + 16 * q, v);
                tc::tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    f32x2 s0, s1;
                    asm volatile("ld.shared.v2.b64 {%0,%1}, [%2];" : "=l"(s0), "=l"(s1) : "r"(scales + (16 * q + 4 * e) * 4) : "memory");
                    asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(s0) : "l"(sw2));
                    asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(s1) : "l"(sw2));
                    ffma2(acc[8 * q + 2 * e], pack2(__uint_as_float(v[4 * e]), __uint_as_float(v[4 * e + 1])), s0);
                    ffma2(acc[8 * q + 2 * e + 1], pack2(__uint_as_float(v[4 * e + 2]), __uint_as_float(v[4 * e + 3])), s1);
                }
            }
            // The scales have been read before the next copy into this stage: generic reads before asynchronous writes, which
            // the barrier alone does not order (without the fence some builds read a later block's last scales).
            tc::fence_proxy_async_smem();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(d_empty + 8 * buf.at);
                mbar_arrive(empty + 8 * st.at);
            }
            st.next();
            buf.next();
            sw = ahead;
        }
        __syncwarp();  // (the barriers below are the warp's)
        // Sums to the CTAs that store them: [CTA that they come from][row / S][128 rows of the weights].
        const float *const part = reinterpret_cast<const float *>(sm + (S == 1 ? 0 : C::kParts));
        const uint32_t part_addr = smem_addr(part) + 4 * r;
        const int log_s = 31 - __clz(S), per = TN >> log_s;
        if (S == 1) {
            asm volatile("bar.sync 1, 128;" ::: "memory");  // (the last block's scales have been read)
#pragma unroll
            for (int c = 0; c < TN; c += 2) {
                const float2 f = unpack2(acc[c / 2]);
                asm volatile("st.shared.f32 [%0], %1;" ::"r"(part_addr + c * 512), "f"(f.x) : "memory");
                asm volatile("st.shared.f32 [%0], %1;" ::"r"(part_addr + c * 512 + 512), "f"(f.y) : "memory");
            }
            asm volatile("bar.sync 1, 128;" ::: "memory");
        } else {
            cluster_wait();  // the other CTAs' barriers are there
            const uint32_t to = part_addr + rank * per * 512;
#pragma unroll
            for (int q = 0; q < TN; q += 16) {
                if (q < rows) {
#pragma unroll
                    for (int c = q; c < q + 16; ++c) {
                        const float2 f = unpack2(acc[c / 2]);
                        if (c < rows) send(to + (c >> log_s) * 512, parts, c & (S - 1), c & 1 ? f.y : f.x);
                    }
                }
            }
            // (the others always send theirs, also after a wait of their own ran out: no CTA ends before)
            if (mine > 0 && !mbar_wait_spin_cluster(parts, 0, a.wait_budget)) {
                fail();
                mbar_wait_spin_cluster(parts, 0, kDrain);
            }
        }
        // A row a warp at a time, four columns a lane.
        const int n0 = nt * 128 + 4 * lane, i0 = warp - 2;
        const bool whole = a.out.stride % 4 == 0 && (!a.add.p || a.add.stride % 4 == 0) && n0 + 4 <= a.N;
#pragma unroll 2
        for (int i = i0; i < mine; i += 4) {
            const int64_t row = (int64_t)t0 + rank + i * S;
            float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            for (int o = 0; o < S; ++o) {
                const float4 x = *reinterpret_cast<const float4 *>(part + (o * per + i) * 128 + 4 * lane);
                v[0] += x.x;
                v[1] += x.y;
                v[2] += x.z;
                v[3] += x.w;
            }
            if (whole) {
                if (a.add.p) add4(a.add, row * a.add.stride + n0, v);
                store4(a.out, row * a.out.stride + n0, v);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (n0 + e < a.N) {
                        if (a.add.p) v[e] += load_value(a.add, row * a.add.stride + n0 + e);
                        store_value(a.out, row * a.out.stride + n0 + e, v[e]);
                    }
            }
        }
    }
    __syncwarp();
    if (warp < 2 || S == 1) cluster_wait();
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        tc::fence_after_sync();
        tc::tmem_dealloc(taddr, TN * C::kBufs);
    }
}

// ---------------------------------------------------------------- CTA pairs
// The four products of a block of 128 columns by a pair of CTAs (M = 256: 128 rows of A and half of B from each one's
// shared memory), by one elected lane of the even CTA's warp.
__device__ __forceinline__ void mma_pair_k128(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc) {
    asm volatile(
        "{\n\t.reg .pred e, p, q;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.u32 p, %10, %10;\n\t"
        "setp.eq.u32 q, %10, %10;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %5, %9, p;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %2, %6, %9, q;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %3, %7, %9, q;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %4, %8, %9, q;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(a + 2), "l"(a + 4), "l"(a + 6), "l"(b), "l"(b + 2), "l"(b + 4), "l"(b + 6), "r"(idesc), "r"(0u)
        : "memory");
}
// Arrive on the mbarrier at this offset in both CTAs once the products that the elected lane issued so far are done.
__device__ __forceinline__ void mma_pair_done(uint32_t mbar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(mbar),
        "h"((uint16_t)3)
        : "memory");
}
// Load a box into this CTA's shared memory that completes on an mbarrier of either CTA of the pair.
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const void *tmap, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 "
        "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
// Arrive on an mbarrier of either CTA of the pair after reads of tensor memory (ordered by the fences of tcgen05): there
// is nothing in other memory to publish, and a release at cluster scope, like an acquire of it by the waiting side,
// would wait for all loads and stores in flight (a block took nine times as long).
__device__ __forceinline__ void mbar_arrive_pair(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
// Eight neighbouring values of `add`, all of them there.
__device__ __forceinline__ void add8(const Mat &m, int64_t at, float (&v)[8]) {
    float r[8];
    if (m.dtype == SI_FP8_F32) widen8<true>(load8<true>(m.p, at), false, r);
    else widen8<false>(load8<false>(m.p, at), m.dtype == SI_FP8_BF16, r);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += r[i];
}

// Rows of `pitch` bytes in a warp's shared memory (16-byte unit u of row r at unit u ^ (r & 7)) to memory, W bytes a lane:
// places are multiples of W bytes.  `bytes` of a row are copied, a multiple of two.
template <int W>
__device__ __forceinline__ void copy_rows_by(uint8_t *dst, int64_t stride, uint32_t stage, int rows, int bytes, int pitch) {
    const int lane = threadIdx.x & 31;
    const int lanes = min(32, pitch / W), step = 32 / lanes, r0 = lane / lanes;  // lanes of a row, rows at a time
    for (int b = lane % lanes * W; b < bytes; b += lanes * W) {
        const bool whole = b + W <= bytes;
        uint8_t *p = dst + r0 * stride + b;
        for (int r = r0; r < rows; r += 8 * step) {  // (eight rows' reads before their stores)
            uint32_t v[8][2];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int row = r + u * step;
                const uint32_t from = stage + row * pitch + (((b >> 4) ^ (row & 7)) << 4) + (b & 15);
                if (row < rows) {
                    if (W == 8) asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v[u][0]), "=r"(v[u][1]) : "r"(from) : "memory");
                    else if (W == 4) asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v[u][0]) : "r"(from) : "memory");
                    else asm volatile("ld.shared.u16 %0, [%1];" : "=r"(v[u][0]) : "r"(from) : "memory");
                }
            }
#pragma unroll
            for (int u = 0; u < 8; ++u, p += step * stride) {
                if (r + u * step >= rows) continue;
                if (whole) {
                    if (W == 8) *reinterpret_cast<uint2 *>(p) = make_uint2(v[u][0], v[u][1]);
                    else if (W == 4) *reinterpret_cast<uint32_t *>(p) = v[u][0];
                    else *reinterpret_cast<uint16_t *>(p) = (uint16_t)v[u][0];
                } else {  // (the row ends within these bytes)
#pragma unroll
                    for (int h = 0; h + 2 < W; h += 2)
                        if (b + h + 2 <= bytes) *reinterpret_cast<uint16_t *>(p + h) = (uint16_t)(v[u][h / 4] >> (h % 4 * 8));
                }
            }
        }
    }
}
__device__ __noinline__ void copy_rows(uint8_t *dst, int64_t stride, uint32_t stage, int rows, int bytes, int pitch) {
    if (stride % 8 == 0) copy_rows_by<8>(dst, stride, stage, rows, bytes, pitch);
    else if (stride % 4 == 0) copy_rows_by<4>(dst, stride, stage, rows, bytes, pitch);
    else copy_rows_by<2>(dst, stride, stage, rows, bytes, pitch);
}
// NC columns of 32 rows, one row a lane, to an `out` whose rows begin anywhere, through a warp's 8 KB of shared memory, so
// that the lanes of a store hold neighbouring columns: rows' pieces are as long as they can be, for the parts of 32 bytes
// at their ends cost most (pieces of 32 columns: 4096 x 5121 x 2048 62 us).
template <int NC>
__device__ __forceinline__ void store_odd(const MatmulArgs &a, uint32_t stage, int row0, int n0, const f32x2 *acc) {
    const int lane = threadIdx.x & 31;
    const int size = a.out.dtype == SI_FP8_F32 ? 4 : 2;
    const int64_t stride = a.out.stride * size;
    const int rows = min(32, a.T - row0), bytes = min(NC, a.N - n0) * size;
    uint8_t *const dst = static_cast<uint8_t *>(a.out.p) + (int64_t)row0 * stride + (int64_t)n0 * size;
    if (size == 2) {
        const bool bf16 = a.out.dtype == SI_FP8_BF16;
#pragma unroll
        for (int u = 0; u < NC / 8; ++u) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = unpack2(acc[4 * u + i]);
                w[i] = pack16(f.x, f.y, bf16);
            }
            asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(stage + lane * (2 * NC) + ((u ^ (lane & 7)) << 4)), "r"(w[0]),
                         "r"(w[1]), "r"(w[2]), "r"(w[3])
                         : "memory");
        }
        __syncwarp();
        copy_rows(dst, stride, stage, rows, bytes, 2 * NC);
    } else {  // (16 rows fit)
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
            if (lane >> 4 == h) {
#pragma unroll
                for (int u = 0; u < NC / 4; ++u) {
                    const float2 x = unpack2(acc[2 * u]), y = unpack2(acc[2 * u + 1]);
                    asm volatile("st.shared.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(stage + (lane & 15) * (4 * NC) + ((u ^ (lane & 7)) << 4)),
                                 "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y)
                                 : "memory");
                }
            }
            __syncwarp();
            copy_rows(dst + 16 * h * stride, stride, stage, min(16, rows - 16 * h), bytes, 4 * NC);
            __syncwarp();
        }
    }
    __syncwarp();
}
// Add eight neighbouring values of `add` (fewer at the end of a row) to eight sums.
__device__ __forceinline__ void add_to(const MatmulArgs &a, bool whole, int64_t row, int n, f32x2 *acc) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = unpack2(acc[i]);
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
    if (whole && n + 8 <= a.N) add8(a.add, row * a.add.stride + n, v);
    else
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (n + i < a.N) v[i] += load_value(a.add, row * a.add.stride + n + i);
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = pack2(v[2 * i], v[2 * i + 1]);
}
// A box of 32 rows x 128 bytes of `out`, one row a lane, from COLS sums a lane, into shared memory as the tensor map of
// `out` swizzles it.
template <int COLS>
__device__ __forceinline__ void fill_box(uint32_t box, const f32x2 *acc, bool bf16) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (COLS == 64) {
                const float2 f = unpack2(acc[4 * u + i]);
                w[i] = pack16(f.x, f.y, bf16);
            } else {
                const float2 f = unpack2(acc[2 * u + i / 2]);
                w[i] = __float_as_uint(i & 1 ? f.y : f.x);
            }
        }
        asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(box + lane * 128 + ((u ^ (lane & 7)) << 4)), "r"(w[0]), "r"(w[1]),
                     "r"(w[2]), "r"(w[3])
                     : "memory");
    }
}
// Add a box of 32 rows x 64 16-bit values, one row a lane, to a lane's sums.
__device__ __forceinline__ void add_box(uint32_t box, f32x2 *acc, bool bf16) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
        uint32_t w[4];
        asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                     : "r"(box + lane * 128 + ((u ^ (lane & 7)) << 4))
                     : "memory");
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = unpack16(w[i], bf16), g = unpack2(acc[4 * u + i]);
            acc[4 * u + i] = pack2(f.x + g.x, f.y + g.y);
        }
    }
}
__device__ __forceinline__ void tma_store(const void *tmap, int x, int y, uint32_t src) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];\n\tcp.async.bulk.commit_group;" ::"l"(
                     reinterpret_cast<uint64_t>(tmap)),
                 "r"(x), "r"(y), "r"(src)
                 : "memory");
}
// Store the NC columns of a warp's 32 rows box by box; two boxes of shared memory in turn, of which the one to be filled
// has been read.  (A tensor-map store writes whole 16 bytes also where the row ends within them, and zeros over what lies
// behind the row: such ends are stored by store_odd.)
template <int NC, int COLS>
__device__ __forceinline__ void store_boxes(const MatmulArgs &a, const void *tmap, uint32_t stage, int row0, int n0, const f32x2 (&acc)[NC / 2]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int q = 0; q < NC / COLS; ++q) {
        const uint32_t box = stage + (q & 1) * 4096;
        const int n = n0 + q * COLS;
        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
        __syncwarp();
        fill_box<COLS>(box, &acc[q * COLS / 2], a.out.dtype == SI_FP8_BF16);
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            if (n < a.N) tma_store(tmap, n, row0, box);
            else asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        }
    }
    if ((NC / COLS) & 1) {  // (the boxes' turns begin anew with each tile)
        if (lane == 0) asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    }
}

// Tile number i of m x n tiles: eight tiles of rows together, so that the tiles at work at one time share operands.
struct TileAt {
    int m, n;
};
__device__ __forceinline__ TileAt tile_at(int i, int m_tiles, int n_tiles) {
    const int group = i / (8 * n_tiles), in = i - group * 8 * n_tiles;
    const int high = min(8, m_tiles - 8 * group);
    return TileAt{8 * group + in % high, in / high};
}

template <int NT>
struct Many {
    static constexpr int kB = NT * 64;                      // bytes of a CTA's half of the weights' tile
    static constexpr int kStage = kTile + kB;
    static constexpr int kStages = NT == 256 ? 5 : 6;
    static constexpr int kBufs = NT == 256 ? 2 : 4;         // sums of a block in tensor memory
    static constexpr int kOut = kStages * kStage;           // 8 KB for each epilogue warp
    static constexpr int kSmem = kOut + 8 * 8192 + 1024;
};
static_assert(Many<256>::kSmem + 512 <= 232448 && Many<128>::kSmem + 512 <= 232448, "shared memory of a CTA");
constexpr int kManyThreads = 384;
// Registers a thread: the launch gives 168 to each of the 12 warps, of which the first four hand on what the epilogue's
// eight need for 128 sums: 4 * 40 + 8 * 232 = 12 * 168.
constexpr int kRegsLoad = 40, kRegsSum = 232;
template <int N>
__device__ __forceinline__ void regs_down() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_up() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// Many rows: a pair of CTAs works on tiles of 256 rows x NT columns, one after the other.  Warp 0 loads this CTA's 128
// rows and its half of the weights' rows, the even CTA's warp 1 issues the products, and warps 4 to 11 add the blocks' sums
// up in registers: a thread has one row and half of the tile's columns.
// What bounds it: a block's products take 512 cycles at NT = 256 (600 beside the copies into shared memory), but with two
// buffers of sums the next but one waits until all of a block's sums have been read, a chain of about 690 cycles a block
// (signal 72, reading about 450, the slower CTA's signal to the issuing warp 259).  4096 x 5120 x 2048: 39 us, 2.2 PFLOP/s;
// 8192^3: 350 us, 3.14 PFLOP/s (in long runs at the power limit 2.5 to 2.9).
// MODE, a kernel for each, as what one does not need costs its loop registers: kPlain stores `out` by boxes; kAddBoxes also
// has `add` by boxes (16-bit values of out's type): a box is fetched while the blocks are added up, into the shared memory
// that its outputs leave from; kAny takes every other case (rows that begin or end anywhere, `add` of another type or one
// row for all).
enum { kPlain, kAddBoxes, kAny };
template <int NT, int MODE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kManyThreads, 1)
    k_matmul_many(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_w,
                  const __grid_constant__ CUtensorMap tm_out, const __grid_constant__ CUtensorMap tm_add, const MatmulArgs a, int boxes,
                  int m_tiles, int n_tiles) {
    using C = Many<NT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ __align__(8) uint64_t s_bar[2 * C::kStages + 2 * C::kBufs + 2 + 16];
    __shared__ uint32_t s_taddr;
    __shared__ int s_err;
    // (the same in all lanes, and known to be: addresses and descriptors stay in the warp's uniform registers)
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int rank = (int)cluster_ctarank(), pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    const int tiles = m_tiles * n_tiles;
    const uint32_t full = smem_addr(s_bar), empty = full + 8 * C::kStages, d_full = empty + 8 * C::kStages, d_empty = d_full + 8 * C::kBufs,
                   fin = d_empty + 8 * C::kBufs, never = fin + 8, add_full = never + 8;  // (two boxes a warp)
    volatile int *err = &s_err;
    if (threadIdx.x == 0) {
        s_err = 0;
        prefetch_tensormap(&tm_a);
        prefetch_tensormap(&tm_w);
        if (MODE != kAny || boxes) prefetch_tensormap(&tm_out);
        if (MODE == kAddBoxes) prefetch_tensormap(&tm_add);
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(full + 8 * s, 1);   // (the even CTA's counts both CTAs' bytes)
            mbar_init(empty + 8 * s, 1);
        }
        for (int b = 0; b < C::kBufs; ++b) {
            mbar_init(d_full + 8 * b, 1);
            mbar_init(d_empty + 8 * b, 16);  // the epilogue warps of both CTAs
        }
        mbar_init(fin, 1);
        mbar_init(never, 1);
        for (int b = 0; b < 16; ++b) mbar_init(add_full + 8 * b, 1);
        fence_mbar_init();
    }
    if (warp == 1) {
        tc::tmem_alloc_pair(smem_addr(&s_taddr), 512);
        tc::tmem_relinquish_pair();
    }
    tc::fence_before_sync();
    __syncthreads();
    cluster_sync();  // both CTAs' barriers are there before anything arrives from the other
    tc::fence_after_sync();
    start_after();
    const uint32_t taddr = __shfl_sync(0xffffffffu, s_taddr, 0);
    auto fail = [&]() {
        set_status(a.status, SI_ERR_TIMEOUT);
        *err = 1;
    };

    if (warp < 4) {
        regs_down<kRegsLoad>();
        if (warp == 0 && lane == 0) {
            const uint32_t lead_full = mapa_shared(full, 0);
            Ring<C::kStages> st;
            int it = 0;
            if (a.fault_wait && !mbar_wait_spin(never, 0, a.wait_budget)) fail();
            for (int i = pair; i < tiles && !*err; i += pairs) {
                const TileAt t = tile_at(i, m_tiles, n_tiles);
                for (int kb = 0; kb < a.KB; ++kb, ++it, st.next()) {
                    const uint32_t bar = 8 * st.at;
                    if (it >= C::kStages && !wait_phase(empty + bar, st.phase ^ 1, a.wait_budget)) {
                        fail();
                        break;
                    }
                    const uint32_t dst = smem_addr(sm) + st.at * C::kStage;
                    if (rank == 0) mbar_arrive_expect_tx(full + bar, 2 * C::kStage);
                    tma_load_pair(dst, &tm_a, kb * 128, t.m * 256 + rank * 128, lead_full + bar);
                    tma_load_pair(dst + kTile, &tm_w, kb * 128, t.n * NT + rank * (NT / 2), lead_full + bar);
                }
            }
            if (rank == 0)  // what both CTAs issued has landed
                for (int q = it > C::kStages ? it - C::kStages : 0; q < it; ++q)
                    mbar_wait_bounded(full + 8 * (q % C::kStages), (q / C::kStages) & 1, kDrain);
            drain<C::kStages>(empty, it, a.wait_budget, err);
        } else if (warp == 1 && rank == 0) {
            const uint64_t desc = tc::sdesc_sw128(smem_addr(sm));
            Ring<C::kStages> st;
            Ring<C::kBufs> buf;
            const int n = (tiles - pair + pairs - 1) / pairs * a.KB;
            for (int it = 0; it < n; ++it) {
                const uint32_t b = buf.at;
                const bool ok = wait_phase(full + 8 * st.at, st.phase, a.wait_budget) &&
                                (it < C::kBufs || wait_phase(d_empty + 8 * b, buf.phase ^ 1, a.wait_budget));
                if (!__all_sync(0xffffffffu, ok)) {
                    if (lane == 0) fail();
                    break;
                }
                tc::fence_after_sync();
                const uint64_t ad = desc + (uint64_t)(st.at * (C::kStage >> 4));
                mma_pair_k128(taddr + NT * b, ad, ad + (kTile >> 4), idesc_e4m3_f32(256, NT));
                mma_pair_done(d_full + 8 * b);
                mma_pair_done(empty + 8 * st.at);
                st.next();
                buf.next();
            }
            mma_pair_done(fin);
        }
        __syncwarp();
    } else {
        regs_up<kRegsSum>();
        constexpr int NC = NT / 2;                            // columns of this warp
        const int quad = warp & 3, half = (warp - 4) >> 2;    // tensor-memory lanes; which columns
        const uint32_t lane_addr = taddr + ((uint32_t)(32 * quad) << 16) + NC * half;
        const uint32_t stage = smem_addr(sm) + C::kOut + (warp - 4) * 8192;
        const uint32_t lead_d_empty = mapa_shared(d_empty, 0);
        const bool add_whole = a.add.stride * (a.add.dtype == SI_FP8_F32 ? 4 : 2) % 16 == 0;
        // A block's scales are fetched four blocks ahead (at a tile's end, for the first blocks of the next one), each into
        // a register of its own: moved from one to another it would be waited for at once.  Rows and columns past the ends
        // take the last one's scale; their sums are not stored.
        struct Scales {
            uint32_t a, w;  // where this thread's row, and this warp's weights, have their first scale
        };
        const uint32_t a_stride = (uint32_t)a.a_stride;
        auto scales_of = [&](int i) {
            const TileAt t = tile_at(min(i, tiles - 1), m_tiles, n_tiles);
            const int row = t.m * 256 + rank * 128 + quad * 32 + lane, nb = (t.n * NT + NC * half) / kBlock;
            return Scales{(uint32_t)min(row, a.T - 1), (uint32_t)min(nb, (a.N - 1) / kBlock) * a.KB};
        };
        float sa[4], sw[4];
        Scales here = scales_of(pair);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t kb = min(j, a.KB - 1);
            sa[j] = a.a_scale[kb * a_stride + here.a];
            sw[j] = a.w_scale[kb + here.w];
        }
        // A block's sums are read in pieces of 16 columns, each while the piece before it is added up (pieces of 32 leave too
        // few registers: 39 -> 67 us for 4096 x 5120 x 2048).  A wait that runs out does not end the loops (a vote of the
        // warp at each block costs 3% of the whole): no later one waits, and what is stored is as good as any.
        f32x2 acc[NC / 2];
        Ring<C::kBufs> buf;
        const uint32_t add_bar = add_full + 16 * (warp - 4);
        uint32_t add_phase = 0;  // a bit for each box
        const int add_at = a.KB > 4 ? 4 : 0;  // (the last tile's boxes have been read by then)
        auto wait_full = [&]() {
            if (!*err && !mbar_wait_spin(d_full + 8 * buf.at, buf.phase, a.wait_budget)) fail();
        };
        for (int i = pair; i < tiles; i += pairs) {
            const TileAt t = tile_at(i, m_tiles, n_tiles);
            const Scales next = scales_of(i + pairs);
#pragma unroll
            for (int c = 0; c < NC / 2; ++c) acc[c] = 0ull;
            const int row0 = t.m * 256 + rank * 128 + quad * 32, n0 = t.n * NT + NC * half;
            for (int kb0 = 0; kb0 < a.KB; kb0 += 4) {
                if (MODE == kAddBoxes && kb0 == add_at && lane == 0 && row0 < a.T && n0 < a.N) {
                    asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
#pragma unroll
                    for (int q = 0; q < NC / 64; ++q)
                        if (n0 + 64 * q < a.N) {
                            mbar_arrive_expect_tx(add_bar + 8 * q, 4096);
                            tma_load_2d_plain(stage + 4096 * q, &tm_add, n0 + 64 * q, row0, add_bar + 8 * q);
                        }
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int kb = kb0 + j;
                    if (kb >= a.KB) break;
                    const float scale = sa[j] * sw[j];
                    const bool more = kb + 4 < a.KB;
                    const uint32_t to = more ? kb + 4 : min(j, a.KB - 1);
                    sa[j] = a.a_scale[to * a_stride + (more ? here.a : next.a)];
                    sw[j] = a.w_scale[to + (more ? here.w : next.w)];
                    const f32x2 scale2 = pack2(scale, scale);
                    if (!mbar_try_wait(d_full + 8 * buf.at, buf.phase)) wait_full();
                    __syncwarp();  // (each lane waited for itself, and the reads below are the warp's)
                    tc::fence_after_sync();
                    const uint32_t from = lane_addr + NT * buf.at;
                    uint32_t v[2][16];
                    tmem_ld16(from, v[0]);
#pragma unroll
                    for (int q = 0; q < NC / 16; ++q) {
                        tc::tmem_wait_ld();
                        if (q + 1 < NC / 16) tmem_ld16(from + 16 * (q + 1), v[(q + 1) & 1]);
                        else {  // all read: the buffer may be written
                            tc::fence_before_sync();
                            __syncwarp();
                            if (lane == 0) mbar_arrive_pair(lead_d_empty + 8 * buf.at);
                        }
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            ffma2(acc[8 * q + e], pack2(__uint_as_float(v[q & 1][2 * e]), __uint_as_float(v[q & 1][2 * e + 1])), scale2);
                    }
                    buf.next();
                }
            }
            here = next;
            if (row0 < a.T && n0 < a.N) {
                if (MODE == kAddBoxes) {
#pragma unroll
                    for (int q = 0; q < NC / 64; ++q)
                        if (n0 + 64 * q < a.N) {
                            if (!mbar_wait_spin(add_bar + 8 * q, (add_phase >> q) & 1, a.wait_budget)) fail();
                            add_phase ^= 1u << q;
                            add_box(stage + 4096 * q, &acc[32 * q], a.add.dtype == SI_FP8_BF16);
                        }
                } else if (MODE == kAny && a.add.p) {
                    const int64_t row = (int64_t)row0 + lane;
#pragma unroll
                    for (int q = 0; q < NC / 8; ++q)
                        if (row < a.T) add_to(a, add_whole, row, n0 + 8 * q, &acc[4 * q]);
                }
                const bool f32 = a.out.dtype == SI_FP8_F32;
                if (MODE != kAny || (boxes && (n0 + NC <= a.N || a.N % (f32 ? 4 : 8) == 0))) {
                    if (f32) store_boxes<NC, 32>(a, &tm_out, stage, row0, n0, acc);
                    else store_boxes<NC, 64>(a, &tm_out, stage, row0, n0, acc);
                } else {
                    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                    __syncwarp();
                    store_odd<NC>(a, stage, row0, n0, acc);
                    tc::fence_proxy_async_smem();  // (the next use may be a copy into it)
                    __syncwarp();
                }
            }
        }
        if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
    tc::fence_before_sync();
    __syncthreads();
    // Every product is done before either CTA gives its memory back, and every signal of the products has arrived: they go
    // to both CTAs, and each waits for its own last ones (the cluster's barrier orders threads, not signals under way).
    if (warp == 1) {
        mbar_wait_spin(fin, 0, kDrain);
        __syncwarp();
    }
    // After a wait that ran out: copies that the even CTA did not wait for (the odd CTA's own, and boxes of `add`) land
    // within microseconds, before either CTA goes.
    if (*err)
        for (const long long t0 = clock64(); clock64() - t0 < kLinger;) __nanosleep(1000);
    __syncwarp();
    cluster_sync();  // (nothing more arrives from the other CTA)
    if (warp == 1) {
        tc::fence_after_sync();
        tc::tmem_dealloc_pair(taddr, 512);
    }
}

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
        cudaGetLastError();
        return (PFN_cuTensorMapEncodeTiled_v12000) nullptr;
    }();
    return fn;
}
// Codes [rows][K] in boxes of 128 columns x box_rows rows, 128-byte swizzle; what lies outside reads as zeros.
bool code_map(const uint8_t *base, int64_t rows, int K, int box_rows, CUtensorMap *tm) {
    const auto enc = encoder();
    if (!enc) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)K};
    const cuuint32_t box[2] = {128, (cuuint32_t)box_rows}, ones[2] = {1, 1};
    return enc(tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t *>(base), dims, strides, box, ones,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// A matrix [T][N] in boxes of 128 bytes x 32 rows, where its rows begin at multiples of 16 bytes: false elsewhere.
bool box_map(const Mat &m, int T, int N, CUtensorMap *tm) {
    const int size = m.dtype == SI_FP8_F32 ? 4 : 2;
    const auto enc = encoder();
    const int64_t stride = T > 1 ? m.stride * size : ((int64_t)N * size + 15) / 16 * 16;
    if (!enc || stride % 16 || stride == 0) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)N, (cuuint64_t)T}, strides[1] = {(cuuint64_t)stride};
    const cuuint32_t box[2] = {(cuuint32_t)(128 / size), 32}, ones[2] = {1, 1};
    return enc(tm, size == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, m.p, dims, strides, box, ones,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

size_t scratch_bytes(const Plan &p, int n_rows) { return kCtrlBytes; }

namespace {
template <int NT>
cudaError_t launch_many(const Plan &p, const MatmulArgs &a, cudaStream_t s) {
    CUtensorMap ta, tw, to{}, tadd{};
    if (!code_map(a.a, a.T, a.K, 128, &ta) || !code_map(a.w, a.N, a.K, NT / 2, &tw)) return cudaErrorNotSupported;
    const bool boxes = box_map(a.out, a.T, a.N, &to);
    const bool whole = boxes && a.N % (a.out.dtype == SI_FP8_F32 ? 4 : 8) == 0;  // (no row ends within 16 bytes)
    const bool add = whole && a.add.p && a.add.dtype == a.out.dtype && a.out.dtype != SI_FP8_F32 && box_map(a.add, a.T, a.N, &tadd);
    const int mode = add ? kAddBoxes : whole && !a.add.p ? kPlain : kAny;
    const auto kernel = mode == kAddBoxes ? k_matmul_many<NT, kAddBoxes> : mode == kPlain ? k_matmul_many<NT, kPlain> : k_matmul_many<NT, kAny>;
    const int m_tiles = (a.T + 255) / 256, n_tiles = (a.N + NT - 1) / NT;
    const cudaError_t e = mode == kAddBoxes ? kv::allow_smem<k_matmul_many<NT, kAddBoxes>>(Many<NT>::kSmem)
                          : mode == kPlain  ? kv::allow_smem<k_matmul_many<NT, kPlain>>(Many<NT>::kSmem)
                                            : kv::allow_smem<k_matmul_many<NT, kAny>>(Many<NT>::kSmem);
    if (e != cudaSuccess) return e;
    const int pairs = (int)std::min<int64_t>(p.sm_count / 2, (int64_t)m_tiles * n_tiles);
    return kv::launch(kernel, dim3(2 * pairs), kManyThreads, Many<NT>::kSmem, s, ta, tw, to, tadd, a, (int)boxes, m_tiles, n_tiles);
}

// How many CTAs share a tile of few rows: a power of two, as many as two CTAs an SM (three are no faster), eight CTAs and
// a block of columns for each leave.  (One CTA more than there is room for costs as much as all: 1 x 5120 x 2048 takes 3.6 us
// with 4; 5.6 with 8, two CTAs an SM.)
int few_share(const Plan &p, const MatmulArgs &a, int TN) {
    const int64_t tiles = (int64_t)((a.N + 127) / 128) * ((a.T + TN - 1) / TN);
    int S = 1;
    while (S < 8 && 2 * S <= a.KB && tiles * S * 2 <= 2 * p.sm_count) S *= 2;
    return S;
}
template <int TN>
cudaError_t launch_few(const Plan &p, const MatmulArgs &a, cudaStream_t s) {
    CUtensorMap ta, tw;
    if (!code_map(a.a, a.T, a.K, TN, &ta) || !code_map(a.w, a.N, a.K, 128, &tw)) return cudaErrorNotSupported;
    const int t_tiles = (a.T + TN - 1) / TN;
    const int64_t tiles = (int64_t)((a.N + 127) / 128) * t_tiles;
    const int S = few_share(p, a, TN);
    const cudaError_t e = kv::allow_smem<k_matmul_few<TN>>(Few<TN>::kSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(tiles * S));
    cfg.blockDim = dim3(192);
    cfg.dynamicSmemBytes = S == 1 ? Few<TN>::kSmemOne : Few<TN>::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)S;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, k_matmul_few<TN>, ta, tw, a, t_tiles, S);
}
}  // namespace

cudaError_t launch_matmul(const Plan &p, const MatmulArgs &a, cudaStream_t s) {
    if (a.T <= 16) return launch_few<16>(p, a, s);
    if (a.T <= 32) return launch_few<32>(p, a, s);
    // Tiles of 64 rows pay as long as four CTAs or more share each of them: 200 x 2048 x 4096 takes 8.9 us so and 11.4 by
    // pairs, 128 x 5120 x 2048 (two CTAs a tile) 9.3 and 7.8.
    if (a.T <= 64 || few_share(p, a, 64) >= 4) return launch_few<64>(p, a, s);
    // A round of tiles of 256 columns takes 1.2 to 1.45 times as long as one of 128 (K = 2048 to 8192).
    const int64_t m = (a.T + 255) / 256, pairs = p.sm_count / 2;
    const int64_t wide = (m * ((a.N + 255) / 256) + pairs - 1) / pairs, narrow = (m * ((a.N + 127) / 128) + pairs - 1) / pairs;
    return 4 * wide <= 3 * narrow ? launch_many<256>(p, a, s) : launch_many<128>(p, a, s);
}

}  // namespace fp8
}  // namespace si
