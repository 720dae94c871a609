// si_fp8_norm.cu -- the passes that write quantised operands: rows (residual
// addition, RMS norm, quantisation for each 128 columns) and weight matrices
// (128 x 128 blocks).
#include <algorithm>

#include "si_fp8_device.cuh"

namespace si {
namespace fp8 {
namespace {

// The largest of V values over each half of a warp, value by value: of 16 neighbouring lanes, lane i * 16/V and the ones
// up to the next multiple of 16/V get value i's.  A lane hands half of its values to the lane that it exchanges with, as
// long as it has more than one: V = 4 takes five exchanges instead of sixteen.
template <int V>
__device__ __forceinline__ uint32_t half_warp_max(uint32_t (&m)[V]) {
    const int lane = threadIdx.x & 31;
    int n = V;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) {
        if (n > 1) {
            n /= 2;
#pragma unroll
            for (int i = 0; i < V / 2; ++i)
                if (i < n) {
                    const uint32_t keep = lane & o ? m[i + n] : m[i], give = lane & o ? m[i] : m[i + n];
                    m[i] = max(keep, __shfl_xor_sync(0xffffffffu, give, o));
                }
        } else {
            m[0] = max(m[0], __shfl_xor_sync(0xffffffffu, m[0], o));
        }
    }
    return m[0];
}

// One row by W warps, R rows a CTA at a time; a thread holds V pieces of eight columns in registers, so a row is read
// once.  16 neighbouring lanes hold the 128 columns of a scale.  RES: 0 no residual, 1 in 16 bits, 2 in 32.
// Many rows: each CTA goes on from row to row, a row's loads are on their way while the row before is reduced, quantised and
// stored, the gain stays in registers, and one division of each kind and one exchange serves the blocks of V pieces.
// 16384 rows of 2048 in bf16 with a residual, 235 MB: 49 us, 71% of the copy rate; without one and without a gain, 6001 rows
// of 4096, 74 MB: 16.4 us, 66%.  Neither memory nor the instructions are what it waits for: with a residual (34 instructions
// a value, 31 warps an SM) the schedulers issue in two thirds of the cycles and DRAM is busy for half, without (14 a value,
// 15 warps) in 59% and for a third.  The rest is the latency of a row's chain, with too few rows under way on an SM.
template <int V, bool X32, int RES>
__global__ void __launch_bounds__(512, V > 2 ? 1 : 2) k_norm(const NormArgs a, int W, int R) {
    __shared__ float s_sum[2][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = (warp % W) * 32 + lane, n = W * 32;
    const int64_t step = (int64_t)gridDim.x * R;
    start_after();

    int64_t row = (int64_t)blockIdx.x * R + warp / W;
    Raw8 xr[V], rr[V];
    auto load = [&](int64_t from) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = (i * n + t) * 8;
            if (from < a.T && c < a.K) {
                xr[i] = load8<X32>(a.x.p, from * a.x.stride + c);
                if (RES) rr[i] = load8<RES == 2>(a.residual.p, from * a.residual.stride + c);
            }
        }
    };
    load(row);
    float g[V][8];
    if (a.gain) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = (i * n + t) * 8;
#pragma unroll
            for (int h = 0; h < 2; ++h)
                *reinterpret_cast<float4 *>(&g[i][4 * h]) =
                    c < a.K ? *reinterpret_cast<const float4 *>(a.gain + c + 4 * h) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
    }
    // (the same number of rounds for all warps of the CTA: they meet in each)
    int turn = 0;
    for (int64_t first = (int64_t)blockIdx.x * R; first < a.T; first += step, row += step, turn ^= 1) {
        const bool live = row < a.T;
        float v[V][8];
        f32x2 sum2 = 0ull;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = (i * n + t) * 8;
            if (live && c < a.K) {
                widen8<X32>(xr[i], a.x.dtype == SI_FP8_BF16, v[i]);
                if (RES) {
                    float r[8];
                    widen8<RES == 2>(rr[i], a.residual.dtype == SI_FP8_BF16, r);
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[i][e] += r[e];
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[i][e] = 0.0f;
            }
        }
        load(row + step);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = (i * n + t) * 8;
            if (a.residual_out.p && live && c < a.K) store8<true>(a.residual_out, row * a.residual_out.stride + c, v[i]);
            if (a.gain) {
#pragma unroll
                for (int e = 0; e < 8; e += 2) ffma2(sum2, pack2(v[i][e], v[i][e + 1]), pack2(v[i][e], v[i][e + 1]));
            }
        }
        if (!a.y.p && !a.codes) continue;
        if (a.gain) {
            const float2 halves = unpack2(sum2);
            float sum = warp_sum(halves.x + halves.y);
            if (W > 1) {
                float *const sums = s_sum[turn];  // (a warp is one round ahead at most)
                if (lane == 0) sums[warp] = sum;
                __syncthreads();
                const int w0 = warp / W * W;
                sum = 0.0f;
                for (int i = 0; i < W; ++i) sum += sums[w0 + i];
            }
            const float scale = rms_scale(sum, a.K, a.eps);
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    f32x2 x;
                    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(x) : "l"(pack2(v[i][e], v[i][e + 1])), "l"(pack2(scale, scale)));
                    asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(x) : "l"(pack2(g[i][e], g[i][e + 1])));
                    const float2 f = unpack2(x);
                    v[i][e] = f.x;
                    v[i][e + 1] = f.y;
                }
        }
        float mul = 0.0f;  // of the block that half_warp_max gives this lane
        if (a.codes) {
            uint32_t amax[V];
#pragma unroll
            for (int i = 0; i < V; ++i) amax[i] = (i * n + t) * 8 < a.K ? amax_bits8(v[i]) : 0u;
            const float scale = block_scale(half_warp_max<V>(amax), mul);
            const int c = ((lane & 15) / (16 / V) * n + t) * 8;  // (within that block)
            if (live && (lane & (16 / V - 1)) == 0 && c / kBlock * kBlock < a.K) a.scales[(c / kBlock) * a.scale_stride + row] = scale;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = (i * n + t) * 8;
            const bool here = live && c < a.K;
            if (a.codes) {
                const float m = __shfl_sync(0xffffffffu, mul, (lane & 16) + i * (16 / V));
                if (here) *reinterpret_cast<uint2 *>(a.codes + row * a.K + c) = codes8(v[i], m);
            }
            if (a.y.p && here) store8<false>(a.y, row * a.y.stride + c, v[i]);
        }
    }
}

// One 128 x 128 block of a weight matrix a CTA: 16 threads a row, eight rows each.
template <bool F32>
__global__ void __launch_bounds__(256) k_pack(const Mat w, uint8_t *codes, float *scales, int N, int K, int KB) {
    __shared__ uint32_t s_max[8];
    const int nb = blockIdx.x / KB, kb = blockIdx.x % KB;
    const int c = kb * kBlock + (threadIdx.x & 15) * 8, r0 = nb * kBlock + (threadIdx.x >> 4);
    start_after();
    Raw8 raw[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        raw[i].a = raw[i].b = make_uint4(0, 0, 0, 0);
        if (r0 + 16 * i < N && c < K) raw[i] = load8<F32>(w.p, (int64_t)(r0 + 16 * i) * w.stride + c);
    }
    uint32_t amax = 0;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        widen8<F32>(raw[i], w.dtype == SI_FP8_BF16, v);
        amax = max(amax, amax_bits8(v));
    }
    amax = __reduce_max_sync(0xffffffffu, amax);
    if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = amax;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = max(amax, s_max[i]);
    float mul;
    const float scale = block_scale(amax, mul);
    if (threadIdx.x == 0) scales[(int64_t)nb * KB + kb] = scale;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (r0 + 16 * i < N && c < K) {
            widen8<F32>(raw[i], w.dtype == SI_FP8_BF16, v);
            *reinterpret_cast<uint2 *>(codes + (int64_t)(r0 + 16 * i) * K + c) = codes8(v, mul);
        }
    }
}

template <int V, bool X32, int RES>
cudaError_t norm_rows(const Plan &p, const NormArgs &a, int W, int R, cudaStream_t s) {
    // as many CTAs as are resident at once, or rows for each once
    int64_t grid = ((int64_t)a.T + R - 1) / R;
    if (grid > p.sm_count) {
        int ctas = 0;
        const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&ctas, k_norm<V, X32, RES>, W * R * 32, 0);
        if (e != cudaSuccess) return e;
        grid = std::min<int64_t>(grid, (int64_t)std::max(1, ctas) * p.sm_count);
    }
    return kv::launch(k_norm<V, X32, RES>, dim3((unsigned)grid), W * R * 32, 0, s, a, W, R);
}
template <bool X32, int RES>
cudaError_t norm_by_size(const Plan &p, const NormArgs &a, cudaStream_t s) {
    // One piece a thread for few rows, where only the time of one row counts (1 x 2048: 2.0 us).  For more, two pieces, or
    // four of one 16-bit operand, as far as a row fills the lanes with them: 16384 x 2048 in bf16 takes 55, 49 and 67 us
    // with one, two and four where there is a residual (which then leaves too few threads), 44, 31 and 29 where there is none.
    // Rows of more than 512, 1024 and 2048 pieces take two, four and eight at least, so that 16 warps hold them.
    const int pieces = (a.K + 7) / 8;  // of eight columns
    const bool few = a.T <= 2 * p.sm_count && pieces <= 512;
    auto fills = [&](int V) { return (pieces + 32 * V - 1) / (32 * V) * 32 * V * 4 <= pieces * 5; };
    const int V = few ? 1 : pieces > 2048 ? 8 : pieces > 1024 || (!X32 && RES == 0 && fills(4)) ? 4 : pieces > 512 || fills(2) ? 2 : 1;
    const int W = (pieces + 32 * V - 1) / (32 * V);
    const int R = W >= 8 ? 1 : 8 / W;
    return V == 1   ? norm_rows<1, X32, RES>(p, a, W, R, s)
           : V == 2 ? norm_rows<2, X32, RES>(p, a, W, R, s)
           : V == 4 ? norm_rows<4, X32, RES>(p, a, W, R, s)
                    : norm_rows<8, X32, RES>(p, a, W, R, s);
}
template <bool X32>
cudaError_t norm_by_residual(const Plan &p, const NormArgs &a, cudaStream_t s) {
    if (!a.residual.p) return norm_by_size<X32, 0>(p, a, s);
    return a.residual.dtype != SI_FP8_F32 ? norm_by_size<X32, 1>(p, a, s) : norm_by_size<X32, 2>(p, a, s);
}

}  // namespace

cudaError_t launch_norm(const Plan &p, const NormArgs &a, cudaStream_t s) {
    return a.x.dtype == SI_FP8_F32 ? norm_by_residual<true>(p, a, s) : norm_by_residual<false>(p, a, s);
}

cudaError_t launch_pack(const Plan &p, const Mat &w, uint8_t *codes, float *scales, cudaStream_t s) {
    const int N = p.desc.out_features, K = p.desc.in_features, KB = (K + kBlock - 1) / kBlock;
    const dim3 grid((unsigned)(((N + kBlock - 1) / kBlock) * KB));
    if (w.dtype == SI_FP8_F32) return kv::launch(k_pack<true>, grid, 256, 0, s, w, codes, scales, N, K, KB);
    return kv::launch(k_pack<false>, grid, 256, 0, s, w, codes, scales, N, K, KB);
}

}  // namespace fp8
}  // namespace si
