// si_kv_decode.cuh -- attention of few rows over the cache (a decode step, the
// verification of drafted tokens): running softmax over key tiles, split over
// the whole GPU along the keys.
//
//   out_r = sum_t p_rt v_t / sum_t p_rt,   p_rt = 2^(s_rt - m_r),   s_rt = f_t (q'_r . code_t)
// where f_t is the product of the page's scale, the row's power of two and
// sm_scale * log2 e, and m_r is a running maximum.
//
// Bound: HBM.  Every cached token is read once for all the rows of its kv
// head, 2D bytes of codes; the arithmetic per byte is 2 x 16 rows of matrix
// work and the codes' conversion to fp16 (about 1.4 half-rate instructions a
// byte), which has to stay below the time that the byte takes to arrive: 23
// bytes a cycle and SM at the measured copy rate.
//  * Work: units of 64 tokens of one (sequence, kv head, row group), numbered in
//    order; each CTA takes an equal share of consecutive units, whatever the
//    sequences' lengths.  A CTA joins its warps' results for each item it
//    touches; an item that lies in several CTAs is joined by the last of them
//    to arrive, in the CTAs' order (the same inputs give the same bits).
//  * A warp owns 16 of a unit's 64 tokens (one page: P >= 16) and copies them
//    into its own ring in shared memory (cp.async, several units ahead): no
//    barrier between warps inside an item.
//  * The maximum is lazy: m moves only when a score passes it by more than 4
//    (a vote a tile instead of shuffles), and p stays below 2^4.
//  * p times the page's V scale is rounded to fp16 for the second product.  The
//    scale is taken relative to the largest so far, so that the products stay
//    inside fp16: p < 2^4, scale/reference <= 1, times 2^11: at most 2^15; a
//    weight of one keeps its eleven bits down to a relative scale of 2^-25.
//    (bf16 weights, without the reference, have eight: half a step of the
//    output's own rounding, or eight steps for an fp16 output.)
#pragma once
#include "si_kv_mma.cuh"

namespace si {
namespace kv {

constexpr int kDecWarps = 4;
constexpr int kDecThreads = kDecWarps * 32;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kLazy = 4.0f, kWeightUnit = 2048.0f;
constexpr float kNoScore = -1e30f;  // a running maximum before the first score

template <int D, int MT>
struct DecodeCfg {
    static constexpr int stage = 32 * D;  // bytes of one warp's 16 keys, K and V
    static constexpr int stages = D == 64 ? 6 : D == 128 ? 4 : 3;
    static constexpr int ring = kDecWarps * stages * stage;
    static constexpr int merge = kDecWarps * 16 * MT * D * 4;
    static constexpr bool q_in_regs = D * MT <= 128;
    static constexpr int q_bytes = q_in_regs ? 0 : MT * (D / 16) * 512;
    static constexpr int ctas = D == 256 ? 2 : MT == 2 ? 2 : D == 64 ? 4 : 3;  // a SM
    static constexpr int smem = (ring > merge ? ring : merge) + q_bytes;
};

// Partial results in the scratch: two slots a CTA (an item that began in an
// earlier CTA, one that goes on in a later one), each [rows][D] sums, then [rows][2]
// maximum and sum.
__host__ __device__ constexpr int64_t partial_floats(int rows, int D) { return (int64_t)rows * (D + 2); }

struct DecodeArgs {
    Ctx c;
    Rows q, out;
    float *lse;
    float scale2;  // sm_scale * log2 e
    int bf16;
    int log_page;
    int32_t *counters;
    float *partial;
};

// Units of sequence b: (pages in tiles of 64 tokens, then the unfinished page) x kv heads x row groups.
__device__ __forceinline__ int seq_tiles(const Ctx &c, int len) {
    const int paged = len & ~(c.P - 1);
    return (paged + 63) / 64 + (paged < len ? 1 : 0);
}

template <int CODE, int D, int MT>
__global__ void __launch_bounds__(kDecThreads, DecodeCfg<D, MT>::ctas) k_kv_decode(const DecodeArgs a) {
    using Cfg = DecodeCfg<D, MT>;
    constexpr int R = 16 * MT;      // rows of an item
    constexpr int NT = D / 8;       // column tiles of the second product
    constexpr int KS = D / 16;      // steps of the first
    constexpr int CH = D / 16;      // 16-byte chunks of a key
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ long long s_scan[kDecWarps];
    __shared__ long long s_off;
    __shared__ int s_b, s_last;
    __shared__ float s_ml[kDecWarps][R][2];
    __shared__ float s_part[R][2];
    const Ctx &c = a.c;
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, g = lane >> 2, j = lane & 3;
    const bool bf16 = a.bf16;

    // ---- this CTA's share of the units
    const int per = (c.B + kDecThreads - 1) / kDecThreads;
    auto units_of = [&](int b) -> long long {
        const Seq s = load_seq(c, b);
        return (long long)seq_tiles(c, s.len) * c.Hk * ((s.n * c.G + R - 1) / R);
    };
    long long mine = 0;
    bool empty = false;
    for (int b = tid * per; b < min(c.B, (tid + 1) * per); ++b) {
        const long long n = units_of(b);
        mine += n;
        empty |= n == 0;
    }
    long long incl = mine;
    for (int o = 1; o < 32; o <<= 1) {
        const long long up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
    }
    if (lane == 31) s_scan[w] = incl;
    const bool some_empty = __syncthreads_or(empty);
    long long before = incl - mine, total = 0;
    for (int k = 0; k < kDecWarps; ++k) {
        if (k < w) before += s_scan[k];
        total += s_scan[k];
    }
    // rows whose sequence has no token at all are in no unit: zeros
    if (some_empty)
        for (int b = blockIdx.x; b < c.B; b += gridDim.x) {
            const Seq s = load_seq(c, b);
            if (s.len > 0) continue;
            for (int k = tid; k < s.n * c.H * (D / 8); k += kDecThreads) {
                const int row = s.row0 + k / (c.H * (D / 8)), head = k / (D / 8) % c.H, d = k % (D / 8) * 8;
                *reinterpret_cast<uint4 *>(a.out.p + row * a.out.row + head * a.out.head + d) = make_uint4(0, 0, 0, 0);
                if (a.lse && d == 0) a.lse[(int64_t)row * c.H + head] = -INFINITY;
            }
        }
    const long long N = total < (long long)gridDim.x ? total : (long long)gridDim.x;
    if (blockIdx.x >= N) return;
    const long long u_begin = blockIdx.x * total / N, u_end = (blockIdx.x + 1) * total / N;
    if (before <= u_begin && u_begin < before + mine) {
        int b = tid * per;
        long long at = before, n;
        while (at + (n = units_of(b)) <= u_begin) {
            at += n;
            ++b;
        }
        s_b = b;
        s_off = u_begin - at;
    }
    __syncthreads();
    int b = s_b;
    long long off = s_off;  // within sequence b
    long long u = u_begin;

    const uint32_t ring = smem_addr(smem) + w * (Cfg::stages * Cfg::stage);
    uint8_t *q_smem = smem + (Cfg::smem - Cfg::q_bytes);

    while (u < u_end) {
        const Seq s = load_seq(c, b);
        const int tiles = seq_tiles(c, s.len);
        const int groups = (s.n * c.G + R - 1) / R;
        const long long n_units = (long long)tiles * c.Hk * groups;
        if (off >= n_units) {  // on to the next sequence (one without units among them)
            off -= n_units;
            ++b;
            continue;
        }
        const int item = (int)(off / tiles), t_first = (int)(off % tiles);
        const int h = item / groups, rb = item % groups;
        const int t_end = (int)min((long long)tiles, t_first + (u_end - u));
        const int rows = min(R, s.n * c.G - rb * R);
        const int paged = s.len & ~(c.P - 1), old = s.len - s.n;
        const int lim_min = old + rb * R / c.G + 1, lim_max = old + (rb * R + rows - 1) / c.G + 1;
        const int paged_tiles = (paged + 63) / 64;

        // ---- q
        uint32_t qa[Cfg::q_in_regs ? MT * KS : 1][4];
        float qf[MT][2];
        int lim[MT][2];
        if (!Cfg::q_in_regs) __syncthreads();  // the last item's readers are done
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = rb * R + mt * 16 + g + 8 * e;
                const bool live = mt * 16 + g + 8 * e < rows;
                const int i = live ? r / c.G : 0, head = live ? h * c.G + r % c.G : 0;
                const uint16_t *src = a.q.p + (s.row0 + i) * a.q.row + head * a.q.head;
                uint4 x[D / 32];
                float amax = 0.0f;
#pragma unroll
                for (int k = 0; k < D / 64; ++k) {
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        x[2 * k + z] = live ? *reinterpret_cast<const uint4 *>(src + k_dim<D>(j, k) + 8 * z) : make_uint4(0, 0, 0, 0);
                        amax = fmaxf(amax, amax8(x[2 * k + z], bf16));
                    }
                }
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
                float mul;
                row_scale(amax, mul, qf[mt][e]);
                qf[mt][e] *= a.scale2;
                lim[mt][e] = live ? old + i + 1 : INT32_MAX;
#pragma unroll
                for (int st = 0; st < KS; ++st) {  // chunk st / 4, four values at 4 * (st % 4)
                    const uint4 &v = x[2 * (st >> 2) + ((st >> 1) & 1)];
                    const uint32_t lo = scale2(st & 1 ? v.z : v.x, mul, bf16), hi = scale2(st & 1 ? v.w : v.y, mul, bf16);
                    if constexpr (Cfg::q_in_regs) {
                        qa[mt * KS + st][e] = lo;
                        qa[mt * KS + st][2 + e] = hi;
                    } else if ((st & 3) == w) {
                        uint32_t *to = reinterpret_cast<uint32_t *>(q_smem + (mt * KS + st) * 512 + lane * 16);
                        to[e] = lo;
                        to[2 + e] = hi;
                    }
                }
            }
        }
        if (!Cfg::q_in_regs) __syncthreads();

        float o[MT][NT][4];
        float m[MT][2], l[MT][2];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
            for (int n = 0; n < NT; ++n) o[mt][n][0] = o[mt][n][1] = o[mt][n][2] = o[mt][n][3] = 0.0f;
            m[mt][0] = m[mt][1] = kNoScore;
            l[mt][0] = l[mt][1] = 0.0f;
        }
        float v_ref = 1e-30f;  // the largest V scale so far: o is in units of v_ref / kWeightUnit

        // Scores to weights: s (raw products) times the columns' factors and the rows', masked at the
        // rows' limits; updates m, l, and o's scale; returns the second product's operand.
        auto weights = [&](float (&sc)[MT][2][4], const float (&kf)[4], const float (&vf)[4], float v_top, int t0,
                           bool masked, uint32_t (&pa)[MT][4]) {
            if (v_top > v_ref) {
                const float f = v_ref / v_top;
                v_ref = v_top;
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[mt][n][e] *= f;
            }
            const float inv = kWeightUnit / v_ref;
            bool over = false;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float z = sc[mt][n][e] * (kf[2 * n + (e & 1)] * qf[mt][e >> 1]);
                        if (masked && t0 + 8 * n + 2 * j + (e & 1) >= lim[mt][e >> 1]) z = -INFINITY;
                        sc[mt][n][e] = z;
                    }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float top = fmaxf(fmaxf(sc[mt][0][2 * e], sc[mt][0][2 * e + 1]),
                                            fmaxf(sc[mt][1][2 * e], sc[mt][1][2 * e + 1]));
                    over |= top > m[mt][e] + kLazy;
                }
            }
            if (__any_sync(0xffffffffu, over)) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    float f[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float top = fmaxf(fmaxf(sc[mt][0][2 * e], sc[mt][0][2 * e + 1]),
                                          fmaxf(sc[mt][1][2 * e], sc[mt][1][2 * e + 1]));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                        top = fmaxf(top, m[mt][e]);
                        f[e] = ex2(m[mt][e] - top);
                        m[mt][e] = top;
                        l[mt][e] *= f[e];
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        o[mt][n][0] *= f[0];
                        o[mt][n][1] *= f[0];
                        o[mt][n][2] *= f[1];
                        o[mt][n][3] *= f[1];
                    }
                }
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float p0 = ex2(sc[mt][n][2 * e] - m[mt][e]), p1 = ex2(sc[mt][n][2 * e + 1] - m[mt][e]);
                        l[mt][e] += p0 + p1;
                        // (a page without a scale makes NaN of the weights that see it, and of no other)
                        const float w0 = p0 == 0.0f ? 0.0f : p0 * (vf[2 * n] * inv);
                        const float w1 = p1 == 0.0f ? 0.0f : p1 * (vf[2 * n + 1] * inv);
                        pa[mt][2 * n + e] = half2_bits(w0, w1);
                    }
        };

        // ---- full pages
        const int t_stop = min(min(t_end, paged_tiles), (lim_max + 63) / 64);  // no row sees a later tile
        const int count = t_stop - t_first;
        // page, K scale and V scale of this warp's 16 tokens, for 32 tiles at a time (a lane a tile), two sets
        int pid[2] = {-2, -2};
        float ksc[2] = {0.0f, 0.0f}, vsc[2] = {0.0f, 0.0f};
        auto fetch = [&](int set, int first) {
            const int t = first + lane, token = (t_first + t) * 64 + 16 * w;
            int p = -2;  // no tokens
            if (t < count && token < paged) p = (int)load_page(c, b, token >> a.log_page);
            const float ks = p >= 0 ? __ldg(c.ks + (int64_t)p * c.Hk + h) : 0.0f;
            const float vs = p >= 0 ? __ldg(c.vs + (int64_t)p * c.Hk + h) : 0.0f;
            if (set) {
                pid[1] = p;
                ksc[1] = ks;
                vsc[1] = vs;
            } else {
                pid[0] = p;
                ksc[0] = ks;
                vsc[0] = vs;
            }
        };
        auto copy = [&](int t) {  // tile t of this item, relative to t_first
            if (t < count) {
                const int p = __shfl_sync(0xffffffffu, (t & 32) ? pid[1] : pid[0], t & 31);
                if (p >= 0) {
                    const int64_t at = page_at(c, p, h) + (int64_t)(((t_first + t) * 64 + 16 * w) & (c.P - 1)) * D;
                    const uint32_t to = ring + (t % Cfg::stages) * Cfg::stage;
#pragma unroll
                    for (int k = 0; k < D / 32; ++k) {
                        const int ci = lane + 32 * k;
                        const uint32_t x = to + tile_at<D>(ci / CH, ci % CH);
                        cp_async16(x, c.kc + at + ci * 16);
                        cp_async16(x + 16 * D, c.vc + at + ci * 16);
                    }
                }
            }
            cp_async_commit();
        };
        if (count > 0) {
            fetch(0, 0);
            fetch(1, 32);
#pragma unroll
            for (int t = 0; t < Cfg::stages - 1; ++t) copy(t);
        }
        for (int t = 0; t < count; ++t) {
            if ((t & 31) == 0 && t > 0) fetch(((t >> 5) + 1) & 1, (t & ~31) + 32);
            copy(t + Cfg::stages - 1);
            cp_async_wait<Cfg::stages - 1>();
            __syncwarp();
            const int p = __shfl_sync(0xffffffffu, (t & 32) ? pid[1] : pid[0], t & 31);
            const float ks = __shfl_sync(0xffffffffu, (t & 32) ? ksc[1] : ksc[0], t & 31);
            const float vs = __shfl_sync(0xffffffffu, (t & 32) ? vsc[1] : vsc[0], t & 31);
            const int t0 = (t_first + t) * 64 + 16 * w;
            if (p == -2 || t0 >= lim_max) continue;
            if (p < 0) {  // not one of the cache's pages: NaN for the rows that see it
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        if (t0 < lim[mt][e]) l[mt][e] = __int_as_float(0x7fc00000);
                continue;
            }
            const uint32_t kt = ring + (t % Cfg::stages) * Cfg::stage, vt = kt + 16 * D;
            float sc[MT][2][4];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int n = 0; n < 2; ++n) sc[mt][n][0] = sc[mt][n][1] = sc[mt][n][2] = sc[mt][n][3] = 0.0f;
#pragma unroll
            for (int i = 0; i < D / 64; ++i) {
                uint4 x[2];
#pragma unroll
                for (int n = 0; n < 2; ++n) x[n] = lds128(kt + tile_at<D>(8 * n + g, k_dim<D>(j, i) / 16));
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int st = 4 * i + q;
                    uint32_t lo[2], hi[2];
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        const uint32_t word = q == 0 ? x[n].x : q == 1 ? x[n].y : q == 2 ? x[n].z : x[n].w;
                        codes_to_half<CODE>(code_bias<CODE>(word), lo[n], hi[n]);
                    }
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        if constexpr (Cfg::q_in_regs) {
                            mma16816(sc[mt][0], qa[mt * KS + st], lo[0], hi[0]);
                            mma16816(sc[mt][1], qa[mt * KS + st], lo[1], hi[1]);
                        } else {
                            const uint4 v = *reinterpret_cast<const uint4 *>(q_smem + (mt * KS + st) * 512 + lane * 16);
                            const uint32_t f[4] = {v.x, v.y, v.z, v.w};
                            mma16816(sc[mt][0], f, lo[0], hi[0]);
                            mma16816(sc[mt][1], f, lo[1], hi[1]);
                        }
                    }
                }
            }
            uint32_t pa[MT][4];
            const float kf[4] = {ks, ks, ks, ks}, vf[4] = {vs, vs, vs, vs};
            if (t0 + 16 <= lim_min)
                weights(sc, kf, vf, vs, t0, false, pa);
            else
                weights(sc, kf, vf, vs, t0, true, pa);
            // V: keys 2j, 2j+1, 2j+8, 2j+9, and for column n of tile nt the value d = n * (16 or 8) + nt
            constexpr int HW = D == 64 ? 2 : 4;  // words of a lane's run of d's
#pragma unroll
            for (int half = 0; half < (D == 256 ? 2 : 1); ++half) {
                uint32_t x[4][HW];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int key = 2 * j + (k & 1) + 8 * (k >> 1);
                    if constexpr (D == 64) {
                        const uint2 v = lds64(vt + tile_at<D>(key, g >> 1) + (g & 1) * 8);
                        x[k][0] = code_bias<CODE>(v.x);
                        x[k][1] = code_bias<CODE>(v.y);
                    } else {
                        const uint4 v = lds128(vt + tile_at<D>(key, 8 * half + g));
                        x[k][0] = code_bias<CODE>(v.x);
                        x[k][1] = code_bias<CODE>(v.y);
                        x[k][2] = code_bias<CODE>(v.z);
                        x[k][3] = code_bias<CODE>(v.w);
                    }
                }
#pragma unroll
                for (int q = 0; q < HW; ++q) {
                    uint32_t b0[4], b1[4];
                    codes_to_half<CODE>(__byte_perm(x[0][q], x[1][q], 0x5140), b0[0], b0[1]);
                    codes_to_half<CODE>(__byte_perm(x[0][q], x[1][q], 0x7362), b0[2], b0[3]);
                    codes_to_half<CODE>(__byte_perm(x[2][q], x[3][q], 0x5140), b1[0], b1[1]);
                    codes_to_half<CODE>(__byte_perm(x[2][q], x[3][q], 0x7362), b1[2], b1[3]);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt) mma16816(o[mt][16 * half + 4 * q + e], pa[mt], b0[e], b1[e]);
                }
            }
            __syncwarp();
        }
        cp_async_wait<0>();

        // ---- the unfinished page's rows, in 16 bits
        const int tail = s.len - paged, key0 = 16 * w;  // this warp's first row of it
        if (t_end > paged_tiles && paged + key0 < min(s.len, lim_max)) {
            float sc[MT][2][4];
            float kf[4], vf[4];
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const int key = key0 + 8 * n + g;
                const bool live = key < tail && s.slot >= 0;
                const uint16_t *src = c.kt + ring_at(c, live ? s.slot : 0, h, paged + (live ? key : 0));
                uint4 x[D / 32];
                float amax = 0.0f;
#pragma unroll
                for (int k = 0; k < D / 64; ++k)
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        x[2 * k + z] = live ? *reinterpret_cast<const uint4 *>(src + k_dim<D>(j, k) + 8 * z) : make_uint4(0, 0, 0, 0);
                        amax = fmaxf(amax, amax8(x[2 * k + z], bf16));
                    }
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
                float mul, f;
                row_scale(amax, mul, f);
                if (s.slot < 0) f = __int_as_float(0x7fc00000);
                kf[2 * n] = __shfl_sync(0xffffffffu, f, 8 * j);          // keys 2j and 2j + 1 of the tile
                kf[2 * n + 1] = __shfl_sync(0xffffffffu, f, 8 * j + 4);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) sc[mt][n][0] = sc[mt][n][1] = sc[mt][n][2] = sc[mt][n][3] = 0.0f;
#pragma unroll
                for (int st = 0; st < KS; ++st) {
                    const uint4 &v = x[2 * (st >> 2) + ((st >> 1) & 1)];
                    const uint32_t lo = scale2(st & 1 ? v.z : v.x, mul, bf16), hi = scale2(st & 1 ? v.w : v.y, mul, bf16);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        if constexpr (Cfg::q_in_regs) {
                            mma16816(sc[mt][n], qa[mt * KS + st], lo, hi);
                        } else {
                            const uint4 q4 = *reinterpret_cast<const uint4 *>(q_smem + (mt * KS + st) * 512 + lane * 16);
                            const uint32_t f4[4] = {q4.x, q4.y, q4.z, q4.w};
                            mma16816(sc[mt][n], f4, lo, hi);
                        }
                    }
                }
            }
            // V rows: a first pass for the keys' scales, a second for the products
            float vmul[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int key = key0 + 2 * j + (k & 1) + 8 * (k >> 1);
                const bool live = key < tail && s.slot >= 0;
                const uint16_t *src = c.vt + ring_at(c, live ? s.slot : 0, h, paged + (live ? key : 0)) + g * (D / 8);
                float amax = 0.0f;
#pragma unroll
                for (int z = 0; z < D / 64; ++z)
                    if (live) amax = fmaxf(amax, amax8(*reinterpret_cast<const uint4 *>(src + 8 * z), bf16));
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 4));
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 8));
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 16));
                row_scale(amax, vmul[k], vf[k]);
                if (!live) vf[k] = 0.0f, vmul[k] = 0.0f;
            }
            float v_top = fmaxf(fmaxf(vf[0], vf[1]), fmaxf(vf[2], vf[3]));  // (NaN leaves it)
            v_top = fmaxf(v_top, __shfl_xor_sync(0xffffffffu, v_top, 1));
            v_top = fmaxf(v_top, __shfl_xor_sync(0xffffffffu, v_top, 2));
            uint32_t pa[MT][4];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)  // rows that pad see no more than the tail's own tokens
                for (int e = 0; e < 2; ++e) lim[mt][e] = min(lim[mt][e], s.len);
            weights(sc, kf, vf, v_top, paged + key0, true, pa);
#pragma unroll
            for (int half = 0; half < (D == 256 ? 2 : 1); ++half) {
                constexpr int HV = D == 64 ? 1 : 2;  // loads of 8 values of a lane's run of d's
#pragma unroll
                for (int z = 0; z < HV; ++z) {
                    uint4 x[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int key = key0 + 2 * j + (k & 1) + 8 * (k >> 1);
                        const bool live = key < tail && s.slot >= 0;
                        const uint16_t *src = c.vt + ring_at(c, live ? s.slot : 0, h, paged + (live ? key : 0)) + 128 * half +
                                              g * (D == 64 ? 8 : 16) + 8 * z;
                        x[k] = live ? *reinterpret_cast<const uint4 *>(src) : make_uint4(0, 0, 0, 0);
                        x[k].x = scale2(x[k].x, vmul[k], bf16);
                        x[k].y = scale2(x[k].y, vmul[k], bf16);
                        x[k].z = scale2(x[k].z, vmul[k], bf16);
                        x[k].w = scale2(x[k].w, vmul[k], bf16);
                    }
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        const uint32_t sel = q & 1 ? 0x7632 : 0x5410;
                        auto word = [&](int k) { return (q >> 1) == 0 ? x[k].x : (q >> 1) == 1 ? x[k].y : (q >> 1) == 2 ? x[k].z : x[k].w; };
                        const uint32_t b0 = __byte_perm(word(0), word(1), sel), b1 = __byte_perm(word(2), word(3), sel);
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt) mma16816(o[mt][16 * half + 8 * z + q], pa[mt], b0, b1);
                    }
                }
            }
        }

        // ---- join the four warps: into shared memory, each in units of its own maximum's share
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float sum = l[mt][e];
                sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                if (j == 0) {
                    s_ml[w][mt * 16 + g + 8 * e][0] = m[mt][e];
                    s_ml[w][mt * 16 + g + 8 * e][1] = sum;
                }
            }
        __syncthreads();  // every warp's ring is idle, and the maxima are there
        float *merge = reinterpret_cast<float *>(smem);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = mt * 16 + g + 8 * e;
                float top = s_ml[0][r][0];
#pragma unroll
                for (int k = 1; k < kDecWarps; ++k) top = fmaxf(top, s_ml[k][r][0]);
                const float f = ex2(m[mt][e] - top) * (v_ref / kWeightUnit);
                float *to = merge + (w * R + r) * D;
                // column 2j (and 2j + 1) of tile nt is d = n * run + nt within its 128 (or 64)
                constexpr int run = D == 64 ? 8 : 16;
#pragma unroll
                for (int n = 0; n < NT; n += 4)
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const int d = (n / 16) * 128 * (D != 64) + (2 * j + q) * run + (D == 64 ? n : n % 16);
                        *reinterpret_cast<float4 *>(to + d) = make_float4(o[mt][n][2 * e + q] * f, o[mt][n + 1][2 * e + q] * f,
                                                                          o[mt][n + 2][2 * e + q] * f, o[mt][n + 3][2 * e + q] * f);
                    }
            }
        if (tid < R) {
            float top = s_ml[0][tid][0], sum = 0.0f;
            for (int k = 1; k < kDecWarps; ++k) top = fmaxf(top, s_ml[k][tid][0]);
            for (int k = 0; k < kDecWarps; ++k) sum += s_ml[k][tid][1] * ex2(s_ml[k][tid][0] - top);
            s_part[tid][0] = top;
            s_part[tid][1] = sum;
        }
        __syncthreads();
        auto merged = [&](int r, int d) {
            float4 x = *reinterpret_cast<const float4 *>(merge + r * D + d);
#pragma unroll
            for (int k = 1; k < kDecWarps; ++k) {
                const float4 y = *reinterpret_cast<const float4 *>(merge + (k * R + r) * D + d);
                x.x += y.x;
                x.y += y.y;
                x.z += y.z;
                x.w += y.w;
            }
            return x;
        };
        auto store = [&](int r, int d, float4 x, float sum) {
            const int rr = rb * R + r, row = s.row0 + rr / c.G, head = h * c.G + rr % c.G;
            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
            uint2 y;
            if (bf16)
                y = make_uint2(pack2<SI_KV_BF16>(x.x * inv, x.y * inv), pack2<SI_KV_BF16>(x.z * inv, x.w * inv));
            else
                y = make_uint2(pack2<SI_KV_F16>(x.x * inv, x.y * inv), pack2<SI_KV_F16>(x.z * inv, x.w * inv));
            *reinterpret_cast<uint2 *>(a.out.p + row * a.out.row + head * a.out.head + d) = y;
        };
        auto store_lse = [&](int r, float top, float sum) {
            const int rr = rb * R + r, row = s.row0 + rr / c.G, head = h * c.G + rr % c.G;
            if (a.lse) a.lse[(int64_t)row * c.H + head] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
        };
        if (t_first == 0 && t_end == tiles) {
            for (int k = tid; k < rows * (D / 4); k += kDecThreads) {
                const int r = k / (D / 4), d = k % (D / 4) * 4;
                store(r, d, merged(r, d), s_part[r][1]);
            }
            if (tid < rows) store_lse(tid, s_part[tid][0], s_part[tid][1]);
            __syncthreads();
        } else {
            const int64_t pf = partial_floats(R, D);
            float *slot = a.partial + (2 * (int64_t)blockIdx.x + (t_first == 0 ? 1 : 0)) * pf;
            for (int k = tid; k < rows * (D / 4); k += kDecThreads) {
                const int r = k / (D / 4), d = k % (D / 4) * 4;
                __stcg(reinterpret_cast<float4 *>(slot + r * D + d), merged(r, d));
            }
            if (tid < rows) __stcg(reinterpret_cast<float2 *>(slot + R * D + 2 * tid), make_float2(s_part[tid][0], s_part[tid][1]));
            // the CTAs that share the item: those of its first and of its last unit
            const long long i0 = u - t_first, i1 = i0 + tiles - 1;
            const long long c0 = ((i0 + 1) * N - 1) / total, c1 = ((i1 + 1) * N - 1) / total;
            __threadfence();
            __syncthreads();
            if (tid == 0) {
                const int n = atomicAdd(a.counters + c0, 1);
                s_last = n == (int)(c1 - c0);
                if (s_last) a.counters[c0] = 0;
                __threadfence();
            }
            __syncthreads();
            if (s_last) {
                const int nc = (int)(c1 - c0) + 1;
                auto slot_of = [&](int k) { return a.partial + (2 * (c0 + k) + (k == 0 ? 1 : 0)) * pf; };
                for (int k = tid; k < rows * (D / 4); k += kDecThreads) {
                    const int r = k / (D / 4), d = k % (D / 4) * 4;
                    float top = kNoScore, sum = 0.0f;
                    for (int q = 0; q < nc; ++q) top = fmaxf(top, __ldcg(slot_of(q) + R * D + 2 * r));
                    float4 x = make_float4(0, 0, 0, 0);
                    for (int q = 0; q < nc; ++q) {
                        const float2 ml = __ldcg(reinterpret_cast<const float2 *>(slot_of(q) + R * D + 2 * r));
                        const float4 y = __ldcg(reinterpret_cast<const float4 *>(slot_of(q) + r * D + d));
                        const float f = ex2(ml.x - top);
                        sum += ml.y * f;
                        x.x = fmaf(y.x, f, x.x);
                        x.y = fmaf(y.y, f, x.y);
                        x.z = fmaf(y.z, f, x.z);
                        x.w = fmaf(y.w, f, x.w);
                    }
                    store(r, d, x, sum);
                    if (d == 0) store_lse(r, top, sum);
                }
            }
            __syncthreads();
        }
        u += t_end - t_first;
        off += t_end - t_first;
    }
}

template <int CODE, int D, int MT>
cudaError_t decode_launch(const Plan &p, const DecodeArgs &a, cudaStream_t s) {
    using Cfg = DecodeCfg<D, MT>;
    cudaError_t e = allow_smem<k_kv_decode<CODE, D, MT>>(p, Cfg::smem);
    if (e != cudaSuccess) return e;
    k_kv_decode<CODE, D, MT><<<p.sm_count * Cfg::ctas, kDecThreads, Cfg::smem, s>>>(a);
    return cudaGetLastError();
}

}  // namespace kv
}  // namespace si
