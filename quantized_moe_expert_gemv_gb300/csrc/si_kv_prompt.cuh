// si_kv_prompt.cuh -- attention of many rows over the cache (a prompt, a chunk
// of one) on the tcgen05 tensor cores, head_dim 64 and 128.
//
// One CTA for 256 rows (query token, query head of the kv head) of one sequence
// and kv head: two tiles of 128 rows, which share every K and V tile.
//   S = Q K^T (fp16 operands, fp32 sums in tensor memory), p = 2^(f S - m),
//   O += (p times the page's V scale, fp16, in tensor memory) V
// The running maximum m is lazy and the V scale is relative to a running
// reference, as in the few-row kernel (si_kv_decode.cuh), so both are rarely
// moved and O is rarely rescaled.
// Roles: warps 0-3 and 4-7 are the softmax of the two row tiles, a thread a row;
// warps 8-11 turn codes into fp16 tiles in shared memory (K with d innermost, V
// with d innermost too: the second product takes V as its transposed operand);
// warps 12 and 13 issue the two row tiles' products; warp 14 looks up pages and
// scales ahead, with the largest V scale up to each (warp 15 only lends its registers).  While one row tile's products
// run, the other's softmax does.
// Bound: at D = 128 a pair of row tiles and 128 keys takes 2048 cycles of the
// tensor cores (32 steps of 128 x 128 x 16, 64 cycles each) beside 1024 of the
// exponential unit (256 x 128 at 32 a cycle) and the tiles' making, 64 KB written to
// shared memory that the products then read; it takes about 3000, the rest being
// the chain from a score to its weight.  At D = 64 the exponential and the products
// are equal.
// Two row tiles a CTA: every K and V tile is made once for 256 rows; with 128 rows
// the making (2 x 128 x D codes) alone would take as long as the products.
// Measured (head_dim 128): prompts of 2900 to 4100 tokens, 32/4 heads, 253 us, 46 %
// of the measured dense rate (causal products only); 1024 tokens behind 24000,
// 32/8 heads, 311 us (E4M3, 69 %) and 343 (int8, whose codes take longer to convert); one prompt of 300, 22 us, of which
// the products are 3: the start, q and the tile with the unfinished page, whose
// rows and factors come one by one, are the rest.
#pragma once
#include "si_kv_decode.cuh"
#include "si_kv_tc.cuh"

namespace si {
namespace kv {

constexpr int kPrRows = 256, kPrKeys = kTileRows;
constexpr int kPrThreads = 16 * 32;
// Registers a thread after the roles part (of 128 each at the launch): 2 x 128 x 176 + 128 x 112 + 128 x 40 = 64512 <= 65536.
constexpr int kPrRegSoftmax = 176, kPrRegTiles = 112, kPrRegMma = 40;
static_assert(kPrRegSoftmax >= 128 && kPrRegTiles <= 128 && kPrRegMma <= 128 &&
                  2 * kPrRegSoftmax + kPrRegTiles + kPrRegMma <= 4 * 128,
              "more than the launch's registers would be waited for without end, and dec only goes down");
constexpr int kPrFactorSlots = 4, kPrInfoSlots = 8;
// What a tile of full pages needs for each 16 tokens: the page (0 where the table names none), K's and V's scale (NaN
// there), and the largest V scale of the 16-token groups before each (NaN left out).
struct PromptInfo {
    int32_t page[8];
    float k[8], v[8], v_upto[9];
    float pad[3];
};

template <int D>
struct PromptCfg {
    static constexpr int tile = kPrKeys * D * 2;  // bytes of one fp16 tile of 128 rows
    static constexpr int q = 0;
    static constexpr int k = 2 * tile;
    static constexpr int v = k + 2 * tile;
    static constexpr int factors = v + 2 * tile;                       // [slots][3][128] floats: K's, V's, V's largest up to there
    static constexpr int info = factors + kPrFactorSlots * 3 * 128 * 4;  // [slots]: PromptInfo
    static constexpr int bars = info + kPrInfoSlots * (int)sizeof(PromptInfo);
    static constexpr int smem = bars + 32 * 8 + 1024;                  // + alignment slack
};
enum PromptBar { kBarQ = 0, kBarKFull = 1, kBarKEmpty = 3, kBarVFull = 5, kBarVEmpty = 7, kBarS = 9, kBarP = 11, kBarO = 13, kBarSFree = 15, kBarInfo = 17, kBarNever = 19, kBarFactors = 21 };
// Tensor memory columns: one S (the row tiles take turns: a softmax thread has its whole row in registers
// before the other tile's product is issued), P of each row tile, O of each.
constexpr int kTmS = 0, kTmP = 128, kTmO = 256;

struct PromptArgs {
    Ctx c;
    Rows q, out;
    float *lse;
    float scale2;
    int bf16;
    int log_page;
    int splits;
    int fault;
    long long budget;
    float *partial;  // [splits][T][H][D], then [splits][T][H][2]
};

// The CTA's first barrier, which each role reaches from its own code once its first loads are under way.
__device__ __forceinline__ void role_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kPrThreads) : "memory"); }
// The largest of the 128 factors at f up to each, to the 128 places behind them (NaN left out): a warp, four a lane.
__device__ __forceinline__ void factors_upto(float *f, int lane) {
    float4 y = reinterpret_cast<const float4 *>(f)[lane];
    y.x = fmaxf(y.x, 0.0f);
    y.y = fmaxf(y.x, y.y);
    y.z = fmaxf(y.y, y.z);
    y.w = fmaxf(y.z, y.w);
    float upto = y.w;
    for (int o = 1; o < 32; o <<= 1) {
        const float up = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto = fmaxf(upto, up);
    }
    const float up = __shfl_up_sync(0xffffffffu, upto, 1), before = lane == 0 ? 0.0f : up;
    reinterpret_cast<float4 *>(f + 128)[lane] = make_float4(fmaxf(before, y.x), fmaxf(before, y.y), fmaxf(before, y.z), upto);
}
template <int N>
__device__ __forceinline__ void reg_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

template <int CODE, int D>
__global__ void __launch_bounds__(kPrThreads, 1) k_kv_prompt(const PromptArgs a) {
    using Cfg = PromptCfg<D>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint32_t s_tmem;
    const Ctx &c = a.c;
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // (uniform)
    const bool bf16 = a.bf16;

    start_after();
    // ---- which rows: the last ones of each sequence first (they see the most keys)
    const int bh = c.B * c.Hk;
    const int split = blockIdx.x % a.splits, id = blockIdx.x / a.splits;
    const int b = id % bh / c.Hk, h = id % c.Hk;
    const Seq s = load_seq(c, b);
    const int blocks = (s.n * c.G + kPrRows - 1) / kPrRows;
    const int rb = blocks - 1 - id / bh;
    if (rb < 0) return;
    const int old = s.len - s.n, paged = s.len & ~(c.P - 1);
    const int rows = min(kPrRows, s.n * c.G - rb * kPrRows);
    int t_to[2];  // where the two row tiles' key tiles end
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const int last = rb * kPrRows + min(rows, 128 * (x + 1)) - 1;
        const int see = rows > 128 * x ? max(0, old + last / c.G + 1) : 0;
        t_to[x] = (see + kPrKeys - 1) / kPrKeys;
    }
    const int nt_all = max(t_to[0], t_to[1]);
    const int t_first = (int)((int64_t)nt_all * split / a.splits), t_last = (int)((int64_t)nt_all * (split + 1) / a.splits);
#pragma unroll
    for (int x = 0; x < 2; ++x) t_to[x] = max(t_first, min(t_to[x], t_last));
    const int nt = max(t_to[0], t_to[1]) - t_first;  // tiles of this CTA
    const int ntx[2] = {t_to[0] - t_first, t_to[1] - t_first};

    const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
    float *factors = reinterpret_cast<float *>(smem_raw + (base - smem_addr(smem_raw)) + Cfg::factors);
    PromptInfo *infos = reinterpret_cast<PromptInfo *>(smem_raw + (base - smem_addr(smem_raw)) + Cfg::info);
    auto bar = [&](int i) { return base + Cfg::bars + 8 * i; };

    bool ok = true;
    // A warp's bounded wait (its lanes give up together).  A role that gives up goes on to the end of
    // the kernel; the others run out in turn.
    auto wait = [&](int i, int parity) {
        if (ok && !mbar_wait_warp(bar(i), (uint32_t)parity, a.budget)) {
            ok = false;
            if (lane == 0) set_status(c.status, SI_ERR_TIMEOUT);
        }
        return ok;
    };
    if (warp < 8) {
        // ================================================= softmax: a thread a row
        reg_inc<kPrRegSoftmax>();
        const int x = warp >> 2, r = tid & 127;
        const int rr = rb * kPrRows + x * 128 + r;
        const bool live = x * 128 + r < rows;
        const int row = s.row0 + (live ? rr / c.G : 0), head = h * c.G + (live ? rr % c.G : 0);
        const int lim = live ? old + rr / c.G + 1 : 0;
        // the warp's 32 rows of q, four lanes a row: a lane a row would touch 32 lines a load (12000 instead of
        // 3000 cycles before the first product)
        float qf = 0.0f;
        {
            RowLoad<D> v[4];
            const int quad = lane >> 2, ch = lane & 3;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int at = x * 128 + 32 * (warp & 3) + 8 * k + quad, rq = rb * kPrRows + at;
                const bool in = at < rows;
                v[k].load(a.q.p + (s.row0 + (in ? rq / c.G : 0)) * a.q.row + (h * c.G + (in ? rq % c.G : 0)) * a.q.head, in, ch);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float f = v[k].store(base + Cfg::q + x * Cfg::tile, 32 * (warp & 3) + 8 * k + quad, ch, bf16);
                const float of = __shfl_sync(0xffffffffu, f, 4 * (lane & 7));
                if (quad >> 1 == k) qf = of;  // (this thread's row is 8 k + lane % 8 of the warp's)
            }
            qf *= a.scale2;
            tc::fence_proxy_async_smem();
        }
        role_sync();
        tc::fence_after_sync();
        const uint32_t tmem = s_tmem;
        mbar_arrive(bar(kBarQ));
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t ts = tmem + lanes + kTmS, tp = tmem + lanes + kTmP + x * 64, to = tmem + lanes + kTmO + x * 128;
        float m = kNoScore, v_ref = 1e-30f, v_inv = kWeightUnit / 1e-30f;
        f32x2 l2 = pk2(0.0f, 0.0f);
        bool far = false;  // a row of the warp has its maximum past kFar
        const int n = ntx[x];
        for (int i = 0; i < n; ++i) {
            const int key0 = (t_first + i) * kPrKeys;
            const float *kf = factors + (i % kPrFactorSlots) * 384, *vf = kf + 128;
            if (!wait(kBarS + x, i & 1)) break;
            tc::fence_after_sync();
            const bool whole = key0 + kPrKeys <= paged;                 // a factor for every 16 keys
            // Rescale of the sums so far where the maximum or the V scales' reference moves.
            auto adjust = [&](float top, float v_top) {
                const bool grow = top > m + kLazy, scale = v_top > v_ref;
                if (!__any_sync(0xffffffffu, grow || scale)) return;
                float f = 1.0f;
                if (grow) {
                    f = ex2(m - top);
                    m = top;
                    l2 = mul2(l2, pk2(f, f));
                }
                if (scale) {
                    f *= v_ref / v_top;
                    v_ref = v_top;
                    v_inv = kWeightUnit / v_top;
                }
                far = __any_sync(0xffffffffu, fabsf(m) > kFar && m != kNoScore);
                if (i > 0) {
#pragma unroll 1
                    for (int q = 0; q < D / 32; ++q) {
                        uint32_t o[32];
                        tc::tmem_ld32(to + 32 * q, o);
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                        tmem_st32(to + 32 * q, o);
                    }
                }
            };
            if (whole) {
                uint32_t z[4][32];
#pragma unroll
                for (int q = 0; q < 4; ++q) tc::tmem_ld32(ts + 32 * q, z[q]);
                const PromptInfo &info = infos[i % kPrInfoSlots];
                // (the largest that the row sees: a later page's scale, however large, takes no bits of its weights)
                const int see = lim - key0;
                const float v_top = info.v_upto[min(max(see + 15, 0) >> 4, 8)];
                tc::tmem_wait_ld();
                tc::fence_before_sync();
                mbar_arrive(bar(kBarSFree + x));
                const bool all = __all_sync(0xffffffffu, !live || see >= kPrKeys);
                f32x2 sum;
                const float top = all ? row_top<false>(z, info.k, qf, see) : row_top<true>(z, info.k, qf, see);
                if (i > 0 && !wait(kBarO + x, (i - 1) & 1)) break;  // P and O are free: the last second product is done
                tc::fence_after_sync();
                adjust(top, v_top);
                if (all && !far)
                    row_weights<false>(z, info.k, info.v, qf, v_inv, m, far, see, tp, sum);
                else
                    row_weights<true>(z, info.k, info.v, qf, v_inv, m, far, see, tp, sum);
                l2 = add2(l2, sum);
            } else {
                // (the factors of four columns a load)
                const float4 *kf4 = reinterpret_cast<const float4 *>(kf), *vf4 = reinterpret_cast<const float4 *>(vf);
                const int see = lim - key0;
                const float v_top = see > 0 ? vf[127 + min(see, kPrKeys)] : 0.0f;  // (the largest up to the row's last column)
                float top = -INFINITY;
#pragma unroll 1
                for (int q = 0; q < 4; ++q) {
                    uint32_t z[32];
                    tc::tmem_ld32(ts + 32 * q, z);
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int k = 0; k < 32; k += 4) {
                        const float4 f = kf4[8 * q + k / 4];
                        const float fs[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (32 * q + k + e < see) top = fmaxf(top, __fmul_rn(__uint_as_float(z[k + e]), fs[e] * qf));
                    }
                }
                if (i > 0 && !wait(kBarO + x, (i - 1) & 1)) break;
                tc::fence_after_sync();
                adjust(top, v_top);
#pragma unroll 1
                for (int q = 0; q < 4; ++q) {
                    uint32_t z[32], p[16];
                    tc::tmem_ld32(ts + 32 * q, z);
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int k = 0; k < 32; k += 4) {
                        const float4 f = kf4[8 * q + k / 4], g = vf4[8 * q + k / 4];
                        const float fs[4] = {f.x, f.y, f.z, f.w}, gs[4] = {g.x, g.y, g.z, g.w};
                        float w[4], pp[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const bool in = 32 * q + k + e < see;
                            pp[e] = in ? ex2(__fmul_rn(__uint_as_float(z[k + e]), fs[e] * qf) - m) : 0.0f;
                            w[e] = in ? pp[e] * (gs[e] * v_inv) : 0.0f;
                        }
                        l2 = add2(l2, pk2(pp[0], pp[1]));
                        l2 = add2(l2, pk2(pp[2], pp[3]));
                        p[k / 2] = half2_bits(w[0], w[1]);
                        p[k / 2 + 1] = half2_bits(w[2], w[3]);
                    }
                    tmem_st16(tp + 16 * q, p);
                }
                tc::fence_before_sync();
                mbar_arrive(bar(kBarSFree + x));
            }
            tmem_wait_st();
            tc::fence_before_sync();
            mbar_arrive(bar(kBarP + x));
        }
        // ---- the rows' results
        if (n > 0) wait(kBarO + x, (n - 1) & 1);
        tc::fence_after_sync();
        float l, l_odd;
        up2(l2, l, l_odd);
        l += l_odd;
        if (ok) {
            const float f = v_ref / kWeightUnit, inv = l == 0.0f ? no_weight(lim - 1) : f / l;
            if (a.splits == 1) {
                uint16_t *dst = a.out.p + row * a.out.row + head * a.out.head;
#pragma unroll
                for (int q = 0; q < D / 32; ++q) {
                    uint32_t o[32];
                    if (n > 0) {
                        tc::tmem_ld32(to + 32 * q, o);
                        tc::tmem_wait_ld();
                    } else {
#pragma unroll
                        for (int k = 0; k < 32; ++k) o[k] = 0;
                    }
#pragma unroll
                    for (int k = 0; k < 32; k += 8) {
                        uint32_t y[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float u = __uint_as_float(o[k + 2 * e]) * inv, v = __uint_as_float(o[k + 2 * e + 1]) * inv;
                            y[e] = bf16 ? pack2<SI_KV_BF16>(u, v) : pack2<SI_KV_F16>(u, v);
                        }
                        if (live) *reinterpret_cast<uint4 *>(dst + 32 * q + k) = make_uint4(y[0], y[1], y[2], y[3]);
                    }
                }
                if (live && a.lse) a.lse[(int64_t)row * c.H + head] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
            } else {
                const int64_t at = ((int64_t)split * c.T + row) * c.H + head;
                float *dst = a.partial + at * D;
#pragma unroll
                for (int q = 0; q < D / 32; ++q) {
                    uint32_t o[32];
                    if (n > 0) {
                        tc::tmem_ld32(to + 32 * q, o);
                        tc::tmem_wait_ld();
                    } else {
#pragma unroll
                        for (int k = 0; k < 32; ++k) o[k] = 0;
                    }
#pragma unroll
                    for (int k = 0; k < 32; k += 4)
                        if (live)
                            *reinterpret_cast<float4 *>(dst + 32 * q + k) =
                                make_float4(__uint_as_float(o[k]) * f, __uint_as_float(o[k + 1]) * f,
                                            __uint_as_float(o[k + 2]) * f, __uint_as_float(o[k + 3]) * f);
                }
                if (live)
                    *reinterpret_cast<float2 *>(a.partial + (int64_t)a.splits * c.T * c.H * D + at * 2) = make_float2(m, l);
            }
        }
        tc::fence_before_sync();
    } else if (warp < 12) {
        // ================================================= codes to fp16 tiles
        reg_dec<kPrRegTiles>();
        const int pt = tid - 256;              // 0..127
        const int ch = pt & 3, r0 = pt >> 2;   // chunks ch, ch + 4 of rows r0 + 32 k
        constexpr int CC = D / 64;             // chunks of 16 codes of one row that a thread takes
        uint4 kx[4 * CC], vx[4 * CC];
        // The codes of a tile of full pages are loaded a tile ahead.
        const uint32_t page_bytes = (uint32_t)c.Hk * c.P * D;
        const uint64_t own = (uint64_t)h * c.P * D + ch * 16;
        const uint8_t *k_own = c.kc + own, *v_own = c.vc + own;
        auto row_at = [&](uint32_t page, int k) -> uint64_t {  // of row r0 + 32 k's codes (a tile starts at a page)
            return (uint64_t)page * page_bytes + (uint32_t)(((r0 + 32 * k) & (c.P - 1)) * D);
        };
        auto load = [&](int i, bool v) {
            if (i >= nt || (t_first + i + 1) * kPrKeys > paged) return;
            const PromptInfo &info = infos[i % kPrInfoSlots];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint8_t *at = (v ? v_own : k_own) + row_at((uint32_t)info.page[(r0 >> 4) + 2 * k], k);
#pragma unroll
                for (int q = 0; q < CC; ++q) {
                    const uint4 y = *reinterpret_cast<const uint4 *>(at + 64 * q);
                    if (v)
                        vx[k * CC + q] = y;
                    else
                        kx[k * CC + q] = y;
                }
            }
        };
        // units 2 ch and 2 ch + 1 of row r0; rows 32 on lie 4096 bytes on, the other half of D 16384
        const uint32_t a0 = f16_tile_at(r0, 2 * ch), a1 = f16_tile_at(r0, 2 * ch + 1);
        auto store = [&](uint32_t tile, int i, bool v) {
            const int key0 = (t_first + i) * kPrKeys;
            float *kf = factors + (i % kPrFactorSlots) * 384;
            if (key0 + kPrKeys <= paged) {
                const uint4(&x)[4 * CC] = v ? vx : kx;
                codes_to_tile<CODE, 0>(x[0], tile + a0, tile + a1);
                codes_to_tile<CODE, 4096>(x[CC], tile + a0, tile + a1);
                codes_to_tile<CODE, 8192>(x[2 * CC], tile + a0, tile + a1);
                codes_to_tile<CODE, 12288>(x[3 * CC], tile + a0, tile + a1);
                if constexpr (CC == 2) {
                    codes_to_tile<CODE, 16384>(x[1], tile + a0, tile + a1);
                    codes_to_tile<CODE, 16384 + 4096>(x[3], tile + a0, tile + a1);
                    codes_to_tile<CODE, 16384 + 8192>(x[5], tile + a0, tile + a1);
                    codes_to_tile<CODE, 16384 + 12288>(x[7], tile + a0, tile + a1);
                }
                return;
            }
            key_rows<CODE, D>(c, s, b, h, v, key0, a.log_page, bf16, tile, kf + (v ? 128 : 0), pt);
        };
        role_sync();
        if (nt > 0) wait(kBarInfo, 0);
        load(0, false);
        load(0, true);
        int slow = 0;  // tiles without a page's scale for each column so far
        for (int i = 0; i < nt; ++i) {
            const int st = i & 1;
            const bool whole = (t_first + i + 1) * kPrKeys <= paged;
            if (i >= 2 && !wait(kBarKEmpty + st, ((i >> 1) - 1) & 1)) break;
            store(base + Cfg::k + st * Cfg::tile, i, false);
            // the softmax reads the tile's V factors with its K factors, so a tile without a page's scale
            // for each column has V in place before K is handed on
            if (!whole) {
                if (i >= 2 && !wait(kBarVEmpty + st, ((i >> 1) - 1) & 1)) break;
                store(base + Cfg::v + st * Cfg::tile, i, true);
                mbar_arrive(bar(kBarFactors));
                if (warp == 8) {
                    if (!wait(kBarFactors, slow & 1)) break;
                    factors_upto(factors + (i % kPrFactorSlots) * 384 + 128, lane);
                }
                ++slow;
            }
            tc::fence_proxy_async_smem();
            mbar_arrive(bar(kBarKFull + st));
            if (i + 1 < nt && !wait(kBarInfo + (st ^ 1), ((i + 1) >> 1) & 1)) break;
            load(i + 1, false);
            if (whole) {
                if (i >= 2 && !wait(kBarVEmpty + st, ((i >> 1) - 1) & 1)) break;
                store(base + Cfg::v + st * Cfg::tile, i, true);
                tc::fence_proxy_async_smem();
            }
            mbar_arrive(bar(kBarVFull + st));
            load(i + 1, true);
        }
    } else {
      reg_dec<kPrRegMma>();
      if (warp == 12) {
        if (lane == 0) {
            mbar_init(bar(kBarQ), 256);
            for (int i = 0; i < 2; ++i) {
                mbar_init(bar(kBarKFull + i), 128);
                mbar_init(bar(kBarKEmpty + i), 2);
                mbar_init(bar(kBarVFull + i), 128);
                mbar_init(bar(kBarVEmpty + i), 2);
                mbar_init(bar(kBarS + i), 1);
                mbar_init(bar(kBarP + i), 128);
                mbar_init(bar(kBarO + i), 1);
                mbar_init(bar(kBarSFree + i), 128);
                mbar_init(bar(kBarInfo + i), 1);
            }
            mbar_init(bar(kBarNever), 1);
            mbar_init(bar(kBarNever + 1), 1);
            mbar_init(bar(kBarFactors), 128);
            fence_mbar_init();
        }
        __syncwarp();
        tc::tmem_alloc(smem_addr(&s_tmem), 512);
        tc::tmem_relinquish();
        tc::fence_before_sync();
      }
      role_sync();
      if (warp < 14) {
        tc::fence_after_sync();
        const uint32_t tmem = s_tmem;
        const int x = warp - 12;  // a warp for each row tile: neither's waits hold up the other's products
        const int n = x ? ntx[1] : ntx[0], n0 = ntx[0], n1 = ntx[1];
        // ================================================= the products
        constexpr uint32_t id_qk = tc::idesc_f16_f32(128, kPrKeys);
        constexpr uint32_t id_pv = tc::idesc_f16_f32(128, D) | (1u << 16);  // V: transposed operand
        const uint64_t q_desc = tc::sdesc_sw128(base + Cfg::q), k_desc = tc::sdesc_sw128(base + Cfg::k);
        const uint64_t v_desc = sdesc_sw128_mn(base + Cfg::v, 16384);
        auto qk = [&](int st) {
            const uint64_t qd = q_desc + (x * Cfg::tile >> 4), kd = k_desc + (st * Cfg::tile >> 4);
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                constexpr int half = 16384 >> 4;
                mma_ss(tmem + kTmS, qd + ((k >> 2) * half + (k & 3) * 2), kd + ((k >> 2) * half + (k & 3) * 2), id_qk, k > 0);
            }
            mma_done(bar(kBarS + x));
        };
        auto pv = [&](int st, bool acc) {
            const uint64_t vd = v_desc + (st * Cfg::tile >> 4);
#pragma unroll
            for (int k = 0; k < kPrKeys / 16; ++k)
                mma_ts(tmem + kTmO + x * 128, tmem + kTmP + x * 64 + 8 * k, vd + k * (2048 >> 4), id_pv, acc || k > 0);
            mma_done(bar(kBarO + x));
        };
        // S is used in the order (tile 0, x 0), (tile 0, x 1), (tile 1, x 0) .. (row tile 0 has no more key tiles
        // than row tile 1, or the latter has none).  Before use, the last user's rows are in registers.  Each
        // row tile says so on its own barrier, of which one warp sees every phase (a barrier of both would be
        // taken for free two phases early).
        auto s_free = [&](int i) {
            if (x == 0) return i == 0 || wait(kBarSFree + (n1 > 0), (i - 1) & 1);
            if (i < n0) return wait(kBarSFree, i & 1);
            return i == 0 || wait(kBarSFree + 1, (i - 1) & 1);
        };
        if (a.fault) wait(kBarNever, 0);
        if (nt > 0 && wait(kBarQ, 0)) {
            // S of step i, then the second product of step i - 1
            for (int i = 0; i <= nt; ++i) {
                const int st = i & 1;
                if (i < nt) {
                    if (!wait(kBarKFull + st, (i >> 1) & 1)) break;
                    if (i < n) {
                        if (!s_free(i)) break;
                        tc::fence_after_sync();
                        qk(st);
                    }
                    // (only what the producers will wait for: nothing arrives after the CTA's end)
                    if (i + 2 < nt) mma_done(bar(kBarKEmpty + st));
                }
                if (i > 0) {
                    if (!wait(kBarVFull + (st ^ 1), ((i - 1) >> 1) & 1)) break;
                    if (i - 1 < n) {
                        if (!wait(kBarP + x, (i - 1) & 1)) break;
                        tc::fence_after_sync();
                        pv(st ^ 1, i > 1);
                    }
                    if (i + 1 < nt) mma_done(bar(kBarVEmpty + (st ^ 1)));
                }
            }
        }
        // whatever was issued is over before the tensor memory goes back
        if (!ok) {
            mma_done(bar(kBarNever + x));
            mbar_wait_bounded(bar(kBarNever + x), 0, 4000000000LL);
        }
        tc::fence_before_sync();
      } else if (warp == 14) {
        // ================================================= pages and scales, two tiles ahead of K's
        // (tile j's once K's tile j - 2 is made: by then no one reads the slot or the phase that it takes)
        auto look = [&](int j, int &page, float &ks, float &vs) {
            const int key0 = (t_first + j) * kPrKeys;
            if (lane >= 8 || j >= nt || key0 + kPrKeys > paged) return;
            const int64_t p = load_page(c, b, (key0 + 16 * lane) >> a.log_page);
            page = p < 0 ? 0 : (int)p;
            ks = p < 0 ? __int_as_float(0x7fc00000) : c.ks[p * c.Hk + h];
            vs = p < 0 ? __int_as_float(0x7fc00000) : c.vs[p * c.Hk + h];
        };
        int page = 0;
        float ks = 0.0f, vs = 0.0f;
        look(0, page, ks, vs);
        for (int j = 0; j < nt; ++j) {
            if (j >= 2 && !wait(kBarKFull + (j & 1), ((j - 2) >> 1) & 1)) break;
            float upto = fmaxf(vs, 0.0f);
            for (int o = 1; o < 8; o <<= 1) {
                const float up = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto = fmaxf(upto, up);
            }
            if (lane < 8) {
                PromptInfo &info = infos[j % kPrInfoSlots];
                info.page[lane] = page;
                info.k[lane] = ks;
                info.v[lane] = vs;
                info.v_upto[lane + 1] = upto;
                if (lane == 0) info.v_upto[0] = 0.0f;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kBarInfo + (j & 1)));
            look(j + 1, page, ks, vs);
        }
      }
    }
    __syncwarp();
    __syncthreads();
    if (warp == 12) {
        tc::fence_after_sync();
        tc::tmem_dealloc(s_tmem, 512);
    }
}

// The splits' partial sums joined in their order: a thread four values of a row.
template <int D>
__global__ void __launch_bounds__(256) k_kv_join(const PromptArgs a) {
    start_after();
    const Ctx &c = a.c;
    const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t rh = at / (D / 4);
    if (rh >= (int64_t)c.T * c.H) return;
    const int d = (int)(at % (D / 4)) * 4;
    const int row = (int)(rh / c.H), head = (int)(rh % c.H);
    // The sequence of a row is the last one that starts at or before it, where all starts ascend.  One that does not may
    // lead the search astray (and the products' kernel has reported it): then every sequence is tried.  Rows of
    // none were not computed.
    int lo = 0, hi = c.B;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (c.q_start[mid] <= row)
            lo = mid;
        else
            hi = mid;
    }
    Seq s = load_seq(c, lo);
    auto out = [&]() { return row < s.row0 || row >= s.row0 + s.n; };
    if (out()) {
        if (*c.status == SI_OK) return;
        for (int b = 0; b < c.B && out(); ++b) s = load_seq(c, b);
        if (out()) return;
    }
    const float *ml = a.partial + (int64_t)a.splits * c.T * c.H * D;
    float m = kNoScore, l = 0.0f;
    float4 o = make_float4(0, 0, 0, 0);
    for (int k = 0; k < a.splits; ++k) m = fmaxf(m, ml[((int64_t)k * c.T * c.H + rh) * 2]);
    for (int k = 0; k < a.splits; ++k) {
        const int64_t i = (int64_t)k * c.T * c.H + rh;
        const float2 v = *reinterpret_cast<const float2 *>(ml + i * 2);
        const float4 y = *reinterpret_cast<const float4 *>(a.partial + i * D + d);
        const float f = ex2(v.x - m);
        l = fmaf(v.y, f, l);
        o.x = fmaf(y.x, f, o.x);
        o.y = fmaf(y.y, f, o.y);
        o.z = fmaf(y.z, f, o.z);
        o.w = fmaf(y.w, f, o.w);
    }
    const float inv = l == 0.0f ? no_weight(s.len - s.n + row - s.row0) : 1.0f / l;
    uint2 y;
    if (a.bf16)
        y = make_uint2(pack2<SI_KV_BF16>(o.x * inv, o.y * inv), pack2<SI_KV_BF16>(o.z * inv, o.w * inv));
    else
        y = make_uint2(pack2<SI_KV_F16>(o.x * inv, o.y * inv), pack2<SI_KV_F16>(o.z * inv, o.w * inv));
    *reinterpret_cast<uint2 *>(a.out.p + row * a.out.row + head * a.out.head + d) = y;
    if (a.lse && d == 0) a.lse[rh] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
}

template <int CODE, int D>
cudaError_t prompt_launch(const Plan &p, const PromptArgs &a, cudaStream_t s) {
    using Cfg = PromptCfg<D>;
    cudaError_t e = allow_smem<k_kv_prompt<CODE, D>>(Cfg::smem);
    if (e != cudaSuccess) return e;
    const int64_t blocks = ((int64_t)a.c.max_new * a.c.G + kPrRows - 1) / kPrRows * a.c.Hk * a.c.B * a.splits;
    if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
    e = launch(k_kv_prompt<CODE, D>, dim3((unsigned)blocks), kPrThreads, Cfg::smem, s, a);
    if (e != cudaSuccess || a.splits == 1) return e;
    const int64_t n = (int64_t)a.c.T * a.c.H * (D / 4);
    return launch(k_kv_join<D>, dim3((unsigned)((n + 255) / 256)), 256, 0, s, a);
}

}  // namespace kv
}  // namespace si
