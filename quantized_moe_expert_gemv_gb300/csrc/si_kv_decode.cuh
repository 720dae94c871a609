// si_kv_decode.cuh -- attention of few rows over the cache (a decode step, the
// verification of drafted tokens): running softmax over key tiles, split over
// the whole GPU along the keys.
//
//   out_r = sum_t p_rt v_t / sum_t p_rt,   p_rt = 2^(s_rt - m_r),   s_rt = f_t (q'_r . code_t)
// where f_t is the product of the page's scale, the row's power of two and
// sm_scale * log2 e, and m_r is a running maximum.
//
// Bound: HBM.  Every cached token is read once for all the rows of its kv
// head, 2D bytes of codes; the arithmetic per byte is the matrix work for 8
// rows and the codes' conversion to fp16 (1.4 instructions a byte, at half
// rate), which has to stay below the time that the byte takes to arrive: 23
// bytes a cycle and SM at the measured copy rate.  Measured (head_dim 128, bytes
// that cannot be spared over the time): 64 sequences of 200 to 16300 tokens, 32/8
// heads, 177 us, 88 % of the copy rate.  Two of 90000 to 131000, 64/8 heads of 64,
// 54 us, 75 %.  24 of up to 6000 with 2 to 6 new tokens, 16/8 heads of 256, where
// the sums' registers leave half the warps: 84 us, 58 %.  Short calls are latency:
// 12.1 us for one sequence of 1000 tokens (11.7 in a graph): start and lengths 2,
// pages and codes 2, a warp's and the CTA's sums 4, the join of 16 CTAs 3.
//  * Products: keys are the 16 rows of the warp-level product and q's rows its 8
//    columns (S^T = K Q^T, then O^T = V^T P^T), so a step of 8 query heads for
//    a kv head wastes none of it; with q's rows as the 16 rows, 4 heads used a
//    quarter of the matrix and softmax work, and a batch of 64 sequences took
//    273 us.  Between the two products P^T is transposed in registers.
//  * Work: units of 64 tokens of one (sequence, kv head, row group), numbered in
//    order; each CTA (two an SM, so that one copies while the other joins its
//    warps) takes an equal share of consecutive units, whatever the sequences'
//    lengths.  A CTA joins its warps' results for each
//    item it touches; an item that lies in several CTAs is joined by the last of
//    them to arrive (in groups of 16 where there are many), in the CTAs' order:
//    the same inputs give the same bits.
//  * A warp takes pieces of 16 tokens (one page: P >= 16), every W-th, and copies
//    them into its own ring in shared memory (cp.async, some pieces ahead): no
//    barrier between warps inside an item.
//  * The maximum is lazy: m moves only when a score passes it by more than 4
//    (a vote a piece instead of shuffles), and p stays below 2^4.
//  * p times the page's V scale is rounded to fp16 for the second product.  The
//    scale is taken relative to the largest so far that the row sees, so that the products stay
//    inside fp16: p < 2^4, scale/reference <= 1, times 2^11: at most 2^15; a
//    weight of one keeps its eleven bits down to a relative scale of 2^-25.
//    (bf16 weights, without the reference, have eight: half a step of the
//    output's own rounding, or eight steps for an fp16 output.)
#pragma once
#include "si_kv_mma.cuh"

namespace si {
namespace kv {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kLazy = 4.0f, kWeightUnit = 2048.0f;
// A running maximum before the first score: the lowest value, which any score that is a number moves (or equals).
// What is past the range (-inf, of a score that its row sees) has no weight; a row of such scores alone is NaN.
constexpr float kNoScore = -3.4028234663852886e38f;

// R8: column tiles of 8 rows.  As many warps as the registers allow (the second product's sums are
// D R8 / 4 a lane), then as many stages as fit 96 KB a CTA.
template <int D, int R8>
struct DecodeCfg {
    static constexpr int ctas = 2;  // a SM
    static constexpr int warps = D * R8 <= 128 ? 8 : D * R8 <= 256 ? 6 : 4;
    static constexpr int stage = 32 * D;  // bytes of one piece, K and V
    static constexpr int stages = 96 * 1024 / (warps * stage);
    static constexpr int ring = warps * stages * stage;
    static constexpr bool q_in_regs = D * R8 <= 256;
    static constexpr int q_bytes = q_in_regs ? 0 : R8 * (D / 16) * 256;
    static constexpr int smem = ring + q_bytes;
    static_assert(warps * 8 * R8 * D * 4 <= ring, "the warps' results are joined in the ring's place");
};

// What a row's sums are multiplied by where they have no weight at all: zero for a row that sees no token (the
// last that it sees is `last`), NaN for one whose scores are all below the range.
__device__ __forceinline__ float no_weight(int last) { return last < 0 ? 0.0f : __int_as_float(0x7fc00000); }

// Partial results in the scratch: two slots a CTA (an item that began in an
// earlier CTA, one that goes on in a later one), each [rows][D] sums, then [rows][2]
// maximum and sum.
__host__ __device__ constexpr int64_t partial_floats(int rows, int D) { return (int64_t)rows * (D + 2); }
constexpr int kMaxDecodeCtas = 1024;  // arrival counters: one an item's first CTA, then two a CTA for groups
constexpr int kJoinGroup = 16;
static_assert(3 * kMaxDecodeCtas <= kCounters, "");

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

// Units of 64 tokens of a sequence: its full pages, then the unfinished page.
__device__ __forceinline__ int seq_tiles(const Ctx &c, int len) {
    const int paged = len & ~(c.P - 1);
    return (paged + 63) / 64 + (paged < len ? 1 : 0);
}

// An item's start and end (its first pages' addresses, q, the join) take a CTA as long as some units of
// tokens: that many units without tokens go before each item's own, so that a share of many short sequences
// costs no more than one of a long one.  (64 sequences of 200 to 16300 tokens: 225 us with 4, 207 with 6, 187
// with 14, 176 with 24, 180 with 44.)
constexpr int kDecodeOver = 24, kWeighOver = 12, kDecodeAlone = 8;
struct Segment {  // what a share takes of an item: its tiles [first, end) of `tiles`
    int item, first, end, step;       // step: units that the share has used up
    long long unit0, unit1;           // the units of the item's first and last tile
};
__device__ __forceinline__ Segment take_segment(int tiles, int over, long long off, long long u, long long u_end) {
    Segment s;
    const int all = tiles + over;
    // (a 64-bit division takes a hundred instructions: only where the numbers need it)
    s.item = off < (1ll << 31) ? (int)((uint32_t)off / (uint32_t)all) : (int)(off / all);
    const int x0 = (int)(off - (long long)s.item * all), x1 = (int)min((long long)all, x0 + (u_end - u));
    s.first = max(0, x0 - over);
    s.end = max(0, x1 - over);
    s.step = x1 - x0;
    s.unit0 = u - x0 + over;
    s.unit1 = u - x0 + all - 1;
    return s;
}

// k of n parts of a total, and the part that unit u lies in (k n fits 32 bits for totals up to 2^21).
__device__ __forceinline__ long long part_of(uint32_t k, long long total, long long n) {
    if (total < (1 << 21)) return (uint32_t)(k * (uint32_t)total) / (uint32_t)n;
    return k * total / n;
}
__device__ __forceinline__ int part_with(long long u, long long total, long long n) {
    if (total < (1 << 21)) return (int)(((uint32_t)(u + 1) * (uint32_t)n - 1) / (uint32_t)total);
    return (int)(((u + 1) * n - 1) / total);
}
static_assert(kMaxDecodeCtas <= 2047, "k and n of part_of and part_with");

// A CTA's equal share [begin, end) of all units, and the sequence that `begin` lies in.  `units_of(b)`:
// units of sequence b.  All threads call this; `some_empty`: whether a sequence has none.
struct Share {
    long long total, ctas, begin, end, off;  // off: begin's place within sequence b
    int b;
    bool some_empty;
};
// Where items are short (`alone` units or fewer on average) there are no more CTAs than items, `items_of(b)` of
// sequence b: an item in one CTA needs no join.  (One sequence, 4 kv heads, in a graph: 8.1 us in one CTA an
// item and 10.7 split at 100 tokens, 10.0 and 11.1 at 300; at 1000, where the rule splits, 13.7 and 11.9.)
template <int WARPS, typename F, typename G>
__device__ __forceinline__ Share take_share(int B, F units_of, G items_of, int alone) {
    __shared__ long long s_scan[WARPS];
    __shared__ long long s_off;
    __shared__ int s_b, s_items[WARPS];
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const int per = (B + WARPS * 32 - 1) / (WARPS * 32);
    long long mine = 0;
    bool empty = false;
    int items = 0;
    for (int b = tid * per; b < min(B, (tid + 1) * per); ++b) {
        const long long n = units_of(b);
        mine += n;
        items += n == 0 ? 0 : items_of(b);
        empty |= n == 0;
    }
    long long incl = mine;
    for (int o = 1; o < 32; o <<= 1) {
        const long long up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
    }
    if (lane == 31) s_scan[w] = incl;
    items = __reduce_add_sync(0xffffffffu, items);
    if (lane == 0) s_items[w] = items;
    Share s;
    s.some_empty = __syncthreads_or(empty);
    long long before = incl - mine;
    s.total = 0;
#pragma unroll
    for (int k = 0; k < WARPS; ++k) {
        if (k < w) before += s_scan[k];
        s.total += s_scan[k];
    }
    items = 0;
#pragma unroll
    for (int k = 0; k < WARPS; ++k) items += s_items[k];
    s.ctas = s.total <= (long long)items * alone ? items : s.total;
    s.ctas = s.ctas < (long long)gridDim.x ? s.ctas : (long long)gridDim.x;
    s.begin = s.end = 0;
    if (blockIdx.x < s.ctas) {
        s.begin = part_of(blockIdx.x, s.total, s.ctas);
        s.end = part_of(blockIdx.x + 1, s.total, s.ctas);
        if (before <= s.begin && s.begin < before + mine) {
            int b = tid * per;
            long long at = before, n;
            while (at + (n = units_of(b)) <= s.begin) {
                at += n;
                ++b;
            }
            s_b = b;
            s_off = s.begin - at;
        }
    }
    __syncthreads();
    s.b = s_b;
    s.off = s_off;
    return s;
}

template <int CODE, int D, int R8>
__global__ void __launch_bounds__(DecodeCfg<D, R8>::warps * 32, DecodeCfg<D, R8>::ctas) k_kv_decode(const DecodeArgs a) {
    using Cfg = DecodeCfg<D, R8>;
    constexpr int W = Cfg::warps, THREADS = W * 32;
    constexpr int R = 8 * R8;       // rows of an item
    constexpr int MT = D / 16;      // row tiles of the second product
    constexpr int KS = D / 16;      // steps of the first
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int s_last;
    __shared__ __align__(8) float s_ml[W][R][2];
    __shared__ __align__(8) float s_part[R][2];
    const Ctx &c = a.c;
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, g = lane >> 2, j = lane & 3;
    const bool bf16 = a.bf16;

    start_after();
    const Share share = take_share<W>(c.B, [&](int b) -> long long {
        const Seq s = load_seq(c, b);
        const int tiles = seq_tiles(c, s.len);
        return tiles == 0 ? 0ll : (long long)(tiles + kDecodeOver) * c.Hk * ((s.n * c.G + R - 1) / R);
    }, [&](int b) { return c.Hk * ((load_seq(c, b).n * c.G + R - 1) / R); }, kDecodeOver + kDecodeAlone);
    // rows whose sequence has no token at all are in no unit: zeros, a row a CTA at a time
    if (share.some_empty) {
        const int lanes = min((int)gridDim.x, c.B);  // sequences at a time
        if (blockIdx.x < gridDim.x / lanes * lanes)
            for (int b = blockIdx.x % lanes; b < c.B; b += lanes) {
                const Seq s = load_seq(c, b);
                if (s.len > 0) continue;
                for (int i = blockIdx.x / lanes; i < s.n; i += gridDim.x / lanes)
                    for (int k = tid; k < c.H * (D / 8); k += THREADS) {
                        const int row = s.row0 + i, head = k / (D / 8), d = k % (D / 8) * 8;
                        *reinterpret_cast<uint4 *>(a.out.p + row * a.out.row + head * a.out.head + d) = make_uint4(0, 0, 0, 0);
                        if (a.lse && d == 0) a.lse[(int64_t)row * c.H + head] = -INFINITY;
                    }
            }
    }
    if (blockIdx.x >= share.ctas) return;
    int b = share.b;
    long long off = share.off, u = share.begin;
    const long long u_end = share.end;

    const uint32_t ring = smem_addr(smem) + w * (Cfg::stages * Cfg::stage);
    uint8_t *q_smem = smem + Cfg::ring;
    PieceCopy<D> piece;
    piece.init(lane);
    KeyLoad<D> keys;
    keys.init(g, j);
    // V: keys 2j and 2j + 1 (and eight on), this lane's run of d's
    const uint32_t v_at0 = D == 64 ? tile_at<D>(2 * j, g >> 1) + (g & 1) * 8 : tile_at<D>(2 * j, g);
    const uint32_t v_at1 = D == 64 ? tile_at<D>(2 * j + 1, g >> 1) + (g & 1) * 8 : tile_at<D>(2 * j + 1, g);

    while (u < u_end) {
        const Seq s = load_seq(c, b);
        const int tiles = seq_tiles(c, s.len);
        const int groups = (s.n * c.G + R - 1) / R;
        const long long n_units = tiles == 0 ? 0ll : (long long)(tiles + kDecodeOver) * c.Hk * groups;
        if (off >= n_units) {  // on to the next sequence (one without units among them)
            off -= n_units;
            ++b;
            continue;
        }
        const Segment seg = take_segment(tiles, kDecodeOver, off, u, u_end);
        u += seg.step;
        off += seg.step;
        const int t_first = seg.first, t_end = seg.end;
        if (t_first == t_end) continue;
        const int h = seg.item / groups, rb = seg.item % groups;
        const int rows = min(R, s.n * c.G - rb * R);
        const int paged = s.len & ~(c.P - 1), old = s.len - s.n;
        const int lim_min = old + rb * R / c.G + 1, lim_max = old + (rb * R + rows - 1) / c.G + 1;
        const int paged_tiles = (paged + 63) / 64;

        // q's rows are on their way first: nothing else waits for them
        RowPart<D> q_part[Cfg::q_in_regs ? R8 : 1];
        auto q_load = [&](int n, RowPart<D> &to) {
            const int r = rb * R + n * 8 + g;
            const bool live = n * 8 + g < rows;
            to.load(a.q.p + (s.row0 + (live ? r / c.G : 0)) * a.q.row + (h * c.G + (live ? r % c.G : 0)) * a.q.head, live, j);
        };
        if constexpr (Cfg::q_in_regs) {
#pragma unroll
            for (int n = 0; n < R8; ++n) q_load(n, q_part[n]);
        }

        // and the unfinished page's rows on their way to the second-level cache
        if (t_end > paged_tiles && w >= W - 4 && s.slot >= 0) {
            constexpr int LINES = D / 64;  // of 128 bytes in a row
#pragma unroll
            for (int k = lane; k < 16 * LINES; k += 32) {
                const int t = paged + 16 * (w - (W - 4)) + k / LINES;
                if (t < s.len) {
                    const int64_t at = ring_at(c, s.slot, h, t) + k % LINES * 64;
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(c.kt + at));
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(c.vt + at));
                }
            }
        }

        // this warp's pieces of full pages: page and scales of 32 pieces at a time (a lane a piece), two sets
        const int p_first = 4 * t_first + w;
        const int p_stop = min(min(4 * t_end, paged >> 4), (lim_max + 15) >> 4);  // no row sees a later piece
        const int count = p_stop > p_first ? (p_stop - p_first + W - 1) / W : 0;
        int pid0 = 0, pid1 = 0;
        float ks0 = 0.0f, ks1 = 0.0f, vs0 = 0.0f, vs1 = 0.0f;
        auto fetch = [&](int set, int first) {
            const int i = first + lane;
            int p = 0;
            float ks = 0.0f, vs = 0.0f;
            if (i < count) {
                p = (int)load_page(c, b, (p_first + W * i) >> (a.log_page - 4));
                ks = vs = __int_as_float(0x7fc00000);
                if (p >= 0) {
                    ks = c.ks[(int64_t)p * c.Hk + h];
                    vs = c.vs[(int64_t)p * c.Hk + h];
                }
                p = max(p, 0);  // (not one of the cache's pages: the first one's codes, and NaN for what sees them)
            }
            if (set) {
                pid1 = p;
                ks1 = ks;
                vs1 = vs;
            } else {
                pid0 = p;
                ks0 = ks;
                vs0 = vs;
            }
        };
        auto copy = [&](int i, int stage) {
            if (i < count) {
                const int p = __shfl_sync(0xffffffffu, (i & 32) ? pid1 : pid0, i & 31);
                const int64_t at = page_at(c, p, h) + (uint32_t)((((p_first + W * i) << 4) & (c.P - 1)) * D + lane * 16);
                const uint32_t to = ring + stage * Cfg::stage;
                piece.template run<0>(to, c.kc + at);
                piece.template run<16 * D>(to, c.vc + at);
            }
            cp_async_commit();
        };
        if (count > 0) {
            fetch(0, 0);
#pragma unroll
            for (int i = 0; i < Cfg::stages - 1; ++i) copy(i, i);
            if (count > 32) fetch(1, 32);
        }

        // ---- q (while the first copies are under way)
        uint2 qb[Cfg::q_in_regs ? R8 : 1][KS];
        float qf[R8][2];   // of rows 2j, 2j + 1 of each column tile
        int lim[R8][2];    // the tokens that they see
        if (!Cfg::q_in_regs) __syncthreads();  // the last item's readers are done
#pragma unroll
        for (int n = 0; n < R8; ++n) {
            uint2 op[KS];
            if constexpr (!Cfg::q_in_regs) q_load(n, q_part[0]);
            const float f = q_part[Cfg::q_in_regs ? n : 0].operand(bf16, op) * a.scale2;
            if constexpr (Cfg::q_in_regs) {
#pragma unroll
                for (int st = 0; st < KS; ++st) qb[n][st] = op[st];
            } else {
#pragma unroll
                for (int st = 0; st < KS; ++st)
                    if (st % W == w) *reinterpret_cast<uint2 *>(q_smem + (n * KS + st) * 256 + lane * 8) = op[st];
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                qf[n][e] = __shfl_sync(0xffffffffu, f, 4 * (2 * j + e));
                const int rr = n * 8 + 2 * j + e;
                lim[n][e] = rr < rows ? old + (rb * R + rr) / c.G + 1 : INT32_MAX;
            }
        }
        if (!Cfg::q_in_regs) __syncthreads();

        float o[R8][MT][4];  // (d, row): d of rows g and g + 8 of row tile mt, rows 2j and 2j + 1 of the column tile
        float m[R8][2], l[R8][2];
#pragma unroll
        for (int n = 0; n < R8; ++n) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) o[n][mt][0] = o[n][mt][1] = o[n][mt][2] = o[n][mt][3] = 0.0f;
            m[n][0] = m[n][1] = kNoScore;
            l[n][0] = l[n][1] = 0.0f;
        }
        // the largest V scale so far, and its inverse: o is in units of v_ref / kWeightUnit
        float v_ref = 1e-30f, v_inv = kWeightUnit / 1e-30f;

        // S^T of one step (k = 16) of 16 keys: ka is the keys' operand
        auto scores = [&](float (&sc)[R8][4], const uint32_t (&ka)[4], int st) {
#pragma unroll
            for (int n = 0; n < R8; ++n) {
                if constexpr (Cfg::q_in_regs) {
                    mma16816(sc[n], ka, qb[n][st].x, qb[n][st].y);
                } else {
                    const uint2 q2 = *reinterpret_cast<const uint2 *>(q_smem + (n * KS + st) * 256 + lane * 8);
                    mma16816(sc[n], ka, q2.x, q2.y);
                }
            }
        };
        auto raise = [&](float v_top) {
            if (v_top > v_ref) {
                const float f = v_ref / v_top;
                v_ref = v_top;
                v_inv = kWeightUnit / v_top;
#pragma unroll
                for (int n = 0; n < R8; ++n)
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[n][mt][e] *= f;
            }
        };
        // Raw scores of keys t0 + g, t0 + g + 8 to the second product's operand: factors kf of the two
        // keys, vf of their V, v_inv of the rows (a function of n and e); updates m, l and o.
        auto weights = [&](float (&sc)[R8][4], float kf0, float kf1, float vf0, float vf1, auto inv_of, int t0, bool masked,
                           uint32_t (&pb)[R8][2]) {
            bool over = false;
#pragma unroll
            for (int n = 0; n < R8; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    sc[n][e] = __fmul_rn(sc[n][e], kf0 * qf[n][e]);  // (rounded, as the maximum is: see row_weights)
                    sc[n][2 + e] = __fmul_rn(sc[n][2 + e], kf1 * qf[n][e]);
                    if (masked) {
                        if (t0 + g >= lim[n][e]) sc[n][e] = -INFINITY;
                        if (t0 + g + 8 >= lim[n][e]) sc[n][2 + e] = -INFINITY;
                    }
                    over |= fmaxf(sc[n][e], sc[n][2 + e]) > m[n][e] + kLazy;
                }
            if (__any_sync(0xffffffffu, over)) {
#pragma unroll
                for (int n = 0; n < R8; ++n) {
                    float f[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float top = fmaxf(sc[n][e], sc[n][2 + e]);
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
                        top = fmaxf(top, m[n][e]);
                        f[e] = ex2(m[n][e] - top);
                        m[n][e] = top;
                        l[n][e] *= f[e];
                    }
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        o[n][mt][0] *= f[0];
                        o[n][mt][1] *= f[1];
                        o[n][mt][2] *= f[0];
                        o[n][mt][3] *= f[1];
                    }
                }
            }
#pragma unroll
            for (int n = 0; n < R8; ++n) {
                const float w[4] = {vf0 * inv_of(n, 0), vf0 * inv_of(n, 1), vf1 * inv_of(n, 0), vf1 * inv_of(n, 1)};
                float p[4], y[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    p[e] = ex2(sc[n][e] - m[n][e & 1]);
                    y[e] = p[e] * w[e];
                    // (a page without a scale makes NaN of what sees it, however small its weight, and of no other)
                    if (masked && t0 + g + 8 * (e >> 1) >= lim[n][e & 1]) y[e] = 0.0f;
                }
                l[n][0] += p[0] + p[2];
                l[n][1] += p[1] + p[3];
                pb[n][0] = transpose8x8(half2_bits(y[0], y[1]));
                pb[n][1] = transpose8x8(half2_bits(y[2], y[3]));
            }
        };

        // ---- full pages
        int stage = 0;
        for (int i = 0; i < count; ++i) {
            if ((i & 31) == 0 && i > 0 && i + 32 < count) fetch(((i >> 5) + 1) & 1, i + 32);
            copy(i + Cfg::stages - 1, stage == 0 ? Cfg::stages - 1 : stage - 1);
            cp_async_wait<Cfg::stages - 1>();
            __syncwarp();
            const float ks = __shfl_sync(0xffffffffu, (i & 32) ? ks1 : ks0, i & 31);
            const float vs = __shfl_sync(0xffffffffu, (i & 32) ? vs1 : vs0, i & 31);
            const int t0 = (p_first + W * i) << 4;
            const uint32_t kt = ring + stage * Cfg::stage;
            stage = stage + 1 == Cfg::stages ? 0 : stage + 1;
            float sc[R8][4];
#pragma unroll
            for (int n = 0; n < R8; ++n) sc[n][0] = sc[n][1] = sc[n][2] = sc[n][3] = 0.0f;
            auto chunk = [&](const uint4 &x, const uint4 &y, int q) {
                const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    uint32_t ka[4];
                    codes_to_half<CODE>(code_bias<CODE>(xs[e]), ka[0], ka[2]);
                    codes_to_half<CODE>(code_bias<CODE>(ys[e]), ka[1], ka[3]);
                    scores(sc, ka, 4 * q + e);
                }
            };
            chunk(keys.template load<0, 0>(kt), keys.template load<0, 1>(kt), 0);
            if constexpr (D > 64) chunk(keys.template load<1, 0>(kt), keys.template load<1, 1>(kt), 1);
            if constexpr (D > 128) {
                chunk(keys.template load<2, 0>(kt), keys.template load<2, 1>(kt), 2);
                chunk(keys.template load<3, 0>(kt), keys.template load<3, 1>(kt), 3);
            }
            uint32_t pb[R8][2];
            raise(vs);  // (rows that do not see the page see no later one of this warp's either)
            weights(sc, ks, ks, vs, vs, [&](int, int) { return v_inv; }, t0, t0 + 16 > lim_min, pb);
            // V^T: keys 2j, 2j+1 and 2j+8, 2j+9; rows g and g + 8 of a row tile are two of this lane's run of d's
            constexpr int HW = D == 64 ? 2 : 4;  // words of a lane's run of d's (8 or 16 of each 64 or 128)
            auto values = [&](const uint32_t (&x)[4][HW], int half) {
#pragma unroll
                for (int q = 0; q < HW; ++q) {  // d = 4 q + e of the run: row tile (4 q + e) / 2, its rows g or g + 8
                    uint32_t b0[4], b1[4];
                    codes_to_half<CODE>(__byte_perm(x[0][q], x[1][q], 0x5140), b0[0], b0[1]);
                    codes_to_half<CODE>(__byte_perm(x[0][q], x[1][q], 0x7362), b0[2], b0[3]);
                    codes_to_half<CODE>(__byte_perm(x[2][q], x[3][q], 0x5140), b1[0], b1[1]);
                    codes_to_half<CODE>(__byte_perm(x[2][q], x[3][q], 0x7362), b1[2], b1[3]);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t va[4] = {b0[2 * e], b0[2 * e + 1], b1[2 * e], b1[2 * e + 1]};
#pragma unroll
                        for (int n = 0; n < R8; ++n) mma16816(o[n][8 * half + 2 * q + e], va, pb[n][0], pb[n][1]);
                    }
                }
            };
            constexpr int VT = 16 * D;  // V's tile lies behind K's
            if constexpr (D == 64) {
                uint32_t x[4][HW];
                codes2<CODE>(lds64<VT>(kt + v_at0), x[0]);
                codes2<CODE>(lds64<VT>(kt + v_at1), x[1]);
                codes2<CODE>(lds64<VT + 8 * D>(kt + v_at0), x[2]);
                codes2<CODE>(lds64<VT + 8 * D>(kt + v_at1), x[3]);
                values(x, 0);
            } else {
                uint32_t x[4][HW];
                codes4<CODE>(lds128<VT>(kt + v_at0), x[0]);
                codes4<CODE>(lds128<VT>(kt + v_at1), x[1]);
                codes4<CODE>(lds128<VT + 8 * D>(kt + v_at0), x[2]);
                codes4<CODE>(lds128<VT + 8 * D>(kt + v_at1), x[3]);
                values(x, 0);
                if constexpr (D == 256) {
                    codes4<CODE>(lds128<VT + 128>(kt + v_at0), x[0]);
                    codes4<CODE>(lds128<VT + 128>(kt + v_at1), x[1]);
                    codes4<CODE>(lds128<VT + 8 * D + 128>(kt + v_at0), x[2]);
                    codes4<CODE>(lds128<VT + 8 * D + 128>(kt + v_at1), x[3]);
                    values(x, 1);
                }
            }
            __syncwarp();
        }
        cp_async_wait<0>();

        // ---- the unfinished page's rows, in 16 bits: 16 of them for each of the last four warps
        const int tail = s.len - paged, key0 = 16 * (w - (W - 4));
        if (t_end > paged_tiles && key0 >= 0 && paged + key0 < min(s.len, lim_max)) {
            constexpr bool AT_ONCE = D * R8 <= 64;   // K's and V's loads together, as far as the registers go
            constexpr int VW = D / 64;               // loads of 8 values of a V row that a lane makes (in halves of a 128)
            float sc[R8][4];
            float kf[2], vmul[4], vf[4];
            RowPart<D> k_part[2];
            uint4 v_part[4][VW];
            auto key_of = [&](int k) { return key0 + 2 * j + (k & 1) + 8 * (k >> 1); };
            auto v_row = [&](int k) {
                const int key = key_of(k);
                return c.vt + ring_at(c, s.slot >= 0 ? s.slot : 0, h, paged + (key < tail ? key : 0));
            };
            auto load_v = [&]() {
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int z = 0; z < VW; ++z) {
                        const int d = D == 64 ? g * 8 : 128 * (z >> 1) + g * 16 + 8 * (z & 1);
                        v_part[k][z] = key_of(k) < tail && s.slot >= 0 ? *reinterpret_cast<const uint4 *>(v_row(k) + d) : make_uint4(0, 0, 0, 0);
                    }
            };
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int key = key0 + 8 * e + g;
                const bool live = key < tail && s.slot >= 0;
                k_part[e].load(c.kt + ring_at(c, live ? s.slot : 0, h, paged + (live ? key : 0)), live, j);
            }
            if constexpr (AT_ONCE) load_v();
            {
                uint32_t ka[KS][4];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    uint2 op[KS];
                    kf[e] = k_part[e].operand(bf16, op);
                    if (s.slot < 0) kf[e] = __int_as_float(0x7fc00000);
#pragma unroll
                    for (int st = 0; st < KS; ++st) {
                        ka[st][e] = op[st].x;
                        ka[st][2 + e] = op[st].y;
                    }
                }
#pragma unroll
                for (int n = 0; n < R8; ++n) sc[n][0] = sc[n][1] = sc[n][2] = sc[n][3] = 0.0f;
#pragma unroll
                for (int st = 0; st < KS; ++st) scores(sc, ka[st], st);
            }
            if constexpr (!AT_ONCE) load_v();
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float amax = 0.0f;
#pragma unroll
                for (int z = 0; z < VW; ++z) amax = fmaxf(amax, amax8(v_part[k][z], bf16));
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 4));
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 8));
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 16));
                row_scale(amax, vmul[k], vf[k]);
                if (!(key_of(k) < tail && s.slot >= 0)) vf[k] = 0.0f, vmul[k] = 0.0f;
            }
            // those of this lane's scores' keys, g and g + 8, are with the lanes of j = g / 2
            float of[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) of[k] = __shfl_sync(0xffffffffu, vf[k], g >> 1);
#pragma unroll
            for (int n = 0; n < R8; ++n)  // rows that pad see no more than the tail's own tokens
#pragma unroll
                for (int e = 0; e < 2; ++e) lim[n][e] = min(lim[n][e], s.len);
            // The weights are relative to the largest V scale so far, or, where rows see different tokens, to the largest
            // that each row sees: a later token's, however large, takes no bits of them.  (Those of the rows lie in the
            // place of the maxima that the join is about to get: registers are short here.)
            const float vk[2] = {g & 1 ? of[1] : of[0], g & 1 ? of[3] : of[2]};
            auto top_of = [&](float x) {
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
            };
            const bool alike = lim_min >= s.len;
            if (alike) {
                raise(top_of(fmaxf(vk[0], vk[1])));  // (NaN leaves it)
            } else {
#pragma unroll
                for (int n = 0; n < R8; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float x = paged + key0 + g < lim[n][e] ? fmaxf(vk[0], 0.0f) : 0.0f;
                        const float vr = fmaxf(v_ref, top_of(paged + key0 + 8 + g < lim[n][e] ? fmaxf(vk[1], x) : x));
                        const float f = v_ref / vr;
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt) {
                            o[n][mt][e] *= f;
                            o[n][mt][2 + e] *= f;
                        }
                        if (g == 0) *reinterpret_cast<float2 *>(s_ml[w][n * 8 + 2 * j + e]) = make_float2(vr / kWeightUnit, kWeightUnit / vr);
                    }
                __syncwarp();
            }
            uint32_t pb[R8][2];
            weights(sc, kf[0], kf[1], vk[0], vk[1], [&](int n, int e) { return alike ? v_inv : s_ml[w][n * 8 + 2 * j + e][1]; },
                    paged + key0, true, pb);
#pragma unroll
            for (int z = 0; z < VW; ++z) {  // values d = 8 z .. of the lane's run: row tiles 4 z ..
                uint32_t x[4][4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    x[k][0] = scale2(v_part[k][z].x, vmul[k], bf16);
                    x[k][1] = scale2(v_part[k][z].y, vmul[k], bf16);
                    x[k][2] = scale2(v_part[k][z].z, vmul[k], bf16);
                    x[k][3] = scale2(v_part[k][z].w, vmul[k], bf16);
                }
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint32_t va[4] = {__byte_perm(x[0][q], x[1][q], 0x5410), __byte_perm(x[0][q], x[1][q], 0x7632),
                                            __byte_perm(x[2][q], x[3][q], 0x5410), __byte_perm(x[2][q], x[3][q], 0x7632)};
#pragma unroll
                    for (int n = 0; n < R8; ++n) mma16816(o[n][4 * z + q], va, pb[n][0], pb[n][1]);
                }
            }
            if (!alike) {  // these tokens are the warp's last: its sums go on in their own units
#pragma unroll
                for (int n = 0; n < R8; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float f = s_ml[w][n * 8 + 2 * j + e][0];
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt) {
                            o[n][mt][e] *= f;
                            o[n][mt][2 + e] *= f;
                        }
                    }
                v_ref = kWeightUnit;
                __syncwarp();
            }
        }

        // ---- join the warps: into shared memory, each in units of the common maximum
#pragma unroll
        for (int n = 0; n < R8; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float sum = l[n][e];
                sum += __shfl_xor_sync(0xffffffffu, sum, 4);
                sum += __shfl_xor_sync(0xffffffffu, sum, 8);
                sum += __shfl_xor_sync(0xffffffffu, sum, 16);
                if (g == 0) *reinterpret_cast<float2 *>(s_ml[w][n * 8 + 2 * j + e]) = make_float2(m[n][e], sum);
            }
        __syncthreads();  // every warp's ring is idle, and the maxima are there
        float *merge = reinterpret_cast<float *>(smem);
#pragma unroll
        for (int n = 0; n < R8; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = n * 8 + 2 * j + e;
                float top = s_ml[0][r][0];
#pragma unroll
                for (int k = 1; k < W; ++k) top = fmaxf(top, s_ml[k][r][0]);
                const float f = ex2(m[n][e] - top) * (v_ref / kWeightUnit);
                float *to = merge + (w * R + r) * D;
                constexpr int run = D == 64 ? 8 : 16;  // a lane's d's: g * run + 2 mt (row g), + 1 (row g + 8)
                if (r < rows) {
#pragma unroll
                    for (int mt = 0; mt < MT; mt += 2)
                        *reinterpret_cast<float4 *>(to + (mt / 8) * 128 + g * run + 2 * (mt % 8)) =
                            make_float4(o[n][mt][e] * f, o[n][mt][2 + e] * f, o[n][mt + 1][e] * f, o[n][mt + 1][2 + e] * f);
                }
            }
        if (tid < R) {
            float top = s_ml[0][tid][0], sum = 0.0f;
            for (int k = 1; k < W; ++k) top = fmaxf(top, s_ml[k][tid][0]);
            for (int k = 0; k < W; ++k) sum += s_ml[k][tid][1] * ex2(s_ml[k][tid][0] - top);
            s_part[tid][0] = top;
            s_part[tid][1] = sum;
        }
        __syncthreads();
        auto merged = [&](int r, int d) {
            float4 x = *reinterpret_cast<const float4 *>(merge + r * D + d);
#pragma unroll
            for (int k = 1; k < W; ++k) {
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
            const float inv = sum == 0.0f ? no_weight(old + rr / c.G) : 1.0f / sum;
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
            for (int k = tid; k < rows * (D / 4); k += THREADS) {
                const int r = k / (D / 4), d = k % (D / 4) * 4;
                store(r, d, merged(r, d), s_part[r][1]);
            }
            if (tid < rows) store_lse(tid, s_part[tid][0], s_part[tid][1]);
            __syncthreads();
        } else {
            // The CTAs that share the item: those of its first and of its last unit.  Each leaves its part in
            // the scratch and counts itself; the last of a group joins the group's parts (in the place of the
            // group's first), the last group's the groups'.
            const long long N = share.ctas, total = share.total;
            const int c0 = part_with(seg.unit0, total, N), c1 = part_with(seg.unit1, total, N);
            const int nc = c1 - c0 + 1, me = (int)blockIdx.x - c0;
            const int64_t pf = partial_floats(R, D);
            auto slot_of = [&](int k) { return a.partial + (2 * (int64_t)(c0 + k) + (k == 0 ? 1 : 0)) * pf; };
            float *slot = slot_of(me);
            for (int k = tid; k < rows * (D / 4); k += THREADS) {
                const int r = k / (D / 4), d = k % (D / 4) * 4;
                __stcg(reinterpret_cast<float4 *>(slot + r * D + d), merged(r, d));
            }
            if (tid < rows) __stcg(reinterpret_cast<float2 *>(slot + R * D + 2 * tid), make_float2(s_part[tid][0], s_part[tid][1]));
            const bool two = nc > 2 * kJoinGroup;
            // `n` parts from part `first`, `step` apart, joined: onto part `first`, or into the result
            auto join = [&](int first, int n, int step, bool last) {
                float2 *ml = reinterpret_cast<float2 *>(smem);  // [n][rows] maximum, sum
                auto at_of = [&](int k) { return k / (D / 4) * D + k % (D / 4) * 4; };
                // the sums of this thread's first place, eight parts: on their way beside the maxima
                float4 v[8];
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    v[q] = q < n && tid < rows * (D / 4)
                               ? __ldcg(reinterpret_cast<const float4 *>(slot_of(first + q * step) + at_of(tid))) : make_float4(0, 0, 0, 0);
                for (int k = tid; k < n * rows; k += THREADS)
                    ml[k] = __ldcg(reinterpret_cast<const float2 *>(slot_of(first + k / rows * step) + R * D) + k % rows);
                __syncthreads();
                auto top_of = [&](int r) {
                    float top = kNoScore;
#pragma unroll 8
                    for (int q = 0; q < n; ++q) top = fmaxf(top, ml[q * rows + r].x);
                    return top;
                };
                for (int k = tid; k < rows * (D / 4); k += THREADS) {
                    const int r = k / (D / 4), d = k % (D / 4) * 4;
                    // (every thread forms its row's maximum and sum itself: no barrier, nothing in turn)
                    const float top = top_of(r);
                    float sum = 0.0f;
                    float4 x = make_float4(0, 0, 0, 0);
                    auto add = [&](const float4 &v, int q) {
                        const float f = ex2(ml[q * rows + r].x - top);
                        sum = fmaf(ml[q * rows + r].y, f, sum);
                        x.x = fmaf(v.x, f, x.x);
                        x.y = fmaf(v.y, f, x.y);
                        x.z = fmaf(v.z, f, x.z);
                        x.w = fmaf(v.w, f, x.w);
                    };
                    int q0 = 0;
                    if (k == tid) {
#pragma unroll
                        for (int q = 0; q < 8; ++q)
                            if (q < n) add(v[q], q);
                        q0 = 8;
                    }
#pragma unroll 8
                    for (int q = q0; q < n; ++q) add(__ldcg(reinterpret_cast<const float4 *>(slot_of(first + q * step) + at_of(k))), q);
                    if (last)
                        store(r, d, x, sum);
                    else
                        __stcg(reinterpret_cast<float4 *>(slot_of(first) + at_of(k)), x);
                    if (d == 0) {
                        if (last)
                            store_lse(r, top, sum);
                        else
                            __stcg(reinterpret_cast<float2 *>(slot_of(first) + R * D) + r, make_float2(top, sum));
                    }
                }
            };
            auto arrive = [&](int32_t *counter, int n) {  // whether this CTA is the last of n
                __syncthreads();
                if (tid == 0) {
                    __threadfence();  // (the CTA's writes, which the barrier has put before)
                    const int k = atomicAdd(counter, 1);
                    s_last = k == n - 1;
                    __threadfence();
                    if (k == n - 1) *counter = 0;  // (its next use is another call's)
                }
                __syncthreads();
                return s_last != 0;
            };
            if (!two) {
                if (arrive(a.counters + c0, nc)) join(0, nc, 1, true);
            } else {
                const int first = me / kJoinGroup * kJoinGroup, n = min(kJoinGroup, nc - first);
                if (arrive(a.counters + kMaxDecodeCtas + 2 * (c0 + first) + (first == 0), n)) {
                    join(first, n, 1, false);
                    const int parts = (nc + kJoinGroup - 1) / kJoinGroup;
                    if (arrive(a.counters + c0, parts)) join(0, parts, kJoinGroup, true);
                }
            }
            __syncthreads();
        }
    }
}

template <int CODE, int D, int R8>
cudaError_t decode_launch(const Plan &p, const DecodeArgs &a, cudaStream_t s) {
    using Cfg = DecodeCfg<D, R8>;
    const cudaError_t e = allow_smem<k_kv_decode<CODE, D, R8>>(Cfg::smem);
    if (e != cudaSuccess) return e;
    return launch(k_kv_decode<CODE, D, R8>, dim3(p.sm_count * Cfg::ctas), Cfg::warps * 32, Cfg::smem, s, a);
}

}  // namespace kv
}  // namespace si
