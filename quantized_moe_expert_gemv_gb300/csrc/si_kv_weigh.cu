// si_kv_weigh.cu -- the attention weights of each cached token, added to its
// running sum:
//   acc_out_t = decay acc_in_t + sum over the rows r that see t of 2^(f S_tr - lse_r log2 e).
// A token's sum is taken by one thread (or four neighbours) in the rows' order:
// no atomics, the same bits for the same inputs.
//
// Few rows (k_kv_weigh_few): bound by HBM, D bytes of K codes a token.  The
// warp-level product has the keys as its 16 rows and q's rows as its 8 columns,
// so that a step of 8 query heads wastes none of it; units of 64 tokens are
// dealt out evenly over the GPU as in the few-row attention, and nothing has to
// be joined.  Measured: a row for each of 32 sequences of 500 to 9000 tokens, 32/8
// heads, 39 us, 64 % of the copy rate (a unit is two chains long and short of loads).
// A window of rows (k_kv_weigh_window, 65 to 512, head_dim 64 and 128): bound by
// the exponential (32 a cycle and SM) and the products.  S^T = K Q^T on the tcgen05
// tensor cores, 128 tokens by 128 rows; all of q's rows stay in shared memory while
// the CTA's share of a kv head's tokens goes by, and a thread holds one token's sum
// and walks every other block's columns in tensor memory.  Measured: 512 rows a kv
// head over 4 sequences of 9000 to 16000 tokens, 4 kv heads of 128, 39 us, where the
// products alone need 14: q's rows into shared memory 4 us a segment (two a CTA), a
// tile 2500 cycles of exponentials and sums (five a score and scheduler) of 3900.
// Many rows (k_kv_weigh_many): one CTA for 128 tokens, whose K tile stays while
// q's tiles of 128 rows follow each other through two stages; for 512 rows it
// takes 112 us where the window kernel takes 39 (most of it in a CTA's start).
#include "si_kv_decode.cuh"
#include "si_kv_tc.cuh"

namespace si {
namespace kv {

struct WeighArgs {
    Ctx c;
    Rows q;
    const float *lse, *acc_in;
    float *acc_out;
    int64_t acc_stride;
    float decay, scale2;
    int bf16, log_page, fault;
    long long budget;
};

// The barrier of the window kernel's softmax warps.
__device__ __forceinline__ void softmax_sync() { asm volatile("bar.sync 2, 256;" ::: "memory"); }
// Tiles that a segment's start counts as in the window kernel's even split.  (512 rows a kv head over four sequences of
// 12500 tokens, 4 kv heads: 43.1 us with 1, 38.7 with 3, 39.4 with 6.)
constexpr int kWindowOver = 3;
constexpr int kWeighRows = 64;  // rows whose operand lies in shared memory at a time

template <int D>
struct WeighCfg {
    static constexpr int ctas = 2;  // a SM
    static constexpr int warps = D == 256 ? 4 : 8;
    static constexpr int stage = 16 * D;  // a piece of 16 keys
    static constexpr int stages = 64 * 1024 / (warps * stage);
    static constexpr int ring = warps * stages * stage;
    static constexpr int q_bytes = kWeighRows / 8 * (D / 16) * 256;
    static constexpr int sums = warps * 32 * 16 * 4;  // the sums of a warp's last 32 pieces
    static constexpr int smem = ring + q_bytes + sums + kWeighRows * 8;
};

template <int CODE, int D>
__global__ void __launch_bounds__(WeighCfg<D>::warps * 32, WeighCfg<D>::ctas) k_kv_weigh_few(const WeighArgs a) {
    using Cfg = WeighCfg<D>;
    constexpr int W = Cfg::warps, KS = D / 16;
    extern __shared__ __align__(128) uint8_t smem[];
    const Ctx &c = a.c;
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, g = lane >> 2, j = lane & 3;
    const bool bf16 = a.bf16;

    start_after();
    const Share share = take_share<W>(c.B, [&](int b) -> long long {
        const int tiles = seq_tiles(c, load_seq(c, b).len);
        return tiles == 0 ? 0ll : (long long)(tiles + kWeighOver) * c.Hk;
    }, [&](int) { return c.Hk; }, 0);
    if (blockIdx.x >= share.ctas) return;
    int b = share.b;
    long long off = share.off, u = share.begin;
    const uint32_t ring = smem_addr(smem) + w * (Cfg::stages * Cfg::stage);
    uint8_t *q_smem = smem + Cfg::ring;
    float *sums = reinterpret_cast<float *>(smem + Cfg::ring + Cfg::q_bytes) + w * 512;
    float2 *rowf = reinterpret_cast<float2 *>(smem + Cfg::ring + Cfg::q_bytes + Cfg::sums);  // factor, lse log2 e
    PieceCopy<D> piece;
    piece.init(lane);
    KeyLoad<D> keys;
    keys.init(g, j);

    while (u < share.end) {
        const Seq s = load_seq(c, b);
        const int tiles = seq_tiles(c, s.len);
        const long long n_units = tiles == 0 ? 0ll : (long long)(tiles + kWeighOver) * c.Hk;
        if (off >= n_units) {
            off -= n_units;
            ++b;
            continue;
        }
        const Segment seg = take_segment(tiles, kWeighOver, off, u, share.end);
        u += seg.step;
        off += seg.step;
        const int h = seg.item, t_first = seg.first, t_end = seg.end;
        if (t_first == t_end) continue;
        const int paged = s.len & ~(c.P - 1), old = s.len - s.n, paged_tiles = (paged + 63) / 64;
        const int all_rows = s.n * c.G;
        const int64_t acc_at = ((int64_t)b * c.Hk + h) * a.acc_stride;
        // this warp's pieces: every W-th of those of the units' full pages
        const int p_first = 4 * t_first + w, p_stop = min(4 * t_end, paged >> 4);
        const int count = p_stop > p_first ? (p_stop - p_first + W - 1) / W : 0;

        // rows in blocks of 64 (one block, but for many rows of 256 values): the first takes up the earlier sums
        for (int rb = 0; rb == 0 || rb * kWeighRows < all_rows; ++rb) {
            const int rows = min(kWeighRows, all_rows - rb * kWeighRows), nts = (rows + 7) / 8;
            const int lim_min = old + rb * kWeighRows / c.G + 1;
            int pid0 = 0, pid1 = 0;
            float ks0 = 0.0f, ks1 = 0.0f;
            auto fetch = [&](int set, int first) {
                const int i = first + lane;
                int p = 0;
                float f = 0.0f;
                if (i < count) {
                    p = (int)load_page(c, b, (p_first + W * i) >> (a.log_page - 4));
                    f = p >= 0 ? c.ks[(int64_t)p * c.Hk + h] : __int_as_float(0x7fc00000);
                    p = max(p, 0);  // (not one of the cache's pages: the first one's codes, and NaN for their weights)
                }
                if (set) {
                    pid1 = p;
                    ks1 = f;
                } else {
                    pid0 = p;
                    ks0 = f;
                }
            };
            auto copy = [&](int i, int stage) {
                if (i < count) {
                    const int p = __shfl_sync(0xffffffffu, (i & 32) ? pid1 : pid0, i & 31);
                    const uint8_t *kc = c.kc + page_at(c, p, h) + (uint32_t)((((p_first + W * i) << 4) & (c.P - 1)) * D + lane * 16);
                    piece.template run<0>(ring + stage * Cfg::stage, kc);
                }
                cp_async_commit();
            };
            if (count > 0) {
                fetch(0, 0);
#pragma unroll
                for (int i = 0; i < Cfg::stages - 1; ++i) copy(i, i);
                if (count > 32) fetch(1, 32);
            }
            __syncthreads();  // the last block's readers of q are done
            for (int nt = w; nt < nts; nt += W) {
                const int r = nt * 8 + g, rr = rb * kWeighRows + r;
                const bool live = r < rows;
                const int i = live ? rr / c.G : 0, head = h * c.G + (live ? rr % c.G : 0);
                uint2 op[KS];
                RowPart<D> part;
                part.load(a.q.p + (s.row0 + i) * a.q.row + head * a.q.head, live, j);
                const float f = part.operand(bf16, op);
                if (j == 0)  // (a row that pads weighs nothing)
                    rowf[r] = live ? make_float2(f * a.scale2, a.lse[(int64_t)(s.row0 + i) * c.H + head] * kLog2e)
                                   : make_float2(0.0f, INFINITY);
#pragma unroll
                for (int st = 0; st < KS; ++st) *reinterpret_cast<uint2 *>(q_smem + (nt * KS + st) * 256 + lane * 8) = op[st];
            }
            __syncthreads();

            // the rows' weights of 16 keys from t0 on, into 16 places of `to`
            auto weigh = [&](const uint32_t (&ka)[KS][4], float kf0, float kf1, int t0, bool masked, float *to) {
                float sum[2] = {0.0f, 0.0f};
                for (int nt = 0; nt < nts; ++nt) {
                    float sc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int st = 0; st < KS; ++st) {
                        const uint2 q2 = *reinterpret_cast<const uint2 *>(q_smem + (nt * KS + st) * 256 + lane * 8);
                        mma16816(sc, ka[st], q2.x, q2.y);
                    }
                    const float4 rf = *reinterpret_cast<const float4 *>(rowf + nt * 8 + 2 * j);
                    float p[4] = {ex2(fmaf(sc[0], kf0 * rf.x, -rf.y)), ex2(fmaf(sc[1], kf0 * rf.z, -rf.w)),
                                  ex2(fmaf(sc[2], kf1 * rf.x, -rf.y)), ex2(fmaf(sc[3], kf1 * rf.z, -rf.w))};
                    if (masked) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int r = rb * kWeighRows + nt * 8 + 2 * j + (e & 1);
                            if (t0 + g + 8 * (e >> 1) > old + r / c.G || r >= all_rows) p[e] = 0.0f;
                        }
                    }
                    sum[0] += p[0] + p[1];
                    sum[1] += p[2] + p[3];
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], 1);
                    sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], 2);
                }
                if (j < 2) to[g + 8 * j] = j ? sum[1] : sum[0];
            };
            // n sums (of pieces p_first + W i from i = first on, or of the tokens from t0 on) onto the earlier ones
            auto flush = [&](int n, int first, int t0) {
                __syncwarp();
                float was[16];  // (all of the earlier sums' loads at once)
                const float *from = rb > 0 ? a.acc_out : a.acc_in;
                const int stop = rb > 0 ? s.len : a.acc_in ? old : 0;
                auto token = [&](int k) { return t0 >= 0 ? t0 + k : ((p_first + W * (first + k / 16)) << 4) + k % 16; };
#pragma unroll
                for (int q = 0; q < 16; ++q) {
                    const int k = 32 * q + lane, t = token(k);
                    was[q] = k < n && t < stop ? from[acc_at + t] : 0.0f;
                }
                const float decay = rb > 0 ? 1.0f : a.decay;
#pragma unroll
                for (int q = 0; q < 16; ++q) {
                    const int k = 32 * q + lane, t = token(k);
                    if (k < n && t < s.len) a.acc_out[acc_at + t] = decay * was[q] + sums[k];
                }
                __syncwarp();
            };

            int stage = 0;
            for (int i = 0; i < count; ++i) {
                if ((i & 31) == 0 && i > 0) {
                    flush(512, i - 32, -1);
                    if (i + 32 < count) fetch(((i >> 5) + 1) & 1, i + 32);
                }
                copy(i + Cfg::stages - 1, stage == 0 ? Cfg::stages - 1 : stage - 1);
                cp_async_wait<Cfg::stages - 1>();
                __syncwarp();
                const float ks = __shfl_sync(0xffffffffu, (i & 32) ? ks1 : ks0, i & 31);
                const int t0 = (p_first + W * i) << 4;
                const uint32_t kt = ring + stage * Cfg::stage;
                stage = stage + 1 == Cfg::stages ? 0 : stage + 1;
                uint32_t ka[KS][4];
                auto chunk = [&](const uint4 &x, int q, int n) {
                    codes_to_half<CODE>(code_bias<CODE>(x.x), ka[4 * q][n], ka[4 * q][2 + n]);
                    codes_to_half<CODE>(code_bias<CODE>(x.y), ka[4 * q + 1][n], ka[4 * q + 1][2 + n]);
                    codes_to_half<CODE>(code_bias<CODE>(x.z), ka[4 * q + 2][n], ka[4 * q + 2][2 + n]);
                    codes_to_half<CODE>(code_bias<CODE>(x.w), ka[4 * q + 3][n], ka[4 * q + 3][2 + n]);
                };
                chunk(keys.template load<0, 0>(kt), 0, 0);
                chunk(keys.template load<0, 1>(kt), 0, 1);
                if constexpr (D > 64) {
                    chunk(keys.template load<1, 0>(kt), 1, 0);
                    chunk(keys.template load<1, 1>(kt), 1, 1);
                }
                if constexpr (D > 128) {
                    chunk(keys.template load<2, 0>(kt), 2, 0);
                    chunk(keys.template load<2, 1>(kt), 2, 1);
                    chunk(keys.template load<3, 0>(kt), 3, 0);
                    chunk(keys.template load<3, 1>(kt), 3, 1);
                }
                if (t0 + 16 <= lim_min)
                    weigh(ka, ks, ks, t0, false, sums + (i & 31) * 16);
                else
                    weigh(ka, ks, ks, t0, true, sums + (i & 31) * 16);
                __syncwarp();
            }
            cp_async_wait<0>();
            if (count > 0) flush(((count - 1) % 32 + 1) * 16, (count - 1) & ~31, -1);

            // ---- the unfinished page's rows, 16 for each of the last four warps
            const int tail = s.len - paged, key0 = 16 * (w - (W - 4));
            if (t_end > paged_tiles && key0 >= 0 && key0 < tail) {
                uint32_t ka[KS][4];
                float kf[2];
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const int key = key0 + 8 * n + g;
                    const bool live = key < tail && s.slot >= 0;
                    uint2 op[KS];
                    RowPart<D> part;
                    part.load(c.kt + ring_at(c, live ? s.slot : 0, h, paged + (live ? key : 0)), live, j);
                    kf[n] = part.operand(bf16, op);
                    if (s.slot < 0) kf[n] = __int_as_float(0x7fc00000);
#pragma unroll
                    for (int st = 0; st < KS; ++st) {
                        ka[st][n] = op[st].x;
                        ka[st][2 + n] = op[st].y;
                    }
                }
                weigh(ka, kf[0], kf[1], paged + key0, true, sums);
                flush(16, 0, paged + key0);
            }
        }
    }
}

// ------------------------------------------------------------------ a window of rows
constexpr int kWwRows = 512, kWwThreads = 13 * 32;
template <int D>
struct WeighWindowCfg {
    static constexpr int block = 256 * D * 2;                  // 256 rows of q: [D / 64][256 rows][128 bytes]
    static constexpr int tile = kTileRows * D * 2;
    static constexpr int k = 2 * block;
    static constexpr int lse = k + 2 * tile;                   // [512] -lse log2 e, then [512] each row's factor
    static constexpr int keyf = lse + 2 * kWwRows * 4;         // [4][128]
    static constexpr int part = keyf + 4 * 128 * 4;            // [2][128]
    static constexpr int bars = part + 2 * 128 * 4;
    static constexpr int smem = bars + 16 * 8 + 1024;
};
enum WindowBar { kXbQ = 0, kXbKFull = 1, kXbKEmpty = 3, kXbSFull = 5, kXbSEmpty = 9, kXbNever = 13 };

// The rows of a segment have one power of two where their largest values lie within 2^8 of one another (a score is then off
// by less than 2^-23 of what the row's largest value makes of it, as much as its sum in 32 bits); else each its own, and a
// factor for each column.
constexpr float kWindowApart = 256.0f;
// 128 columns of a lane's token: 2^(kf S - lse), added up.  MASK: columns below r_min see nothing of it; APART: columns
// have factors, behind the 512 lse.
template <bool MASK, bool APART>
__device__ __forceinline__ void window_sums(uint32_t ts, const float4 *rl, f32x2 kf2, int r_min, f32x2 &sum, f32x2 &sum1) {
    uint32_t z[2][32];
    tc::tmem_ld32(ts, z[0]);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        tc::tmem_wait_ld();
        if (e < 3) tc::tmem_ld32(ts + 32 * e + 32, z[(e + 1) & 1]);
        const uint32_t(&y)[32] = z[e & 1];
#pragma unroll
        for (int k = 0; k < 32; k += 4) {
            const float4 l = rl[8 * e + k / 4];
            f32x2 f0 = kf2, f1 = kf2;
            if constexpr (APART) {
                const float4 f = rl[kWwRows / 4 + 8 * e + k / 4];
                f0 = mul2(kf2, pk2(f.x, f.y));
                f1 = mul2(kf2, pk2(f.z, f.w));
            }
            float w[4];
            up2(fma2(pk2(__uint_as_float(y[k]), __uint_as_float(y[k + 1])), f0, pk2(l.x, l.y)), w[0], w[1]);
            up2(fma2(pk2(__uint_as_float(y[k + 2]), __uint_as_float(y[k + 3])), f1, pk2(l.z, l.w)), w[2], w[3]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                w[i] = ex2(w[i]);
                if (MASK && 32 * e + k + i < r_min) w[i] = 0.0f;
            }
            sum = add2(sum, pk2(w[0], w[1]));
            sum1 = add2(sum1, pk2(w[2], w[3]));
        }
    }
}

// Tiles of 128 tokens of a sequence (the unfinished page is in the last).
__device__ __forceinline__ int window_tiles(int len) { return (len + kTileRows - 1) / kTileRows; }

template <int CODE, int D>
__global__ void __launch_bounds__(kWwThreads, 1) k_kv_weigh_window(const WeighArgs a) {
    using Cfg = WeighWindowCfg<D>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint32_t s_tmem;
    __shared__ uint32_t s_top, s_low;  // the largest and the smallest of the rows' largest magnitudes (bits; without zeros)
    const Ctx &c = a.c;
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // (uniform)
    const bool bf16 = a.bf16;
    const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
    uint8_t *at = smem_raw + (base - smem_addr(smem_raw));
    float *lse_s = reinterpret_cast<float *>(at + Cfg::lse), *keyf = reinterpret_cast<float *>(at + Cfg::keyf);
    float *part = reinterpret_cast<float *>(at + Cfg::part);
    auto bar = [&](int i) { return base + Cfg::bars + 8 * i; };

    start_after();
    const Share share = take_share<kWwThreads / 32>(c.B, [&](int b) -> long long {
        const int tiles = window_tiles(load_seq(c, b).len);
        return tiles == 0 ? 0ll : (long long)(tiles + kWindowOver) * c.Hk;
    }, [&](int) { return c.Hk; }, 0);
    if (blockIdx.x >= share.ctas) return;
    if (tid == 0) {
        mbar_init(bar(kXbQ), 256);
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(kXbKFull + i), 128);
            mbar_init(bar(kXbKEmpty + i), 1);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(bar(kXbSFull + i), 1);
            mbar_init(bar(kXbSEmpty + i), 128);
        }
        mbar_init(bar(kXbNever), 1);
        fence_mbar_init();
        s_top = 0;
        s_low = 0x7f800000;
    }
    if (warp == 12) {
        tc::tmem_alloc(smem_addr(&s_tmem), 512);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = s_tmem;
    bool ok = true;
    auto wait = [&](int i, int parity) {
        if (ok && !mbar_wait_warp(bar(i), (uint32_t)parity, a.budget)) {
            ok = false;
            if (lane == 0) set_status(c.status, SI_ERR_TIMEOUT);
        }
        return ok;
    };

    // Every role walks the same segments (a run of one kv head's tiles), tiles (numbered over all of them) and
    // blocks of 128 rows, each with a quarter of the tensor memory; a tile's blocks are those with a row that sees
    // its first key.  Warps 0-3 take the even blocks, warps 4-7 the odd ones.  A segment without rows is the softmax
    // warps' alone and is in no one's count of tiles or segments: its tiles have no block whose barrier would hold them
    // until the product warp has seen q's (two such segments in a row could pass that warp by a phase).  With rows,
    // every tile has a block.
    int seq = share.b;
    long long off = share.off, u = share.begin;
    int tile_no = 0, seg_no = 0;
    struct Place {
        Seq s;
        int b, h, first, end, rows, old;
    };
    auto next = [&](Place &p) {  // the next segment; false at the end
        while (u < share.end) {
            p.s = load_seq(c, seq);
            const int tiles = window_tiles(p.s.len);
            const long long n = tiles == 0 ? 0ll : (long long)(tiles + kWindowOver) * c.Hk;
            if (off >= n) {
                off -= n;
                ++seq;
                continue;
            }
            const Segment seg = take_segment(tiles, kWindowOver, off, u, share.end);
            u += seg.step;
            off += seg.step;
            if (seg.first == seg.end) continue;
            p.b = seq;
            p.h = seg.item;
            p.first = seg.first;
            p.end = seg.end;
            p.rows = p.s.n * c.G;
            p.old = p.s.len - p.s.n;
            return true;
        }
        return false;
    };
    auto first_block = [&](const Place &p, int t) { return max(0, t * kTileRows - p.old) * c.G / 128; };
    auto blocks_of = [&](const Place &p) { return (p.rows + 127) / 128; };
    uint32_t s_use = 0;  // a bit a quarter: its uses so far are odd
    Place p;

    if (warp < 8) {
        // ================================================= q, then a thread a key and half of the blocks
        const int x = warp >> 2, ch = tid & 3;
        const uint32_t ts = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        while (next(p)) {
            if (p.rows == 0) {  // the earlier sums' decay is all: half of the tiles for each half of the warps
                for (int t = p.first + x; t < p.end; t += 2) {
                    const int token = t * kTileRows + (tid & 127);
                    const int64_t acc_at = ((int64_t)p.b * c.Hk + p.h) * a.acc_stride + token;
                    if (token < p.s.len) a.acc_out[acc_at] = a.acc_in ? a.decay * a.acc_in[acc_at] : 0.0f;
                }
                continue;
            }
            // the rows' values times a power of two (one for all, if they are of a size), a row that is not finite as
            // zeros with the lse NaN
            const int passes = (p.rows + 255) / 256 * 4;  // of 64 rows, to the end of the last block
            auto row_ptr = [&](int r) -> const uint16_t * {
                return a.q.p + (p.s.row0 + r / c.G) * a.q.row + (p.h * c.G + r % c.G) * a.q.head;
            };
            uint32_t top = 0, low = 0x7f800000, fine = 0;  // a bit a pass
            float *rowf = lse_s + kWwRows;  // first each row's largest, then its factor
            auto place = [&](int r, int q, int e) {
                const int unit = 2 * (ch + 4 * q) + e;
                return base + (r >> 8) * Cfg::block + (unit >> 3) * 32768 + (r & 255) * 128 + (((unit ^ r) & 7) << 4);
            };
            // the values as they are into their places, four passes' loads under way, and the largest ...
            for (int k0 = 0; k0 < passes; k0 += 4) {
                RowLoad<D> v[4];
                float l[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int r = 64 * (k0 + k) + (tid >> 2);
                    v[k].load(r < p.rows ? row_ptr(r) : a.q.p, r < p.rows, ch);
                    l[k] = ch == 0 && r < p.rows
                               ? a.lse[(int64_t)(p.s.row0 + r / c.G) * c.H + p.h * c.G + r % c.G] : INFINITY;
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int r = 64 * (k0 + k) + (tid >> 2);
                    float m = 0.0f;
#pragma unroll
                    for (int q = 0; q < D / 64; ++q)
                        m = fmaxf(m, fmaxf(amax8(v[k].y[q][0], bf16), amax8(v[k].y[q][1], bf16)));
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
                    if (m <= 3.4e38f) {
                        top = max(top, __float_as_uint(m));
                        if (m > 0.0f) low = min(low, __float_as_uint(m));
                        fine |= 1u << (k0 + k);
                    }
#pragma unroll
                    for (int q = 0; q < D / 64; ++q)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            sts128(place(r, q, e), v[k].y[q][e].x, v[k].y[q][e].y, v[k].y[q][e].z, v[k].y[q][e].w);
                    if (ch == 0) {  // (a row that pads weighs nothing)
                        lse_s[r] = m <= 3.4e38f ? -l[k] * kLog2e : __int_as_float(0x7fc00000);
                        rowf[r] = m;
                    }
                }
            }
            top = __reduce_max_sync(0xffffffffu, top);
            low = __reduce_min_sync(0xffffffffu, low);
            if (lane == 0) {  // (extremes: the order does not matter)
                atomicMax(&s_top, top);
                atomicMin(&s_low, low);
            }
            softmax_sync();
            // ... then each thread's own places scaled
            float mul, f;
            row_scale(__uint_as_float(s_top), mul, f);
            const bool apart = __uint_as_float(s_top) * (1.0f / kWindowApart) > __uint_as_float(s_low);
            for (int k = 0; k < passes; ++k) {
                const int r = 64 * k + (tid >> 2);
                float by = fine >> k & 1 ? mul : 0.0f;
                if (apart) {
                    float own;
                    row_scale(rowf[r], by, own);
                    __syncwarp();
                    if (ch == 0) rowf[r] = own;
                }
#pragma unroll
                for (int q = 0; q < D / 64; ++q)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint4 y = *reinterpret_cast<const uint4 *>(at + (place(r, q, e) - base));
                        sts128(place(r, q, e), scale2(y.x, by, bf16), scale2(y.y, by, bf16), scale2(y.z, by, bf16),
                               scale2(y.w, by, bf16));
                    }
            }
            tc::fence_proxy_async_smem();
            softmax_sync();
            if (tid == 0) s_top = 0, s_low = 0x7f800000;  // (read by everyone; their next use is a barrier away)
            mbar_arrive(bar(kXbQ));
            const int blocks = blocks_of(p);
            const float scale = (apart ? 1.0f : f) * a.scale2;
            // (a warp whose wait ran out goes on through the tiles, without waits, for the barriers' sake)
            for (int t = p.first; t < p.end; ++t, ++tile_no) {
                const int token = t * kTileRows + (tid & 127), r_min = max(0, token - p.old) * c.G;
                const int64_t acc_at = ((int64_t)p.b * c.Hk + p.h) * a.acc_stride + token;
                const float was = x == 0 && a.acc_in && token < p.old ? a.decay * a.acc_in[acc_at] : 0.0f;
                f32x2 sum = pk2(0.0f, 0.0f), sum1 = sum;
                float kf = 0.0f;
                int q = first_block(p, t);
                for (q += (q ^ x) & 1; q < blocks; q += 2) {
                    const int quarter = q & 3;
                    if (!wait(kXbSFull + quarter, s_use >> quarter & 1)) break;
                    s_use ^= 1u << quarter;
                    tc::fence_after_sync();
                    kf = keyf[(tile_no & 3) * 128 + (tid & 127)] * scale;
                    const f32x2 kf2 = pk2(kf, kf);
                    const int r0 = q * 128;
                    const float4 *rl = reinterpret_cast<const float4 *>(lse_s + r0);
                    if (apart)
                        window_sums<true, true>(ts + quarter * 128, rl, kf2, r_min - r0, sum, sum1);
                    else if (__all_sync(0xffffffffu, r0 >= r_min))
                        window_sums<false, false>(ts + quarter * 128, rl, kf2, 0, sum, sum1);
                    else
                        window_sums<true, false>(ts + quarter * 128, rl, kf2, r_min - r0, sum, sum1);
                    tc::fence_before_sync();
                    mbar_arrive(bar(kXbSEmpty + quarter));
                }
                float s0, s1;
                up2(add2(sum, sum1), s0, s1);
                if (x) part[(tile_no & 1) * 128 + (tid & 127)] = s0 + s1;
                softmax_sync();
                if (x == 0 && ok && token < p.s.len) a.acc_out[acc_at] = was + ((s0 + s1) + part[(tile_no & 1) * 128 + tid]);
            }
        }
    } else if (warp < 12) {
        // ================================================= K's tiles
        const int pt = tid - 256, ch = pt & 3, r0 = pt >> 2;
        constexpr int CC = D / 64;
        const uint32_t a0 = f16_tile_at(r0, 2 * ch), a1 = f16_tile_at(r0, 2 * ch + 1);
        while (next(p)) {
            if (p.rows == 0) continue;
            const int paged = p.s.len & ~(c.P - 1);
            const int32_t *table = c.table + (int64_t)p.b * c.table_stride;
            int pg[5];
            uint4 kx[4 * CC];
            float kfx = 0.0f;
            auto whole = [&](int t) { return (t + 1) * kTileRows <= paged; };
            auto named = [&](int v) { return (uint32_t)v < (uint32_t)c.n_pages; };
            auto pages = [&](int t) {
                if (t >= p.end || !whole(t)) return;
#pragma unroll
                for (int k = 0; k < 5; ++k) pg[k] = table[(t * kTileRows + (k < 4 ? r0 + 32 * k : pt)) >> a.log_page];
            };
            auto load = [&](int t) {
                if (t >= p.end || !whole(t)) return;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint8_t *from = c.kc + page_at(c, named(pg[k]) ? pg[k] : 0, p.h) + ((r0 + 32 * k) & (c.P - 1)) * D + ch * 16;
#pragma unroll
                    for (int q = 0; q < CC; ++q) kx[k * CC + q] = *reinterpret_cast<const uint4 *>(from + 64 * q);
                }
                kfx = c.ks[(int64_t)(named(pg[4]) ? pg[4] : 0) * c.Hk + p.h];
                if (!named(pg[4])) {
                    set_status(c.status, SI_ERR_DEVICE);
                    kfx = __int_as_float(0x7fc00000);
                }
            };
            pages(p.first);
            load(p.first);
            pages(p.first + 1);
            for (int t = p.first; t < p.end; ++t, ++tile_no) {
                const int st = tile_no & 1;
                if (tile_no >= 2 && !wait(kXbKEmpty + st, ((tile_no >> 1) - 1) & 1)) break;
                const uint32_t tile = base + Cfg::k + st * Cfg::tile;
                float *kf = keyf + (tile_no & 3) * 128;
                if (whole(t)) {
                    codes_to_tile<CODE, 0>(kx[0], tile + a0, tile + a1);
                    codes_to_tile<CODE, 4096>(kx[CC], tile + a0, tile + a1);
                    codes_to_tile<CODE, 8192>(kx[2 * CC], tile + a0, tile + a1);
                    codes_to_tile<CODE, 12288>(kx[3 * CC], tile + a0, tile + a1);
                    if constexpr (CC == 2) {
                        codes_to_tile<CODE, 16384>(kx[1], tile + a0, tile + a1);
                        codes_to_tile<CODE, 16384 + 4096>(kx[3], tile + a0, tile + a1);
                        codes_to_tile<CODE, 16384 + 8192>(kx[5], tile + a0, tile + a1);
                        codes_to_tile<CODE, 16384 + 12288>(kx[7], tile + a0, tile + a1);
                    }
                    kf[pt] = kfx;
                } else {
                    key_rows<CODE, D>(c, p.s, p.b, p.h, false, t * kTileRows, a.log_page, bf16, tile, kf, pt);
                }
                tc::fence_proxy_async_smem();
                mbar_arrive(bar(kXbKFull + st));
                load(t + 1);
                pages(t + 2);
            }
            if (!ok) break;
        }
    } else {
        // ================================================= the products: 128 keys by 128 rows
        constexpr uint32_t id = tc::idesc_f16_f32(128, 128);
        const uint64_t k_desc = tc::sdesc_sw128(base + Cfg::k), q_desc = tc::sdesc_sw128(base);
        if (a.fault) wait(kXbNever, 0);
        while (ok && next(p)) {
            if (p.rows == 0) continue;
            if (!wait(kXbQ, seg_no & 1)) break;
            const int blocks = blocks_of(p);
            for (int t = p.first; t < p.end; ++t, ++tile_no) {
                const int st = tile_no & 1;
                if (!wait(kXbKFull + st, (tile_no >> 1) & 1)) break;
                tc::fence_after_sync();
                const uint64_t kd = k_desc + (st * Cfg::tile >> 4);
                for (int q = first_block(p, t); q < blocks; ++q) {
                    const int quarter = q & 3;
                    if (!wait(kXbSEmpty + quarter, ~s_use >> quarter & 1)) break;  // (the first use waits for nothing)
                    s_use ^= 1u << quarter;
                    tc::fence_after_sync();
                    const uint64_t qd = q_desc + ((q >> 1) * Cfg::block + (q & 1) * 128 * 128 >> 4);
#pragma unroll
                    for (int k = 0; k < D / 16; ++k)
                        mma_ss(tmem + quarter * 128, kd + ((k >> 2) * (16384 >> 4) + (k & 3) * 2),
                               qd + ((k >> 2) * (32768 >> 4) + (k & 3) * 2), id, k > 0);
                    mma_done(bar(kXbSFull + quarter));
                }
                if (!ok) break;
                mma_done(bar(kXbKEmpty + st));
            }
            ++seg_no;
        }
        // whatever was issued is over before the tensor memory goes back (and the last commits, which no one waits for)
        mma_done(bar(kXbNever));
        mbar_wait_bounded(bar(kXbNever), 0, 4000000000LL);
        tc::fence_before_sync();
    }
    __syncwarp();
    __syncthreads();
    if (warp == 12) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, 512);
    }
}

// ------------------------------------------------------------------ many rows
constexpr int kWmThreads = 9 * 32;
template <int D>
struct WeighManyCfg {
    static constexpr int tile = kTileRows * D * 2;
    static constexpr int q = tile;
    static constexpr int rows = q + 2 * tile;                 // [4][2][128] factor, -lse log2 e
    static constexpr int keyf = rows + 4 * 128 * 8;           // [128]
    static constexpr int bars = keyf + 128 * 4;
    static constexpr int smem = bars + 16 * 8 + 1024;
};
enum WeighBar { kWbK = 0, kWbQFull = 1, kWbQEmpty = 3, kWbSFull = 5, kWbSEmpty = 7, kWbNever = 9 };

template <int CODE, int D>
__global__ void __launch_bounds__(kWmThreads, 2) k_kv_weigh_many(const WeighArgs a) {
    using Cfg = WeighManyCfg<D>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint32_t s_tmem;
    const Ctx &c = a.c;
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // (uniform)
    start_after();
    const int b = blockIdx.z, h = blockIdx.y, key0 = blockIdx.x * kTileRows;
    const Seq s = load_seq(c, b);
    if (key0 >= s.len) return;
    const int old = s.len - s.n, all_rows = s.n * c.G;
    // the first row that sees the tile's first key, in tiles of 128 rows
    const int first = max(0, key0 - old) * c.G / kTileRows;
    const int nt = max(0, (all_rows + kTileRows - 1) / kTileRows - first);

    const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
    uint8_t *aligned = smem_raw + (base - smem_addr(smem_raw));
    float *rowf = reinterpret_cast<float *>(aligned + Cfg::rows);  // [4][2][128]: factor, -lse log2 e
    float *keyf = reinterpret_cast<float *>(aligned + Cfg::keyf);
    auto bar = [&](int i) { return base + Cfg::bars + 8 * i; };
    if (tid == 0) {
        mbar_init(bar(kWbK), 128);
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(kWbQFull + i), 128);
            mbar_init(bar(kWbQEmpty + i), 1);
            mbar_init(bar(kWbSFull + i), 1);
            mbar_init(bar(kWbSEmpty + i), 128);
        }
        mbar_init(bar(kWbNever), 1);
        fence_mbar_init();
    }
    if (warp == 8) {
        tc::tmem_alloc(smem_addr(&s_tmem), 256);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = s_tmem;
    bool ok = true;
    auto wait = [&](int i, int parity) {
        if (ok && !mbar_wait_warp(bar(i), (uint32_t)parity, a.budget)) {
            ok = false;
            if (lane == 0) set_status(c.status, SI_ERR_TIMEOUT);
        }
        return ok;
    };

    if (warp < 4) {
        // ================================================= a thread a key
        const int t = key0 + tid;
        const int64_t at = ((int64_t)b * c.Hk + h) * a.acc_stride + t;
        const float was = t < old && a.acc_in ? a.decay * a.acc_in[at] : 0.0f;
        const int r_min = max(0, t - old) * c.G;  // the first row that sees the key
        const uint32_t ts = tmem + ((uint32_t)(32 * warp) << 16);
        f32x2 sum = pk2(0.0f, 0.0f), sum1 = sum;
        float kf = 0.0f;
        if (wait(kWbK, 0)) kf = keyf[tid];
        const f32x2 kf2 = pk2(kf, kf);
        for (int i = 0; i < nt; ++i) {
            if (!wait(kWbSFull + (i & 1), (i >> 1) & 1)) break;
            tc::fence_after_sync();
            const int r0 = (first + i) * kTileRows;
            const float4 *rf = reinterpret_cast<const float4 *>(rowf + (i & 3) * 256), *rl = rf + 32;  // four rows each
            const bool all = __all_sync(0xffffffffu, r0 >= r_min);
            uint32_t z[2][32];
            tc::tmem_ld32(ts + (i & 1) * 128, z[0]);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                tc::tmem_wait_ld();
                if (q < 3) tc::tmem_ld32(ts + (i & 1) * 128 + 32 * q + 32, z[(q + 1) & 1]);
                const uint32_t(&y)[32] = z[q & 1];
#pragma unroll
                for (int k = 0; k < 32; k += 4) {
                    const float4 f = rf[8 * q + k / 4], l = rl[8 * q + k / 4];
                    const f32x2 e0 = fma2(pk2(__uint_as_float(y[k]), __uint_as_float(y[k + 1])), mul2(kf2, pk2(f.x, f.y)), pk2(l.x, l.y));
                    const f32x2 e1 = fma2(pk2(__uint_as_float(y[k + 2]), __uint_as_float(y[k + 3])), mul2(kf2, pk2(f.z, f.w)), pk2(l.z, l.w));
                    float p[4];
                    up2(e0, p[0], p[1]);
                    up2(e1, p[2], p[3]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        p[e] = ex2(p[e]);
                        if (!all && r0 + 32 * q + k + e < r_min) p[e] = 0.0f;
                    }
                    sum = add2(sum, pk2(p[0], p[1]));
                    sum1 = add2(sum1, pk2(p[2], p[3]));
                }
            }
            tc::fence_before_sync();
            mbar_arrive(bar(kWbSEmpty + (i & 1)));
        }
        float x, y;
        up2(add2(sum, sum1), x, y);
        if (ok && t < s.len) a.acc_out[at] = was + (x + y);
    } else if (warp < 8) {
        // ================================================= K's tile, then q's
        const int pt = tid - 128, ch = pt & 3;
        key_rows<CODE, D>(c, s, b, h, false, key0, a.log_page, a.bf16, base, keyf, pt);
        tc::fence_proxy_async_smem();
        mbar_arrive(bar(kWbK));
        RowLoad<D> x[4];
        float lse = 0.0f;  // of row pt of the tile
        auto load = [&](int i) {  // this thread's part of four rows of q tile i, and a row's lse
            if (i >= nt) return;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int rr = (first + i) * kTileRows + (pt >> 2) + 32 * k;
                const bool live = rr < all_rows;
                const int row = s.row0 + (live ? rr / c.G : 0), head = h * c.G + (live ? rr % c.G : 0);
                x[k].load(a.q.p + row * a.q.row + head * a.q.head, live, ch);
            }
            const int rr = (first + i) * kTileRows + pt;
            lse = rr < all_rows ? a.lse[(int64_t)(s.row0 + rr / c.G) * c.H + h * c.G + rr % c.G] : INFINITY;
        };
        load(0);
        for (int i = 0; i < nt; ++i) {
            if (i >= 2 && !wait(kWbQEmpty + (i & 1), ((i >> 1) - 1) & 1)) break;
            float *rf = rowf + (i & 3) * 256;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int r = (pt >> 2) + 32 * k;
                const float f = x[k].store(base + Cfg::q + (i & 1) * Cfg::tile, r, ch, a.bf16);
                if (ch == 0) rf[r] = f * a.scale2;
            }
            rf[128 + pt] = -lse * kLog2e;  // (a row that pads weighs nothing)
            tc::fence_proxy_async_smem();
            mbar_arrive(bar(kWbQFull + (i & 1)));
            load(i + 1);
        }
    } else {
        // ================================================= the products
        constexpr uint32_t id = tc::idesc_f16_f32(128, kTileRows);
        const uint64_t k_desc = tc::sdesc_sw128(base), q_desc = tc::sdesc_sw128(base + Cfg::q);
        if (a.fault) wait(kWbNever, 0);
        if (wait(kWbK, 0))
            for (int i = 0; i < nt; ++i) {
                const int st = i & 1;
                if (!wait(kWbQFull + st, (i >> 1) & 1)) break;
                if (i >= 2 && !wait(kWbSEmpty + st, ((i >> 1) - 1) & 1)) break;
                tc::fence_after_sync();
                const uint64_t qd = q_desc + (st * Cfg::tile >> 4);
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    constexpr int half = 16384 >> 4;
                    mma_ss(tmem + st * 128, k_desc + ((k >> 2) * half + (k & 3) * 2), qd + ((k >> 2) * half + (k & 3) * 2), id, k > 0);
                }
                mma_done(bar(kWbSFull + st));
                if (i + 2 < nt) mma_done(bar(kWbQEmpty + st));
            }
        if (!ok) {  // whatever was issued is over before the tensor memory goes back
            mma_done(bar(kWbNever));
            mbar_wait_bounded(bar(kWbNever), 0, 4000000000LL);
        }
        tc::fence_before_sync();
    }
    __syncwarp();
    __syncthreads();
    if (warp == 8) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, 256);
    }
}

template <int CODE, int D>
static cudaError_t few(const Plan &p, const WeighArgs &a, cudaStream_t s) {
    using Cfg = WeighCfg<D>;
    cudaError_t e = allow_smem<k_kv_weigh_few<CODE, D>>(Cfg::smem);
    if (e != cudaSuccess) return e;
    return launch(k_kv_weigh_few<CODE, D>, dim3(p.sm_count * Cfg::ctas), Cfg::warps * 32, Cfg::smem, s, a);
}
template <int CODE, int D>
static cudaError_t many(const Plan &p, const WeighArgs &a, cudaStream_t s) {
    using Cfg = WeighManyCfg<D>;
    cudaError_t e = allow_smem<k_kv_weigh_many<CODE, D>>(Cfg::smem);
    if (e != cudaSuccess) return e;
    const dim3 grid((a.c.max_len + kTileRows - 1) / kTileRows, a.c.Hk, a.c.B);
    return launch(k_kv_weigh_many<CODE, D>, grid, kWmThreads, Cfg::smem, s, a);
}
template <int CODE, int D>
static cudaError_t window(const Plan &p, const WeighArgs &a, cudaStream_t s) {
    using Cfg = WeighWindowCfg<D>;
    cudaError_t e = allow_smem<k_kv_weigh_window<CODE, D>>(Cfg::smem);
    if (e != cudaSuccess) return e;
    return launch(k_kv_weigh_window<CODE, D>, dim3(p.sm_count), kWwThreads, Cfg::smem, s, a);
}
template <int CODE>
static cudaError_t weigh(const Plan &p, const WeighArgs &a, cudaStream_t s) {
    const int64_t rows = (int64_t)a.c.max_new * a.c.G;
    switch (p.desc.head_dim) {
        case 64: return rows > kWwRows ? many<CODE, 64>(p, a, s) : rows > kWeighRows ? window<CODE, 64>(p, a, s) : few<CODE, 64>(p, a, s);
        case 128: return rows > kWwRows ? many<CODE, 128>(p, a, s) : rows > kWeighRows ? window<CODE, 128>(p, a, s) : few<CODE, 128>(p, a, s);
        default: return few<CODE, 256>(p, a, s);
    }
}

cudaError_t launch_weigh(const Plan &p, const Ctx &c, Rows q, const float *lse, const float *acc_in, float *acc_out,
                         int64_t acc_stride, float decay, float sm, cudaStream_t s) {
    WeighArgs a{};
    a.c = c;
    a.q = q;
    a.lse = lse;
    a.acc_in = acc_in;
    a.acc_out = acc_out;
    a.acc_stride = acc_stride;
    a.decay = decay;
    a.scale2 = sm * kLog2e;
    a.bf16 = p.desc.dtype == SI_KV_BF16;
    a.log_page = p.desc.page_tokens == 16 ? 4 : p.desc.page_tokens == 32 ? 5 : 6;
    a.fault = p.fault_wait;
    a.budget = p.wait_budget;
    return p.desc.code == SI_KV_INT8 ? weigh<SI_KV_INT8>(p, a, s) : weigh<SI_KV_E4M3>(p, a, s);
}

}  // namespace kv
}  // namespace si
