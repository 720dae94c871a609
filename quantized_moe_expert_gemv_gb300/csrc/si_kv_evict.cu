// si_kv_evict.cu -- eviction by accumulated attention weight: the choice of
// each kv head's pages, and their move.
//
// Choice (k_kv_choose, one CTA for each sequence and kv head).  A page's score
// is the sum of acc over its tokens, in whole numbers (a page that is kept by a
// last-bit difference would depend on the order of the sum).  Scores
// become 64-bit keys whose unsigned order is the scores' order, the protected
// pages get the largest key, and a radix selection finds the key of the last
// page that stays: 8 bits a pass from the top, a histogram of the keys that
// still share the prefix, until the digit's bin holds exactly the pages still
// wanted.  Equal keys go to the lower page, by a count over the pages in order.
// Move (k_kv_move, one CTA for each new page, and one for the rest): codes,
// scale and sums are copied as they are; the unfinished page's rows only where
// no other sequence's lie or go.
// Bound: HBM for the move (each kept byte read and written once); the choice reads
// acc once and is a chain of block-wide steps.  Measured: 8 sequences of 20000 to
// 32700 tokens, 8 heads of 128, down to 128 pages of 64: 128 us, 80 % of the copy
// rate, with the kept pages read back (evict alone 65, of which 25 remain with a
// budget of ten pages); one of 1500 tokens 9 us, two launches' latency.
#include "si_kv_device.cuh"

namespace si {
namespace kv {

constexpr int kChooseMost = 1024;
constexpr int kMoveThreads = 256;

// Order-preserving key of a score; NaN counts as largest, -0 as +0.
__device__ __forceinline__ unsigned long long score_key(double x) {
    if (x != x) return ~0ull - 1;
    const unsigned long long u = (unsigned long long)__double_as_longlong(x == 0.0 ? 0.0 : x);
    return u >> 63 ? ~u : u | 0x8000000000000000ull;
}

// A page's sum, in whole units of 2^(top - 182), where top is the largest exponent field of its values: a value is its
// 24 bits shifted by what its exponent is below the top (up to 32 to the left, bits further down are cut off), below 2^56, so
// 64 of them fit 64 bits.  Whole numbers add up to the same in any order: pages of the same values tie.  The sum is
// exact where the values lie within 2^32 of one another, and else off by less than 2^-49 of the largest.  (In 64-bit floating
// point, of two lanes a cycle and SM, 32768 tokens took 17 us.)
__device__ __forceinline__ int exponent_of(float x) { return (__float_as_uint(x) >> 23) & 255; }
__device__ __forceinline__ long long in_units(float x, int top) {
    const uint32_t u = __float_as_uint(x);
    const int e = exponent_of(x), down = top - max(e, 1);
    const unsigned long long m = (unsigned long long)((u & 0x7fffffu) | (e ? 0x800000u : 0u)) << 32;
    const long long v = down < 64 ? (long long)(m >> down) : 0;
    return u >> 31 ? -v : v;
}

// score_key of such a sum (its 53 leading bits), by its bits: the 64-bit unit's conversion and product take longer.
__device__ __forceinline__ unsigned long long units_key(long long v, int top) {
    if (v == 0) return 0x8000000000000000ull;
    const unsigned long long mag = v < 0 ? 0ull - (unsigned long long)v : (unsigned long long)v;
    const int zeros = __clzll((long long)mag);
    const unsigned long long u = (unsigned long long)(63 - zeros + top - 182 + 1023) << 52 | (mag << zeros << 1) >> 12;
    return v < 0 ? ~(u | 0x8000000000000000ull) : u | 0x8000000000000000ull;
}

// Exclusive prefix of a 0/1 flag over the CTA's threads in order; `total` = their sum.
__device__ __forceinline__ int block_prefix(bool flag, int *s_warp, int &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const unsigned m = __ballot_sync(0xffffffffu, flag);
    __syncthreads();  // s_warp's earlier use is over
    if (lane == 0) s_warp[warp] = __popc(m);
    __syncthreads();
    const int mine = lane < warps ? s_warp[lane] : 0;
    total = __reduce_add_sync(0xffffffffu, mine);
    return __reduce_add_sync(0xffffffffu, lane < warp ? mine : 0) + __popc(m & ((1u << lane) - 1));
}

__global__ void __launch_bounds__(kChooseMost) k_kv_choose(Ctx c, const float *acc, int64_t acc_stride, int budget,
                                                              int sink, int recent, int32_t *keep, int32_t *lens_out) {
    extern __shared__ unsigned long long s_key[];  // [max_len / P]
    __shared__ int s_hist[256], s_warp[kChooseMost / 32], s_digit, s_above, s_in;
    const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, threads = blockDim.x, P = c.P;
    start_after();
    const Seq s = load_seq(c, b, false);
    const int F = s.len / P, n_keep = min(F, budget);
    keep += ((int64_t)b * c.Hk + h) * budget;
    if (h == 0 && tid == 0) lens_out[b] = n_keep * P + s.len % P;
    for (int i = n_keep + tid; i < budget; i += threads) keep[i] = -1;
    if (F <= budget) {
        for (int i = tid; i < F; i += threads) keep[i] = i;
        return;
    }
    // 16 lanes a page, 8 pages' loads at a time under way (four a lane and page at most)
    const float *a = acc + ((int64_t)b * c.Hk + h) * acc_stride;
    const int l16 = tid & 15, step = threads / 16;
    const unsigned half = 0xffffu << (tid & 16);
    for (int j0 = tid >> 4; j0 < F; j0 += 8 * step) {
        float x[8][4];
#pragma unroll
        for (int q = 0; q < 8; ++q)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int j = j0 + q * step, t = l16 + 16 * e;
                x[q][e] = j < F && t < P ? a[(int64_t)j * P + t] : 0.0f;
            }
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const int j = j0 + q * step;
            if (j >= F) break;
            int top = max(max(exponent_of(x[q][0]), exponent_of(x[q][1])), max(exponent_of(x[q][2]), exponent_of(x[q][3])));
            top = max(__reduce_max_sync(half, top), 1);
            unsigned long long key;
            if (top < 255) {
                const unsigned long long v = (in_units(x[q][0], top) + in_units(x[q][1], top)) +
                                             (in_units(x[q][2], top) + in_units(x[q][3], top));
                // (16 lanes' sum modulo 2^64, by 22 bits at a time)
                const unsigned long long a0 = __reduce_add_sync(half, (unsigned)(v & 0x3fffff));
                const unsigned long long a1 = __reduce_add_sync(half, (unsigned)(v >> 22 & 0x3fffff));
                const unsigned long long a2 = __reduce_add_sync(half, (unsigned)(v >> 44));
                key = units_key((long long)(a0 + (a1 << 22) + (a2 << 44)), top);
            } else {  // a value that is not finite
                double sum = ((double)x[q][0] + (double)x[q][1]) + ((double)x[q][2] + (double)x[q][3]);
                for (int o = 8; o; o >>= 1) sum += __shfl_xor_sync(half, sum, o);
                key = score_key(sum);
            }
            if (l16 == 0) s_key[j] = j < sink || j >= F - recent ? ~0ull : key;
        }
    }
    __syncthreads();
    unsigned long long prefix = 0, mask = 0;
    int want = n_keep;  // pages still to be taken among those that share the prefix
    bool ties = true;
    for (int shift = 56; shift >= 0; shift -= 8) {
        for (int i = tid; i < 256; i += threads) s_hist[i] = 0;
        __syncthreads();
        for (int j = tid; j < F; j += threads)
            if ((s_key[j] & mask) == prefix) atomicAdd(&s_hist[(s_key[j] >> shift) & 255], 1);
        __syncthreads();
        if (tid < 32) {  // the digit whose bin the last wanted page falls in, from the top
            int mine[8], sum = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) sum += mine[e] = s_hist[255 - (tid * 8 + e)];
            int before = sum;
            for (int o = 1; o < 32; o <<= 1) {
                const int up = __shfl_up_sync(0xffffffffu, before, o);
                if (tid >= o) before += up;
            }
            before -= sum;
            if (before < want && want <= before + sum) {
                int e = 0;
                while (before + mine[e] < want) before += mine[e++];
                s_digit = 255 - (tid * 8 + e);
                s_above = before;
                s_in = mine[e];
            }
        }
        __syncthreads();
        prefix |= (unsigned long long)s_digit << shift;
        mask |= 255ull << shift;
        want -= s_above;
        if (s_in == want) {  // all of the bin stay: the lower bits do not matter
            ties = false;
            break;
        }
    }
    // Taken: keys above the prefix, and of those that share it all, or the first `want`.
    int kept = 0, tied = 0;
    for (int j0 = 0; j0 < F; j0 += threads) {
        const int j = j0 + tid;
        const unsigned long long k = j < F ? s_key[j] & mask : 0;
        bool take = j < F && k >= prefix;
        int total;
        if (ties) {
            const bool eq = j < F && k == prefix;
            const int at = tied + block_prefix(eq, s_warp, total);
            tied += total;
            if (eq) take = at < want;
        }
        const int at = kept + block_prefix(take, s_warp, total);
        if (take) keep[at] = j;
        kept += total;
    }
}

__global__ void __launch_bounds__(kMoveThreads) k_kv_move(Ctx c, const float *acc_in, float *acc_out, int64_t acc_stride,
                                                          int budget, int most, const int32_t *new_table,
                                                          const int32_t *new_slots, const int32_t *keep) {
    const int i = blockIdx.x, h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x, P = c.P;
    start_after();
    const Seq s = load_seq(c, b, false);
    const int F = s.len / P, n_keep = min(F, budget);
    const int64_t bh = (int64_t)b * c.Hk + h;
    if (i < n_keep) {
        const int j = keep[bh * budget + i];
        const int64_t src = load_page(c, b, j);
        const int dst = new_table[(int64_t)b * budget + i];
        if (tid < P) acc_out[bh * acc_stride + i * P + tid] = acc_in[bh * acc_stride + (int64_t)j * P + tid];
        if (dst < 0 || dst >= c.n_pages) {
            if (tid == 0) set_status(c.status, SI_ERR_DEVICE);
            return;
        }
        const int units = P * c.D / 16;
        const int64_t from = page_at(c, src < 0 ? 0 : src, h), to = page_at(c, dst, h);
        const uint4 zero = make_uint4(0, 0, 0, 0);
        for (int u = tid; u < units; u += kMoveThreads) {
            const uint4 k = src < 0 ? zero : *reinterpret_cast<const uint4 *>(c.kc + from + u * 16);
            const uint4 v = src < 0 ? zero : *reinterpret_cast<const uint4 *>(c.vc + from + u * 16);
            *reinterpret_cast<uint4 *>(c.kc + to + u * 16) = k;
            *reinterpret_cast<uint4 *>(c.vc + to + u * 16) = v;
        }
        if (tid < 2) {
            float *sc = tid ? c.vs : c.ks;
            sc[(int64_t)dst * c.Hk + h] = src < 0 ? __int_as_float(0x7fc00000) : sc[src * c.Hk + h];
        }
        return;
    }
    if (i != most) return;
    // the unfinished page: its sums, and its rows where their ring place changes
    const int r = s.len - F * P;
    if (tid < r) acc_out[bh * acc_stride + n_keep * P + tid] = acc_in[bh * acc_stride + (int64_t)F * P + tid];
    const int slot = new_slots ? new_slots[b] : s.slot;
    if (slot < 0 || slot >= c.n_slots) {
        if (tid == 0) set_status(c.status, SI_ERR_DEVICE);
        return;
    }
    if (s.slot < 0 || r == 0 || (slot == s.slot && ((F ^ n_keep) & 1) == 0)) return;
    if (slot != s.slot) {
        // all sequences' rows move at once: the slot may hold no other's (which may have to be read yet, or stay), nor be
        // another's new one
        bool taken = false;
        for (int k = tid; k < c.B; k += kMoveThreads) {
            const int len = c.lens[k], own = c.slots ? c.slots[k] : k;
            if (k != b && len >= 0 && len <= c.max_len && len % P != 0) taken |= own == slot || new_slots[k] == slot;
        }
        if (__syncthreads_or(taken)) {
            if (tid == 0) set_status(c.status, SI_ERR_DEVICE);
            return;
        }
    }
    const int upr = c.D / 8;
    for (int u = tid; u < r * upr; u += kMoveThreads) {
        const int t = u / upr, d = u % upr * 8;
        const int64_t from = ring_at(c, s.slot, h, F * P + t) + d, to = ring_at(c, slot, h, n_keep * P + t) + d;
        *reinterpret_cast<uint4 *>(c.kt + to) = *reinterpret_cast<const uint4 *>(c.kt + from);
        *reinterpret_cast<uint4 *>(c.vt + to) = *reinterpret_cast<const uint4 *>(c.vt + from);
    }
}

cudaError_t launch_evict(const Plan &p, const Ctx &c, const float *acc_in, float *acc_out, int64_t acc_stride, int budget,
                         int sink, int recent, const int32_t *new_table, const int32_t *new_slots, int32_t *keep,
                         int32_t *lens_out, cudaStream_t s) {
    const size_t smem = (size_t)(c.max_len / c.P) * sizeof(unsigned long long);
    cudaError_t e = allow_smem<k_kv_choose>(SI_KV_MAX_EVICT_PAGES * (int)sizeof(unsigned long long));
    if (e != cudaSuccess) return e;
    // as many threads as half-warps for a page, up to 1024 (a small cache's block-wide steps are quicker with few)
    const int threads = c.max_len / c.P <= 64 ? 256 : kChooseMost;
    e = launch(k_kv_choose, dim3(c.Hk, c.B), threads, smem, s, c, acc_in, acc_stride, budget, sink, recent, keep, lens_out);
    if (e != cudaSuccess) return e;
    const int most = min(budget, c.max_len / c.P);  // no sequence keeps more
    return launch(k_kv_move, dim3(most + 1, c.Hk, c.B), kMoveThreads, 0, s, c, acc_in, acc_out, acc_stride, budget, most,
                  new_table, new_slots, keep);
}

}  // namespace kv
}  // namespace si
