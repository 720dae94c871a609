// si_kv_attend.cu -- which kernel a call of si_kv_attend takes, and the scratch it needs.
#include <algorithm>
#include <cmath>

#include "si_kv_prompt.cuh"

namespace si {
namespace kv {

cudaError_t launch_decode_int8(const Plan &p, const DecodeArgs &a, int r8, cudaStream_t s);
cudaError_t launch_decode_e4m3(const Plan &p, const DecodeArgs &a, int r8, cudaStream_t s);
cudaError_t launch_prompt_int8(const Plan &p, const PromptArgs &a, cudaStream_t s);
cudaError_t launch_prompt_e4m3(const Plan &p, const PromptArgs &a, cudaStream_t s);

// Many rows: the tensor-core kernel's tile of 128 rows is at least half full.
static bool many_rows(const Plan &p, int max_new) {
    return p.desc.head_dim <= 128 && (int64_t)max_new * (p.desc.n_heads / p.desc.n_kv_heads) > 64;
}
// Its CTAs are split along the keys into as many parts as the estimate below
// makes the call shortest with, from bounds that the host has: the longest CTA,
// the waves of CTAs over the SMs (a CTA an SM), the mean work; a key tile takes
// 1.6 us, a wave's start and end 8, the join of parts 6 and 0.9 for each MB of
// partial results (measured at head_dim 128).  In a graph, int8, one part against
// the chosen number: 300 new tokens behind 20000, 8/8 heads: 264 and 57 us (8 parts);
// 512 behind 8000, 32/8 heads: 124 and 94 us (2).  Where it stays at one part, two would
// take: 1349 new tokens, 16/8 heads: 51 instead of 33 us; 1024 behind 24000, 32/8 heads:
// 376 instead of 343, and 289 instead of 277 at head_dim 64.
// The estimate takes the call's rows as full blocks of kPrRows.  A call of one chunk and
// many steps has more CTAs than that, each nearly empty, and is better made as two: 512 new
// tokens behind 8000 and a token of each of 63 sequences of 8000, 32/8 heads, took 551 us in
// one call and 286 in two.
// The partial results are bounded: kPartialRows rows (query heads counted) for an SM.
constexpr int kMaxSplits = 32, kPartialRows = 4 * kPrRows;
static int prompt_splits(const Plan &p, int total_new, int max_new, int max_len) {
    const int64_t G = p.desc.n_heads / p.desc.n_kv_heads, row_heads = (int64_t)total_new * p.desc.n_heads;
    const int64_t blocks = (total_new * G + kPrRows - 1) / kPrRows * p.desc.n_kv_heads, sms = p.sm_count;
    const float longest = (float)max_len / kPrKeys, shortest = (float)(max_len - max_new) / kPrKeys;
    const float even = 0.5f * (longest + shortest) * blocks / sms;
    int best = 1;
    float least = INFINITY;
    for (int n = 1; n <= kMaxSplits; ++n) {
        if (n > 1 && n * row_heads > sms * kPartialRows) break;
        const float waves = (float)((blocks * n + sms - 1) / sms);
        float us = 1.6f * std::max({longest / n, waves * shortest / n, even}) + 8.0f * waves;
        if (n > 1) us += 6.0f + 0.9e-6f * 4 * (p.desc.head_dim + 2) * n * row_heads;
        if (us < least) {
            least = us;
            best = n;
        }
    }
    return best;
}

// Column tiles of 8 rows in a row group of the few-row kernel: the fewest that hold a sequence's rows,
// as far as the registers go.
static int row_tiles(const Plan &p, int max_new) {
    const int64_t rows = (int64_t)max_new * (p.desc.n_heads / p.desc.n_kv_heads);
    return rows <= 8 ? 1 : rows <= 16 || p.desc.head_dim == 256 ? 2 : 4;
}

size_t scratch_bytes(const Plan &p, int, int total_new, int max_new, int) {
    // A buffer for larger bounds serves smaller ones, so this takes the most that any call within the bounds needs:
    // a call with fewer rows may be split more.
    const size_t D = p.desc.head_dim;
    size_t most = (size_t)p.sm_count * DecodeCfg<64, 1>::ctas * 2 * (size_t)partial_floats(8 * row_tiles(p, max_new), p.desc.head_dim) * sizeof(float);
    if (many_rows(p, max_new)) {
        const size_t row_heads = (size_t)total_new * p.desc.n_heads, cap = (size_t)p.sm_count * kPartialRows;
        size_t n = row_heads * kMaxSplits;
        n = n < cap ? n : cap;
        n = n * (D + 2) * sizeof(float);
        most = n > most ? n : most;
    }
    return kCtrlBytes + most;
}

cudaError_t launch_attend(const Plan &p, const Ctx &c, Rows q, Rows out, float *lse, float sm, void *scratch, cudaStream_t s) {
    const int log_page = p.desc.page_tokens == 16 ? 4 : p.desc.page_tokens == 32 ? 5 : 6;
    if (many_rows(p, c.max_new)) {
        PromptArgs a{};
        a.c = c;
        a.q = q;
        a.out = out;
        a.lse = lse;
        a.scale2 = sm * kLog2e;
        a.bf16 = p.desc.dtype == SI_KV_BF16;
        a.log_page = log_page;
        a.splits = prompt_splits(p, c.T, c.max_new, c.max_len);
        a.fault = p.fault_wait;
        a.budget = p.wait_budget;
        a.partial = reinterpret_cast<float *>(static_cast<uint8_t *>(scratch) + kCtrlBytes);
        return p.desc.code == SI_KV_INT8 ? launch_prompt_int8(p, a, s) : launch_prompt_e4m3(p, a, s);
    }
    DecodeArgs a{};
    a.c = c;
    a.q = q;
    a.out = out;
    a.lse = lse;
    a.scale2 = sm * kLog2e;
    a.bf16 = p.desc.dtype == SI_KV_BF16;
    a.log_page = log_page;
    a.counters = static_cast<int32_t *>(scratch) + kCtrlWords;
    a.partial = reinterpret_cast<float *>(static_cast<uint8_t *>(scratch) + kCtrlBytes);
    const int r8 = row_tiles(p, c.max_new);
    return p.desc.code == SI_KV_INT8 ? launch_decode_int8(p, a, r8, s) : launch_decode_e4m3(p, a, r8, s);
}

}  // namespace kv
}  // namespace si
