// si_kv_api.cu -- the attention block's C ABI (include/si_kv.h): plans,
// argument checks and stream-ordered launches.  Every argument error is
// returned before anything is launched.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstdlib>
#include <new>

#include "si_kv.h"

using si::kv::Ctx;
using si::kv::Plan;
using si::kv::Rows;

struct si_kv_plan_s {
    Plan p;
};

namespace {

// Rows of one sequence and kv head, query heads counted: more break a bound (SI_ERR_DEVICE).  A sequence of
// SI_KV_MAX_LEN rows and 256 query heads for a kv head has as many.
constexpr int32_t kMaxRowHeads = 1 << 30;

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool overlap(const void *a, size_t na, const void *b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

si_status validate_desc(const si_kv_desc *d) {
    if (!d) return SI_ERR_INVALID_ARG;
    if (d->n_heads < 1 || d->n_kv_heads < 1 || d->n_heads % d->n_kv_heads) return SI_ERR_INVALID_ARG;
    if (d->n_heads > SI_KV_MAX_HEADS) return SI_ERR_UNSUPPORTED;
    if (d->head_dim != 64 && d->head_dim != 128 && d->head_dim != 256) return SI_ERR_UNSUPPORTED;
    if (d->page_tokens != 16 && d->page_tokens != 32 && d->page_tokens != 64) return SI_ERR_UNSUPPORTED;
    if (d->code != SI_KV_INT8 && d->code != SI_KV_E4M3) return SI_ERR_UNSUPPORTED;
    if (d->dtype != SI_KV_BF16 && d->dtype != SI_KV_F16) return SI_ERR_UNSUPPORTED;
    return SI_OK;
}

// The bounds of a call; `rows`: the call has q, k or v rows.
si_status check_bounds(int32_t n_seqs, int32_t total_new, int32_t max_new, int32_t max_len) {
    if (n_seqs < 1 || total_new < 0 || max_new < 0 || max_len < 0) return SI_ERR_INVALID_ARG;
    if (n_seqs > SI_KV_MAX_SEQS || max_len > SI_KV_MAX_LEN) return SI_ERR_UNSUPPORTED;
    return SI_OK;
}

si_status check_cache(const si_kv_cache *c) {
    if (!c || !c->k_codes || !c->v_codes || !c->k_scale || !c->v_scale || !c->k_tail || !c->v_tail)
        return SI_ERR_INVALID_ARG;
    if (c->n_pages < 1 || c->n_pages > INT32_MAX || c->n_slots < 1) return SI_ERR_INVALID_ARG;
    if (!aligned(c->k_codes, 16) || !aligned(c->v_codes, 16) || !aligned(c->k_scale, 16) || !aligned(c->v_scale, 16) ||
        !aligned(c->k_tail, 16) || !aligned(c->v_tail, 16))
        return SI_ERR_MISALIGNED;
    return SI_OK;
}

si_status check_scratch(const Plan &p, const si_kv_batch *b, const void *scratch, size_t bytes) {
    if (!scratch) return SI_ERR_INVALID_ARG;
    if (!aligned(scratch, 16)) return SI_ERR_MISALIGNED;
    const size_t need = b ? si::kv::scratch_bytes(p, b->n_seqs, b->total_new, b->max_new, b->max_len)
                          : si::kv::kCtrlBytes;
    return bytes < need ? SI_ERR_SCRATCH_TOO_SMALL : SI_OK;
}

si_status check_batch(const Plan &p, const si_kv_batch *b, bool rows) {
    if (!b) return SI_ERR_INVALID_ARG;
    const si_status st = check_bounds(b->n_seqs, rows ? b->total_new : 0, rows ? b->max_new : 0, b->max_len);
    if (st != SI_OK) return st;
    if (!b->lens || (rows && !b->q_start)) return SI_ERR_INVALID_ARG;
    const int32_t pages = b->max_len / p.desc.page_tokens;
    if (b->table_stride < pages || (pages > 0 && !b->page_table)) return SI_ERR_INVALID_ARG;
    if (!aligned(b->lens, 4) || !aligned(b->q_start, 4) || !aligned(b->page_table, 4) || !aligned(b->slots, 4))
        return SI_ERR_MISALIGNED;
    return SI_OK;
}

// (without rows there may be no data)
si_status check_rows(const Plan &p, const si_kv_rows *r, const si_kv_batch *b, bool written) {
    if (!r || (!r->data && b->total_new > 0)) return SI_ERR_INVALID_ARG;
    if (r->row_stride < 0 || r->head_stride < 0) return SI_ERR_INVALID_ARG;
    if (written && (r->row_stride < p.desc.head_dim || r->head_stride < p.desc.head_dim)) return SI_ERR_INVALID_ARG;
    if (!aligned(r->data, 16) || r->row_stride % 8 || r->head_stride % 8) return SI_ERR_MISALIGNED;
    return SI_OK;
}

// Whether D values at elements x + r row + h head and D at y + r' row + h' head can share one, for |r - r'| < T and
// |h - h'| < H; `self`: the same operand, in which r = r' and h = h' is one place.
bool strides_meet(int64_t apart, int64_t row, int64_t head, int64_t T, int64_t H, int64_t D, bool self) {
    for (int64_t h = 1 - H; h < H; ++h) {
        const int64_t at = apart + h * head;  // of which multiples of row, up to T - 1 of them, may make less than D
        const int64_t near = row == 0 ? 0 : -at / row;
        for (int64_t r = std::max(near - 1, 1 - T); r <= std::min(near + 1, T - 1); ++r)
            if ((!self || r != 0 || h != 0) && std::abs(at + r * row) < D) return true;
    }
    return false;
}
// out's rows and heads may not meet one another; nor q's, as far as their strides are alike (else only the places of
// which both have the first).
si_status check_out(const Plan &p, const si_kv_rows *q, const si_kv_rows *out, int64_t T) {
    const int64_t D = p.desc.head_dim, H = p.desc.n_heads;
    const bool spans = out->row_stride >= (H - 1) * out->head_stride + D || out->head_stride >= (T - 1) * out->row_stride + D;
    if (!spans && strides_meet(0, out->row_stride, out->head_stride, T, H, D, true)) return SI_ERR_INVALID_ARG;
    const int64_t apart = (int64_t)(reinterpret_cast<intptr_t>(out->data) - reinterpret_cast<intptr_t>(q->data)) / 2;
    const bool alike = (q->row_stride == out->row_stride || T == 1) && (q->head_stride == out->head_stride || H == 1);
    const int64_t reach = (T - 1) * out->row_stride + (H - 1) * out->head_stride + D;
    if (alike ? std::abs(apart) < reach && strides_meet(apart, out->row_stride, out->head_stride, T, H, D, false)
              : std::abs(apart) < D)
        return SI_ERR_INVALID_ARG;
    return SI_OK;
}

Ctx make_ctx(const Plan &p, const si_kv_cache *c, const si_kv_batch *b, void *scratch) {
    Ctx x{};
    x.kc = static_cast<uint8_t *>(c->k_codes);
    x.vc = static_cast<uint8_t *>(c->v_codes);
    x.ks = c->k_scale;
    x.vs = c->v_scale;
    x.kt = static_cast<uint16_t *>(c->k_tail);
    x.vt = static_cast<uint16_t *>(c->v_tail);
    x.n_pages = c->n_pages;
    x.n_slots = c->n_slots;
    x.status = static_cast<int32_t *>(scratch);
    x.H = p.desc.n_heads;
    x.Hk = p.desc.n_kv_heads;
    x.G = x.H / x.Hk;
    x.D = p.desc.head_dim;
    x.P = p.desc.page_tokens;
    if (b) {
        x.q_start = b->q_start;
        x.lens = b->lens;
        x.table = b->page_table;
        x.slots = b->slots;
        x.table_stride = b->table_stride;
        x.B = b->n_seqs;
        x.T = b->total_new;
        // (what max_new leaves open, total_new may not; and the kernels number a kv head's rows in 32 bits)
        x.max_new = std::min({b->max_new, b->total_new, kMaxRowHeads / x.G});
        x.max_len = b->max_len;
    }
    return x;
}

Rows make_rows(const si_kv_rows *r) { return Rows{static_cast<uint16_t *>(r->data), r->row_stride, r->head_stride}; }

si_status launched(cudaError_t e) {
    if (e == cudaSuccess) return SI_OK;
    cudaGetLastError();
    return SI_ERR_CUDA;
}

}  // namespace

#define SI_KV_TRY(x)                      \
    do {                                  \
        const si_status st_ = (x);        \
        if (st_ != SI_OK) return st_;     \
    } while (0)

extern "C" {

si_status si_kv_plan(const si_kv_desc *desc, int cuda_device, si_kv_plan_t *out) {
    if (!out) return SI_ERR_INVALID_ARG;
    *out = nullptr;
    SI_KV_TRY(validate_desc(desc));
    int sms = 0, khz = 0;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, cuda_device) != cudaSuccess ||
        cudaDeviceGetAttribute(&khz, cudaDevAttrClockRate, cuda_device) != cudaSuccess) {
        cudaGetLastError();
        return SI_ERR_CUDA;
    }
    si_kv_plan_s *h = new (std::nothrow) si_kv_plan_s();
    if (!h) return SI_ERR_CUDA;
    h->p.desc = *desc;
    h->p.device = cuda_device;
    h->p.sm_count = sms;
    h->p.wait_budget = khz > 0 ? (long long)khz * 1000 : 2000000000ll;  // about one second
    // SI_FAULT_WAIT_BUDGET as for si_moe_plan: its cycle count is the budget, and a wait runs out for certain
    h->p.fault_wait = false;
    if (const char *env = std::getenv("SI_FAULT_WAIT_BUDGET")) {
        char *end = nullptr;
        const long long v = std::strtoll(env, &end, 10);
        if (end && end != env && *end == '\0' && v >= 0) {
            h->p.wait_budget = v;
            h->p.fault_wait = true;
        }
    }
    *out = h;
    return SI_OK;
}

void si_kv_plan_destroy(si_kv_plan_t plan) { delete plan; }

si_status si_kv_scratch_bytes(si_kv_plan_t plan, int32_t n_seqs, int32_t total_new, int32_t max_new, int32_t max_len,
                              size_t *bytes) {
    if (!plan || !bytes) return SI_ERR_INVALID_ARG;
    SI_KV_TRY(check_bounds(n_seqs, total_new, max_new, max_len));
    *bytes = si::kv::scratch_bytes(plan->p, n_seqs, total_new, max_new, max_len);
    return SI_OK;
}

si_status si_kv_scratch_init(si_kv_plan_t plan, void *scratch, size_t scratch_bytes, si_stream_t stream) {
    if (!plan || !scratch) return SI_ERR_INVALID_ARG;
    if (!aligned(scratch, 16)) return SI_ERR_MISALIGNED;
    if (scratch_bytes < si::kv::kCtrlBytes) return SI_ERR_SCRATCH_TOO_SMALL;
    return launched(cudaMemsetAsync(scratch, 0, si::kv::kCtrlBytes, (cudaStream_t)stream));
}

si_status si_kv_append(si_kv_plan_t plan, const si_kv_cache *cache, const si_kv_batch *batch, const si_kv_rows *k,
                       const si_kv_rows *v, int32_t *lens_out, void *scratch, size_t scratch_bytes,
                       si_stream_t stream) {
    if (!plan || !lens_out) return SI_ERR_INVALID_ARG;
    SI_KV_TRY(check_cache(cache));
    SI_KV_TRY(check_batch(plan->p, batch, true));
    SI_KV_TRY(check_rows(plan->p, k, batch, false));
    SI_KV_TRY(check_rows(plan->p, v, batch, false));
    if (!aligned(lens_out, 4)) return SI_ERR_MISALIGNED;
    const size_t n = (size_t)batch->n_seqs * sizeof(int32_t);
    if (overlap(lens_out, n, batch->lens, n)) return SI_ERR_INVALID_ARG;
    SI_KV_TRY(check_scratch(plan->p, batch, scratch, scratch_bytes));
    return launched(si::kv::launch_append(plan->p, make_ctx(plan->p, cache, batch, scratch), make_rows(k), make_rows(v),
                                          lens_out, (cudaStream_t)stream));
}

si_status si_kv_read(si_kv_plan_t plan, const si_kv_cache *cache, const int32_t *pages, int32_t n, void *k_out,
                     void *v_out, void *scratch, size_t scratch_bytes, si_stream_t stream) {
    if (!plan || n < 0 || (n > 0 && (!pages || !k_out || !v_out))) return SI_ERR_INVALID_ARG;
    SI_KV_TRY(check_cache(cache));
    if (!aligned(pages, 4) || !aligned(k_out, 16) || !aligned(v_out, 16)) return SI_ERR_MISALIGNED;
    SI_KV_TRY(check_scratch(plan->p, nullptr, scratch, scratch_bytes));
    if (n == 0) return SI_OK;
    return launched(si::kv::launch_read(plan->p, make_ctx(plan->p, cache, nullptr, scratch), pages, n,
                                        static_cast<uint16_t *>(k_out), static_cast<uint16_t *>(v_out),
                                        (cudaStream_t)stream));
}

si_status si_kv_attend(si_kv_plan_t plan, const si_kv_cache *cache, const si_kv_batch *batch, const si_kv_rows *q,
                       const si_kv_rows *out, float *lse, float sm_scale, void *scratch, size_t scratch_bytes,
                       si_stream_t stream) {
    if (!plan || !(sm_scale >= 0.0f) || !std::isfinite(sm_scale)) return SI_ERR_INVALID_ARG;
    SI_KV_TRY(check_cache(cache));
    SI_KV_TRY(check_batch(plan->p, batch, true));
    SI_KV_TRY(check_rows(plan->p, q, batch, false));
    SI_KV_TRY(check_rows(plan->p, out, batch, true));
    if (!aligned(lse, 4)) return SI_ERR_MISALIGNED;
    SI_KV_TRY(check_scratch(plan->p, batch, scratch, scratch_bytes));
    if (batch->total_new == 0 || batch->max_new == 0) return SI_OK;
    SI_KV_TRY(check_out(plan->p, q, out, batch->total_new));
    return launched(si::kv::launch_attend(plan->p, make_ctx(plan->p, cache, batch, scratch), make_rows(q),
                                          make_rows(out), lse, sm_scale, scratch, (cudaStream_t)stream));
}

si_status si_kv_weigh(si_kv_plan_t plan, const si_kv_cache *cache, const si_kv_batch *batch, const si_kv_rows *q,
                      const float *lse, const float *acc_in, float *acc_out, int64_t acc_stride, float decay,
                      float sm_scale, void *scratch, size_t scratch_bytes, si_stream_t stream) {
    if (!plan || !acc_out || !(sm_scale >= 0.0f) || !std::isfinite(sm_scale) || !std::isfinite(decay))
        return SI_ERR_INVALID_ARG;
    SI_KV_TRY(check_cache(cache));
    SI_KV_TRY(check_batch(plan->p, batch, true));
    SI_KV_TRY(check_rows(plan->p, q, batch, false));
    if (acc_stride < batch->max_len || (!lse && batch->total_new > 0)) return SI_ERR_INVALID_ARG;
    if (!aligned(lse, 4) || !aligned(acc_in, 4) || !aligned(acc_out, 4)) return SI_ERR_MISALIGNED;
    if (acc_in && acc_in != acc_out) {  // the same array, or arrays apart
        const size_t n = (size_t)batch->n_seqs * plan->p.desc.n_kv_heads * (size_t)acc_stride * sizeof(float);
        if (overlap(acc_in, n, acc_out, n)) return SI_ERR_INVALID_ARG;
    }
    SI_KV_TRY(check_scratch(plan->p, batch, scratch, scratch_bytes));
    if (batch->max_len == 0) return SI_OK;
    return launched(si::kv::launch_weigh(plan->p, make_ctx(plan->p, cache, batch, scratch), make_rows(q), lse, acc_in,
                                         acc_out, acc_stride, decay, sm_scale, (cudaStream_t)stream));
}

si_status si_kv_evict(si_kv_plan_t plan, const si_kv_cache *cache, const si_kv_batch *batch, const float *acc_in,
                      float *acc_out, int64_t acc_stride, int32_t budget, int32_t sink, int32_t recent,
                      const int32_t *new_table, const int32_t *new_slots, int32_t *keep, int32_t *lens_out,
                      void *scratch, size_t scratch_bytes, si_stream_t stream) {
    if (!plan || !acc_in || !acc_out || !new_table || !keep || !lens_out) return SI_ERR_INVALID_ARG;
    if (budget < 1 || sink < 0 || recent < 0 || (int64_t)sink + recent > budget) return SI_ERR_INVALID_ARG;
    SI_KV_TRY(check_cache(cache));
    SI_KV_TRY(check_batch(plan->p, batch, false));
    if (batch->max_len / plan->p.desc.page_tokens > SI_KV_MAX_EVICT_PAGES) return SI_ERR_UNSUPPORTED;
    if (acc_stride < batch->max_len) return SI_ERR_INVALID_ARG;
    if (!aligned(acc_in, 4) || !aligned(acc_out, 4) || !aligned(new_table, 4) || !aligned(new_slots, 4) ||
        !aligned(keep, 4) || !aligned(lens_out, 4))
        return SI_ERR_MISALIGNED;
    const size_t n = (size_t)batch->n_seqs * plan->p.desc.n_kv_heads * (size_t)acc_stride * sizeof(float);
    const size_t m = (size_t)batch->n_seqs * sizeof(int32_t);
    if (overlap(acc_in, n, acc_out, n) || overlap(lens_out, m, batch->lens, m)) return SI_ERR_INVALID_ARG;
    SI_KV_TRY(check_scratch(plan->p, nullptr, scratch, scratch_bytes));
    Ctx c = make_ctx(plan->p, cache, batch, scratch);
    c.T = 0;
    c.max_new = 0;
    return launched(si::kv::launch_evict(plan->p, c, acc_in, acc_out, acc_stride, budget, sink, recent, new_table,
                                         new_slots, keep, lens_out, (cudaStream_t)stream));
}

si_status si_kv_read_status(si_kv_plan_t plan, const void *scratch, si_stream_t stream) {
    if (!plan || !scratch) return SI_ERR_INVALID_ARG;
    if (!aligned(scratch, 16)) return SI_ERR_MISALIGNED;
    int32_t word = 0;
    SI_KV_TRY(launched(cudaStreamSynchronize((cudaStream_t)stream)));
    SI_KV_TRY(launched(cudaMemcpy(&word, scratch, sizeof(word), cudaMemcpyDeviceToHost)));
    if (word == 0) return SI_OK;
    // (cleared in the stream's order: a call that follows in it may report at once)
    SI_KV_TRY(launched(cudaMemsetAsync(const_cast<void *>(scratch), 0, sizeof(word), (cudaStream_t)stream)));
    return (si_status)word;
}

}  // extern "C"
