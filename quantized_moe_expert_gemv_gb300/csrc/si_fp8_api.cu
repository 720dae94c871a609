// si_fp8_api.cu -- the dense block's C ABI (include/si_fp8.h): plans, argument
// checks and stream-ordered launches.  Every argument error is returned
// before anything is launched.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstdlib>
#include <new>

#include "si_fp8.h"

using si::fp8::Mat;
using si::fp8::MatmulArgs;
using si::fp8::NormArgs;
using si::fp8::Plan;

struct si_fp8_plan_s {
    Plan p;
};

namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int64_t size_of(int32_t dtype) { return dtype == SI_FP8_F32 ? 4 : 2; }

si_status validate_desc(const si_fp8_desc *d) {
    if (!d || d->in_features < 1 || d->out_features < 1) return SI_ERR_INVALID_ARG;
    if (d->in_features % 16 || d->in_features > SI_FP8_MAX_IN || d->out_features > SI_FP8_MAX_OUT) return SI_ERR_UNSUPPORTED;
    return SI_OK;
}

// The launches go to the current device: it has to be the plan's.
si_status check_device(const Plan &p) {
    int device = -1;
    if (cudaGetDevice(&device) != cudaSuccess) {
        cudaGetLastError();
        return SI_ERR_CUDA;
    }
    return device == p.device ? SI_OK : SI_ERR_INVALID_ARG;
}

// A device's SMs and clock.  The clock takes the driver most of a millisecond, and a program makes a plan for each shape
// of its layers: it is asked for once a device.
bool device_numbers(int device, int &sms, int &khz) {
    static std::atomic<int> known[64];  // kHz
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess) return false;
    const bool kept = device >= 0 && device < 64;
    khz = kept ? known[device].load(std::memory_order_relaxed) : 0;
    if (khz > 0) return true;
    if (cudaDeviceGetAttribute(&khz, cudaDevAttrClockRate, device) != cudaSuccess) return false;
    if (kept) known[device].store(khz, std::memory_order_relaxed);
    return true;
}

si_status check_rows_count(int32_t n_rows) {
    if (n_rows < 0) return SI_ERR_INVALID_ARG;
    return n_rows > SI_FP8_MAX_ROWS ? SI_ERR_UNSUPPORTED : SI_OK;
}

// A matrix of T rows of `cols` values; `whole`: rows start at multiples of 16 bytes.
si_status check_mat(const si_fp8_mat *m, int64_t T, int64_t cols, bool written, bool whole) {
    if (!m->data && T > 0) return SI_ERR_INVALID_ARG;
    if (m->dtype != SI_FP8_BF16 && m->dtype != SI_FP8_F16 && m->dtype != SI_FP8_F32) return SI_ERR_UNSUPPORTED;
    if (m->row_stride < 0 || m->row_stride > (int64_t)1 << 38) return SI_ERR_INVALID_ARG;
    // (rows of an input may lie on one another; T = 1 has one row)
    if (written && T > 1 && m->row_stride < cols) return SI_ERR_INVALID_ARG;
    if (!aligned(m->data, 16) || (whole && T > 1 && m->row_stride * size_of(m->dtype) % 16)) return SI_ERR_MISALIGNED;
    return SI_OK;
}

// The bytes of a matrix: `rows` pieces of `len`, `step` apart.
struct Span {
    uintptr_t at;
    int64_t rows, step, len;
};
Span span(const si_fp8_mat *m, int64_t T, int64_t cols) {
    const int64_t e = size_of(m->dtype);
    return Span{reinterpret_cast<uintptr_t>(m->data), m->row_stride ? T : 1, m->row_stride * e, cols * e};
}
Span span(const void *p, int64_t bytes) { return Span{reinterpret_cast<uintptr_t>(p), 1, bytes, bytes}; }

// Whether the two share a byte.  Pieces the same distance apart are told apart exactly (two halves of each row of one
// buffer do not meet); of others, what lies between the pieces counts as theirs.
bool meet(const Span &a, const Span &b) {
    if (a.rows < 1 || b.rows < 1) return false;
    const int64_t ea = (a.rows - 1) * a.step + a.len, eb = (b.rows - 1) * b.step + b.len;
    if (a.at + ea <= b.at || b.at + eb <= a.at) return false;
    if (a.rows > 1 && b.rows > 1 && a.step == b.step && a.len <= a.step && b.len <= a.step) {
        const int64_t d = (int64_t)(b.at - a.at), off = ((d % a.step) + a.step) % a.step;  // b's piece in a's rows
        return off < a.len || off + b.len > a.step;
    }
    return true;
}
// An output that is the very matrix that an input is: each value is read before it is written, by the same thread.
bool same(const si_fp8_mat *a, const si_fp8_mat *b, int64_t T) {
    return a->data == b->data && (T <= 1 || a->row_stride == b->row_stride) && size_of(a->dtype) == size_of(b->dtype);
}

Mat make_mat(const si_fp8_mat *m) { return m ? Mat{m->data, m->row_stride, m->dtype} : Mat{nullptr, 0, 0}; }

int blocks_of(int64_t n) { return (int)((n + SI_FP8_BLOCK - 1) / SI_FP8_BLOCK); }

si_status check_q_rows(const si_fp8_rows *r, int32_t n_rows) {
    if (!r || (n_rows > 0 && (!r->codes || !r->scales))) return SI_ERR_INVALID_ARG;
    if (r->scale_stride < n_rows) return SI_ERR_INVALID_ARG;
    if (r->scale_stride > SI_FP8_MAX_ROWS) return SI_ERR_UNSUPPORTED;  // (the kernels number the scales in 32 bits)
    if (!aligned(r->codes, 16) || !aligned(r->scales, 16) || r->scale_stride % 4) return SI_ERR_MISALIGNED;
    return SI_OK;
}

si_status check_weight(const si_fp8_weight *w) {
    if (!w || !w->codes || !w->scales) return SI_ERR_INVALID_ARG;
    return aligned(w->codes, 16) && aligned(w->scales, 16) ? SI_OK : SI_ERR_MISALIGNED;
}

si_status launched(cudaError_t e) {
    if (e == cudaSuccess) return SI_OK;
    cudaGetLastError();
    return SI_ERR_CUDA;
}

}  // namespace

#define SI_FP8_TRY(x)                     \
    do {                                  \
        const si_status st_ = (x);        \
        if (st_ != SI_OK) return st_;     \
    } while (0)

extern "C" {

si_status si_fp8_plan(const si_fp8_desc *desc, int cuda_device, si_fp8_plan_t *out) {
    if (!out) return SI_ERR_INVALID_ARG;
    *out = nullptr;
    SI_FP8_TRY(validate_desc(desc));
    int sms = 0, khz = 0;
    if (!device_numbers(cuda_device, sms, khz)) {
        cudaGetLastError();
        return SI_ERR_CUDA;
    }
    si_fp8_plan_s *h = new (std::nothrow) si_fp8_plan_s();
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

void si_fp8_plan_destroy(si_fp8_plan_t plan) { delete plan; }

si_status si_fp8_scratch_bytes(si_fp8_plan_t plan, int32_t n_rows, size_t *bytes) {
    if (!plan || !bytes) return SI_ERR_INVALID_ARG;
    SI_FP8_TRY(check_rows_count(n_rows));
    *bytes = si::fp8::scratch_bytes(plan->p, n_rows);
    return SI_OK;
}

si_status si_fp8_scratch_init(si_fp8_plan_t plan, void *scratch, size_t scratch_bytes, si_stream_t stream) {
    if (!plan || !scratch) return SI_ERR_INVALID_ARG;
    if (!aligned(scratch, 16)) return SI_ERR_MISALIGNED;
    if (scratch_bytes < si::fp8::kCtrlBytes) return SI_ERR_SCRATCH_TOO_SMALL;
    SI_FP8_TRY(check_device(plan->p));
    return launched(cudaMemsetAsync(scratch, 0, si::fp8::kCtrlBytes, (cudaStream_t)stream));
}

si_status si_fp8_pack(si_fp8_plan_t plan, const si_fp8_mat *w, const si_fp8_weight *out, si_stream_t stream) {
    if (!plan || !w) return SI_ERR_INVALID_ARG;
    const int64_t N = plan->p.desc.out_features, K = plan->p.desc.in_features;
    SI_FP8_TRY(check_mat(w, N, K, false, true));
    SI_FP8_TRY(check_weight(out));
    const Span codes = span(out->codes, N * K), scales = span(out->scales, 4ll * blocks_of(N) * blocks_of(K));
    if (meet(codes, scales) || meet(codes, span(w, N, K)) || meet(scales, span(w, N, K))) return SI_ERR_INVALID_ARG;
    SI_FP8_TRY(check_device(plan->p));
    return launched(si::fp8::launch_pack(plan->p, make_mat(w), static_cast<uint8_t *>(out->codes), out->scales,
                                         (cudaStream_t)stream));
}

si_status si_fp8_norm(si_fp8_plan_t plan, const si_fp8_mat *x, const si_fp8_mat *residual, const float *gain, float eps,
                      const si_fp8_mat *residual_out, const si_fp8_mat *y, const si_fp8_rows *rows, int32_t n_rows,
                      si_stream_t stream) {
    if (!plan || !x || (!residual_out && !y && !rows)) return SI_ERR_INVALID_ARG;
    if (gain && (!(eps >= 0.0f) || !std::isfinite(eps))) return SI_ERR_INVALID_ARG;
    SI_FP8_TRY(check_rows_count(n_rows));
    const int64_t T = n_rows, K = plan->p.desc.in_features;
    SI_FP8_TRY(check_mat(x, T, K, false, true));
    if (residual) SI_FP8_TRY(check_mat(residual, T, K, false, true));
    if (residual_out) SI_FP8_TRY(check_mat(residual_out, T, K, true, true));
    if (y) SI_FP8_TRY(check_mat(y, T, K, true, true));
    if (rows) SI_FP8_TRY(check_q_rows(rows, n_rows));
    if (!aligned(gain, 16)) return SI_ERR_MISALIGNED;
    if (n_rows == 0) return SI_OK;
    // outputs meet neither one another nor, but as the very same matrix, an input
    Span outs[4];
    int n_out = 0;
    for (const si_fp8_mat *m : {residual_out, y}) {
        if (!m) continue;
        const Span s = span(m, T, K);
        for (const si_fp8_mat *in : {x, residual})
            if (in && !same(m, in, T) && meet(s, span(in, T, K))) return SI_ERR_INVALID_ARG;
        outs[n_out++] = s;
    }
    if (rows) {
        outs[n_out++] = span(rows->codes, T * K);
        outs[n_out++] = Span{reinterpret_cast<uintptr_t>(rows->scales), blocks_of(K), 4 * rows->scale_stride, 4 * T};
        for (const si_fp8_mat *in : {x, residual})
            if (in && (meet(outs[n_out - 2], span(in, T, K)) || meet(outs[n_out - 1], span(in, T, K)))) return SI_ERR_INVALID_ARG;
    }
    for (int i = 0; i < n_out; ++i) {
        if (gain && meet(outs[i], span(gain, 4 * K))) return SI_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (meet(outs[i], outs[j])) return SI_ERR_INVALID_ARG;
    }
    SI_FP8_TRY(check_device(plan->p));
    NormArgs a{};
    a.x = make_mat(x);
    a.residual = make_mat(residual);
    a.residual_out = make_mat(residual_out);
    a.y = make_mat(y);
    a.gain = gain;
    a.eps = eps;
    if (rows) {
        a.codes = static_cast<uint8_t *>(rows->codes);
        a.scales = rows->scales;
        a.scale_stride = rows->scale_stride;
    }
    a.T = n_rows;
    a.K = (int32_t)K;
    return launched(si::fp8::launch_norm(plan->p, a, (cudaStream_t)stream));
}

si_status si_fp8_matmul(si_fp8_plan_t plan, const si_fp8_rows *rows, const si_fp8_weight *weight, const si_fp8_mat *add,
                        const si_fp8_mat *out, int32_t n_rows, void *scratch, size_t scratch_bytes, si_stream_t stream) {
    if (!plan || !out) return SI_ERR_INVALID_ARG;
    SI_FP8_TRY(check_rows_count(n_rows));
    const int64_t T = n_rows, K = plan->p.desc.in_features, N = plan->p.desc.out_features;
    SI_FP8_TRY(check_q_rows(rows, n_rows));
    SI_FP8_TRY(check_weight(weight));
    SI_FP8_TRY(check_mat(out, T, N, true, false));
    if (add) SI_FP8_TRY(check_mat(add, T, N, false, false));
    if (!scratch) return SI_ERR_INVALID_ARG;
    if (!aligned(scratch, 16)) return SI_ERR_MISALIGNED;
    if (scratch_bytes < si::fp8::scratch_bytes(plan->p, n_rows)) return SI_ERR_SCRATCH_TOO_SMALL;
    if (n_rows == 0) return SI_OK;
    const Span o = span(out, T, N);
    const Span in[5] = {span(rows->codes, T * K),
                        Span{reinterpret_cast<uintptr_t>(rows->scales), blocks_of(K), 4 * rows->scale_stride, 4 * T},
                        span(weight->codes, N * K), span(weight->scales, 4ll * blocks_of(N) * blocks_of(K)),
                        span(scratch, (int64_t)std::min<size_t>(scratch_bytes, (size_t)1 << 40))};
    for (const Span &s : in)
        if (meet(o, s)) return SI_ERR_INVALID_ARG;
    // (add's very matrix: each value is read and then written by the same thread)
    if (add && !(same(out, add, T) && out->dtype == add->dtype) && meet(o, span(add, T, N))) return SI_ERR_INVALID_ARG;
    SI_FP8_TRY(check_device(plan->p));
    MatmulArgs a{};
    a.a = static_cast<const uint8_t *>(rows->codes);
    a.a_scale = rows->scales;
    a.a_stride = rows->scale_stride;
    a.w = static_cast<const uint8_t *>(weight->codes);
    a.w_scale = weight->scales;
    a.add = make_mat(add);
    a.out = make_mat(out);
    a.T = n_rows;
    a.N = (int32_t)N;
    a.K = (int32_t)K;
    a.KB = blocks_of(K);
    a.status = static_cast<int32_t *>(scratch);
    a.wait_budget = plan->p.wait_budget;
    a.fault_wait = plan->p.fault_wait;
    return launched(si::fp8::launch_matmul(plan->p, a, (cudaStream_t)stream));
}

si_status si_fp8_read_status(si_fp8_plan_t plan, const void *scratch, si_stream_t stream) {
    if (!plan || !scratch) return SI_ERR_INVALID_ARG;
    if (!aligned(scratch, 16)) return SI_ERR_MISALIGNED;
    SI_FP8_TRY(check_device(plan->p));
    int32_t word = 0;
    SI_FP8_TRY(launched(cudaStreamSynchronize((cudaStream_t)stream)));
    SI_FP8_TRY(launched(cudaMemcpy(&word, scratch, sizeof(word), cudaMemcpyDeviceToHost)));
    if (word == 0) return SI_OK;
    // (cleared in the stream's order: a call that follows in it may report at once)
    SI_FP8_TRY(launched(cudaMemsetAsync(const_cast<void *>(scratch), 0, sizeof(word), (cudaStream_t)stream)));
    return (si_status)word;
}

}  // extern "C"
