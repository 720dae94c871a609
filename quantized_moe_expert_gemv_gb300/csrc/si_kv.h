// si_kv.h -- the attention block's internals: the plan, the scratch layout,
// the arguments every kernel gets, and the launchers.
#pragma once
#include <atomic>
#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/si_kv.h"

namespace si {
namespace kv {

// Scratch: control words (the status first), then arrival counters of the
// attention's split rows (one for each CTA; the last to arrive puts its counter
// back to zero), then partial results.
constexpr int kCtrlWords = 64;
constexpr int kCounters = 4096;
constexpr size_t kCtrlBytes = (kCtrlWords + kCounters) * sizeof(int32_t);

struct Plan {
    si_kv_desc desc;
    int device;
    int sm_count;
    long long wait_budget;  // SM cycles a device-side wait may spin before reporting SI_ERR_TIMEOUT
    bool fault_wait;        // test mode: the many-row attention first waits on a barrier nothing arrives at
};

// What every kernel knows of the cache and the call.
struct Ctx {
    uint8_t *kc, *vc;
    float *ks, *vs;
    uint16_t *kt, *vt;
    const int32_t *q_start, *lens, *table, *slots;
    int32_t *status;
    int64_t n_pages;
    int32_t n_slots, table_stride;
    int32_t B, T, max_new, max_len;
    int32_t H, Hk, G, D, P;
};

struct Rows {
    uint16_t *p;
    int64_t row, head;  // strides in elements
};

// Allow kernel F `smem` bytes of dynamic shared memory on the current device (the one that a launch goes to,
// whatever the plan's is), once a device: F and smem are the caller's constants, and the attribute stays with
// the function.
template <auto F>
cudaError_t allow_smem(int smem) {
    static std::atomic<unsigned long long> done{0};
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = device < 64 ? 1ull << device : 0;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(reinterpret_cast<const void *>(F), cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// Launch with programmatic dependent launch: the kernel may start while the one
// before it in the stream ends, and every kernel here waits for that one's end
// (start_after) before it touches global memory.
template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, A... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

size_t scratch_bytes(const Plan &p, int n_seqs, int total_new, int max_new, int max_len);

cudaError_t launch_append(const Plan &p, const Ctx &c, Rows k, Rows v, int32_t *lens_out, cudaStream_t s);
cudaError_t launch_read(const Plan &p, const Ctx &c, const int32_t *pages, int n, uint16_t *k_out, uint16_t *v_out,
                        cudaStream_t s);
cudaError_t launch_attend(const Plan &p, const Ctx &c, Rows q, Rows out, float *lse, float sm_scale, void *scratch,
                          cudaStream_t s);
cudaError_t launch_weigh(const Plan &p, const Ctx &c, Rows q, const float *lse, const float *acc_in, float *acc_out,
                         int64_t acc_stride, float decay, float sm_scale, cudaStream_t s);
cudaError_t launch_evict(const Plan &p, const Ctx &c, const float *acc_in, float *acc_out, int64_t acc_stride,
                         int budget, int sink, int recent, const int32_t *new_table, const int32_t *new_slots,
                         int32_t *keep, int32_t *lens_out, cudaStream_t s);

}  // namespace kv
}  // namespace si
