// si_kv_weigh.cu -- the attention weights of each cached token, added to its running sum.
#include "si_kv_device.cuh"

namespace si {
namespace kv {

constexpr int kThreads = 128;

// One CTA for each (sequence, kv head, 128 tokens), a thread a token, the rows one after the other.
template <int CODE, int DT>
__global__ void __launch_bounds__(kThreads) k_kv_weigh(Ctx c, Rows q, const float *lse, const float *acc_in,
                                                       float *acc_out, int64_t acc_stride, float decay, float sm) {
    __shared__ float s_q[256];
    const int h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x, D = c.D, P = c.P;
    const Seq s = load_seq(c, b);
    const int t = blockIdx.x * kThreads + tid;
    if (blockIdx.x * kThreads >= s.len) return;
    const bool live = t < s.len;
    const int old = s.len - s.n, paged = s.len / P * P;
    const int64_t page = live && t < paged ? load_page(c, b, t / P) : -1;
    float sum = 0.0f;
    for (int i = 0; i < s.n; ++i)
        for (int g = 0; g < c.G; ++g) {
            const int head = h * c.G + g, row = s.row0 + i;
            __syncthreads();
            for (int d = tid; d < D; d += kThreads) s_q[d] = to_float<DT>(q.p[row * q.row + head * q.head + d]);
            __syncthreads();
            if (!live || t > old + i) continue;
            float dot = 0.0f;
            if (t < paged) {
                if (page < 0) dot = NAN;
                else {
                    const uint8_t *k = c.kc + page_at(c, page, h) + (int64_t)(t % P) * D;
                    for (int d = 0; d < D; ++d) dot = fmaf(s_q[d], code_value<CODE>(k[d]), dot);
                    dot *= c.ks[page * c.Hk + h];
                }
            } else if (s.slot < 0) dot = NAN;
            else {
                const uint16_t *k = c.kt + ring_at(c, s.slot, h, t);
                for (int d = 0; d < D; ++d) dot = fmaf(s_q[d], to_float<DT>(k[d]), dot);
            }
            sum += expf(dot * sm - lse[(int64_t)row * c.H + head]);
        }
    if (!live) return;
    const int64_t at = ((int64_t)b * c.Hk + h) * acc_stride + t;
    acc_out[at] = (acc_in && t < old ? decay * acc_in[at] : 0.0f) + sum;
}

cudaError_t launch_weigh(const Plan &p, const Ctx &c, Rows q, const float *lse, const float *acc_in, float *acc_out,
                         int64_t acc_stride, float decay, float sm, cudaStream_t s) {
    const dim3 grid((c.max_len + kThreads - 1) / kThreads, c.Hk, c.B);
    if (p.desc.code == SI_KV_INT8) {
        if (p.desc.dtype == SI_KV_BF16) k_kv_weigh<SI_KV_INT8, SI_KV_BF16><<<grid, kThreads, 0, s>>>(c, q, lse, acc_in, acc_out, acc_stride, decay, sm);
        else k_kv_weigh<SI_KV_INT8, SI_KV_F16><<<grid, kThreads, 0, s>>>(c, q, lse, acc_in, acc_out, acc_stride, decay, sm);
    } else {
        if (p.desc.dtype == SI_KV_BF16) k_kv_weigh<SI_KV_E4M3, SI_KV_BF16><<<grid, kThreads, 0, s>>>(c, q, lse, acc_in, acc_out, acc_stride, decay, sm);
        else k_kv_weigh<SI_KV_E4M3, SI_KV_F16><<<grid, kThreads, 0, s>>>(c, q, lse, acc_in, acc_out, acc_stride, decay, sm);
    }
    return cudaGetLastError();
}

}  // namespace kv
}  // namespace si
