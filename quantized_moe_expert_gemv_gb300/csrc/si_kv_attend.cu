// si_kv_attend.cu -- causal attention over the cache.
#include "si_kv_device.cuh"

namespace si {
namespace kv {

size_t scratch_bytes(const Plan &, int, int, int, int) { return kCtrlBytes; }

constexpr int kThreads = 128;

// One CTA for each (row, query head); tiles of 128 tokens, a thread a token for the scores and a
// thread a dimension (or two) for the sums; running maximum and sum.
template <int CODE, int DT>
__global__ void __launch_bounds__(kThreads) k_kv_attend(Ctx c, Rows q, Rows out, float *lse, float sm) {
    __shared__ float s_q[256], s_p[kThreads], s_red[4];
    const int i = blockIdx.x, head = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
    const Seq s = load_seq(c, b);
    if (i >= s.n) return;
    const int h = head / c.G, D = c.D, P = c.P, row = s.row0 + i;
    const int see = s.len - s.n + i + 1, paged = s.len / P * P;
    for (int d = tid; d < D; d += kThreads) s_q[d] = to_float<DT>(q.p[row * q.row + head * q.head + d]);
    __syncthreads();
    float m = -INFINITY, l = 0.0f, o[2] = {0.0f, 0.0f};
    for (int t0 = 0; t0 < see; t0 += kThreads) {
        const int t = t0 + tid;
        float z = -INFINITY;
        if (t < see) {
            float dot = 0.0f;
            if (t < paged) {
                const int64_t page = load_page(c, b, t / P);
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
            z = dot * sm;
        }
        float top = z;
        for (int k = 16; k; k >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, k));
        if ((tid & 31) == 0) s_red[tid >> 5] = top;
        __syncthreads();
        const float m2 = fmaxf(m, fmaxf(fmaxf(s_red[0], s_red[1]), fmaxf(s_red[2], s_red[3])));
        const float keep = m == -INFINITY ? 0.0f : expf(m - m2);
        s_p[tid] = t < see ? expf(z - m2) : 0.0f;
        m = m2;
        __syncthreads();
        l *= keep;
        o[0] *= keep;
        o[1] *= keep;
        const int n = min(kThreads, see - t0);
        for (int k = 0; k < n; ++k) {
            const int u = t0 + k;
            const float p = s_p[k];
            l += p;
            for (int e = 0; e < 2; ++e) {
                const int d = tid + e * kThreads;
                if (d >= D) break;
                float v = NAN;
                if (u < paged) {
                    const int64_t page = load_page(c, b, u / P);
                    if (page >= 0) v = code_value<CODE>(c.vc[page_at(c, page, h) + (int64_t)(u % P) * D + d]) * c.vs[page * c.Hk + h];
                } else if (s.slot >= 0) v = to_float<DT>(c.vt[ring_at(c, s.slot, h, u) + d]);
                o[e] = fmaf(p, v, o[e]);
            }
        }
        __syncthreads();
    }
    for (int e = 0; e < 2; ++e) {
        const int d = tid + e * kThreads;
        if (d < D) out.p[row * out.row + head * out.head + d] = from_float<DT>(see > 0 ? o[e] / l : 0.0f);
    }
    if (lse && tid == 0) lse[(int64_t)row * c.H + head] = see > 0 ? m + logf(l) : -INFINITY;
}

cudaError_t launch_attend(const Plan &p, const Ctx &c, Rows q, Rows out, float *lse, float sm, void *, cudaStream_t s) {
    const dim3 grid(c.max_new, c.H, c.B);
    if (p.desc.code == SI_KV_INT8) {
        if (p.desc.dtype == SI_KV_BF16) k_kv_attend<SI_KV_INT8, SI_KV_BF16><<<grid, kThreads, 0, s>>>(c, q, out, lse, sm);
        else k_kv_attend<SI_KV_INT8, SI_KV_F16><<<grid, kThreads, 0, s>>>(c, q, out, lse, sm);
    } else {
        if (p.desc.dtype == SI_KV_BF16) k_kv_attend<SI_KV_E4M3, SI_KV_BF16><<<grid, kThreads, 0, s>>>(c, q, out, lse, sm);
        else k_kv_attend<SI_KV_E4M3, SI_KV_F16><<<grid, kThreads, 0, s>>>(c, q, out, lse, sm);
    }
    return cudaGetLastError();
}

}  // namespace kv
}  // namespace si
