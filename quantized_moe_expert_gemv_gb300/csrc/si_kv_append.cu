// si_kv_append.cu -- writing the cache (append) and reading pages back.
//
// Append.  One CTA for each (sequence, page that the call completes, kv head, K
// or V).  A page is complete when its last token has come, so its amax over
// P*D values is taken once, from values that the CTA holds in registers:
// each element is read once and each code written once.
//   scale = amax / Q,  code = round(x * fp32(Q / amax))
// The CTA of a sequence's first page also writes the ring (the new rows of the
// unfinished page and of the page before): the ring place of the unfinished
// page may be the one that the first page's old rows lie in (a call of more
// than one page), so these writes come after that CTA's own reads, and no
// other CTA reads the ring.
// Bound: HBM (2 bytes in, 1 byte out for each value of a completed page); a
// decode step completes few pages and is bound by latency (9 us with the launch
// from Python).  Maxima and conversions are packed, four values an instruction or
// two: with one value at a time the issue slots bounded it (74 us for what takes 56).
// Measured: 5 prompts of 1500 to 7000 tokens, 8 heads of 128, then their pages read back,
// 56 us together, 80 % of the copy rate.
#include "si_kv_mma.cuh"

namespace si {
namespace kv {

constexpr int kAppendThreads = 256;

// UN: units of 16 values that a thread holds of one page's P*D values; PG: pages of a CTA (their loads are
// under way together: with one page of 8 KB a CTA, the chain of loads, maximum and stores reached 4 TB/s).
template <int CODE, int DT, int UN, int PG>
__global__ void __launch_bounds__(kAppendThreads) k_kv_append(Ctx c, Rows k, Rows v, int32_t *lens_out) {
    __shared__ float s_max[PG][kAppendThreads / 32];
    start_after();
    const int j = blockIdx.x * PG, h = blockIdx.y >> 1, b = blockIdx.z;
    const bool is_v = blockIdx.y & 1;
    const int tid = threadIdx.x;
    Seq s = load_seq(c, b);
    if ((int64_t)s.len + s.n > c.max_len) {  // the new tokens do not fit the host's bound
        if (tid == 0) set_status(c.status, SI_ERR_DEVICE);
        s.n = 0;
    }
    if (s.slot < 0) s.n = 0;
    if (j == 0 && blockIdx.y == 0 && tid == 0) lens_out[b] = s.len + s.n;
    if (s.n == 0) return;
    const int P = c.P, D = c.D;
    const int first = s.len / P, last = (s.len + s.n) / P;
    const int count = min(PG, last - first - j);  // pages to quantise here
    if (count <= 0 && j > 0) return;
    const Rows in = is_v ? v : k;
    uint16_t *ring = is_v ? c.vt : c.kt;
    const int upr = D / 16;  // units in a row

    if (count > 0) {
        uint4 x[PG][UN][2];
        int64_t dst[PG];
#pragma unroll
        for (int g = 0; g < PG; ++g) dst[g] = g < count ? load_page(c, b, first + j + g) : -1;
#pragma unroll
        for (int g = 0; g < PG; ++g)
#pragma unroll
            for (int u = 0; u < UN; ++u) {
                const int unit = u * kAppendThreads + tid;
                x[g][u][0] = x[g][u][1] = make_uint4(0, 0, 0, 0);
                if (g < count && unit < P * upr) {
                    const int t = (first + j + g) * P + unit / upr, d = unit % upr * 16;
                    const uint16_t *src = t < s.len ? ring + ring_at(c, s.slot, h, t) + d
                                                    : in.p + (int64_t)(s.row0 + t - s.len) * in.row + h * in.head + d;
                    x[g][u][0] = *reinterpret_cast<const uint4 *>(src);
                    x[g][u][1] = *reinterpret_cast<const uint4 *>(src + 8);
                }
            }
#pragma unroll
        for (int g = 0; g < PG; ++g) {
            float amax = 0.0f;  // (infinite where a value is not finite)
#pragma unroll
            for (int u = 0; u < UN; ++u)
                amax = fmaxf(amax, fmaxf(amax8(x[g][u][0], DT == SI_KV_BF16), amax8(x[g][u][1], DT == SI_KV_BF16)));
            for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            if ((tid & 31) == 0) s_max[g][tid >> 5] = amax;
        }
        __syncthreads();
#pragma unroll
        for (int g = 0; g < PG; ++g) {
            if (dst[g] < 0) continue;
            float amax = s_max[g][0];
#pragma unroll
            for (int i = 1; i < kAppendThreads / 32; ++i) amax = fmaxf(amax, s_max[g][i]);
            const float Q = CODE == SI_KV_INT8 ? kQInt8 : kQE4m3;
            const bool live = amax >= 0x1p-100f && amax <= 3.4e38f;
            const float inv = live ? __fdiv_rn(Q, amax) : 0.0f;
            const float scale = amax > 3.4e38f ? __int_as_float(0x7fc00000) : live ? __fdiv_rn(amax, Q) : 0.0f;
            if (tid == 0) (is_v ? c.vs : c.ks)[dst[g] * c.Hk + h] = scale;
            uint8_t *codes = (is_v ? c.vc : c.kc) + page_at(c, dst[g], h);
#pragma unroll
            for (int u = 0; u < UN; ++u) {
                const int unit = u * kAppendThreads + tid;
                if (unit >= P * upr) continue;
                uint4 o = make_uint4(0, 0, 0, 0);
                if (live) {
                    o.x = to_codes<CODE, DT>(x[g][u][0].x, x[g][u][0].y, inv);
                    o.y = to_codes<CODE, DT>(x[g][u][0].z, x[g][u][0].w, inv);
                    o.z = to_codes<CODE, DT>(x[g][u][1].x, x[g][u][1].y, inv);
                    o.w = to_codes<CODE, DT>(x[g][u][1].z, x[g][u][1].w, inv);
                }
                *reinterpret_cast<uint4 *>(codes + (int64_t)unit * 16) = o;
            }
        }
    }
    if (j > 0) return;
    __syncthreads();  // every old row of the ring has been read
    const int from = max(s.len, (last - 1) * P), rows = s.len + s.n - from;
    for (int unit = tid; unit < rows * upr; unit += kAppendThreads) {
        const int t = from + unit / upr, d = unit % upr * 16;
        const uint16_t *src = in.p + (int64_t)(s.row0 + t - s.len) * in.row + h * in.head + d;
        uint16_t *to = ring + ring_at(c, s.slot, h, t) + d;
        *reinterpret_cast<uint4 *>(to) = *reinterpret_cast<const uint4 *>(src);
        *reinterpret_cast<uint4 *>(to + 8) = *reinterpret_cast<const uint4 *>(src + 8);
    }
}

template <int CODE, int DT>
static cudaError_t append_units(const Ctx &c, Rows k, Rows v, int32_t *lens_out, cudaStream_t s) {
    // a call of n rows completes at most (P - 1 + n) / P pages of a sequence
    // (the bound on n may be any number: the tokens have to fit max_len too)
    const int pages = max(1, (c.P - 1 + min(c.max_new, c.max_len)) / c.P);
    const int units = c.P * c.D / 16;
    const bool many = pages >= 8;  // a prompt: several pages a CTA (a step has one page at most, and the fewest registers)
    auto go = [&](auto kernel, int pg) {
        return launch(kernel, dim3((pages + pg - 1) / pg, 2 * c.Hk, c.B), kAppendThreads, 0, s, c, k, v, lens_out);
    };
    if (units <= kAppendThreads) return many ? go(k_kv_append<CODE, DT, 1, 4>, 4) : go(k_kv_append<CODE, DT, 1, 1>, 1);
    if (units <= 2 * kAppendThreads) return many ? go(k_kv_append<CODE, DT, 2, 2>, 2) : go(k_kv_append<CODE, DT, 2, 1>, 1);
    return go(k_kv_append<CODE, DT, 4, 1>, 1);
}

cudaError_t launch_append(const Plan &p, const Ctx &c, Rows k, Rows v, int32_t *lens_out, cudaStream_t s) {
    if (p.desc.code == SI_KV_INT8)
        return p.desc.dtype == SI_KV_BF16 ? append_units<SI_KV_INT8, SI_KV_BF16>(c, k, v, lens_out, s)
                                          : append_units<SI_KV_INT8, SI_KV_F16>(c, k, v, lens_out, s);
    return p.desc.dtype == SI_KV_BF16 ? append_units<SI_KV_E4M3, SI_KV_BF16>(c, k, v, lens_out, s)
                                      : append_units<SI_KV_E4M3, SI_KV_F16>(c, k, v, lens_out, s);
}

// Read: a thread takes 16 codes of K and the same 16 of V; bound by HBM (1 byte
// in, 2 bytes out for each value).
constexpr int kReadThreads = 256;

template <int CODE, int DT>
__global__ void __launch_bounds__(kReadThreads) k_kv_read(Ctx c, const int32_t *pages, int64_t units, uint16_t *k_out,
                                                          uint16_t *v_out) {
    start_after();
    const int64_t unit = (int64_t)blockIdx.x * kReadThreads + threadIdx.x;  // of 16 values, in the output's order
    if (unit >= units) return;
    const int per = c.P * c.D / 16;
    const int64_t ph = unit / per;
    const int i = (int)(ph / c.Hk), h = (int)(ph % c.Hk);
    const int page = pages[i];
    const bool ok = page >= 0 && page < c.n_pages;
    if (!ok) set_status(c.status, SI_ERR_DEVICE);
    const int64_t at = page_at(c, ok ? page : 0, h) + (unit % per) * 16;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        const float nan = __int_as_float(0x7fc00000);
        const float scale = ok ? (which ? c.vs : c.ks)[(int64_t)page * c.Hk + h] : nan;
        const uint4 x = *reinterpret_cast<const uint4 *>((which ? c.vc : c.kc) + at);
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
        uint32_t o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t two = w[e >> 1] >> (16 * (e & 1));
            o[e] = pack2<DT>(code_value<CODE>((uint8_t)two) * scale, code_value<CODE>((uint8_t)(two >> 8)) * scale);
        }
        uint4 *to = reinterpret_cast<uint4 *>((which ? v_out : k_out) + unit * 16);
        to[0] = make_uint4(o[0], o[1], o[2], o[3]);
        to[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
}

cudaError_t launch_read(const Plan &p, const Ctx &c, const int32_t *pages, int n, uint16_t *k_out, uint16_t *v_out,
                        cudaStream_t s) {
    const int64_t units = (int64_t)n * c.Hk * c.P * c.D / 16;
    const int64_t grid = (units + kReadThreads - 1) / kReadThreads;
    if (grid > INT32_MAX) return cudaErrorInvalidConfiguration;
    auto go = [&](auto kernel) { return launch(kernel, dim3((unsigned)grid), kReadThreads, 0, s, c, pages, units, k_out, v_out); };
    const bool bf16 = p.desc.dtype == SI_KV_BF16;
    if (p.desc.code == SI_KV_INT8) return bf16 ? go(k_kv_read<SI_KV_INT8, SI_KV_BF16>) : go(k_kv_read<SI_KV_INT8, SI_KV_F16>);
    return bf16 ? go(k_kv_read<SI_KV_E4M3, SI_KV_BF16>) : go(k_kv_read<SI_KV_E4M3, SI_KV_F16>);
}

}  // namespace kv
}  // namespace si
