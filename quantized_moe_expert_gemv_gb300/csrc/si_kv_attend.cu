// si_kv_attend.cu -- which kernel a call of si_kv_attend takes, and the scratch it needs.
#include "si_kv_decode.cuh"

namespace si {
namespace kv {

cudaError_t launch_decode_int8(const Plan &p, const DecodeArgs &a, int mt, cudaStream_t s);
cudaError_t launch_decode_e4m3(const Plan &p, const DecodeArgs &a, int mt, cudaStream_t s);

// Row groups of 16 (one group for a decode step) or 32 rows.
static int row_tiles(const Plan &p, int max_new) {
    const int64_t rows = (int64_t)max_new * (p.desc.n_heads / p.desc.n_kv_heads);
    return rows > 16 && p.desc.head_dim <= 128 ? 2 : 1;
}
static int decode_ctas(const Plan &p, int mt) {
    const int D = p.desc.head_dim;
    return p.sm_count * (D == 256 ? DecodeCfg<256, 1>::ctas
                                  : D == 128 ? (mt == 1 ? DecodeCfg<128, 1>::ctas : DecodeCfg<128, 2>::ctas)
                                             : (mt == 1 ? DecodeCfg<64, 1>::ctas : DecodeCfg<64, 2>::ctas));
}

size_t scratch_bytes(const Plan &p, int, int, int, int) {
    size_t most = 0;
    for (int mt = 1; mt <= 2; ++mt) {
        const size_t n = (size_t)decode_ctas(p, mt) * 2 * (size_t)partial_floats(16 * mt, p.desc.head_dim) * sizeof(float);
        most = n > most ? n : most;
    }
    return kCtrlBytes + most;
}

cudaError_t launch_attend(const Plan &p, const Ctx &c, Rows q, Rows out, float *lse, float sm, void *scratch, cudaStream_t s) {
    DecodeArgs a{};
    a.c = c;
    a.q = q;
    a.out = out;
    a.lse = lse;
    a.scale2 = sm * kLog2e;
    a.bf16 = p.desc.dtype == SI_KV_BF16;
    a.log_page = p.desc.page_tokens == 16 ? 4 : p.desc.page_tokens == 32 ? 5 : 6;
    a.counters = static_cast<int32_t *>(scratch) + kCtrlWords;
    a.partial = reinterpret_cast<float *>(static_cast<uint8_t *>(scratch) + kCtrlBytes);
    const int mt = row_tiles(p, c.max_new);
    return p.desc.code == SI_KV_INT8 ? launch_decode_int8(p, a, mt, s) : launch_decode_e4m3(p, a, mt, s);
}

}  // namespace kv
}  // namespace si
