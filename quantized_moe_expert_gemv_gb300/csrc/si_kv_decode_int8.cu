// si_kv_decode_int8.cu -- the few-row attention kernel over int8 codes.
#include "si_kv_decode.cuh"

namespace si {
namespace kv {

template <int D>
static cudaError_t by_rows(const Plan &p, const DecodeArgs &a, int r8, cudaStream_t s) {
    if (r8 == 1) return decode_launch<SI_KV_INT8, D, 1>(p, a, s);
    if constexpr (D <= 128)
        if (r8 == 4) return decode_launch<SI_KV_INT8, D, 4>(p, a, s);
    return decode_launch<SI_KV_INT8, D, 2>(p, a, s);
}

cudaError_t launch_decode_int8(const Plan &p, const DecodeArgs &a, int r8, cudaStream_t s) {
    switch (p.desc.head_dim) {
        case 64: return by_rows<64>(p, a, r8, s);
        case 128: return by_rows<128>(p, a, r8, s);
        default: return by_rows<256>(p, a, r8, s);
    }
}

}  // namespace kv
}  // namespace si
