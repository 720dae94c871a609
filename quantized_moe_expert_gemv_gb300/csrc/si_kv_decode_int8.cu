// si_kv_decode_int8.cu -- the few-row attention kernel over int8 codes.
#include "si_kv_decode.cuh"

namespace si {
namespace kv {

cudaError_t launch_decode_int8(const Plan &p, const DecodeArgs &a, int mt, cudaStream_t s) {
    switch (p.desc.head_dim) {
        case 64: return mt == 1 ? decode_launch<SI_KV_INT8, 64, 1>(p, a, s) : decode_launch<SI_KV_INT8, 64, 2>(p, a, s);
        case 128: return mt == 1 ? decode_launch<SI_KV_INT8, 128, 1>(p, a, s) : decode_launch<SI_KV_INT8, 128, 2>(p, a, s);
        default: return decode_launch<SI_KV_INT8, 256, 1>(p, a, s);
    }
}

}  // namespace kv
}  // namespace si
