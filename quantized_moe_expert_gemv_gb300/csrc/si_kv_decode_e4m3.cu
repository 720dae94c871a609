// si_kv_decode_e4m3.cu -- the few-row attention kernel over e4m3 codes.
#include "si_kv_decode.cuh"

namespace si {
namespace kv {

cudaError_t launch_decode_e4m3(const Plan &p, const DecodeArgs &a, int mt, cudaStream_t s) {
    switch (p.desc.head_dim) {
        case 64: return mt == 1 ? decode_launch<SI_KV_E4M3, 64, 1>(p, a, s) : decode_launch<SI_KV_E4M3, 64, 2>(p, a, s);
        case 128: return mt == 1 ? decode_launch<SI_KV_E4M3, 128, 1>(p, a, s) : decode_launch<SI_KV_E4M3, 128, 2>(p, a, s);
        default: return decode_launch<SI_KV_E4M3, 256, 1>(p, a, s);
    }
}

}  // namespace kv
}  // namespace si
