// si_kv_prompt_int8.cu -- the many-row attention kernel over int8 codes.
#include "si_kv_prompt.cuh"

namespace si {
namespace kv {

cudaError_t launch_prompt_int8(const Plan &p, const PromptArgs &a, cudaStream_t s) {
    return p.desc.head_dim == 64 ? prompt_launch<SI_KV_INT8, 64>(p, a, s) : prompt_launch<SI_KV_INT8, 128>(p, a, s);
}

}  // namespace kv
}  // namespace si
