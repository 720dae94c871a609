// si_kv_prompt_e4m3.cu -- the many-row attention kernel over e4m3 codes.
#include "si_kv_prompt.cuh"

namespace si {
namespace kv {

cudaError_t launch_prompt_e4m3(const Plan &p, const PromptArgs &a, cudaStream_t s) {
    return p.desc.head_dim == 64 ? prompt_launch<SI_KV_E4M3, 64>(p, a, s) : prompt_launch<SI_KV_E4M3, 128>(p, a, s);
}

}  // namespace kv
}  // namespace si
