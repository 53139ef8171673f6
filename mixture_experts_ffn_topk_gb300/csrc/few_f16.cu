// few_f16.cu -- the layer for a few tokens, F16 activations.
#include "few.cuh"

namespace moe {

cudaError_t launch_few_f16(const FewArgs &a, cudaStream_t s)
{
    return a.gate_scales != nullptr ? launch_few_form<DT_F16, true>(a, s) : launch_few_form<DT_F16, false>(a, s);
}

}  // namespace moe
