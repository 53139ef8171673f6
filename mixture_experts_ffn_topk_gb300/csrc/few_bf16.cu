// few_bf16.cu -- the layer for a few tokens, BF16 activations.
#include "few.cuh"

namespace moe {

cudaError_t launch_few_bf16(const FewArgs &a, cudaStream_t s)
{
    return a.gate_scales != nullptr ? launch_few_form<DT_BF16, true>(a, s) : launch_few_form<DT_BF16, false>(a, s);
}

}  // namespace moe
