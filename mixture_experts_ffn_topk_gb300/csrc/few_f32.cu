// few_f32.cu -- the layer for a few tokens, F32 activations.
#include "few.cuh"

namespace moe {

cudaError_t launch_few_f32(const FewArgs &a, cudaStream_t s) { return launch_few_form<DT_F32, false>(a, s); }

}  // namespace moe
