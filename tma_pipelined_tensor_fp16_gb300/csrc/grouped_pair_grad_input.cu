// grouped_pair_grad_input.cu -- the GROUPED_GRAD_INPUT form of the grouped product on CTA pairs.
#include "kernel_grouped_pair.cuh"

namespace tg {

template cudaError_t launch_grouped_pair<GROUPED_GRAD_INPUT>(const GroupedSpec&, cudaStream_t);

}  // namespace tg
