// grouped_pair_grad_weight.cu -- the GROUPED_GRAD_WEIGHT form of the grouped product on CTA pairs.
#include "kernel_grouped_pair.cuh"

namespace tg {

template cudaError_t launch_grouped_pair<GROUPED_GRAD_WEIGHT>(const GroupedSpec&, cudaStream_t);

}  // namespace tg
