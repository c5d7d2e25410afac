// grouped_forward.cu -- the GROUPED_FORWARD form of the grouped product.
#include "kernel_grouped.cuh"
#include "kernel_grouped_pair.cuh"

namespace tg {

template cudaError_t launch_grouped_op<GROUPED_FORWARD>(const GroupedSpec&, cudaStream_t);

}  // namespace tg
