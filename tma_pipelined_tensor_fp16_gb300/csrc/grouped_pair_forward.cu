// grouped_pair_forward.cu -- the GROUPED_FORWARD form of the grouped product on CTA pairs.
#include "kernel_grouped_pair.cuh"

namespace tg {

template cudaError_t launch_grouped_pair<GROUPED_FORWARD>(const GroupedSpec&, cudaStream_t);

}  // namespace tg
