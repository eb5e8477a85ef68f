// The kernels of agmm_prefix_kernel.h for bf16.
#include "agmm_prefix_kernel.h"

namespace agmm {

hipError_t launch_prefix_bf16(const PrefixParams& p, int storage, int grid, hipStream_t s) {
  return prefix_by_storage<AGMM_BF16>(p, storage, grid, s);
}

}  // namespace agmm
