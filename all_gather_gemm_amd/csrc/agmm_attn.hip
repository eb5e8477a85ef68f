// The kernels of the attention of one new token: agmm_attn_kernel.h.
#include "agmm_attn_kernel.h"

namespace agmm {

hipError_t launch_attn(const AttnParams& p, int dtype, int storage, int grid, hipStream_t s) {
  if (dtype == AGMM_F16)
    by_storage<AGMM_F16, kPlain>(p, storage, grid, s);
  else
    by_storage<AGMM_BF16, kPlain>(p, storage, grid, s);
  return hipGetLastError();
}

}  // namespace agmm
