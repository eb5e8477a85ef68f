// The kernels of the attention of one new token: agmm_attn_kernel.h, with a page table for each kv head.
#include "agmm_attn_kernel.h"

namespace agmm {

hipError_t launch_attn_heads(const AttnParams& p, int dtype, int storage, int grid, hipStream_t s) {
  if (dtype == AGMM_F16)
    by_storage<AGMM_F16, kHeads>(p, storage, grid, s);
  else
    by_storage<AGMM_BF16, kHeads>(p, storage, grid, s);
  return hipGetLastError();
}

}  // namespace agmm
