// Attention over the paged cache for many rows a KV head: prefix and own units
// of more than 16 rows, one line.
#include "paged_many.cuh"

namespace palu {

template <bool BF16>
__global__ void __launch_bounds__(kManyThreads, 1)
    paged_many_kernel(const AttnParams p, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ PlanScratch plan;
  grid_dep_launch();
  many_stretch<BF16, false, false>(p, p.part, &kmap, &vmap, plan, many_smem(smem_raw),
                     [&] { plan_start<kManyRows, kManyRows, kManyThreads - 256>(p, &plan, threadIdx.x - 256); });
}

palu_status launch_many(const AttnParams& p, const CUtensorMap& km, const CUtensorMap& vm, bool bf16, cudaStream_t stream) {
  return bf16 ? launch(paged_many_kernel<true>, device_sm_count(), kManyThreads, kManySmemBytes, false, stream,
                       "paged_many_kernel launch", p, km, vm)
              : launch(paged_many_kernel<false>, device_sm_count(), kManyThreads, kManySmemBytes, false, stream,
                       "paged_many_kernel launch", p, km, vm);
}

}  // namespace palu
