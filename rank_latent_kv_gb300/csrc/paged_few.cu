// Attention over the paged cache for few rows a KV head, of the prefix as of own
// units: one line.
#include "paged_few.cuh"

namespace palu {

template <bool BF16, int NT>
__global__ void __launch_bounds__(kFewThreads, 1)
    paged_few_kernel(const AttnParams p, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ PlanScratch plan;
  uint8_t* smem = few_smem(smem_raw);
  grid_dep_launch();
  if (threadIdx.x == 0) few_init(few_shared(smem));
  plan_start<8 * NT, 8 * NT, kFewThreads>(p, &plan, threadIdx.x);  // all threads meet in it
  few_stretch<BF16, NT, false>(p, p.part, kmap, vmap, plan, smem);
}

template <bool BF16>
static palu_status launch_type(const AttnParams& p, const CUtensorMap& km, const CUtensorMap& vm, cudaStream_t s) {
  return p.part.R == 8 ? launch(paged_few_kernel<BF16, 1>, device_sm_count(), kFewThreads, kFewSmemBytes, false, s,
                                "paged_few_kernel launch", p, km, vm)
                       : launch(paged_few_kernel<BF16, 2>, device_sm_count(), kFewThreads, kFewSmemBytes, false, s,
                                "paged_few_kernel launch", p, km, vm);
}

palu_status launch_few(const AttnParams& p, const CUtensorMap& km, const CUtensorMap& vm, bool bf16, cudaStream_t stream) {
  return bf16 ? launch_type<true>(p, km, vm, stream) : launch_type<false>(p, km, vm, stream);
}

}  // namespace palu
