// Attention over the 4-bit paged cache for many rows a KV head: prefix and own
// units of more than 16 rows, one line.
#include "paged_many.cuh"

namespace palu {

template <bool BF16>
__global__ void __launch_bounds__(kMany4Threads, 1) paged4_many_kernel(const AttnParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ PlanScratch plan;
  grid_dep_launch();
  many_stretch<BF16, false, true>(p, p.part, nullptr, nullptr, plan, many_smem(smem_raw), [&] {
    plan_start<kManyRows, kManyRows, kMany4Threads - 256, true>(p, &plan, threadIdx.x - 256);
  });
}

palu_status launch_many4(const AttnParams& p, bool bf16, cudaStream_t stream) {
  return bf16 ? launch(paged4_many_kernel<true>, device_sm_count(), kMany4Threads, kMany4SmemBytes, false, stream,
                       "paged4_many_kernel launch", p)
              : launch(paged4_many_kernel<false>, device_sm_count(), kMany4Threads, kMany4SmemBytes, false, stream,
                       "paged4_many_kernel launch", p);
}

}  // namespace palu
