// Attention over the 4-bit paged cache for few rows a KV head, of the prefix as
// of own units: one line.
#include "paged4_few.cuh"

namespace palu {

template <bool BF16, int NT>
__global__ void __launch_bounds__(kFew4Threads<NT>, 1) paged4_few_kernel(const AttnParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ PlanScratch plan;
  uint8_t* smem = few4_smem(smem_raw);
  grid_dep_launch();
  if (threadIdx.x == 0) few4_init<NT>(few4_shared<NT>(smem));
  plan_start<8 * NT, 8 * NT, kFew4Threads<NT>, true>(p, &plan, threadIdx.x);  // all threads meet in it
  if (threadIdx.x < 32 * kFew4Warps<NT>)
    few4_work<BF16, NT>(p, p.part, plan, smem);
  else
    few4_load<NT, false>(p, p.part, plan, smem);
}

template <bool BF16, int NT>
static palu_status launch_rows(const AttnParams& p, cudaStream_t s) {
  return launch(paged4_few_kernel<BF16, NT>, device_sm_count(), kFew4Threads<NT>, kFew4SmemBytes<NT>, false, s,
                "paged4_few_kernel launch", p);
}

palu_status launch_few4(const AttnParams& p, bool bf16, cudaStream_t stream) {
  if (p.part.R == 8) return bf16 ? launch_rows<true, 1>(p, stream) : launch_rows<false, 1>(p, stream);
  return bf16 ? launch_rows<true, 2>(p, stream) : launch_rows<false, 2>(p, stream);
}

}  // namespace palu
