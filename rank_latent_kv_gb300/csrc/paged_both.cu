// Attention over the paged cache behind a shared prefix that many rows attend
// to, where each sequence has few: a CTA works on the prefix as those of
// paged_many_kernel do, or on own units as those of paged_few_kernel.  Which,
// the lengths decide (split_ctas).  Products for the prefix are far from the
// tensor cores' bound here; own units have half the beginning and end that they
// have on the other kernel (32 sequences of 777 behind 8192, 24 heads of 8: 42
// us, all on one line 50; 256 sequences of 300 behind 4096, 28 of 4: 75 and 95).
#include "paged_few.cuh"
#include "paged_many.cuh"

namespace palu {

constexpr int kBothSmemBytes = kFewSmemBytes > kManySmemBytes ? kFewSmemBytes : kManySmemBytes;
static_assert(kFewThreads <= kManyThreads, "threads of paged_both_kernel");

template <bool BF16, int NT>
__global__ void __launch_bounds__(kManyThreads, 1)
    paged_both_kernel(const AttnParams p, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ PlanScratch plan;
  grid_dep_launch();
  plan_start<8 * NT, kManyRows, kManyThreads>(p, &plan, threadIdx.x);
  if (plan.has_prefix) {
    many_stretch<BF16, true, false>(p, p.prefix, &kmap, &vmap, plan, many_smem(smem_raw), [] {});
  } else {
    uint8_t* smem = few_smem(smem_raw);
    if (threadIdx.x == 0) few_init(few_shared(smem));
    __syncthreads();
    if (threadIdx.x < kFewThreads) few_stretch<BF16, NT, true>(p, p.part, kmap, vmap, plan, smem);
  }
}

template <bool BF16>
static palu_status launch_type(const AttnParams& p, const CUtensorMap& km, const CUtensorMap& vm, cudaStream_t s) {
  return p.part.R == 8 ? launch(paged_both_kernel<BF16, 1>, device_sm_count(), kManyThreads, kBothSmemBytes, false, s,
                                "paged_both_kernel launch", p, km, vm)
                       : launch(paged_both_kernel<BF16, 2>, device_sm_count(), kManyThreads, kBothSmemBytes, false, s,
                                "paged_both_kernel launch", p, km, vm);
}

palu_status launch_both(const AttnParams& p, const CUtensorMap& km, const CUtensorMap& vm, bool bf16, cudaStream_t stream) {
  return bf16 ? launch_type<true>(p, km, vm, stream) : launch_type<false>(p, km, vm, stream);
}

}  // namespace palu
