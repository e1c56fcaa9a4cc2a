// Attention over the 4-bit paged cache behind a shared prefix that many rows
// attend to, where each sequence has few: a CTA works on the prefix as those of
// paged4_many_kernel do, or on own units as those of paged4_few_kernel.  Which,
// the lengths decide (split_ctas).
#include "paged4_few.cuh"
#include "paged_many.cuh"

namespace palu {

template <int NT>
constexpr int kBoth4SmemBytes = kFew4SmemBytes<NT> > kMany4SmemBytes ? kFew4SmemBytes<NT> : kMany4SmemBytes;
static_assert(kFew4Threads<1> <= kMany4Threads && kFew4Threads<2> <= kMany4Threads, "threads of paged4_both_kernel");
static_assert(kBoth4SmemBytes<1> + sizeof(PlanScratch) <= 232448 && kBoth4SmemBytes<2> + sizeof(PlanScratch) <= 232448,
              "shared memory of paged4_both_kernel");

template <bool BF16, int NT>
__global__ void __launch_bounds__(kMany4Threads, 1) paged4_both_kernel(const AttnParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ PlanScratch plan;
  grid_dep_launch();
  plan_start<8 * NT, kManyRows, kMany4Threads, true>(p, &plan, threadIdx.x);
  if (plan.has_prefix) {
    many_stretch<BF16, true, true>(p, p.prefix, nullptr, nullptr, plan, many_smem(smem_raw), [] {});
  } else {
    uint8_t* smem = few4_smem(smem_raw);
    if (threadIdx.x == 0) few4_init<NT>(few4_shared<NT>(smem));
    __syncthreads();
    // Of the launch's 96 registers a thread the warps that compute take 112 of 16 warps, or 168 of 8, by warpgroups.
    if (NT == 1 && threadIdx.x < 512) {
      asm volatile("setmaxnreg.inc.sync.aligned.u32 112;");
      if (threadIdx.x < 32 * kFew4Warps<NT>)
        few4_work<BF16, NT>(p, p.part, plan, smem);
      else
        few4_load<NT, true>(p, p.part, plan, smem);
    } else if (NT == 1) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 24;");
    } else if (threadIdx.x < 256) {
      asm volatile("setmaxnreg.inc.sync.aligned.u32 168;");
      few4_work<BF16, NT>(p, p.part, plan, smem);
    } else {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
      if (threadIdx.x < kFew4Threads<NT>) few4_load<NT, true>(p, p.part, plan, smem);
    }
  }
}

template <bool BF16, int NT>
static palu_status launch_rows(const AttnParams& p, cudaStream_t s) {
  return launch(paged4_both_kernel<BF16, NT>, device_sm_count(), kMany4Threads, kBoth4SmemBytes<NT>, false, s,
                "paged4_both_kernel launch", p);
}

palu_status launch_both4(const AttnParams& p, bool bf16, cudaStream_t stream) {
  if (p.part.R == 8) return bf16 ? launch_rows<true, 1>(p, stream) : launch_rows<false, 1>(p, stream);
  return bf16 ? launch_rows<true, 2>(p, stream) : launch_rows<false, 2>(p, stream);
}

}  // namespace palu
