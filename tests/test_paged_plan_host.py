"""The work plan of the paged attention, without a GPU: the shared memory in
which a CTA's warps add up the line has a place for each of them, in every
kernel that plans."""
import os
import subprocess
import tempfile

import pytest

from rank_latent_kv_gb300 import build as B

PROLOGUE = """
#include "paged_few.cuh"
#include "paged4_few.cuh"
#include "paged_many.cuh"
using namespace palu;
constexpr int kSums = sizeof(PlanScratch::warp_sum) / sizeof(long long), kLongest = sizeof(PlanScratch::warp_longest) / sizeof(int);
constexpr int kPlaces = kSums < kLongest ? kSums : kLongest;
"""


def compiles(body):
    """Whether these lines compile behind the kernels' headers, and what the compiler says."""
    try:
        cc = B.nvcc()
    except RuntimeError:
        pytest.skip("needs nvcc")
    with tempfile.TemporaryDirectory() as d:
        src = os.path.join(d, "t.cu")
        with open(src, "w") as f:
            f.write(PROLOGUE + body)
        r = subprocess.run([cc, *B.ARCH, "-std=c++17", "-I", B.INCLUDE, "-I", B.CSRC, "-cubin", src, "-o", os.path.join(d, "t.cubin")],
                           capture_output=True, text=True)
    return r.returncode == 0, r.stderr


def test_every_planning_warp_has_a_place():
    ok, said = compiles("""
template <int THREADS>
constexpr bool fits = THREADS / 32 <= kPlaces;
static_assert(fits<kFewThreads>, "paged_few_kernel");
static_assert(fits<kManyThreads>, "paged_both_kernel, and more than paged_many_kernel");
static_assert(fits<kFew4Threads<1>> && fits<kFew4Threads<2>>, "paged4_few_kernel");
static_assert(fits<kMany4Threads>, "paged4_both_kernel, and more than paged4_many_kernel");
""")
    assert ok, said


def test_more_warps_than_places_are_refused_by_the_compiler():
    plan = """
__global__ void plan_kernel(const AttnParams p) {
  __shared__ PlanScratch plan;
  plan_start<8, kManyRows, 32 * (kPlaces + %d), true>(p, &plan, threadIdx.x);
}
"""
    ok, said = compiles(plan % 0)
    assert ok, said
    ok, said = compiles(plan % 1)
    assert not ok and "place for each warp" in said
