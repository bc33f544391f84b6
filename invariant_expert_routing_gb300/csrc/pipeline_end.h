// How a pipelined GEMM's CTA ends after a bounded wait gave up.
//
// Whichever role gives up, the producer may have asked for operand loads that
// no MMA has consumed.  They write this CTA's shared memory, so the CTA (or a
// CTA pair) leaves only after they have landed: it waits for the full barriers
// of its last `stages` loads once every role is done.  Load i fills stage i %
// stages in the barrier's phase i / stages.  A run that ends in the usual way
// has consumed every load and waits for nothing.
//
// In a pair both CTAs' loads complete on the even CTA's full barriers, which the
// even CTA arms for both CTAs' bytes.  The CTAs may have given up after
// different numbers of loads, at most `stages` apart (a stage is filled again
// only after the MMAs have read both CTAs' parts of it), so for each load that
// one of them issued alone that CTA makes up for the other: the even one
// completes the bytes that will not come, the odd one arms the barrier for its
// own.
#pragma once

#ifdef __CUDACC__
#define MOE_HD __host__ __device__ __forceinline__
#else
#define MOE_HD inline
#endif

namespace moe {

// wait(stage, parity) for the last loads of `issued`.
template <class Wait>
MOE_HD void wait_last_loads(int issued, int stages, Wait wait) {
  for (int i = issued > stages ? issued - stages : 0; i < issued; ++i) wait(i % stages, (unsigned)(i / stages) & 1u);
}

// A CTA of a pair, `mine` and `peer` the loads that it and the other issued:
// complete(load) on the even CTA, arm(load) on the odd one.
template <class Complete, class Arm>
MOE_HD void settle_pair_loads(bool even, int mine, int peer, Complete complete, Arm arm) {
  for (int i = peer; i < mine; ++i) {
    if (even)
      complete(i);
    else
      arm(i);
  }
}

}  // namespace moe
