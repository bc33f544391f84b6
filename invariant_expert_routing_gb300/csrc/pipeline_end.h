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

// The same where several warps of a CTA request loads in turn: load i is of warp
// i % parts, and count[w] says how many of its own warp w issued.  An issued
// load that no MMA has consumed is one of the `stages` before the highest.
MOE_HD bool load_issued(const int* count, int parts, int i) { return i / parts < count[i % parts]; }
MOE_HD int loads_top(const int* count, int parts) {
  int top = 0;
  for (int w = 0; w < parts; ++w) {
    const int t = count[w] ? (count[w] - 1) * parts + w + 1 : 0;
    top = t > top ? t : top;
  }
  return top;
}
MOE_HD int loads_top(const int* mine, const int* peer, int parts) {
  const int a = loads_top(mine, parts), b = loads_top(peer, parts);
  return a > b ? a : b;
}
template <class Complete, class Arm>
MOE_HD void settle_pair_parts(bool even, const int* mine, const int* peer, int parts, int stages, Complete complete, Arm arm) {
  const int top = loads_top(mine, peer, parts);
  for (int i = top > stages ? top - stages : 0; i < top; ++i) {
    if (!load_issued(mine, parts, i) || load_issued(peer, parts, i)) continue;
    if (even)
      complete(i);
    else
      arm(i);
  }
}
template <class Wait>
MOE_HD void wait_pair_parts(const int* mine, const int* peer, int parts, int stages, Wait wait) {
  const int top = loads_top(mine, peer, parts);
  for (int i = top > stages ? top - stages : 0; i < top; ++i)
    if (load_issued(mine, parts, i) || load_issued(peer, parts, i)) wait(i % stages, (unsigned)(i / stages) & 1u);
}

}  // namespace moe
