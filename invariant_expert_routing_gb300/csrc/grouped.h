// Products grouped by expert with ragged sizes, and the weight gradient:
// arguments and launchers.  Internal, not part of the C ABI.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <cstdint>

namespace moe {

// Expert e's rows: counts[e] of them from start[e], the sum of the earlier
// experts' counts, each rounded up to a multiple of B.
struct GroupArgs {
  const int32_t* counts;   // [N] on the device
  int N, B;
  long long max_rows;      // rows of the grouped tensors
  const int32_t* ids;      // route of each row; read for gathered operands only
  int T, slots;            // a gathered operand has T rows, row ids[p] / slots
  int K, F;                // inner and outer sizes (multiples of 8)
  int* status;
  unsigned long long wait_ns;   // limit of the pipeline waits; 0: the default
};

struct GroupedGemmArgs {
  GroupArgs g;
  const uint16_t *x, *w;
  uint16_t* y;
  int gather, transposed;
};

struct GroupedWgradArgs {
  GroupArgs g;
  const uint16_t *x, *dy;
  const float* add;        // or null
  void* dw;
  int gather_x, gather_dy, fp32;
};

// false: a tensor map could not be made
bool launch_grouped_gemm(const GroupedGemmArgs& a, PFN_cuTensorMapEncodeTiled_v12000 encode, int sms, cudaStream_t s);
bool launch_grouped_wgrad(const GroupedWgradArgs& a, PFN_cuTensorMapEncodeTiled_v12000 encode, int sms, cudaStream_t s);

}  // namespace moe
