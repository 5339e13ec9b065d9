// Matrix instructions of the attention operators (HIP sources only): products of 16 x 16 tiles whose operands
// are 16 bytes a lane.
#pragma once
#include "sequence_device.h"

namespace sc {

typedef float F4 __attribute__((ext_vector_type(4)));

// A lane's part of an operand: N consecutive values of the summed index of row (or column) lane & 15, from
// N * (lane >> 4) on, out of kDepth.  The result's lane has column lane & 15 and rows 4 (lane >> 4) + 0..3.
template <class T>
struct Frag {
  static constexpr int N = 16 / sizeof(T);
  static constexpr int kDepth = 4 * N;
  typedef T type __attribute__((ext_vector_type(N)));
};

__device__ __forceinline__ F4 mma(Frag<__bf16>::type a, Frag<__bf16>::type b, F4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ F4 mma(Frag<_Float16>::type a, Frag<_Float16>::type b, F4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}
// fp32: four instructions of depth 4; the order of the summed index is free as long as both operands agree.
__device__ __forceinline__ F4 mma(Frag<float>::type a, Frag<float>::type b, F4 c) {
#pragma unroll
  for (int i = 0; i < 4; i++) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[i], b[i], c, 0, 0, 0);
  return c;
}

}  // namespace sc
