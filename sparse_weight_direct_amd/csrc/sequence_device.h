// Device helpers of the sequence operators (HIP sources only).
#pragma once
#include <hip/hip_runtime.h>

#include "sequence.h"

namespace sc {

// V values of T at any multiple of T's size: one wide load or store, which the hardware takes
// at every address (rows of odd length start at odd offsets).
template <class T, int V>
struct Pack {
  typedef T type __attribute__((ext_vector_type(V), aligned(sizeof(T))));
};

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float exp2_fast(float v) { return __builtin_amdgcn_exp2f(v); }

// v * sigmoid(v).  exp2 and rcp are exact to 1 ulp, well inside what the fp32 sums before it carry.
__device__ __forceinline__ float silu(float v) {
  return v * __builtin_amdgcn_rcpf(1.0f + exp2_fast(-kLog2e * v));
}

// log(1 + exp(v)).  The small results matter (time steps of 1e-3), so log1p is the exact one: 1 + e
// would keep only the bits of e above 2^-24.
__device__ __forceinline__ float softplus(float v) { return fmaxf(v, 0.0f) + log1pf(exp2_fast(-kLog2e * fabsf(v))); }

// Slot of sequence b; negative where it is idle.
__device__ __forceinline__ int slot_of(const int32_t* slots, int num_slots, int b) {
  if (!slots) return b;
  const int s = slots[b];
  return s >= 0 && s < num_slots ? s : -1;
}

__device__ __forceinline__ int length_of(const int32_t* lengths, int L, int b) {
  return lengths ? min(max(lengths[b], 0), L) : L;
}

}  // namespace sc
