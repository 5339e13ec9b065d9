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

// V values at p of which the first n exist; the others are 0 and not read.
template <class T, int V>
__device__ __forceinline__ typename Pack<T, V>::type load_some(const T* p, int n) {
  typedef typename Pack<T, V>::type Vec;
  if (n >= V) return *reinterpret_cast<const Vec*>(p);
  Vec v;
#pragma unroll
  for (int i = 0; i < V; i++) v[i] = i < n ? p[i] : T(0.0f);
  return v;
}

template <class T, int V>
__device__ __forceinline__ void store_some(T* p, int n, typename Pack<T, V>::type v) {
  typedef typename Pack<T, V>::type Vec;
  if (n >= V) {
    *reinterpret_cast<Vec*>(p) = v;
  } else {
#pragma unroll
    for (int i = 0; i < V; i++)
      if (i < n) p[i] = v[i];
  }
}

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float exp2_fast(float v) { return __builtin_amdgcn_exp2f(v); }

// v * sigmoid(v).  exp2 and rcp are exact to 1 ulp, well inside what the fp32 sums before it carry.  From v = -87.4
// down the result is 0 (rcp makes no denormals): off by 1.3e-36 at most.
__device__ __forceinline__ float silu(float v) {
  return v * __builtin_amdgcn_rcpf(1.0f + exp2_fast(-kLog2e * v));
}

// log(1 + exp(v)) = max(v, 0) + log1p(e), e = exp(-|v|), to 4.7 x 2^-24 of every result (4 million values
// over -40..25): the small ones count (time steps of 1e-3).  With u = 1 + e rounded, e - (u - 1) is what the
// rounding lost, exactly, and log1p(e) = log(u) + that / u, where / u changes less than a rounding.
// exp2's argument carries its rounding error along; |v| is bounded for that (e is 0 from 88 on), or the
// product would be infinite at the ends of the range and the error no number: softplus(-inf) is 0 and
// softplus(inf) is inf.  The maximum keeps a NaN.  14 instructions; the math library's log1p alone is
// 110, which was half of the whole scan's time (scan_prompt's shape: 259 us, and 175 with a polynomial of
// 18 in its place).
__device__ __forceinline__ float softplus(float v) {
  const float m = __builtin_elementwise_maximum(-fabsf(v), -126.0f), p = m * kLog2e;
  const float rest = fmaf(m, 1.92596299e-8f, fmaf(m, kLog2e, -p));  // log2(e) - kLog2e = 1.926e-8
  float e = exp2_fast(p);
  e = fmaf(e * 0.69314718f, rest, e);
  const float u = 1.0f + e;
  return fmaf(__builtin_amdgcn_logf(u), 0.69314718f, e - (u - 1.0f)) + fmaxf(v, 0.0f);
}

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
