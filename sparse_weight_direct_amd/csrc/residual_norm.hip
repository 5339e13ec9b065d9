// The norms around a block with its residual sum (sparseconv_residual_norm).
//
//   r = x + scale gate post(y),  out = norm(r) weight + bias,  over the channels of each position
#include <hip/hip_runtime.h>

#include "attention.h"
#include "attention_plan.h"
#include "sequence_device.h"
#include "xcd.h"

namespace sc {

namespace {

// Sums over the workgroup's 16 rows of threads, for each of its 16 positions.
__device__ __forceinline__ float over_rows(float v, float (*part)[16]) {
  const int col = threadIdx.x & 15, row = threadIdx.x >> 4;
  __syncthreads();
  part[row][col] = v;
  __syncthreads();
  float s = 0.0f;
#pragma unroll
  for (int k = 0; k < 16; k++) s += part[k][col];
  return s;
}

// Any sizes: 16 positions a workgroup, what it needs again it reads again.
template <class T>
__global__ __launch_bounds__(256) void norm_any(const sc_residual_norm a, int tiles) {
  __shared__ float part[16][16];
  const int col = threadIdx.x & 15, row = threadIdx.x >> 4;
  const int id = xcd_logical(blockIdx.x, gridDim.x);
  const int l = id % tiles * 16 + col, b = id / tiles;
  const bool live = l < a.L;
  const int at = live ? l : a.L - 1;
  const bool center = a.flags & SC_NORM_CENTER;
  const float per = 1.0f / a.C;
  const T* x = static_cast<const T*>(a.x) + b * a.x_batch + at;
  const T* y = static_cast<const T*>(a.y) + b * a.y_batch + at;
  const T* gate = static_cast<const T*>(a.gate) + b * a.gate_batch + (a.gate_position ? at : 0);
  auto statistics = [&](auto value, float& mean, float& by) {
    mean = 0.0f;
    float s = 0.0f;
    if (center) {
      for (int c = row; c < a.C; c += 16) s += value(c);
      mean = over_rows(s, part) * per;
    }
    s = 0.0f;
    for (int c = row; c < a.C; c += 16) {
      const float d = value(c) - mean;
      s = fmaf(d, d, s);
    }
    by = 1.0f / sqrtf(over_rows(s, part) * per + a.eps);
  };
  float post_mean = 0.0f, post_by = 1.0f, mean = 0.0f, by = 1.0f;
  if (a.post_weight) statistics([&](int c) { return (float)y[c * a.y_channel]; }, post_mean, post_by);
  auto summed = [&](int c) {
    const float v = (float)x[c * a.x_channel];
    if (!a.y) return v;
    float w = (float)y[c * a.y_channel];
    if (a.post_weight) w = (w - post_mean) * post_by * a.post_weight[c] + (a.post_bias ? a.post_bias[c] : 0.0f);
    if (a.gate) w *= (float)gate[c * a.gate_channel];
    return fmaf(a.scale, w, v);
  };
  if (a.out) statistics(summed, mean, by);
  __syncthreads();
  if (!live) return;
  T* sum = static_cast<T*>(a.sum) + b * a.sum_batch + l;
  T* out = static_cast<T*>(a.out) + b * a.out_batch + l;
  for (int c = row; c < a.C; c += 16) {
    const float r = summed(c);
    if (a.sum) sum[c * a.sum_channel] = T(r);
    if (a.out) out[c * a.out_channel] = T((r - mean) * by * (a.weight ? a.weight[c] : 1.0f) + (a.bias ? a.bias[c] : 0.0f));
  }
}

template <class T>
int launch_type(const sc_residual_norm& a, int cus, hipStream_t st) {
  const int tiles = (int)ceil_div(a.L, 16);
  hipLaunchKernelGGL(norm_any<T>, dim3((unsigned)((int64_t)a.B * tiles)), dim3(256), 0, st, a, tiles);
  return (int)hipGetLastError();
}

}  // namespace

int launch_residual_norm(const sc_residual_norm& a, int cus, void* stream) {
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if (a.dtype == SC_F32) return launch_type<float>(a, cus, st);
  if (a.dtype == SC_BF16) return launch_type<__bf16>(a, cus, st);
  return launch_type<_Float16>(a, cus, st);
}

}  // namespace sc
