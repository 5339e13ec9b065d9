// Selective state space scan (sparseconv_selective_scan).
//
//   h_t[n] = exp(s_t A[d,n]) h_{t-1}[n] + s_t b_t[n] x_t,   out_t = (sum_n c_t[n] h_t[n] + skip[d] x_t) silu(z_t)
#include <hip/hip_runtime.h>

#include "sequence_device.h"

namespace sc {

namespace {

// One wavefront per (sequence, channel), its lanes over the states, one position after another.
template <class T>
__global__ __launch_bounds__(256) void scan_rows(const sc_selective_scan a) {
  const int lane = threadIdx.x & 63;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (row >= (int64_t)a.B * a.D) return;
  const int b = row / a.D, d = row - (int64_t)b * a.D, g = d / (a.D / a.G);
  const int slot = slot_of(a.slots, a.num_slots, b);
  const int len = slot < 0 ? 0 : length_of(a.lengths, a.L, b);
  const T* x = static_cast<const T*>(a.x) + b * a.x_batch + d * a.x_channel;
  const T* dt = static_cast<const T*>(a.dt) + b * a.dt_batch + d * a.dt_channel;
  const T* z = a.z ? static_cast<const T*>(a.z) + b * a.z_batch + d * a.z_channel : nullptr;
  const T* bm = static_cast<const T*>(a.b) + b * a.b_batch + g * a.b_group;
  const T* cm = static_cast<const T*>(a.c) + b * a.c_batch + g * a.c_group;
  T* out = static_cast<T*>(a.out) + b * a.out_batch + d * a.out_channel;
  const float skip = a.skip ? a.skip[d] : 0.0f, bias = a.dt_bias ? a.dt_bias[d] : 0.0f;
  float A[4], h[4];
#pragma unroll
  for (int j = 0; j < 4; j++) {
    const int n = lane + 64 * j;
    A[j] = n < a.N ? a.A[(int64_t)d * a.N + n] * kLog2e : 0.0f;
    h[j] = n < a.N && a.initial_state && slot >= 0 ? a.initial_state[slot * a.initial_stride + (int64_t)d * a.N + n] : 0.0f;
  }
  for (int t = 0; t < len; t++) {
    const float xt = (float)x[t], raw = (float)dt[t] + bias;
    const float s = a.flags & SC_SEQ_SOFTPLUS ? softplus(raw) : raw;
    float y = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; j++) {
      const int n = lane + 64 * j;
      if (n < a.N) {
        h[j] = fmaf(exp2_fast(s * A[j]), h[j], s * xt * (float)bm[n * a.b_state + t]);
        y = fmaf((float)cm[n * a.c_state + t], h[j], y);
      }
    }
    for (int m = 32; m; m >>= 1) y += __shfl_xor(y, m);
    y = fmaf(skip, xt, y);
    if (z) y *= silu((float)z[t]);
    if (lane == 0) out[t] = T(y);
  }
  for (int t = len + lane; t < a.L; t += 64) out[t] = T(0.0f);
  if (a.final_state && slot >= 0)
#pragma unroll
    for (int j = 0; j < 4; j++) {
      const int n = lane + 64 * j;
      if (n < a.N) a.final_state[slot * a.final_stride + (int64_t)d * a.N + n] = h[j];
    }
}

template <class T>
int launch_type(const sc_selective_scan& a, hipStream_t st) {
  const int64_t rows = (int64_t)a.B * a.D;
  hipLaunchKernelGGL((scan_rows<T>), dim3((unsigned)((rows + 3) / 4)), dim3(256), 0, st, a);
  return (int)hipGetLastError();
}

}  // namespace

int64_t scan_workspace(const sc_selective_scan&, int) { return 0; }

int launch_selective_scan(const sc_selective_scan& a, int, void* stream) {
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if (a.dtype == SC_F32) return launch_type<float>(a, st);
  if (a.dtype == SC_BF16) return launch_type<__bf16>(a, st);
  return launch_type<_Float16>(a, st);
}

}  // namespace sc
