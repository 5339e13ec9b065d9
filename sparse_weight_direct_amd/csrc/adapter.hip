// Low-rank adapters of many requests beside a shared projection (sparseconv_adapter_apply).
//
//   out[b] = base[b] + scale[r] up[r] (down[r] x[b]),  r = index[b]
#include <hip/hip_runtime.h>

#include "sequence_device.h"

namespace sc {

namespace {

__device__ __forceinline__ int adapter_of(const sc_adapter& a, int b) {
  const int r = a.index[b];
  return r >= 0 && r < a.adapters ? r : -1;
}

// low[b][r][l] = scale * sum_c down[r][c] x[b][c][l], fp32.
template <class T>
__global__ __launch_bounds__(256) void adapter_down(const sc_adapter a, float* low) {
  const int l = blockIdx.x * 256 + threadIdx.x, r = blockIdx.y, b = blockIdx.z;
  const int ad = adapter_of(a, b);
  if (l >= a.L || ad < 0) return;
  const T* w = static_cast<const T*>(a.down) + ((int64_t)ad * a.R + r) * a.C;
  const T* x = static_cast<const T*>(a.x) + b * a.x_batch + l;
  float v = 0.0f;
  for (int c = 0; c < a.C; c++) v = fmaf((float)w[c], (float)x[c * a.x_channel], v);
  low[((int64_t)b * a.R + r) * a.L + l] = a.scale ? a.scale[ad] * v : v;
}

template <class T>
__global__ __launch_bounds__(256) void adapter_up(const sc_adapter a, const float* low) {
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int b = blockIdx.z;
  if (id >= (int64_t)a.M * a.L) return;
  const int m = id / a.L, l = id - (int64_t)m * a.L;
  const int ad = adapter_of(a, b);
  float v = a.base ? (float)static_cast<const T*>(a.base)[b * a.base_batch + m * a.base_channel + l] : 0.0f;
  if (ad >= 0) {
    const T* w = static_cast<const T*>(a.up) + ((int64_t)ad * a.M + m) * a.R;
    for (int r = 0; r < a.R; r++) v = fmaf((float)w[r], low[((int64_t)b * a.R + r) * a.L + l], v);
  }
  static_cast<T*>(a.out)[b * a.out_batch + m * a.out_channel + l] = T(v);
}

template <class T>
int launch_type(const sc_adapter& a, hipStream_t st) {
  float* low = static_cast<float*>(a.workspace);
  hipLaunchKernelGGL((adapter_down<T>), dim3((a.L + 255) / 256, a.R, a.B), dim3(256), 0, st, a, low);
  if (const int e = (int)hipGetLastError()) return e;
  hipLaunchKernelGGL((adapter_up<T>), dim3((unsigned)(((int64_t)a.M * a.L + 255) / 256), 1, a.B), dim3(256), 0, st, a,
                     low);
  return (int)hipGetLastError();
}

}  // namespace

int64_t adapter_workspace(const sc_adapter& a, int) { return (int64_t)a.B * a.R * a.L * 4; }

int launch_adapter(const sc_adapter& a, int, void* stream) {
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if (a.dtype == SC_F32) return launch_type<float>(a, st);
  if (a.dtype == SC_BF16) return launch_type<__bf16>(a, st);
  return launch_type<_Float16>(a, st);
}

}  // namespace sc
