// The norms around a block with its residual sum (sparseconv_residual_norm).
//
//   r = x + scale gate post(y),  out = norm(r) weight + bias,  over the channels of each position
//
// Bound by memory, in phases: a workgroup loads, makes statistics, stores the sum, makes statistics, stores the norm, and holds its
// values in so many registers that no other shares its CU.  8 x 2048 channels x 2048 positions, bf16, gated: 93 us, 2.9 TB/s
// (read and written once, by the counters; a copy: 5.1).  64 single positions of 4096 channels: 6.2 us.
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

// ---- Values in registers: every input is read once
//
// A thread has PASS channels of V consecutive positions; LP lanes side by side along the positions, THREADS / LP rows of channels. The block's
// output stays in registers from its statistics to the sum, the sum (in fp32) from its statistics to the norm.
// (The channels' weights and gates in LDS beside the first loads gained nothing, and cost registers.)

// Sums over the workgroup's rows of channels, for each of a lane's positions.  (part: LDS, THREADS / 64 x LP x V.)
template <int V, int THREADS>
__device__ __forceinline__ void over_channels(float (&v)[V], int lp, float* part) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1)
    if (m >= lp)
#pragma unroll
      for (int j = 0; j < V; j++) v[j] += __shfl_xor(v[j], m);
  __syncthreads();  // the sums before have been read
  if (lane < lp)
#pragma unroll
    for (int j = 0; j < V; j++) part[(wave * lp + lane) * V + j] = v[j];
  __syncthreads();
#pragma unroll
  for (int j = 0; j < V; j++) v[j] = 0.0f;
#pragma unroll 1
  for (int w = 0; w < THREADS / 64; w++)
#pragma unroll
    for (int j = 0; j < V; j++) v[j] += part[(w * lp + (lane & (lp - 1))) * V + j];
}

template <int V, int PASS, int THREADS>
__device__ __forceinline__ void statistics(const float (&v)[PASS][V], bool center, float eps, int channels, int rows, int C, int lp, float* part,
                                           float (&mean)[V], float (&by)[V]) {
  const float per = 1.0f / C;
#pragma unroll
  for (int j = 0; j < V; j++) mean[j] = 0.0f;
  if (center) {  // (what lies past the channels is 0)
#pragma unroll
    for (int p = 0; p < PASS; p++)
#pragma unroll
      for (int j = 0; j < V; j++) mean[j] += v[p][j];
    over_channels<V, THREADS>(mean, lp, part);
#pragma unroll
    for (int j = 0; j < V; j++) mean[j] *= per;
  }
#pragma unroll
  for (int j = 0; j < V; j++) by[j] = 0.0f;
#pragma unroll
  for (int p = 0; p < PASS; p++) {
    const bool there = channels + p * rows < C;
#pragma unroll
    for (int j = 0; j < V; j++) {
      const float d = there ? v[p][j] - mean[j] : 0.0f;
      by[j] = fmaf(d, d, by[j]);
    }
  }
  over_channels<V, THREADS>(by, lp, part);
#pragma unroll
  for (int j = 0; j < V; j++) by[j] = 1.0f / sqrtf(by[j] * per + eps);
}

// Prompts: positions are contiguous.
template <class T, int V, int PASS, int THREADS>
__global__ __launch_bounds__(THREADS) void norm_prompt(const sc_residual_norm a, int tiles, int lp_shift) {
  extern __shared__ float part[];
  typedef typename Pack<T, V>::type Vec;
  const int lp = 1 << lp_shift, rows = THREADS >> lp_shift, row = threadIdx.x >> lp_shift;
  const int id = xcd_logical(blockIdx.x, gridDim.x), b = id / tiles;
  const int l = ((id % tiles << lp_shift) + (threadIdx.x & (lp - 1))) * V, n = min(max(a.L - l, 0), V);
  const int at = n ? l : 0;  // lanes past the end read nothing
  const bool center = a.flags & SC_NORM_CENTER;
  const T* x = static_cast<const T*>(a.x) + b * a.x_batch + at;
  const T* y = static_cast<const T*>(a.y) + b * a.y_batch + at;
  const T* gate = static_cast<const T*>(a.gate) + b * a.gate_batch + (a.gate_position ? at : 0);
  T* sum = static_cast<T*>(a.sum) + b * a.sum_batch + at;
  T* out = static_cast<T*>(a.out) + b * a.out_batch + at;
  Vec xr[PASS];
  float v[PASS][V], mean[V], by[V];
#pragma unroll
  for (int p = 0; p < PASS; p++) {
    const int c = row + p * rows;
    Vec yr = {};
    xr[p] = Vec{};
    if (a.y && c < a.C) yr = load_some<T, V>(y + c * a.y_channel, n);
#pragma unroll
    for (int j = 0; j < V; j++) v[p][j] = (float)yr[j];
  }
#pragma unroll
  for (int p = 0; p < PASS; p++) {
    const int c = row + p * rows;
    if (c < a.C) xr[p] = load_some<T, V>(x + c * a.x_channel, n);
  }
  if (a.post_weight) {
    statistics<V, PASS, THREADS>(v, center, a.eps, row, rows, a.C, lp, part, mean, by);
#pragma unroll
    for (int p = 0; p < PASS; p++) {
      const int c = min(row + p * rows, a.C - 1);
      const float w = a.post_weight[c], bias = a.post_bias ? a.post_bias[c] : 0.0f;
#pragma unroll
      for (int j = 0; j < V; j++) v[p][j] = (v[p][j] - mean[j]) * by[j] * w + bias;
    }
  }
#pragma unroll
  for (int p = 0; p < PASS; p++) {
    const int c = row + p * rows;
    if (a.gate && c < a.C) {
      if (a.gate_position) {
        const Vec g = load_some<T, V>(gate + c * a.gate_channel, n);
#pragma unroll
        for (int j = 0; j < V; j++) v[p][j] *= (float)g[j];
      } else {
        const float g = (float)gate[c * a.gate_channel];
#pragma unroll
        for (int j = 0; j < V; j++) v[p][j] *= g;
      }
    }
    const bool there = c < a.C;
#pragma unroll
    for (int j = 0; j < V; j++) {
      const float xv = (float)xr[p][j], s = a.y ? fmaf(a.scale, v[p][j], xv) : xv;
      v[p][j] = there ? s : 0.0f;
    }
    if (a.sum && there) {
      Vec r;
#pragma unroll
      for (int j = 0; j < V; j++) r[j] = T(v[p][j]);
      store_some<T, V>(sum + c * a.sum_channel, n, r);
    }
  }
  if (!a.out) return;
  statistics<V, PASS, THREADS>(v, center, a.eps, row, rows, a.C, lp, part, mean, by);
#pragma unroll
  for (int p = 0; p < PASS; p++) {
    const int c = row + p * rows;
    if (c >= a.C) continue;
    const float w = a.weight ? a.weight[c] : 1.0f, bias = a.bias ? a.bias[c] : 0.0f;
    Vec r;
#pragma unroll
    for (int j = 0; j < V; j++) r[j] = T((v[p][j] - mean[j]) * by[j] * w + bias);
    store_some<T, V>(out + c * a.out_channel, n, r);
  }
}

// Single positions whose channels are contiguous: a workgroup has one, a thread 8 channels at a time.
template <class T, int PASS, int THREADS>
__global__ __launch_bounds__(THREADS) void norm_token(const sc_residual_norm a) {
  typedef typename Pack<T, 8>::type Vec;
  typedef typename Pack<float, 8>::type F8;
  __shared__ float part[THREADS / 64];
  const int b = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const bool center = a.flags & SC_NORM_CENTER;
  const float per = 1.0f / a.C;
  const T* x = static_cast<const T*>(a.x) + b * a.x_batch;
  const T* y = static_cast<const T*>(a.y) + b * a.y_batch;
  const T* gate = static_cast<const T*>(a.gate) + b * a.gate_batch;
  T* sum = static_cast<T*>(a.sum) + b * a.sum_batch;
  T* out = static_cast<T*>(a.out) + b * a.out_batch;
  auto everywhere = [&](float s) {
#pragma unroll
    for (int m = 32; m; m >>= 1) s += __shfl_xor(s, m);
    __syncthreads();
    if (lane == 0) part[wave] = s;
    __syncthreads();
    s = 0.0f;
#pragma unroll
    for (int w = 0; w < THREADS / 64; w++) s += part[w];
    return s;
  };
  float v[PASS][8], w1[PASS][8], b1[PASS][8], xv[PASS][8], gv[PASS][8];
  int left[PASS];
#pragma unroll
  for (int p = 0; p < PASS; p++) {  // everything is asked for at once
    const int c = (threadIdx.x + p * THREADS) * 8;
    left[p] = min(max(a.C - c, 0), 8);
    const int at = left[p] ? c : 0;
    const Vec yr = a.y ? load_some<T, 8>(y + at, left[p]) : Vec{}, xr = load_some<T, 8>(x + at, left[p]);
    Vec gr = {};
    if (a.gate)
#pragma unroll
      for (int j = 0; j < 8; j++) gr[j] = j < left[p] ? gate[(at + j) * a.gate_channel] : T(0.0f);
    const F8 wr = a.post_weight ? load_some<float, 8>(a.post_weight + at, left[p]) : F8{}, br = a.post_bias ? load_some<float, 8>(a.post_bias + at, left[p]) : F8{};
#pragma unroll
    for (int j = 0; j < 8; j++) v[p][j] = (float)yr[j], xv[p][j] = (float)xr[j], gv[p][j] = (float)gr[j], w1[p][j] = wr[j], b1[p][j] = br[j];
  }
  auto stats = [&](float& mean, float& by) {
    mean = 0.0f;
    float s = 0.0f;
    if (center) {
#pragma unroll
      for (int p = 0; p < PASS; p++)
#pragma unroll
        for (int j = 0; j < 8; j++) s += v[p][j];
      mean = everywhere(s) * per;
      s = 0.0f;
    }
#pragma unroll
    for (int p = 0; p < PASS; p++)
#pragma unroll
      for (int j = 0; j < 8; j++) {
        const float d = j < left[p] ? v[p][j] - mean : 0.0f;
        s = fmaf(d, d, s);
      }
    by = 1.0f / sqrtf(everywhere(s) * per + a.eps);
  };
  float mean, by;
  if (a.post_weight) {
    stats(mean, by);
#pragma unroll
    for (int p = 0; p < PASS; p++)
#pragma unroll
      for (int j = 0; j < 8; j++) v[p][j] = (v[p][j] - mean) * by * w1[p][j] + b1[p][j];
  }
#pragma unroll
  for (int p = 0; p < PASS; p++) {
    const int c = (threadIdx.x + p * THREADS) * 8;
    Vec r;
#pragma unroll
    for (int j = 0; j < 8; j++) {
      const float u = a.gate ? v[p][j] * gv[p][j] : v[p][j], s = a.y ? fmaf(a.scale, u, xv[p][j]) : xv[p][j];
      v[p][j] = j < left[p] ? s : 0.0f;
      r[j] = T(v[p][j]);
    }
    if (a.sum && left[p]) store_some<T, 8>(sum + c, left[p], r);
  }
  if (!a.out) return;
#pragma unroll
  for (int p = 0; p < PASS; p++) {
    const int at = left[p] ? (threadIdx.x + p * THREADS) * 8 : 0;
    const F8 one = {1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f};
    const F8 wr = a.weight ? load_some<float, 8>(a.weight + at, left[p]) : one, br = a.bias ? load_some<float, 8>(a.bias + at, left[p]) : F8{};
#pragma unroll
    for (int j = 0; j < 8; j++) w1[p][j] = wr[j], b1[p][j] = br[j];
  }
  stats(mean, by);
#pragma unroll
  for (int p = 0; p < PASS; p++) {
    Vec r;
#pragma unroll
    for (int j = 0; j < 8; j++) r[j] = T((v[p][j] - mean) * by * w1[p][j] + b1[p][j]);
    if (left[p]) store_some<T, 8>(out + (threadIdx.x + p * THREADS) * 8, left[p], r);
  }
}

// Any sizes (more channels than registers hold, single positions with channels apart): 16 positions a workgroup, what it
// needs again it reads again.
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

template <class T, int V, int PASS, int THREADS>
int launch_prompt(const sc_residual_norm& a, const NormPlan& p, hipStream_t st) {
  const int lds = THREADS / 64 * (V << p.lp_shift) * 4;
  hipLaunchKernelGGL((norm_prompt<T, V, PASS, THREADS>), dim3((unsigned)((int64_t)a.B * p.tiles)), dim3(THREADS), lds, st, a, p.tiles, p.lp_shift);
  return (int)hipGetLastError();
}

template <class T, int PASS, int THREADS>
int launch_token(const sc_residual_norm& a, hipStream_t st) {
  hipLaunchKernelGGL((norm_token<T, PASS, THREADS>), dim3((unsigned)a.B), dim3(THREADS), 0, st, a);
  return (int)hipGetLastError();
}

template <class T>
int launch_type(const sc_residual_norm& a, int cus, hipStream_t st) {
  constexpr int V = 16 / sizeof(T);
  const NormPlan p = norm_plan(a, cus);
  switch (p.form) {
    case kNormToken: return p.threads == 256 ? launch_token<T, 1, 256>(a, st) : p.threads == 512 ? launch_token<T, 1, 512>(a, st) : launch_token<T, 1, 1024>(a, st);
    case kNormPrompt:
      if (p.threads == 256)
        return p.pass == 4 ? launch_prompt<T, V, 4, 256>(a, p, st) : p.pass == 8 ? launch_prompt<T, V, 8, 256>(a, p, st) : launch_prompt<T, V, 16, 256>(a, p, st);
      return p.pass == 4 ? launch_prompt<T, V, 4, 512>(a, p, st) : p.pass == 8 ? launch_prompt<T, V, 8, 512>(a, p, st) : launch_prompt<T, V, 16, 512>(a, p, st);
    default: break;
  }
  hipLaunchKernelGGL(norm_any<T>, dim3((unsigned)((int64_t)a.B * p.tiles)), dim3(256), 0, st, a, p.tiles);
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
