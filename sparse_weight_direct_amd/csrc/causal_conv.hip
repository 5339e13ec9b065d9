// Short causal convolution of each channel (sparseconv_causal_conv).
//
//   out[b,d,t] = act(bias[d] + sum_k w[d,k] u[b,d,t-K+1+k]),  u = the initial state, then x.
//
// Bound by memory: every input is read and every output written once, 2 K + 10 instructions a value.
// Measured (bf16, K = 4): 8 x 2048 rows of 2048 positions 28.2 us, 4.8 TB/s of x and out, where a copy of
// 1 GiB runs at 5.1; 4 x 2048 rows in fp32 at 5.8 TB/s.  Two or four rows a thread in flight were slower
// (30.3 and 32.1 us).  Single positions: 128 x 4096 channels 4.4 us, a launch.
#include <hip/hip_runtime.h>

#include "sequence_device.h"
#include "sequence_plan.h"

namespace sc {

namespace {

constexpr int kV = kConvV;  // positions per thread

// A thread makes kV positions of one row from them and the kV before them (the second read comes from
// L1).  ROW: a workgroup stays in one row (of `blocks` workgroups), so everything but the positions is
// scalar; otherwise, for rows that would leave its threads idle, each thread has a place of its own.  (L may be
// 2^31 - 1: nothing here may pass it, and t0 is compared by what is left of the row.)
template <class T, int K, bool SILU, bool ROW>
__global__ __launch_bounds__(256) void causal_conv_rows(const sc_causal_conv a, int blocks, int nv) {
  typedef typename Pack<T, kV>::type Vec;
  int row, t0;
  if (ROW) {
    row = blockIdx.x / blocks;
    const int v = (blockIdx.x - row * blocks) * 256 + threadIdx.x;
    if (v >= nv) return;
    t0 = v * kV;
  } else {
    const uint32_t id = blockIdx.x * 256u + threadIdx.x;
    if (id >= (uint32_t)a.B * a.D * nv) return;
    row = id / nv;
    t0 = (id - row * nv) * kV;
  }
  const int b = row / a.D, d = row - b * a.D;
  const T* x = static_cast<const T*>(a.x) + b * a.x_batch + d * a.x_channel;
  const int here = min(a.L - t0, kV);
  const Vec now = load_some<T, kV>(x + t0, here);
  Vec before = {};
  if (t0 > 0) before = *reinterpret_cast<const Vec*>(x + t0 - kV);
  const int slot = slot_of(a.slots, a.num_slots, b);
  const int len = slot < 0 ? 0 : length_of(a.lengths, a.L, b);
  float w[K];
#pragma unroll
  for (int k = 0; k < K; k++) w[k] = a.weight[(int64_t)d * K + k];
  const float bias = a.bias ? a.bias[d] : 0.0f;
  T u[K - 1 + kV];  // positions t0-K+1 .. t0+kV-1
#pragma unroll
  for (int i = 0; i < kV; i++) u[K - 1 + i] = now[i];
#pragma unroll
  for (int j = 0; j < K - 1; j++) u[j] = before[kV - K + 1 + j];
  if (t0 == 0 && slot >= 0) {
    if (a.initial_state) {
      const T* first = static_cast<const T*>(a.initial_state) + slot * a.initial_stride + (int64_t)d * (K - 1);
#pragma unroll
      for (int j = 0; j < K - 1; j++) u[j] = first[j];
    }
    // The state is read (above) and written by this thread alone, so it may be updated in place.
    if (K > 1 && a.final_state) {
      T* last = static_cast<T*>(a.final_state) + slot * a.final_stride + (int64_t)d * (K - 1);
#pragma unroll
      for (int j = 0; j < K - 1; j++) {
        const int t = len - (K - 1) + j;
        T v = t >= 0 ? x[t] : T(0.0f);
#pragma unroll
        for (int i = 0; i < K - 1; i++)
          if (t == i - (K - 1)) v = u[i];
        last[j] = v;
      }
    }
  }
  float f[K - 1 + kV];
#pragma unroll
  for (int i = 0; i < K - 1 + kV; i++) f[i] = (float)u[i];
  Vec y;
#pragma unroll
  for (int i = 0; i < kV; i++) {
    float v = bias;
#pragma unroll
    for (int k = 0; k < K; k++) v = fmaf(w[k], f[i + k], v);
    y[i] = T(SILU ? silu(v) : v);
  }
  if (len - t0 < kV)
#pragma unroll
    for (int i = 0; i < kV; i++) y[i] = t0 + i < len ? y[i] : T(0.0f);
  store_some<T, kV>(static_cast<T*>(a.out) + b * a.out_batch + d * a.out_channel + t0, here, y);
}

// Single positions: a thread takes kC channels, whose states lie together.
constexpr int kC = kConvC;

template <class T, int K, bool SILU>
__global__ __launch_bounds__(256) void causal_conv_token(const sc_causal_conv a, int per_row) {
  typedef typename Pack<T, kC>::type Vec;
  const uint32_t id = blockIdx.x * 256u + threadIdx.x;
  const int b = id / (uint32_t)per_row, d = (id - (uint32_t)b * per_row) * kC;
  if (b >= a.B) return;
  const int slot = slot_of(a.slots, a.num_slots, b), n = min(a.D - d, kC);
  const bool on = slot >= 0 && length_of(a.lengths, 1, b) == 1;
  const T* x = static_cast<const T*>(a.x) + b * a.x_batch + d * a.x_channel;
  T* out = static_cast<T*>(a.out) + b * a.out_batch + d * a.out_channel;
  Vec now;
  if (a.x_channel == 1)
    now = load_some<T, kC>(x, n);
  else
#pragma unroll
    for (int i = 0; i < kC; i++) now[i] = i < n ? x[i * a.x_channel] : T(0.0f);
  T u[kC][K];  // a channel's last K - 1 inputs, and the present one
  const T* from = a.initial_state && slot >= 0 ? static_cast<const T*>(a.initial_state) + slot * a.initial_stride + (int64_t)d * (K - 1)
                                               : nullptr;
  const int held = n * (K - 1);
#pragma unroll
  for (int r = 0; r < K - 1; r++) {
    const Vec v = load_some<T, kC>(from + r * kC, from ? held - r * kC : 0);
#pragma unroll
    for (int i = 0; i < kC; i++) u[(r * kC + i) / (K - 1)][(r * kC + i) % (K - 1)] = v[i];
  }
  Vec y;
#pragma unroll
  for (int i = 0; i < kC; i++) {
    u[i][K - 1] = now[i];
    const int c = min(d + i, a.D - 1);
    float v = a.bias ? a.bias[c] : 0.0f;
#pragma unroll
    for (int k = 0; k < K; k++) v = fmaf(a.weight[(int64_t)c * K + k], (float)u[i][k], v);
    if (SILU) v = silu(v);
    y[i] = T(on ? v : 0.0f);
  }
  if (a.out_channel == 1)
    store_some<T, kC>(out, n, y);
  else
#pragma unroll
    for (int i = 0; i < kC; i++)
      if (i < n) out[i * a.out_channel] = y[i];
  if (K > 1 && a.final_state && slot >= 0) {
    T* to = static_cast<T*>(a.final_state) + slot * a.final_stride + (int64_t)d * (K - 1);
#pragma unroll
    for (int r = 0; r < K - 1; r++) {
      Vec v;
#pragma unroll
      for (int i = 0; i < kC; i++) {
        const int c = (r * kC + i) / (K - 1), k = (r * kC + i) % (K - 1);
        v[i] = on ? u[c][k + 1] : u[c][k];
      }
      store_some<T, kC>(to + r * kC, held - r * kC, v);
    }
  }
}

template <class T, int K, bool SILU>
int launch_one(const sc_causal_conv& a, hipStream_t st) {
  if (a.L == 1) {
    const int per_row = (int)ceil_div(a.D, kC);
    hipLaunchKernelGGL((causal_conv_token<T, K, SILU>), dim3((unsigned)(((int64_t)a.B * per_row + 255) / 256)), dim3(256), 0,
                       st, a, per_row);
    return (int)hipGetLastError();
  }
  const int nv = (int)conv_places(a), blocks = (nv + 255) / 256;
  const int64_t rows = (int64_t)a.B * a.D;
  if (conv_own_rows(a))
    hipLaunchKernelGGL((causal_conv_rows<T, K, SILU, true>), dim3((unsigned)(rows * blocks)), dim3(256), 0, st, a, blocks, nv);
  else
    hipLaunchKernelGGL((causal_conv_rows<T, K, SILU, false>), dim3((unsigned)((rows * nv + 255) / 256)), dim3(256), 0, st, a,
                       blocks, nv);
  return (int)hipGetLastError();
}

template <class T, int K>
int launch_act(const sc_causal_conv& a, hipStream_t st) {
  return a.flags & SC_SEQ_SILU ? launch_one<T, K, true>(a, st) : launch_one<T, K, false>(a, st);
}

template <class T>
int launch_taps(const sc_causal_conv& a, hipStream_t st) {
  switch (a.K) {
    case 1: return launch_act<T, 1>(a, st);
    case 2: return launch_act<T, 2>(a, st);
    case 3: return launch_act<T, 3>(a, st);
    case 4: return launch_act<T, 4>(a, st);
    case 5: return launch_act<T, 5>(a, st);
    case 6: return launch_act<T, 6>(a, st);
    case 7: return launch_act<T, 7>(a, st);
    default: return launch_act<T, 8>(a, st);
  }
}

}  // namespace

int launch_causal_conv(const sc_causal_conv& a, void* stream) {
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if (a.dtype == SC_F32) return launch_taps<float>(a, st);
  if (a.dtype == SC_BF16) return launch_taps<__bf16>(a, st);
  return launch_taps<_Float16>(a, st);
}

}  // namespace sc
