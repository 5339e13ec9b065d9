// Low-rank adapters of many requests beside a shared projection (sparseconv_adapter_apply).
//
//   out[b] = base[b] + scale[r] up[r] (down[r] x[b]),  r = index[b]
#include <hip/hip_runtime.h>

#include <algorithm>

#include "sequence_device.h"
#include "xcd.h"

namespace sc {

namespace {

typedef float F4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ int adapter_of(const sc_adapter& a, int b) {
  const int r = a.index[b];
  return r >= 0 && r < a.adapters ? r : -1;
}

// ---- Prompts: two products on the matrix cores around R values a position.
//
// Both products have 16 rows of weights as one operand and positions as the other.  A lane loads
// V = 16 bytes' worth of consecutive positions of a row (V matrix columns 16 apart in the tile, so
// column 16 q + j of the tile is position V j + q) and a wavefront 16 V positions: 256 bytes of
// every row.  The order of the summed index within an instruction is free as long as both operands
// agree, so weights come in 16-byte loads too.

template <class T>
struct Tile {
  static constexpr int V = 16 / sizeof(T);    // positions per lane
  static constexpr int L = 16 * V;            // positions per tile
  static constexpr int K = sizeof(T) == 4 ? 4 : 8;  // summed rows per lane and block
  typedef typename Pack<T, V>::type Vec;
  typedef typename Pack<T, K>::type KVec;
};

// acc += a b over the 4 K rows that the wavefront's lanes hold, K values a lane.
__device__ __forceinline__ F4 mfma(Tile<__bf16>::KVec a, Tile<__bf16>::KVec b, F4 acc) {
  typedef __bf16 B8 __attribute__((ext_vector_type(8)));
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16((B8)a, (B8)b, acc, 0, 0, 0);
}
__device__ __forceinline__ F4 mfma(Tile<_Float16>::KVec a, Tile<_Float16>::KVec b, F4 acc) {
  typedef _Float16 H8 __attribute__((ext_vector_type(8)));
  return __builtin_amdgcn_mfma_f32_16x16x32_f16((H8)a, (H8)b, acc, 0, 0, 0);
}
__device__ __forceinline__ F4 mfma(Tile<float>::KVec a, Tile<float>::KVec b, F4 acc) {
#pragma unroll
  for (int i = 0; i < 4; i++) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a[i], b[i], acc, 0, 0, 0);
  return acc;
}

// low[seg][b][r][l] = scale sum over the segment's c of down[r][c] x[b][c][l], fp32.  Four wavefronts
// take every fourth block of 4 K channels and add up in LDS, in order.
template <class T, int RT>
__global__ __launch_bounds__(256) void adapter_down(const sc_adapter a, float* low, int segments, int ltiles) {
  typedef Tile<T> X;
  typedef typename X::Vec Vec;
  typedef typename X::KVec KVec;
  __shared__ float sum[RT * 16][X::L];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 15, part = lane >> 4;
  int id = xcd_logical(blockIdx.x, gridDim.x);
  const int l0 = id % ltiles * X::L;
  id /= ltiles;
  const int seg = id % segments, b = id / segments;
  const int ad = adapter_of(a, b);
  if (ad < 0) return;
  const int blocks = (a.C + 4 * X::K - 1) / (4 * X::K), per = (blocks + segments - 1) / segments;
  const int end = min(blocks, (seg + 1) * per);
  const T* w = static_cast<const T*>(a.down) + (int64_t)ad * a.R * a.C;
  const int l = l0 + X::V * col, nl = a.L - l;
  const T* x = static_cast<const T*>(a.x) + b * a.x_batch + l;
  F4 acc[RT][X::V];
#pragma unroll
  for (int t = 0; t < RT; t++)
#pragma unroll
    for (int q = 0; q < X::V; q++) acc[t][q] = F4{0.0f, 0.0f, 0.0f, 0.0f};
  for (int blk = seg * per + wave; blk < end; blk += 4) {
    const int c = blk * 4 * X::K + part * X::K, nc = a.C - c;
    Vec xv[X::K];
    KVec wv[RT];
#pragma unroll
    for (int i = 0; i < X::K; i++) xv[i] = load_some<T, X::V>(x + (int64_t)(c + i) * a.x_channel, i < nc ? nl : 0);
#pragma unroll
    for (int t = 0; t < RT; t++) {
      const int r = t * 16 + col;
      wv[t] = load_some<T, X::K>(w + (int64_t)r * a.C + c, r < a.R ? nc : 0);
    }
#pragma unroll
    for (int q = 0; q < X::V; q++) {
      KVec xq;
#pragma unroll
      for (int i = 0; i < X::K; i++) xq[i] = xv[i][q];
#pragma unroll
      for (int t = 0; t < RT; t++) acc[t][q] = mfma(wv[t], xq, acc[t][q]);
    }
  }
  for (int k = 0; k < 4; k++) {
    if (wave == k)
#pragma unroll
      for (int t = 0; t < RT; t++)
#pragma unroll
        for (int i = 0; i < 4; i++)
#pragma unroll
          for (int q = 0; q < X::V; q++) {
            float& s = sum[t * 16 + part * 4 + i][X::V * col + q];
            s = k ? s + acc[t][q][i] : acc[t][q][i];
          }
    __syncthreads();
  }
  const float scale = a.scale ? a.scale[ad] : 1.0f;
  float* to = low + ((int64_t)seg * a.B + b) * a.R * a.L;
  for (int i = threadIdx.x; i < a.R * X::L; i += 256) {
    const int r = i / X::L, j = i % X::L;
    if (l0 + j < a.L) to[(int64_t)r * a.L + l0 + j] = scale * sum[r][j];
  }
}

// The sum over the segments of 8 rows of low from r0 on, at one position; 0 past R.
__device__ __forceinline__ void low_rows(const sc_adapter& a, const float* low, int segments, int b, int r0, int l,
                                         float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; i++) {
    v[i] = 0.0f;
    if (r0 + i < a.R && l < a.L)
      for (int s = 0; s < segments; s++) v[i] += low[(((int64_t)s * a.B + b) * a.R + r0 + i) * a.L + l];
  }
}

// out = base + up low for `mrows` output channels of one tile of positions.  low is held in LDS as the
// matrix cores take it: fp32 as it is; for 16-bit types as the sum of two 16-bit values, which share
// one instruction (its 32 summed rows are 16 high parts and the same 16 low parts), so the
// intermediate keeps 16 bits.  fp16's narrow exponent is met by a power of two per position.
template <class T>
__global__ __launch_bounds__(256) void adapter_up(const sc_adapter a, const float* low, int segments, int ltiles,
                                                  int mtiles, int mrows) {
  typedef Tile<T> X;
  typedef typename X::Vec Vec;
  typedef typename X::KVec KVec;
  extern __shared__ float lds[];
  constexpr bool kWide = sizeof(T) == 4;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, col = lane & 15, part = lane >> 4;
  int id = xcd_logical(blockIdx.x, gridDim.x);
  const int m_begin = id % mtiles * mrows;
  id /= mtiles;
  const int l0 = id % ltiles * X::L, b = id / ltiles;
  const int ad = adapter_of(a, b);
  const int R16 = (a.R + 15) / 16;
  float back[X::V];  // 2^e of the lane's positions
#pragma unroll
  for (int q = 0; q < X::V; q++) back[q] = 1.0f;
  if (ad >= 0) {
    if constexpr (kWide) {
      for (int i = tid; i < R16 * 2 * X::L; i += 256) {
        const int j = i % X::L, r0 = i / X::L * 8;
        float v[8];
        low_rows(a, low, segments, b, r0, l0 + j, v);
#pragma unroll
        for (int k = 0; k < 8; k++) lds[(r0 + k) * X::L + j] = v[k];
      }
      __syncthreads();
    } else {
      // two threads a position, each with every other 8 rows
      const int j = tid & 127, half = tid >> 7;
      float forth = 1.0f;
      if constexpr (__is_same(T, _Float16)) {
        float* most = lds;  // [2][128], before the operands take the place
        float m = 0.0f;
        for (int k = 0; k < R16; k++) {
          float v[8];
          low_rows(a, low, segments, b, k * 16 + half * 8, l0 + j, v);
#pragma unroll
          for (int i = 0; i < 8; i++) m = fmaxf(m, fabsf(v[i]));
        }
        most[half * 128 + j] = m;
        __syncthreads();
        m = fmaxf(most[j], most[128 + j]);
        // the largest lands in [2^9, 2^10): its low part is exact, and no product overflows fp32
        const int e = m > 0.0f && m < __builtin_inff() ? 10 - __builtin_amdgcn_frexp_expf(m) : 0;
        forth = __builtin_ldexpf(1.0f, min(e, 126));
        __syncthreads();
        if (half == 0) most[j] = __builtin_ldexpf(1.0f, -min(e, 126));
        __syncthreads();
#pragma unroll
        for (int q = 0; q < X::V; q++) back[q] = most[X::V * col + q];
        __syncthreads();
      }
      KVec* op = reinterpret_cast<KVec*>(lds);  // [R16][8 tiles][64 lanes]
      for (int k = 0; k < R16; k++) {
        float v[8];
        low_rows(a, low, segments, b, k * 16 + half * 8, l0 + j, v);
        KVec hi, lo;
#pragma unroll
        for (int i = 0; i < 8; i++) {
          const float s = v[i] * forth;
          hi[i] = T(s);
          const float rest = s - (float)hi[i];
          lo[i] = T(__builtin_isfinite(rest) ? rest : 0.0f);
        }
        KVec* to = op + (k * 8 + j % 8) * 64 + j / 8 + half * 16;
        to[0] = hi;
        to[32] = lo;
      }
      __syncthreads();
    }
  }
  const T* w = static_cast<const T*>(a.up) + (int64_t)max(ad, 0) * a.M * a.R;
  const int l = l0 + X::V * col, nl = a.L - l;
  const T* base = static_cast<const T*>(a.base);
  if (base) base += b * a.base_batch + l;
  T* out = static_cast<T*>(a.out) + b * a.out_batch + l;
  const int m_end = min(a.M, m_begin + mrows);
  for (int m0 = m_begin + wave * 16; m0 < m_end; m0 += 64) {
    Vec bv[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const int m = m0 + part * 4 + i;
      bv[i] = load_some<T, X::V>(base + (int64_t)m * a.base_channel, base && m < m_end ? nl : 0);
    }
    F4 acc[X::V];
#pragma unroll
    for (int q = 0; q < X::V; q++) acc[q] = F4{0.0f, 0.0f, 0.0f, 0.0f};
    if (ad >= 0) {
      const int m = m0 + col;
      for (int k = 0; k < R16; k++) {
        const int r = k * 16 + (kWide ? part * 4 : (part & 1) * 8);
        const KVec wv = load_some<T, X::K>(w + (int64_t)m * a.R + r, m < m_end ? a.R - r : 0);
        if constexpr (kWide) {
          F4 lv[4];
#pragma unroll
          for (int i = 0; i < 4; i++) lv[i] = *reinterpret_cast<const F4*>(lds + (r + i) * X::L + 4 * col);
#pragma unroll
          for (int q = 0; q < X::V; q++) acc[q] = mfma(wv, KVec{lv[0][q], lv[1][q], lv[2][q], lv[3][q]}, acc[q]);
        } else {
          const KVec* op = reinterpret_cast<const KVec*>(lds) + k * 8 * 64 + lane;
#pragma unroll
          for (int q = 0; q < X::V; q++) acc[q] = mfma(wv, op[q * 64], acc[q]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const int m = m0 + part * 4 + i;
      Vec v;
#pragma unroll
      for (int q = 0; q < X::V; q++) v[q] = T(fmaf(acc[q][i], back[q], (float)bv[i][q]));
      if (m < m_end) store_some<T, X::V>(out + (int64_t)m * a.out_channel, nl, v);
    }
  }
}

// ---- Single positions: one launch.  A workgroup takes one position's `mrows` output channels and
// makes the R values for itself (down[r] comes from L2 after the first workgroup has read it), which
// costs less than a second launch.
constexpr int kToken = 512;

template <class T>
__global__ __launch_bounds__(kToken) void adapter_token(const sc_adapter a, int mtiles, int mrows) {
  constexpr int V = 16 / sizeof(T);
  typedef typename Pack<T, V>::type Vec;
  __shared__ float low[128];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int id = xcd_logical(blockIdx.x, gridDim.x);
  const int mt = id % mtiles;
  id /= mtiles;
  const int l = id % a.L, b = id / a.L;
  const int ad = adapter_of(a, b);
  if (ad >= 0) {
    const T* x = static_cast<const T*>(a.x) + b * a.x_batch + l;
    const T* w = static_cast<const T*>(a.down) + (int64_t)ad * a.R * a.C;
    const float scale = a.scale ? a.scale[ad] : 1.0f;
    for (int r = wave; r < a.R; r += kToken / 64) {
      const T* wr = w + (int64_t)r * a.C;
      float v = 0.0f;
      for (int c = lane * V; c < a.C; c += 64 * V) {
        const int n = a.C - c;
        const Vec wv = load_some<T, V>(wr + c, n);
        Vec xv;
        if (a.x_channel == 1) {
          xv = load_some<T, V>(x + c, n);
        } else {
#pragma unroll
          for (int i = 0; i < V; i++) xv[i] = i < n ? x[(c + i) * a.x_channel] : T(0.0f);
        }
#pragma unroll
        for (int i = 0; i < V; i++) v = fmaf((float)wv[i], (float)xv[i], v);
      }
#pragma unroll
      for (int m = 32; m; m >>= 1) v += __shfl_xor(v, m);
      if (lane == 0) low[r] = scale * v;
    }
  }
  __syncthreads();
  const int m_end = min(a.M, (mt + 1) * mrows);
  for (int m = mt * mrows + threadIdx.x; m < m_end; m += kToken) {
    float v = a.base ? (float)static_cast<const T*>(a.base)[b * a.base_batch + m * a.base_channel + l] : 0.0f;
    if (ad >= 0) {
      const T* w = static_cast<const T*>(a.up) + ((int64_t)ad * a.M + m) * a.R;
      float s = 0.0f;
      for (int r = 0; r < a.R; r += V) {
        const Vec wv = load_some<T, V>(w + r, a.R - r);
#pragma unroll
        for (int i = 0; i < V; i++)
          if (r + i < a.R) s = fmaf((float)wv[i], low[r + i], s);
      }
      v += s;
    }
    static_cast<T*>(a.out)[b * a.out_batch + m * a.out_channel + l] = T(v);
  }
}

struct Plan {
  bool token;
  int ltiles, segments;  // positions' tiles; pieces of C
  int mtiles, mrows;     // output channels' pieces
};

Plan plan_of(const sc_adapter& a, int cus) {
  Plan p{};
  const bool wide = a.dtype == SC_F32;
  p.token = a.L <= 4;
  if (p.token) {
    p.mtiles = (a.M + 2 * kToken - 1) / (2 * kToken);
    p.mrows = (a.M + p.mtiles - 1) / p.mtiles;
    return p;
  }
  p.ltiles = (a.L + (wide ? 64 : 128) - 1) / (wide ? 64 : 128);
  const int64_t tiles = (int64_t)a.B * p.ltiles;
  const int blocks = (a.C + (wide ? 16 : 32) - 1) / (wide ? 16 : 32);
  p.segments = (int)std::clamp<int64_t>((2 * cus + tiles - 1) / tiles, 1, std::max(1, std::min(blocks / 8, 8)));
  // an empty last piece would leave its part of the workspace unwritten
  const int per = (blocks + p.segments - 1) / p.segments;
  p.segments = (blocks + per - 1) / per;
  p.mtiles = (int)std::clamp<int64_t>((8 * cus + tiles - 1) / tiles, 1, (a.M + 63) / 64);
  p.mrows = ((a.M + p.mtiles - 1) / p.mtiles + 63) / 64 * 64;
  p.mtiles = (a.M + p.mrows - 1) / p.mrows;
  return p;
}

template <class T>
int launch_type(const sc_adapter& a, int cus, hipStream_t st) {
  const Plan p = plan_of(a, cus);
  if (p.token) {
    const int64_t n = (int64_t)a.B * a.L * p.mtiles;
    hipLaunchKernelGGL((adapter_token<T>), dim3((unsigned)n), dim3(kToken), 0, st, a, p.mtiles, p.mrows);
    return (int)hipGetLastError();
  }
  float* low = static_cast<float*>(a.workspace);
  const int64_t nd = (int64_t)a.B * p.ltiles * p.segments, nu = (int64_t)a.B * p.ltiles * p.mtiles;
  const dim3 gd((unsigned)nd), gu((unsigned)nu), block(256);
  if (a.R <= 16)
    hipLaunchKernelGGL((adapter_down<T, 1>), gd, block, 0, st, a, low, p.segments, p.ltiles);
  else if (a.R <= 32)
    hipLaunchKernelGGL((adapter_down<T, 2>), gd, block, 0, st, a, low, p.segments, p.ltiles);
  else if (a.R <= 64)
    hipLaunchKernelGGL((adapter_down<T, 4>), gd, block, 0, st, a, low, p.segments, p.ltiles);
  else
    hipLaunchKernelGGL((adapter_down<T, 8>), gd, block, 0, st, a, low, p.segments, p.ltiles);
  if (const int e = (int)hipGetLastError()) return e;
  const int R16 = (a.R + 15) / 16;
  const int lds = sizeof(T) == 4 ? R16 * 16 * 64 * 4 : R16 * 8 * 64 * 16;
  hipLaunchKernelGGL((adapter_up<T>), gu, block, lds, st, a, low, p.segments, p.ltiles, p.mtiles, p.mrows);
  return (int)hipGetLastError();
}

}  // namespace

int64_t adapter_workspace(const sc_adapter& a, int cus) {
  const Plan p = plan_of(a, cus);
  return p.token ? 0 : (int64_t)p.segments * a.B * a.R * a.L * 4;
}

int launch_adapter(const sc_adapter& a, int cus, void* stream) {
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if (a.dtype == SC_F32) return launch_type<float>(a, cus, st);
  if (a.dtype == SC_BF16) return launch_type<__bf16>(a, cus, st);
  return launch_type<_Float16>(a, cus, st);
}

}  // namespace sc
