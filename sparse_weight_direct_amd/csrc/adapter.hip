// Low-rank adapters of many requests beside a shared projection (sparseconv_adapter_apply).
//
//   out[b] = base[b] + scale[r] up[r] (down[r] x[b]),  r = index[b]
//
// Bound by memory: x and base are read and out is written once; the R values a position between the two
// products are a workspace that stays in L2 (R / (C + 2 M) of the rest).  Measured: fp32, 8 x 2048 -> 4096
// channels x 1024 positions, R = 16: 72 us (16 and 56 for the two products), 4.7 TB/s, where a copy of 1 GiB
// runs at 5.1; bf16, 12 x 1001 -> 1500 x 333, R = 24: 19.0 us (7 and 12): each of a tile's 12
// workgroups of the second product reads all R values of the four pieces of C again, 64 KB from L2.  64 single positions of 4096 -> 4096 channels, 32 adapters, bf16: 8.2 us in one launch.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "sequence_device.h"
#include "sequence_plan.h"
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

// A tile's lane starts at position l0 + V col, or where its V positions would pass the row's end at
// L - V: every access is whole, and what two lanes then share only the first of them stores.  (L >= V.)
__device__ __forceinline__ int lane_start(int l0, int V, int col, int L) { return min(l0 + V * col, L - V); }

// low[seg][b][r][l] = scale sum over the segment's c of down[r][c] x[b][c][l], fp32.  NW wavefronts
// take every NW-th block of 4 K channels; their sums are added in LDS, in order.
template <class T, int RT, int NW>
__global__ __launch_bounds__(64 * NW) void adapter_down(const sc_adapter a, float* low, int segments, int ltiles, int rpieces) {
  typedef Tile<T> X;
  typedef typename X::Vec Vec;
  typedef typename X::KVec KVec;
  __shared__ float sum[NW][16][X::L];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 15, part = lane >> 4;
  int id = xcd_logical(blockIdx.x, gridDim.x);
  const int l0 = id % ltiles * X::L;
  id /= ltiles;
  const int r0 = id % rpieces * (16 * RT);
  id /= rpieces;
  const int seg = id % segments, b = id / segments;
  const int ad = adapter_of(a, b);
  if (ad < 0) return;
  const int blocks = (a.C + 4 * X::K - 1) / (4 * X::K), per = (blocks + segments - 1) / segments;
  const int end = min(blocks, (seg + 1) * per);
  const T* x = static_cast<const T*>(a.x) + b * a.x_batch + lane_start(l0, X::V, col, a.L);
  const T* w[RT];  // rows past R repeat the last one, and their sums are dropped
#pragma unroll
  for (int t = 0; t < RT; t++)
    w[t] = static_cast<const T*>(a.down) + ((int64_t)ad * a.R + min(r0 + t * 16 + col, a.R - 1)) * a.C;
  F4 acc[RT][X::V];
#pragma unroll
  for (int t = 0; t < RT; t++)
#pragma unroll
    for (int q = 0; q < X::V; q++) acc[t][q] = F4{0.0f, 0.0f, 0.0f, 0.0f};
  auto product = [&](const Vec(&xv)[X::K], const KVec(&wv)[RT]) {
#pragma unroll
    for (int q = 0; q < X::V; q++) {
      KVec xq;
#pragma unroll
      for (int i = 0; i < X::K; i++) xq[i] = xv[i][q];
#pragma unroll
      for (int t = 0; t < RT; t++) acc[t][q] = mfma(wv[t], xq, acc[t][q]);
    }
  };
  int blk = seg * per + wave;
  const int whole = min(end, a.C / (4 * X::K));
#pragma unroll 2
  for (; blk < whole; blk += NW) {
    const int c = blk * 4 * X::K + part * X::K;
    Vec xv[X::K];
    KVec wv[RT];
#pragma unroll
    for (int i = 0; i < X::K; i++) xv[i] = *reinterpret_cast<const Vec*>(x + (c + i) * a.x_channel);
#pragma unroll
    for (int t = 0; t < RT; t++) wv[t] = *reinterpret_cast<const KVec*>(w[t] + c);
    product(xv, wv);
  }
  if (blk < end) {  // the last channels; past them the last one is read, and zeros take its place
    const int c = blk * 4 * X::K + part * X::K;
    Vec xv[X::K];
    KVec wv[RT];
#pragma unroll
    for (int i = 0; i < X::K; i++) {
      xv[i] = *reinterpret_cast<const Vec*>(x + min(c + i, a.C - 1) * a.x_channel);
#pragma unroll
      for (int t = 0; t < RT; t++) wv[t][i] = w[t][min(c + i, a.C - 1)];
    }
#pragma unroll
    for (int i = 0; i < X::K; i++)
      if (c + i >= a.C) {
        xv[i] = Vec{};
#pragma unroll
        for (int t = 0; t < RT; t++) wv[t][i] = T(0.0f);
      }
    product(xv, wv);
  }
  const float scale = a.scale ? a.scale[ad] : 1.0f;
  float* to = low + ((int64_t)seg * a.B + b) * a.R * a.L;
#pragma unroll
  for (int t = 0; t < RT; t++) {
    if (t) __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; i++)
#pragma unroll
      for (int q = 0; q < X::V; q += 4)
        *reinterpret_cast<F4*>(&sum[wave][part * 4 + i][X::V * col + q]) =
            F4{acc[t][q][i], acc[t][q + 1][i], acc[t][q + 2][i], acc[t][q + 3][i]};
    __syncthreads();
    for (int i = threadIdx.x; i < 16 * X::L; i += 64 * NW) {
      const int r = i / X::L, j = i % X::L;
      float v = 0.0f;
#pragma unroll
      for (int k = 0; k < NW; k++) v += sum[k][r][j];
      const int own = l0 + j / X::V * X::V, l = lane_start(l0, X::V, j / X::V, a.L) + j % X::V;
      if (r0 + t * 16 + r < a.R && l >= own) to[(int64_t)(r0 + t * 16 + r) * a.L + l] = scale * v;
    }
  }
}

// The sum over S segments of 8 rows of low from r0 on, at one position; 0 past R (where the last row is
// read instead).  No branch stands between the 8 S loads: they come from L2 and are asked for at once.
template <int S>
__device__ __forceinline__ void low_rows(const sc_adapter& a, const float* low, int b, int r0, int l, float (&v)[8]) {
  float u[S][8];
#pragma unroll
  for (int s = 0; s < S; s++) {
    const float* p = low + ((int64_t)s * a.B + b) * a.R * a.L + l;
#pragma unroll
    for (int i = 0; i < 8; i++) u[s][i] = p[(int64_t)min(r0 + i, a.R - 1) * a.L];
  }
#pragma unroll
  for (int i = 0; i < 8; i++) {
    v[i] = u[0][i];
#pragma unroll
    for (int s = 1; s < S; s++) v[i] += u[s][i];
    v[i] = r0 + i < a.R ? v[i] : 0.0f;
  }
}

// out = base + up low for `mrows` output channels of one tile of positions.  low is held in LDS as the
// matrix cores take it: fp32 as it is; for 16-bit types as the sum of two 16-bit values, which share
// one instruction (its 32 summed rows are 16 high parts and the same 16 low parts), so the
// intermediate keeps 16 bits (bf16) or 22 (fp16): a choice, by which an output is off by up to 2^-16 (2^-22)
// of its terms' magnitudes before its own rounding, which is off by 2^-8 (2^-11) of their sum.  fp16's
// narrow exponent is met by a power of two per position.  Where something infinite meets the parts (a
// weight, whose product with a part that is 0 or has the other sign is NaN, or a value that only fp32
// holds) they are no longer the value: sums that are not finite are made again from the fp32 values.
// The next 16 channels' base is on its way while these are computed and stored.
template <class T, int S, int WL>
__global__ __launch_bounds__(256, 4) void adapter_up(const sc_adapter a, const float* low, int ltiles, int mtiles, int mrows) {
  typedef Tile<T> X;
  typedef typename X::Vec Vec;
  typedef typename X::KVec KVec;
  extern __shared__ float lds[];
  constexpr bool kWide = sizeof(T) == 4;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, col = lane & 15, part = lane >> 4;
  constexpr int WM = 4 / WL;  // wavefronts side by side along the positions, and along the channels
  int id = xcd_logical(blockIdx.x, gridDim.x);
  const int lset = (ltiles + WL - 1) / WL, lt0 = id % lset * WL, mine = wave % WL;
  id /= lset;
  const int m_begin = id % mtiles * mrows, b = id / mtiles;
  const int ad = adapter_of(a, b);
  const int R16 = (a.R + 15) / 16, tile_words = R16 * (kWide ? 16 * X::L : 2048);
  const int l0 = (lt0 + mine) * X::L, own = l0 + X::V * col, l = lane_start(l0, X::V, col, a.L);
  const T* base = static_cast<const T*>(a.base);
  if (base) base += b * a.base_batch + l;
  const int m_end = lt0 + mine < ltiles ? min(a.M, m_begin + mrows) : 0;
  Vec next[4] = {};
  auto fetch = [&](int m0) {
    if (base)
#pragma unroll
      for (int i = 0; i < 4; i++)
        next[i] = *reinterpret_cast<const Vec*>(base + min(m0 + part * 4 + i, m_end - 1) * a.base_channel);
  };
  int m0 = m_begin + wave / WL * 16;
  if (m0 < m_end) fetch(m0);
  float back[X::V];  // 2^e of the lane's positions
#pragma unroll
  for (int q = 0; q < X::V; q++) back[q] = 1.0f;
  if (ad >= 0) {
    if constexpr (kWide) {
      for (int i = tid; i < WL * R16 * 2 * X::L; i += 256) {
        const int j = i % X::L, r0 = i / X::L % (R16 * 2) * 8, tile = i / X::L / (R16 * 2);
        float v[8];
        low_rows<S>(a, low, b, r0, lane_start((lt0 + tile) * X::L, X::V, j / X::V, a.L) + j % X::V, v);
#pragma unroll
        for (int k = 0; k < 8; k++) lds[tile * tile_words + (r0 + k) * X::L + j] = v[k];
      }
      __syncthreads();
    } else {
      // two threads a position, each with every other 8 rows
      const int j = tid & 127, half = tid >> 7;
      for (int tile = 0; tile < WL; tile++) {
        const int at = lane_start((lt0 + tile) * X::L, X::V, j / X::V, a.L) + j % X::V;
        float* at_lds = lds + tile * tile_words;
        float forth = 1.0f;
        if constexpr (__is_same(T, _Float16)) {
          float* most = at_lds;  // [2][128], before the operands take the place
          float m = 0.0f;
          for (int k = 0; k < R16; k++) {
            float v[8];
            low_rows<S>(a, low, b, k * 16 + half * 8, at, v);
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
          if (tile == mine)
#pragma unroll
            for (int q = 0; q < X::V; q++) back[q] = most[X::V * col + q];
          __syncthreads();
        }
        KVec* op = reinterpret_cast<KVec*>(at_lds);  // [R16][8 tiles][64 lanes]
        for (int k = 0; k < R16; k++) {
          float v[8];
          low_rows<S>(a, low, b, k * 16 + half * 8, at, v);
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
      }
      __syncthreads();
    }
  }
  const float* operand = lds + mine * tile_words;
  const T* w = static_cast<const T*>(a.up) + (int64_t)max(ad, 0) * a.M * a.R;
  T* out = static_cast<T*>(a.out) + b * a.out_batch + l;
  for (; m0 < m_end; m0 += 16 * WM) {
    Vec bv[4];
#pragma unroll
    for (int i = 0; i < 4; i++) bv[i] = next[i];
    if (m0 + 16 * WM < m_end) fetch(m0 + 16 * WM);
    F4 acc[X::V];
#pragma unroll
    for (int q = 0; q < X::V; q++) acc[q] = F4{0.0f, 0.0f, 0.0f, 0.0f};
    if (ad >= 0) {
      const T* wm = w + (int64_t)min(m0 + col, m_end - 1) * a.R;
      for (int k = 0; k < R16; k++) {
        const int r = k * 16 + (kWide ? part * 4 : (part & 1) * 8);
        const KVec wv = k * 16 + 16 <= a.R ? *reinterpret_cast<const KVec*>(wm + r) : load_some<T, X::K>(wm + r, a.R - r);
        if constexpr (kWide) {
          F4 lv[4];
#pragma unroll
          for (int i = 0; i < 4; i++) lv[i] = *reinterpret_cast<const F4*>(operand + (r + i) * X::L + 4 * col);
#pragma unroll
          for (int q = 0; q < X::V; q++) acc[q] = mfma(wv, KVec{lv[0][q], lv[1][q], lv[2][q], lv[3][q]}, acc[q]);
        } else {
          const KVec* op = reinterpret_cast<const KVec*>(operand) + k * 8 * 64 + lane;
#pragma unroll
          for (int q = 0; q < X::V; q++) acc[q] = mfma(wv, op[q * 64], acc[q]);
        }
      }
      if constexpr (!kWide) {
        float none = 0.0f;
#pragma unroll
        for (int q = 0; q < X::V; q++)
#pragma unroll
          for (int i = 0; i < 4; i++) none = fmaf(acc[q][i], 0.0f, none);
        if (__builtin_expect(__any(none != 0.0f), false)) {
          int at = l, k = part;
          asm volatile("" : "+v"(at), "+v"(k));  // keeps what follows from them out of the loop's registers
#pragma unroll
          for (int q = 0; q < X::V; q++) {
            F4 again = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
            for (int r0 = 0; r0 < a.R; r0 += 4) {
              const int r = r0 + k;
              float v = 0.0f;
              if (r < a.R)
#pragma unroll 1
                for (int s = 0; s < S; s++) v += low[(((int64_t)s * a.B + b) * a.R + r) * a.L + at + q];
              again = __builtin_amdgcn_mfma_f32_16x16x4f32(r < a.R ? (float)wm[r] : 0.0f, v, again, 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < 4; i++) acc[q][i] = __builtin_isfinite(acc[q][i]) ? acc[q][i] : again[i] / back[q];
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const int m = m0 + part * 4 + i;
      Vec v;
#pragma unroll
      for (int q = 0; q < X::V; q++) v[q] = T(fmaf(acc[q][i], back[q], (float)bv[i][q]));
      if (m >= m_end) continue;
      T* to = out + m * a.out_channel;
      if (l == own) {
        *reinterpret_cast<Vec*>(to) = v;
      } else {
#pragma unroll
        for (int q = 0; q < X::V; q++)
          if (l + q >= own) to[q] = v[q];
      }
    }
  }
}

// ---- Single positions: one launch.  A workgroup takes one position's `mrows` output channels and
// makes the R values for itself (down[r] comes from L2 after the first workgroup has read it), which
// costs less than a second launch.  Its time is latency: what the second half needs (the base and the
// first kFront values of every row of up) is asked for before the first half begins.
constexpr int kToken = kAdapterToken;          // threads
constexpr int kTokenRows = kAdapterTokenRows;  // output channels per thread
constexpr int kFront = 16;  // (what follows takes them in 16s too)

// RW: rows of down per wavefront at a time.
template <class T, int RW>
__global__ __launch_bounds__(kToken) void adapter_token(const sc_adapter a, int mtiles, int mrows) {
  constexpr int V = 16 / sizeof(T), F = kFront / V;
  typedef typename Pack<T, V>::type Vec;
  __shared__ float low[128];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int id = xcd_logical(blockIdx.x, gridDim.x);
  const int mt = id % mtiles;
  id /= mtiles;
  const int l = id % a.L, b = id / a.L;
  const int ad = adapter_of(a, b);
  const T* up = static_cast<const T*>(a.up) + (int64_t)max(ad, 0) * a.M * a.R;
  const T* base = a.base ? static_cast<const T*>(a.base) + b * a.base_batch + l : nullptr;
  T first[kTokenRows];
  Vec front[kTokenRows][F];
#pragma unroll
  for (int k = 0; k < kTokenRows; k++) {
    const int m = min(mt * mrows + (int)threadIdx.x + k * kToken, a.M - 1);
    first[k] = base ? base[m * a.base_channel] : T(0.0f);
    if (ad < 0) continue;
#pragma unroll
    for (int f = 0; f < F; f++)
      front[k][f] = f * V + V <= a.R ? *reinterpret_cast<const Vec*>(up + (int64_t)m * a.R + f * V)
                                     : load_some<T, V>(up + (int64_t)m * a.R + f * V, a.R - f * V);
  }
  if (ad >= 0) {
    const T* x = static_cast<const T*>(a.x) + b * a.x_batch + l;
    const T* w = static_cast<const T*>(a.down) + (int64_t)ad * a.R * a.C;
    const float scale = a.scale ? a.scale[ad] : 1.0f;
    auto x_at = [&](int c) {
      if (a.x_channel == 1) return *reinterpret_cast<const Vec*>(x + c);
      Vec v;
#pragma unroll
      for (int i = 0; i < V; i++) v[i] = x[(c + i) * a.x_channel];
      return v;
    };
    // RW rows at a time, four pieces of each in flight
    for (int r = RW * wave; r < a.R; r += RW * (kToken / 64)) {
      const T* wr[RW];
      float v[RW];
#pragma unroll
      for (int k = 0; k < RW; k++) wr[k] = w + (int64_t)min(r + k, a.R - 1) * a.C, v[k] = 0.0f;
      int c = lane * V;
#pragma unroll 4
      for (; c + V <= a.C; c += 64 * V) {
        const Vec xv = x_at(c);
        Vec wv[RW];
#pragma unroll
        for (int k = 0; k < RW; k++) wv[k] = *reinterpret_cast<const Vec*>(wr[k] + c);
#pragma unroll
        for (int k = 0; k < RW; k++)
#pragma unroll
          for (int i = 0; i < V; i++) v[k] = fmaf((float)wv[k][i], (float)xv[i], v[k]);
      }
      for (int i = c; i < a.C && i < c + V; i++) {
        const float xv = (float)x[i * a.x_channel];
#pragma unroll
        for (int k = 0; k < RW; k++) v[k] = fmaf((float)wr[k][i], xv, v[k]);
      }
#pragma unroll
      for (int m = 32; m; m >>= 1)
#pragma unroll
        for (int k = 0; k < RW; k++) v[k] += __shfl_xor(v[k], m);
      if (lane == 0)
#pragma unroll
        for (int k = 0; k < RW; k++)
          if (r + k < a.R) low[r + k] = scale * v[k];
    }
  }
  __syncthreads();
  float s[kTokenRows] = {};
  if (ad >= 0) {
    const T* um[kTokenRows];
#pragma unroll
    for (int k = 0; k < kTokenRows; k++) {
      um[k] = up + (int64_t)min(mt * mrows + (int)threadIdx.x + k * kToken, a.M - 1) * a.R;
#pragma unroll
      for (int r = 0; r < kFront; r++)
        if (r < a.R) s[k] = fmaf((float)front[k][r / V][r % V], low[r], s[k]);
    }
    int r = kFront;
    for (; r + 16 <= a.R; r += 16) {  // sixteen more of every row at once
      Vec wv[kTokenRows][F];
#pragma unroll
      for (int k = 0; k < kTokenRows; k++)
#pragma unroll
        for (int f = 0; f < F; f++) wv[k][f] = *reinterpret_cast<const Vec*>(um[k] + r + f * V);
#pragma unroll
      for (int k = 0; k < kTokenRows; k++)
#pragma unroll
        for (int i = 0; i < 16; i++) s[k] = fmaf((float)wv[k][i / V][i % V], low[r + i], s[k]);
    }
    for (; r < a.R; r++)
#pragma unroll
      for (int k = 0; k < kTokenRows; k++) s[k] = fmaf((float)um[k][r], low[r], s[k]);
  }
#pragma unroll
  for (int k = 0; k < kTokenRows; k++) {
    const int m = mt * mrows + threadIdx.x + k * kToken;
    if (m < a.M) static_cast<T*>(a.out)[b * a.out_batch + m * a.out_channel + l] = T((float)first[k] + s[k]);
  }
}

template <class T, int S>
int launch_up(const sc_adapter& a, const AdapterPlan& p, int lds, const float* low, hipStream_t st) {
  const dim3 grid((unsigned)p.up_blocks);
  if (p.wide)
    hipLaunchKernelGGL((adapter_up<T, S, 4>), grid, dim3(256), 4 * lds, st, a, low, p.ltiles, p.mtiles, p.mrows);
  else
    hipLaunchKernelGGL((adapter_up<T, S, 1>), grid, dim3(256), lds, st, a, low, p.ltiles, p.mtiles, p.mrows);
  return (int)hipGetLastError();
}

template <class T>
int launch_type(const sc_adapter& a, int cus, hipStream_t st) {
  const AdapterPlan p = adapter_plan(a, cus);
  if (p.token) {
    const dim3 grid((unsigned)p.up_blocks);
    if (a.R <= 16)
      hipLaunchKernelGGL((adapter_token<T, 2>), grid, dim3(kToken), 0, st, a, p.mtiles, p.mrows);
    else
      hipLaunchKernelGGL((adapter_token<T, 4>), grid, dim3(kToken), 0, st, a, p.mtiles, p.mrows);
    return (int)hipGetLastError();
  }
  float* low = static_cast<float*>(a.workspace);
  const dim3 gd((unsigned)p.down_blocks);
  if (a.R <= 16)
    hipLaunchKernelGGL((adapter_down<T, 1, 8>), gd, dim3(512), 0, st, a, low, p.segments, p.ltiles, p.rpieces);
  else if (a.R <= 32)
    hipLaunchKernelGGL((adapter_down<T, 2, 8>), gd, dim3(512), 0, st, a, low, p.segments, p.ltiles, p.rpieces);
  else
    hipLaunchKernelGGL((adapter_down<T, 4, 4>), gd, dim3(256), 0, st, a, low, p.segments, p.ltiles, p.rpieces);
  if (const int e = (int)hipGetLastError()) return e;
  const int R16 = (a.R + 15) / 16;
  const int lds = sizeof(T) == 4 ? R16 * 16 * 64 * 4 : R16 * 8 * 64 * 16;
  if (p.segments == 1) return launch_up<T, 1>(a, p, lds, low, st);
  if (p.segments == 2) return launch_up<T, 2>(a, p, lds, low, st);
  return launch_up<T, 4>(a, p, lds, low, st);
}

}  // namespace

int64_t adapter_workspace(const sc_adapter& a, int cus) {
  const AdapterPlan p = adapter_plan(a, cus);
  return p.token ? 0 : (int64_t)p.segments * a.B * a.R * a.L * 4;
}

int launch_adapter(const sc_adapter& a, int cus, void* stream) {
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if (a.dtype == SC_F32) return launch_type<float>(a, cus, st);
  if (a.dtype == SC_BF16) return launch_type<__bf16>(a, cus, st);
  return launch_type<_Float16>(a, cus, st);
}

}  // namespace sc
