// Attention of new positions over a paged cache (sparseconv_paged_attention).
//
//   out_i = sum_t p_t v_t / sum_t p_t,  p_t = exp(s_t - m),  s_t = f(scale q_i . k_t) - slope |i - t|
//
// One pass over the context with the running maximum m and sum.  Both products are made transposed,
// S^T = K q^T and O^T = V^T P^T: a lane then has one query (column lane & 15) in both, its maximum, sum and
// factors are the lane's own, P^T goes from the first product's result into the second's operand within the lane, and the cache's
// layouts (keys with contiguous dims, values with contiguous positions) are read in whole 16 bytes as the
// matrix cores take them.  For that the 32 keys of a block are dealt to the rows of two S^T tiles so that a
// lane's eight results are eight (fp32: two times four) consecutive keys.
#include <hip/hip_runtime.h>

#include "attention.h"
#include "attention_plan.h"
#include "matrix_device.h"
#include "xcd.h"

namespace sc {

namespace {

constexpr int kBlock = 32;  // keys
constexpr float kInf = __builtin_inff();

struct Cut {
  int pitch, tiles, splits;
  float* sums;   // [rows][splits][D], unnormalised
  float2* tops;  // [rows][splits]: {maximum (log2), sum of weights}
};

// What limits a tile's rows; the same for all its lanes.
struct Reach {
  int past, len, end, prefix;  // end: keys that there are; prefix <= end
  int first, last;             // the rows' positions among the new ones (those that there are)
  bool any;
};

__device__ __forceinline__ Reach reach_of(const sc_paged_attention& a, int b, int row0, int rows, int pitch) {
  Reach r;
  const int cap = a.width * a.P;
  r.past = a.past[b];
  const bool idle = r.past < 0 || r.past > cap;
  r.len = idle ? 0 : length_of(a.lengths, a.L, b);
  r.past = idle ? 0 : r.past;
  r.end = min(r.past + r.len, cap);
  r.prefix = a.prefix ? min(max(a.prefix[b], 0), r.end) : 0;
  const int h0 = row0 / pitch, h1 = (row0 + rows - 1) / pitch;
  r.first = h0 == h1 ? row0 - h0 * pitch : 0;
  r.last = min(h0 == h1 ? row0 + rows - 1 - h1 * pitch : pitch - 1, r.len - 1);
  r.any = r.first <= r.last;
  return r;
}

// max and sum over the four lanes of a column.
__device__ __forceinline__ float column_max(float v) {
  v = fmaxf(v, __shfl_xor(v, 16));
  return fmaxf(v, __shfl_xor(v, 32));
}
__device__ __forceinline__ float column_sum(float v) {
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}

// tanh.  16-bit types: 1 - 2 / (1 + e^2x), off by 2^-23 of 1, far inside what their weights are rounded to.
template <class T>
__device__ __forceinline__ float tanh_of(float x) {
  if constexpr (sizeof(T) == 4) return tanhf(x);
  return 1.0f - 2.0f * __builtin_amdgcn_rcpf(1.0f + exp2_fast(2.0f * kLog2e * x));
}

// A word of one or two values: the sign bits of the result say which exponents are full (infinities and NaN).
template <class T>
__device__ __forceinline__ uint32_t exponents_full(uint32_t w) {
  if constexpr (sizeof(T) == 4) return (w & 0x7f800000u) + 0x00800000u;
  if constexpr (__is_same(T, __bf16)) return (w & 0x7f807f80u) + 0x00800080u;
  return (w & 0x7c007c00u) + 0x04000400u;
}

typedef uint32_t W4 __attribute__((ext_vector_type(4)));

// ---- Few rows: every wavefront has its own blocks of keys
//
// A workgroup has 16 NT rows of one head of keys and a piece of the context; its four wavefronts take its
// blocks in turn, operands straight from the cache to registers (each byte is read once), the next block's on their
// way while one is computed, and their sums are joined at the end.
template <class T, int DT, int NT>
__global__ __launch_bounds__(256, (2 + NT) * DT * (int)sizeof(T) > 1024 ? 1 : 2) void attend_direct(const sc_paged_attention a, const Cut cut) {
  typedef typename Frag<T>::type V;
  constexpr int N = Frag<T>::N, KF = DT / (4 * N), VF = kBlock / (4 * N), DM = DT / 16;
  constexpr bool kWide = sizeof(T) == 4;
  // fp16's weights lie below 2^14: what is 2^-20 of the largest is still a normal number
  constexpr float kLift = __is_same(T, _Float16) ? 6.0f : 0.0f;
  constexpr int kPitch = DT + 4;
  constexpr bool kAhead = DT * sizeof(T) < 1024;  // else a block's keys and values alone fill the registers
  __shared__ float lds[4 * 16 * kPitch > 4 * 16 * NT * 33 ? 4 * 16 * kPitch : 4 * 16 * NT * 33];
  __shared__ float2 tops[4][16];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), col = lane & 15, part = lane >> 4;
  int id = xcd_logical(blockIdx.x, gridDim.x);
  const int split = id % cut.splits;
  id /= cut.splits;
  const int tile = id % cut.tiles;
  id /= cut.tiles;
  const int g = id % a.G, b = id / a.G, share = a.H / a.G, row0 = tile * 16 * NT;
  const Reach r = reach_of(a, b, row0, 16 * NT, cut.pitch);

  // the rows' positions and queries
  int pos[NT], head[NT], low[NT], pre[NT], most_key[NT];
  bool live[NT], there[NT];
  V q[NT][KF];
#pragma unroll
  for (int t = 0; t < NT; t++) {
    const int row = row0 + t * 16 + col, h = row / cut.pitch, i = row - h * cut.pitch;
    there[t] = h < share && i < a.L;
    live[t] = there[t] && i < r.len;
    pos[t] = live[t] ? r.past + i : -1;
    low[t] = a.window ? pos[t] - a.window + 1 : 0;
    pre[t] = live[t] ? r.prefix : 0;
    most_key[t] = min(pos[t], r.end - 1);
    head[t] = min(g * share + h, a.H - 1);
    const T* p = static_cast<const T*>(a.q) + b * a.q_batch + (int64_t)head[t] * a.D * a.q_channel + i;
#pragma unroll
    for (int f = 0; f < KF; f++)
#pragma unroll
      for (int j = 0; j < N; j++) {
        const int d = f * 4 * N + part * N + j;
        q[t][f][j] = live[t] && d < a.D ? p[d * a.q_channel] : T(0.0f);
      }
  }

  // the blocks: those of the prefix, then those that the window leaves
  const int last_pos = r.past + r.last, first_pos = r.past + r.first;
  const int until = r.any ? max(min(last_pos + 1, r.end), r.prefix) : 0;
  const int from = r.any && a.window ? min(max(first_pos - a.window + 1, 0), until) / kBlock : 0;
  const int np = (r.prefix + kBlock - 1) / kBlock, jump = max(from - np, 0);
  const int blocks = r.any ? max((until + kBlock - 1) / kBlock - jump, 0) : 0;
  const int per = (blocks + cut.splits - 1) / cut.splits, stop = min(blocks, (split + 1) * per);
  auto block_at = [&](int n) { return n < np ? n : n + jump; };
  const int shift = 31 - __builtin_clz(a.P);

  // the pages of a block's two halves, negative where there is none (page 0 is read then, and hidden)
  struct Where {
    int first, second, key;
  };
  const int32_t* table = a.table + b * a.table_batch;
  auto page = [&](int at) {
    const int p = at < a.width ? table[at] : -1;
    return p < a.pages ? p : -1;
  };
  auto find = [&](int blk) { return Where{page(blk * kBlock >> shift), page((blk * kBlock + 16) >> shift), blk * kBlock}; };
  // of key `key` of the block: its dims, and its values of dim 0
  const T* k_head = static_cast<const T*>(a.k_pages) + (int64_t)g * a.P * a.D;
  const T* v_head = static_cast<const T*>(a.v_pages) + (int64_t)g * a.P * a.D;
  auto page_of = [&](Where w, int key) { return max(key & 16 ? w.second : w.first, 0); };
  auto key_at = [&](Where w, int key) { return k_head + page_of(w, key) * a.k_page + ((w.key + key) & (a.P - 1)) * a.D; };
  auto value_at = [&](Where w, int key) { return v_head + page_of(w, key) * a.v_page + ((w.key + key) & (a.P - 1)); };
  V kf[2][KF], vf[DM][VF];
  auto load_k = [&](Where w) {
#pragma unroll
    for (int t = 0; t < 2; t++) {
      const int key = kWide ? 16 * t + col : 8 * (col >> 2) + 4 * t + (col & 3);
      const T* p = key_at(w, key);
#pragma unroll
      for (int f = 0; f < KF; f++) kf[t][f] = *reinterpret_cast<const V*>(p + min(f * 4 * N + part * N, a.D - N));
    }
    if (a.D != DT)
#pragma unroll
      for (int t = 0; t < 2; t++)
#pragma unroll
        for (int f = 0; f < KF; f++)
          kf[t][f] = f * 4 * N + part * N < a.D ? kf[t][f] : V{};
  };
  auto load_v = [&](Where w) {
#pragma unroll
    for (int f = 0; f < VF; f++) {
      const int key = f * 4 * N + part * N;
      const T* p = value_at(w, key);
#pragma unroll
      for (int d = 0; d < DM; d++) vf[d][f] = *reinterpret_cast<const V*>(p + min(d * 16 + col, a.D - 1) * a.P);
    }
  };

  F4 o[DM][NT];
  float top[NT], use[NT], sum[NT], slope[NT];
#pragma unroll
  for (int t = 0; t < NT; t++) {
#pragma unroll
    for (int d = 0; d < DM; d++) o[d][t] = F4{0.0f, 0.0f, 0.0f, 0.0f};
    top[t] = -kInf, use[t] = -kLift, sum[t] = 0.0f;
    slope[t] = a.slopes ? a.slopes[head[t]] * kLog2e : 0.0f;
  }
  const float scale = a.cap > 0.0f ? a.scale / a.cap : a.scale * kLog2e, cap = a.cap * kLog2e;

  int n = split * per + wave;
  Where at, next;
  if (n < stop) {
    at = find(block_at(n));
    if (kAhead) {
      load_k(at);
      load_v(at);
    }
  }
  for (; n < stop; n += 4) {
    const int k0 = at.key, miss = (at.first < 0 ? 1 : 0) | (at.second < 0 ? 2 : 0);
    const bool more = n + 4 < stop;
    if (more) next = find(block_at(n + 4));
    if (!kAhead) load_k(at);
    F4 s[2][NT];
#pragma unroll
    for (int u = 0; u < 2; u++)
#pragma unroll
      for (int t = 0; t < NT; t++) {
        s[u][t] = F4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int f = 0; f < KF; f++) s[u][t] = mma(kf[u][f], q[t][f], s[u][t]);
      }
    if (kAhead && more) load_k(next);
    if (!kAhead) load_v(at);
    // scores in units of log 2
    auto key_of = [&](int lanes, int u, int i) { return k0 + (kWide ? 16 * u + 4 * lanes + i : 8 * lanes + 4 * u + i); };
#pragma unroll
    for (int u = 0; u < 2; u++)
#pragma unroll
      for (int t = 0; t < NT; t++)
#pragma unroll
        for (int i = 0; i < 4; i++) {
          float v = s[u][t][i] * scale;
          if (a.cap > 0.0f) v = cap * tanh_of<T>(v);
          if (a.slopes) v -= slope[t] * fabsf((float)(pos[t] - key_of(part, u, i)));
          s[u][t][i] = v;
        }
    const bool whole = !miss && k0 + kBlock <= r.end &&
                       (k0 + kBlock <= r.prefix || (k0 + kBlock - 1 <= first_pos && (!a.window || k0 >= last_pos - a.window + 1)));
    // all of it without branches: elements of a vector that were written under a lane's condition came out wrong here
    auto hidden = [&](int lanes, int u, int t, int i) {
      const int key = key_of(lanes, u, i);
      return (((miss >> (kWide ? u : lanes >> 1)) & 1) != 0) | ((key >= pre[t]) & ((key > most_key[t]) | (key < low[t])));
    };
    if (!whole)
#pragma unroll
      for (int u = 0; u < 2; u++)
#pragma unroll
        for (int t = 0; t < NT; t++) {
          F4 v = s[u][t];
#pragma unroll
          for (int i = 0; i < 4; i++) v[i] = hidden(part, u, t, i) ? -kInf : v[i];
          s[u][t] = v;
        }
    // the maximum moves where a score passes it by 2^8 (the first ones do)
    bool moves = false;
    float most[NT];
#pragma unroll
    for (int t = 0; t < NT; t++) {
      most[t] = -kInf;
#pragma unroll
      for (int i = 0; i < 4; i++) most[t] = fmaxf(most[t], fmaxf(s[0][t][i], s[1][t][i]));
      moves |= most[t] > top[t] + 8.0f;
    }
    if (__any(moves))
#pragma unroll
      for (int t = 0; t < NT; t++) {
        const float m = fmaxf(top[t], column_max(most[t])), u = m == -kInf ? 0.0f : m;
        const float factor = top[t] == -kInf ? 0.0f : exp2_fast(top[t] - u);
        top[t] = m, use[t] = u - kLift;
        sum[t] *= factor;
#pragma unroll
        for (int d = 0; d < DM; d++)
#pragma unroll
          for (int i = 0; i < 4; i++) o[d][t][i] *= factor;
      }
    V p[NT][VF];
#pragma unroll
    for (int t = 0; t < NT; t++)
#pragma unroll
      for (int u = 0; u < 2; u++)
#pragma unroll
        for (int i = 0; i < 4; i++) {
          const float w = exp2_fast(s[u][t][i] - use[t]);
          sum[t] += w;
          s[u][t][i] = w;
          p[t][kWide ? u : 0][kWide ? i : 4 * u + i] = T(w);
        }
    bool odd = false;
    if (!whole) {
      // nothing that is not there reaches the product, and what only some rows see is looked at: 0 times
      // infinity is no 0
      uint32_t full = 0;
#pragma unroll
      for (int f = 0; f < VF; f++) {
        const int key = f * 4 * N + part * N, left = miss >> (key >> 4 & 1) & 1 ? 0 : r.end - k0 - key;
        W4 keep;
#pragma unroll
        for (int j = 0; j < 4; j++) keep[j] = kWide ? (j < left ? ~0u : 0u) : (2 * j + 1 < left ? ~0u : 2 * j < left ? 0xffffu : 0u);
#pragma unroll
        for (int d = 0; d < DM; d++) {
          const W4 v = __builtin_bit_cast(W4, vf[d][f]) & keep;
          vf[d][f] = __builtin_bit_cast(V, v);
#pragma unroll
          for (int j = 0; j < 4; j++) full |= exponents_full<T>(v[j]);
        }
      }
      odd = __any((full & (kWide ? 0x80000000u : 0x80008000u)) != 0);
    }
    if (__builtin_expect(odd, false)) {
      int lanes = part;
      asm volatile("" : "+v"(lanes));  // keeps what is made of it below out of the loop's registers
      float* w = lds + wave * (16 * NT * 33);
#pragma unroll
      for (int t = 0; t < NT; t++)
#pragma unroll
        for (int u = 0; u < 2; u++)
#pragma unroll
          for (int i = 0; i < 4; i++) w[(t * 16 + col) * 33 + key_of(lanes, u, i) - k0] = hidden(lanes, u, t, i) ? -1.0f : s[u][t][i];
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
#pragma unroll 1
      for (int key = 0; key < kBlock; key++) {
        const T* pv = value_at(at, key);
        if (k0 + key >= r.end || (miss >> (key >> 4) & 1)) continue;
        float weight[NT];
#pragma unroll
        for (int t = 0; t < NT; t++) weight[t] = w[(t * 16 + col) * 33 + key];
#pragma unroll
        for (int d = 0; d < DM; d++)
#pragma unroll
          for (int i = 0; i < 4; i++) {
            const float val = (float)pv[min(d * 16 + 4 * lanes + i, a.D - 1) * a.P];
#pragma unroll
            for (int t = 0; t < NT; t++)
              o[d][t][i] = weight[t] >= 0.0f ? fmaf(weight[t], val, o[d][t][i]) : o[d][t][i];
          }
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
      __builtin_amdgcn_wave_barrier();
    } else {
#pragma unroll
      for (int f = 0; f < VF; f++)
#pragma unroll
        for (int d = 0; d < DM; d++)
#pragma unroll
          for (int t = 0; t < NT; t++) o[d][t] = mma(vf[d][f], p[t][f], o[d][t]);
    }
    if (kAhead && more) load_v(next);
    at = next;
  }

  // the four wavefronts' sums, 16 rows at a time
  const int row = threadIdx.x & 15, piece = threadIdx.x >> 4;
#pragma unroll
  for (int t = 0; t < NT; t++) {
    __syncthreads();
#pragma unroll
    for (int d = 0; d < DM; d++) *reinterpret_cast<F4*>(&lds[(wave * 16 + col) * kPitch + d * 16 + part * 4]) = o[d][t];
    const float total = column_sum(sum[t]);
    if (part == 0) tops[wave][col] = make_float2(top[t], total);
    __syncthreads();
    const int at_row = row0 + t * 16 + row, h = at_row / cut.pitch, i = at_row - h * cut.pitch;
    if (h >= share || i >= a.L) continue;
    float m = -kInf, l = 0.0f, f[4];
#pragma unroll
    for (int w = 0; w < 4; w++) m = fmaxf(m, tops[w][row].x);
#pragma unroll
    for (int w = 0; w < 4; w++) {
      f[w] = tops[w][row].x == -kInf ? 0.0f : exp2_fast(tops[w][row].x - m);
      l += f[w] * tops[w][row].y;
    }
    const bool seen = m > -kInf;  // NaN scores have no maximum either, but they have a sum
    bool none = !seen;
#pragma unroll
    for (int w = 0; w < 4; w++) none = none & (tops[w][row].y == 0.0f);
    none = none | (i >= r.len);  // (where whole blocks are seen, rows that are not there saw them too)
    const int64_t ws_row = ((int64_t)(b * a.G + g) * cut.tiles + tile) * (16 * NT) + t * 16 + row;
    const float by = cut.splits > 1 ? 1.0f : none ? 0.0f : seen ? 1.0f / l : __builtin_nanf("");
    if (cut.splits > 1 && piece == 0) cut.tops[ws_row * cut.splits + split] = make_float2(none ? -kInf : m, none ? 0.0f : seen ? l : __builtin_nanf(""));
    const int64_t out = b * a.out_batch + (int64_t)(g * share + h) * a.D * a.out_channel + i;
    for (int d = piece * (DT / 16); d < min((piece + 1) * (DT / 16), a.D); d++) {
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < 4; w++) v += f[w] != 0.0f ? f[w] * lds[(w * 16 + row) * kPitch + d] : 0.0f;
      v = none ? 0.0f : v * by;
      if (cut.splits > 1)
        cut.sums[(ws_row * cut.splits + split) * a.D + d] = v;
      else if (a.flags & SC_ATT_OUT_F32)
        static_cast<float*>(a.out)[out + d * a.out_channel] = v;
      else
        static_cast<T*>(a.out)[out + d * a.out_channel] = T(v);
    }
  }
}

// The pieces of the context, joined: a wavefront has a row.
template <class T>
__global__ __launch_bounds__(256) void attend_join(const sc_paged_attention a, const Cut cut, int rows) {
  const int lane = threadIdx.x & 63;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int64_t per = (int64_t)cut.tiles * rows;  // of a head of keys
  const int g = row / per % a.G, b = row / per / a.G, share = a.H / a.G;
  if (b >= a.B) return;
  const int at = row % per, h = at / cut.pitch, i = at - h * cut.pitch;
  if (h >= share || i >= a.L) return;
  const float2* tops = cut.tops + row * cut.splits;
  float m = -kInf, l = 0.0f;
  float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int s = 0; s < cut.splits; s++) m = fmaxf(m, tops[s].x);
  for (int s = 0; s < cut.splits; s++) {
    const float2 e = tops[s];
    if (e.y == 0.0f) continue;
    const float f = e.x == -kInf ? 1.0f : exp2_fast(e.x - m);  // without a maximum: NaN
    l += f * e.y;
    const float* p = cut.sums + (row * cut.splits + s) * a.D;
#pragma unroll
    for (int k = 0; k < 4; k++)
      if (lane + 64 * k < a.D) v[k] += f * p[lane + 64 * k];
  }
  const float by = l == 0.0f ? 0.0f : 1.0f / l;
  const int64_t out = b * a.out_batch + (int64_t)(g * share + h) * a.D * a.out_channel + i;
#pragma unroll
  for (int k = 0; k < 4; k++) {
    const int d = lane + 64 * k;
    if (d >= a.D) continue;
    if (a.flags & SC_ATT_OUT_F32)
      static_cast<float*>(a.out)[out + d * a.out_channel] = v[k] * by;
    else
      static_cast<T*>(a.out)[out + d * a.out_channel] = T(v[k] * by);
  }
}

template <class T, int DT, int NT>
int launch_direct(const sc_paged_attention& a, const AttendPlan& p, const Cut& cut, hipStream_t st) {
  const int64_t blocks = (int64_t)a.B * a.G * p.groups();
  hipLaunchKernelGGL((attend_direct<T, DT, NT>), dim3((unsigned)blocks), dim3(256), 0, st, a, cut);
  return (int)hipGetLastError();
}

template <class T, int DT>
int launch_dims(const sc_paged_attention& a, const AttendPlan& p, const Cut& cut, hipStream_t st) {
  constexpr int kMost = attend_most_tiles(sizeof(T), DT);
  if constexpr (kMost >= 4)
    if (p.nt == 4) return launch_direct<T, DT, 4>(a, p, cut, st);
  if constexpr (kMost >= 2)
    if (p.nt == 2) return launch_direct<T, DT, 2>(a, p, cut, st);
  return launch_direct<T, DT, 1>(a, p, cut, st);
}

template <class T>
int launch_type(const sc_paged_attention& a, int cus, hipStream_t st) {
  const AttendPlan p = attend_plan(a, cus);
  const int64_t rows = attend_rows(a, p);
  Cut cut{p.pitch, (int)p.tiles, p.splits, nullptr, nullptr};
  if (p.splits > 1) {
    cut.tops = static_cast<float2*>(a.workspace);
    cut.sums = reinterpret_cast<float*>(cut.tops + rows * p.splits);
  }
  const int e = a.D <= 64 ? launch_dims<T, 64>(a, p, cut, st) : a.D <= 128 ? launch_dims<T, 128>(a, p, cut, st) : launch_dims<T, 256>(a, p, cut, st);
  if (e || p.splits == 1) return e;
  hipLaunchKernelGGL(attend_join<T>, dim3((unsigned)ceil_div(rows, 4)), dim3(256), 0, st, a, cut, 16 * p.nt);
  return (int)hipGetLastError();
}

}  // namespace

int launch_paged_attention(const sc_paged_attention& a, int cus, void* stream) {
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if (a.dtype == SC_F32) return launch_type<float>(a, cus, st);
  if (a.dtype == SC_BF16) return launch_type<__bf16>(a, cus, st);
  return launch_type<_Float16>(a, cus, st);
}

}  // namespace sc
