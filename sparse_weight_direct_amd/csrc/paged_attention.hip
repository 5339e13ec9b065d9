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
//
// Two kernels, for few rows (bound by the cache's bytes) and for many (bound by matrix and vector issue together), and one
// that joins pieces of the context.  Measured, with 32 heads over 8 of 128 dims, bf16: 64 single positions after 0 to 8191
// others 230 us, 4.7 TB/s of keys and values (where all have 8191: 357 us uncut, 6.0 TB/s); 2 x 4096 positions 302 us, 911
// TFLOP/s (a product of 8192^3 in the library: 1185), the matrix cores busy 45% of the time, the vector units 50%;
// 512 after 30000: 271 us.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "attention.h"
#include "attention_plan.h"
#include "matrix_device.h"

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

// tanh.  16-bit types: 1 - 2 / (1 + e^2x), off by 2^-22 of 1, which under caps up to kCap is at most 2^-12 of a weight, half a unit of fp16.  Under
// a larger one (LARGE; scores are the cap times this) what counts is the error relative to the tanh, so below 1/8 its series to
// x^5 (the next term is 2^-22 of it): off by 2^-19 of the result everywhere.  Those have kernels of their own: in everybody's it cost 5 x 333
// positions of 80 dims under a cap 2 us of 39, as a branch there twice the time of every prompt (other registers spilled).
constexpr float kCap = 1024.0f;

template <class T, bool LARGE>
__device__ __forceinline__ float tanh_of(float x) {
  if constexpr (sizeof(T) == 4) return tanhf(x);
  const float far = 1.0f - 2.0f * __builtin_amdgcn_rcpf(1.0f + exp2_fast(2.0f * kLog2e * x));
  if constexpr (!LARGE) return far;
  const float z = x * x;
  return z < 0.015625f ? fmaf(x * z, fmaf(z, 2.0f / 15.0f, -1.0f / 3.0f), x) : far;
}

// Words of one or two values.
template <class T>
struct Bits {  // of each value: its sign, its exponent's highest and lowest, the number 1
  static constexpr bool kWide = sizeof(T) == 4, kB = __is_same(T, __bf16);
  static constexpr uint32_t kSigns = kWide ? 0x80000000u : 0x80008000u;
  static constexpr uint32_t kExponents = kWide ? 0x7f800000u : kB ? 0x7f807f80u : 0x7c007c00u;
  static constexpr uint32_t kOnes = kWide ? 0x3f800000u : kB ? 0x3f803f80u : 0x3c003c00u;
  // the signs of these say which exponents are full (infinities and NaN), and which values are NaN
  static __device__ __forceinline__ uint32_t full(uint32_t w) { return (w & kExponents) + (kExponents & ~(kExponents << 1)); }
  static __device__ __forceinline__ uint32_t above_infinity(uint32_t w) { return (w & ~kSigns) + (~kSigns - kExponents); }
  // all bits of the values whose sign is set
  static __device__ __forceinline__ uint32_t spread(uint32_t w) { return kWide ? (uint32_t)((int32_t)w >> 31) : ((w >> 15) & 0x00010001u) * 0xffffu; }
};

typedef uint32_t W4 __attribute__((ext_vector_type(4)));

// ---- What both kernels do with 16 NT rows and 32 keys
//
// A lane has row `col` of each of its NT tiles and, of a block of 32 keys, those that key_of says.
template <class T, int DT, int NT>
struct Rows {
  typedef typename Frag<T>::type V;
  static constexpr int N = Frag<T>::N, KF = DT / (4 * N), VF = kBlock / (4 * N), DM = DT / 16;
  static constexpr bool kWide = sizeof(T) == 4;
  // fp16's weights lie below 2^14: what is 2^-20 of the largest is still a normal number
  static constexpr float kLift = __is_same(T, _Float16) ? 6.0f : 0.0f;

  const sc_paged_attention& a;
  const Reach r;
  const int part, col;
  int head[NT], pos[NT], low[NT], pre[NT], most_key[NT];  // the row's head, position, and the keys that it sees
  float slope[NT];
  V q[NT][KF];
  F4 o[DM][NT];                        // dims 16 d + 4 part + 0..3, unnormalised
  F4 total[NT];                        // sum of the weights (fp32: of the lane's own keys, in the first)
  float top[NT], use[NT];              // the running maximum (in units of log 2), and what is subtracted from scores

  static __device__ __forceinline__ int key_of(int lanes, int u, int i) { return kWide ? 16 * u + 4 * lanes + i : 8 * lanes + 4 * u + i; }
  static __device__ __forceinline__ int key_row(int u, int m) { return kWide ? 16 * u + m : 8 * (m >> 2) + 4 * u + (m & 3); }  // of row m of tile u

  __device__ __forceinline__ Rows(const sc_paged_attention& a_, const Reach& r_, int b, int g, int row0, int pitch, int lane)
      : a(a_), r(r_), part(lane >> 4), col(lane & 15) {
    const int share = a.H / a.G;
#pragma unroll
    for (int t = 0; t < NT; t++) {
      const int row = row0 + t * 16 + col, h = row / pitch, i = row - h * pitch;
      const bool live = h < share && i < r.len;
      pos[t] = live ? r.past + i : -1;
      low[t] = a.window ? pos[t] - a.window + 1 : 0;
      pre[t] = live ? r.prefix : 0;
      most_key[t] = min(pos[t], r.end - 1);
      head[t] = min(g * share + h, a.H - 1);
      slope[t] = a.slopes ? a.slopes[head[t]] * kLog2e : 0.0f;
      // rows that are not there read ones that are: their results are dropped
      const T* p = static_cast<const T*>(a.q) + b * a.q_batch + (int64_t)head[t] * a.D * a.q_channel + min(i, a.L - 1);
#pragma unroll
      for (int f = 0; f < KF; f++) {
        const int d0 = f * 4 * N + part * N;  // D is a multiple of N: all N dims are there or none
        const T* from = p + min(d0, a.D - N) * a.q_channel;
        V v;
        if (a.q_channel == 1) {  // single positions
          const typename Pack<T, N>::type w = *reinterpret_cast<const typename Pack<T, N>::type*>(from);
#pragma unroll
          for (int j = 0; j < N; j++) v[j] = w[j];
        } else {
#pragma unroll
          for (int j = 0; j < N; j++) v[j] = from[j * a.q_channel];
        }
        q[t][f] = d0 < a.D ? v : V{};
      }
    }
    start();
  }

  __device__ __forceinline__ void start() {
#pragma unroll
    for (int t = 0; t < NT; t++) {
#pragma unroll
      for (int d = 0; d < DM; d++) o[d][t] = F4{0.0f, 0.0f, 0.0f, 0.0f};
      total[t] = F4{0.0f, 0.0f, 0.0f, 0.0f};
      top[t] = -kInf, use[t] = -kLift;
    }
  }

  // Whether a row that is there has a sum that is not finite.
  __device__ __forceinline__ bool spoilt() const {
    bool any = false;
#pragma unroll
    for (int t = 0; t < NT; t++) {
      float none = 0.0f;
#pragma unroll
      for (int d = 0; d < DM; d++)
#pragma unroll
        for (int i = 0; i < 4; i++) none = fmaf(o[d][t][i], 0.0f, none);
      any |= pos[t] >= 0 && none != 0.0f;
    }
    return any;
  }

  // Whether every row sees all of `size` keys from k0 on (`miss`: halves of them that are on no page).
  __device__ __forceinline__ bool whole(int k0, int miss, int size = kBlock) const {
    const int first = r.past + r.first, last = r.past + r.last;
    return !miss && k0 + size <= r.end &&
           (k0 + size <= r.prefix || (k0 + size - 1 <= first && (!a.window || k0 >= last - a.window + 1)));
  }
  __device__ __forceinline__ bool hidden(int lanes, int k0, int miss, int u, int t, int i) const {
    const int key = k0 + key_of(lanes, u, i);
    return (((miss >> (kWide ? u : lanes >> 1)) & 1) != 0) | ((key >= pre[t]) & ((key > most_key[t]) | (key < low[t])));
  }

  // From the products q . k of NB blocks of keys from k0 on to the weights, rounded; sums and totals follow the maximum.
  // (`miss`: two bits a block.)  With FINE, 16-bit types get what the rounding lost as a second operand.
  template <int NB, bool FINE, bool LARGE>
  __device__ __forceinline__ void weigh(F4 (&s)[2 * NB][NT], V (&p)[NT][NB * VF], V (&rest)[NT][FINE ? NB * VF : 1], int k0, int miss, bool all) {
    float scale = a.scale * kLog2e;
    if (a.cap > 0.0f || a.slopes || !(scale > 0.0f)) {  // else the maximum is looked for among the products themselves
      const float by = a.cap > 0.0f ? a.scale / a.cap : scale, cap = a.cap * kLog2e;
#pragma unroll
      for (int u = 0; u < 2 * NB; u++)
#pragma unroll
        for (int t = 0; t < NT; t++) {
          F4 v = s[u][t];
#pragma unroll
          for (int i = 0; i < 4; i++) {
            v[i] *= by;
            if (a.cap > 0.0f) v[i] = cap * tanh_of<T, LARGE>(v[i]);
            if (a.slopes) v[i] -= slope[t] * fabsf((float)(pos[t] - k0 - (u / 2) * kBlock - key_of(part, u & 1, i)));
          }
          s[u][t] = v;
        }
      scale = 1.0f;
    }
    // without branches: elements of a vector that were written under a lane's condition came out wrong here
    if (!all)
#pragma unroll
      for (int u = 0; u < 2 * NB; u++)
#pragma unroll
        for (int t = 0; t < NT; t++) {
          F4 v = s[u][t];
#pragma unroll
          for (int i = 0; i < 4; i++) v[i] = hidden(part, k0 + (u / 2) * kBlock, miss >> (u & ~1), u & 1, t, i) ? -kInf : v[i];
          s[u][t] = v;
        }
    // the maximum moves where a score passes it by 2^8 (the first ones do).  (maximum() lets a NaN through, which spoils the row
    // as it would anyway, and takes three operands; fmaxf of matrix results is two instructions more.)
    bool moves = false;
    float most[NT];
#pragma unroll
    for (int t = 0; t < NT; t++) {
      most[t] = -kInf;
#pragma unroll
      for (int u = 0; u < 2 * NB; u++)
#pragma unroll
        for (int i = 0; i < 4; i += 2)
          most[t] = __builtin_elementwise_maximum(most[t], __builtin_elementwise_maximum(s[u][t][i], s[u][t][i + 1]));
      most[t] *= scale;
      moves |= most[t] > top[t] + 8.0f;
    }
    if (__any(moves))
#pragma unroll
      for (int t = 0; t < NT; t++) {
        const float m = fmaxf(top[t], column_max(most[t])), u = m == -kInf ? 0.0f : m;
        const float factor = top[t] == -kInf ? 0.0f : exp2_fast(top[t] - u);
        top[t] = m, use[t] = u - kLift;
        total[t] *= factor;
#pragma unroll
        for (int d = 0; d < DM; d++) o[d][t] *= factor;
      }
#pragma unroll
    for (int t = 0; t < NT; t++)
#pragma unroll
      for (int u = 0; u < 2 * NB; u++) {
        F4 w = s[u][t];
#pragma unroll
        for (int i = 0; i < 4; i++) w[i] = exp2_fast(fmaf(w[i], scale, -use[t]));
        s[u][t] = w;
        if (kWide) total[t][0] += (w[0] + w[1]) + (w[2] + w[3]);
#pragma unroll
        for (int i = 0; i < 4; i++) p[t][kWide ? u : u / 2][kWide ? i : 4 * (u & 1) + i] = T(w[i]);
        if constexpr (FINE && !kWide)
#pragma unroll
          for (int i = 0; i < 4; i++) rest[t][u / 2][4 * (u & 1) + i] = T(w[i] - (float)T(w[i]));
      }
    // the rounded weights are summed as they are used: a sum over rows of ones on the matrix cores
    if constexpr (!kWide) {
      V ones;
#pragma unroll
      for (int j = 0; j < N; j++) ones[j] = T(1.0f);
#pragma unroll
      for (int t = 0; t < NT; t++)
#pragma unroll
        for (int n = 0; n < NB; n++) {
          total[t] = mma(ones, p[t][n], total[t]);
          if constexpr (FINE) total[t] = mma(ones, rest[t][n], total[t]);
        }
    }
  }

  __device__ __forceinline__ float sum_of(int t) const { return kWide ? column_sum(total[t][0]) : total[t][0]; }

  // o += the weights times the values of a block that some rows see in part, with infinities or NaN among them: those only the rows that
  // see them may meet (0 times infinity is no 0).  The finite values as always, and for the others two products of ones
  // and zeros say which rows see a +infinity or NaN, and which a -infinity or NaN.  value(d, f): a lane's values.
  // It takes so many registers that the walk over the context knows nothing of it: where a sum is not finite at
  // its end (which is seldom), the walk is made again with it.
  // (p's from f0 on are the block's)
  template <bool FINE, int NF, int NR, class Value>
  __device__ __forceinline__ void add_odd(const V (&p)[NT][NF], const V (&rest)[NT][NR], int f0, int k0, int miss, Value value) {
    int lanes = part;
    asm volatile("" : "+v"(lanes));  // keeps what is made of it out of the loop's registers
    V seen[NT][VF];
#pragma unroll
    for (int t = 0; t < NT; t++)
#pragma unroll
      for (int u = 0; u < 2; u++)
#pragma unroll
        for (int i = 0; i < 4; i++) seen[t][kWide ? u : 0][kWide ? i : 4 * u + i] = hidden(lanes, k0, miss, u, t, i) ? T(0.0f) : T(1.0f);
#pragma unroll
    for (int d = 0; d < DM; d++)
#pragma unroll
      for (int f = 0; f < VF; f++) {
        __builtin_amdgcn_sched_barrier(0);  // one after another: few registers
        const W4 v = __builtin_bit_cast(W4, value(d, f));
        W4 w, x, y;
#pragma unroll
        for (int j = 0; j < 4; j++) {
          const uint32_t odd = Bits<T>::spread(Bits<T>::full(v[j])), nan = Bits<T>::spread(Bits<T>::above_infinity(v[j])), neg = Bits<T>::spread(v[j]);
          w[j] = v[j] & ~odd;
          x[j] = odd & (nan | ~neg) & Bits<T>::kOnes;
          y[j] = odd & (nan | neg) & Bits<T>::kOnes;
        }
        const V finite = __builtin_bit_cast(V, w), up = __builtin_bit_cast(V, x), down = __builtin_bit_cast(V, y);
#pragma unroll
        for (int t = 0; t < NT; t++) {
          const F4 none = {0.0f, 0.0f, 0.0f, 0.0f}, ups = mma(up, seen[t][f], none), downs = mma(down, seen[t][f], none);
          F4 odd;
#pragma unroll
          for (int i = 0; i < 4; i++) odd[i] = (ups[i] > 0.0f ? kInf : 0.0f) - (downs[i] > 0.0f ? kInf : 0.0f);
          o[d][t] = mma(finite, p[t][f0 + f], o[d][t]) + odd;
          if constexpr (FINE) o[d][t] = mma(finite, rest[t][f0 + f], o[d][t]);
        }
      }
  }
};

// The blocks of `size` keys that a tile's rows see: those of the prefix, then those that the window leaves.
struct Blocks {
  int prefix, jump, count;
  __device__ __forceinline__ Blocks(const sc_paged_attention& a, const Reach& r, int size) {
    const int until = r.any ? max(min(r.past + r.last + 1, r.end), r.prefix) : 0;
    const int from = r.any && a.window ? min(max(r.past + r.first - a.window + 1, 0), until) / size : 0;
    prefix = (r.prefix + size - 1) / size;
    jump = max(from - prefix, 0);
    count = r.any ? max((until + size - 1) / size - jump, 0) : 0;
  }
  __device__ __forceinline__ int at(int n) const { return n < prefix ? n : n + jump; }
};

// Four dims of a row of the output.
template <class T>
__device__ __forceinline__ void put4(const sc_paged_attention& a, int64_t at, F4 v) {
  if (a.flags & SC_ATT_OUT_F32) {
#pragma unroll
    for (int i = 0; i < 4; i++) static_cast<float*>(a.out)[at + i * a.out_channel] = v[i];
    return;
  }
  T* out = static_cast<T*>(a.out) + at;
  if (a.out_channel == 1) {
    typename Pack<T, 4>::type w;
#pragma unroll
    for (int i = 0; i < 4; i++) w[i] = T(v[i]);
    *reinterpret_cast<typename Pack<T, 4>::type*>(out) = w;
  } else {
#pragma unroll
    for (int i = 0; i < 4; i++) out[i * a.out_channel] = T(v[i]);
  }
}

// Page `at` of a sequence's table, negative where there is none.
__device__ __forceinline__ int page_of(const sc_paged_attention& a, const int32_t* table, int at) {
  const int p = at < a.width ? table[at] : -1;
  return p < a.pages ? p : -1;
}

// ---- Few rows: every wavefront has its own blocks of keys
//
// A workgroup has 16 NT rows of one head of keys and a piece of the context; its four wavefronts take its
// blocks in turn, operands straight from the cache to registers (each byte is read once), the next block's on their
// way while one is computed, and their sums are joined at the end.  Bound by the cache's bytes, so the matrix cores have time for
// weights of twice 16 bits: a weight and what its rounding lost are two operands, and an output is as exact as its own rounding.
template <class T, int DT, int NT, bool LARGE>
__global__ __launch_bounds__(256, (2 + NT) * DT * (int)sizeof(T) > 1024 ? 1 : NT > 1 || (DT == 128 && sizeof(T) == 2) ? 2 : 3) void attend_direct(const sc_paged_attention a, const Cut cut) {
  typedef Rows<T, DT, NT> R;
  typedef typename R::V V;
  constexpr int N = R::N, KF = R::KF, VF = R::VF, DM = R::DM;
  constexpr int kPitch = DT + 4;
  constexpr bool kAhead = DT * sizeof(T) < 1024;  // else a block's keys and values alone fill the registers
  __shared__ float lds[4 * 16 * kPitch];
  __shared__ float2 tops[4][16];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), col = lane & 15, part = lane >> 4;
  // the heads of keys side by side, so that every XCD (workgroups go round them) has its part of each sequence, however
  // long; the pieces one after another: those that have no blocks would else leave whole groups of CUs idle
  int id = blockIdx.x;
  const int heads = a.B * a.G, bg = id % heads;
  id /= heads;
  const int tile = id % cut.tiles, split = id / cut.tiles;
  const int g = bg % a.G, b = bg / a.G, share = a.H / a.G, row0 = tile * 16 * NT;
  const Reach r = reach_of(a, b, row0, 16 * NT, cut.pitch);
  const Blocks blocks(a, r, kBlock);
  const int per = (blocks.count + cut.splits - 1) / cut.splits, stop = min(blocks.count, (split + 1) * per);
  const int shift = 31 - __builtin_clz(a.P);

  // the pages of a block's two halves, negative where there is none (page 0 is read then, and hidden)
  struct Where {
    int first, second, key;
  };
  const int32_t* table = a.table + b * a.table_batch;
  auto find = [&](int blk) __attribute__((always_inline)) {
    return Where{page_of(a, table, blk * kBlock >> shift), page_of(a, table, (blk * kBlock + 16) >> shift), blk * kBlock};
  };
  // of key `key` of the block: its dims, and its values of dim 0
  const T* k_head = static_cast<const T*>(a.k_pages) + (int64_t)g * a.P * a.D;
  const T* v_head = static_cast<const T*>(a.v_pages) + (int64_t)g * a.P * a.D;
  auto page_at = [&](Where w, int key) __attribute__((always_inline)) { return max(key & 16 ? w.second : w.first, 0); };
  auto key_at = [&](Where w, int key) __attribute__((always_inline)) { return k_head + page_at(w, key) * a.k_page + ((w.key + key) & (a.P - 1)) * a.D; };
  auto value_at = [&](Where w, int key) __attribute__((always_inline)) { return v_head + page_at(w, key) * a.v_page + ((w.key + key) & (a.P - 1)); };
  V kf[2][KF], vf[DM][VF];
  auto load_k = [&](Where w) __attribute__((always_inline)) {
#pragma unroll
    for (int t = 0; t < 2; t++) {
      const T* p = key_at(w, R::key_row(t, col));
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
  auto load_v = [&](Where w) __attribute__((always_inline)) {
#pragma unroll
    for (int f = 0; f < VF; f++) {
      const T* p = value_at(w, f * 4 * N + part * N);
#pragma unroll
      for (int d = 0; d < DM; d++) vf[d][f] = *reinterpret_cast<const V*>(p + min(d * 16 + col, a.D - 1) * a.P);
    }
  };

  R rows(a, r, b, g, row0, cut.pitch, lane);
  auto walk = [&](auto odd) __attribute__((always_inline)) {
    int n = split * per + wave;
    Where at, next;
    if (n < stop) {
      at = find(blocks.at(n));
      if (kAhead) {
        load_k(at);
        load_v(at);
      }
    }
    for (; n < stop; n += 4) {
      const int k0 = at.key, miss = (at.first < 0 ? 1 : 0) | (at.second < 0 ? 2 : 0);
      const bool more = n + 4 < stop;
      if (more) next = find(blocks.at(n + 4));
      if (!kAhead) load_k(at);
      F4 s[2][NT];
#pragma unroll
      for (int u = 0; u < 2; u++)
#pragma unroll
        for (int t = 0; t < NT; t++) {
          s[u][t] = F4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int f = 0; f < KF; f++) s[u][t] = mma(kf[u][f], rows.q[t][f], s[u][t]);
        }
      if (kAhead && more) load_k(next);
      if (!kAhead) load_v(at);
      const bool whole = rows.whole(k0, miss);
      V p[NT][VF], rest[NT][R::kWide ? 1 : VF];
      rows.template weigh<1, !R::kWide, LARGE>(s, p, rest, k0, miss, whole);
      if (!whole) {  // nothing that is not there reaches the product
#pragma unroll
        for (int f = 0; f < VF; f++) {
          const int key = f * 4 * N + part * N, left = miss >> (key >> 4 & 1) & 1 ? 0 : r.end - k0 - key;
          W4 keep;
#pragma unroll
          for (int j = 0; j < 4; j++) keep[j] = R::kWide ? (j < left ? ~0u : 0u) : (2 * j + 1 < left ? ~0u : 2 * j < left ? 0xffffu : 0u);
#pragma unroll
          for (int d = 0; d < DM; d++) vf[d][f] = __builtin_bit_cast(V, __builtin_bit_cast(W4, vf[d][f]) & keep);
        }
      }
      if (odd && !whole) {
        rows.template add_odd<!R::kWide>(p, rest, 0, k0, miss, [&](int d, int f) { return vf[d][f]; });
      } else {
#pragma unroll
        for (int f = 0; f < VF; f++)
#pragma unroll
          for (int d = 0; d < DM; d++)
#pragma unroll
            for (int t = 0; t < NT; t++) {
              rows.o[d][t] = mma(vf[d][f], p[t][f], rows.o[d][t]);
              if constexpr (!R::kWide) rows.o[d][t] = mma(vf[d][f], rest[t][f], rows.o[d][t]);
            }
      }
      if (kAhead && more) load_v(next);
      at = next;
    }
  };
  walk(std::false_type());
  if (__builtin_expect(__any(rows.spoilt()), false)) {
    rows.start();
    walk(std::true_type());
  }

  // the four wavefronts' sums, 16 rows at a time
  const int row = threadIdx.x & 15, piece = threadIdx.x >> 4;
#pragma unroll
  for (int t = 0; t < NT; t++) {
    __syncthreads();
#pragma unroll
    for (int d = 0; d < DM; d++) *reinterpret_cast<F4*>(&lds[(wave * 16 + col) * kPitch + d * 16 + part * 4]) = rows.o[d][t];
    const float total = rows.sum_of(t);
    if (part == 0) tops[wave][col] = make_float2(rows.top[t], total);
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
    const int64_t ws_row = ((int64_t)bg * cut.tiles + tile) * (16 * NT) + t * 16 + row;
    const float by = none ? 0.0f : cut.splits > 1 ? 1.0f : seen ? 1.0f / l : __builtin_nanf("");
    const int64_t ws = ws_row * cut.splits + split;
    if (cut.splits > 1 && piece == 0) cut.tops[ws] = make_float2(none ? -kInf : m, none ? 0.0f : seen ? l : __builtin_nanf(""));
    const int64_t out = b * a.out_batch + (int64_t)(g * share + h) * a.D * a.out_channel + i;
#pragma unroll
    for (int k = 0; k < DT / 64; k++) {  // four dims at a time, pieces side by side
      const int d = (k * 16 + piece) * 4;
      if (d >= a.D) continue;
      F4 v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int w = 0; w < 4; w++) {
        const F4 u = *reinterpret_cast<const F4*>(&lds[(w * 16 + row) * kPitch + d]) * f[w];
        v += f[w] != 0.0f ? u : F4{0.0f, 0.0f, 0.0f, 0.0f};
      }
      v = none ? F4{0.0f, 0.0f, 0.0f, 0.0f} : v * by;
      if (cut.splits > 1)
        *reinterpret_cast<F4*>(cut.sums + ws * a.D + d) = v;
      else
        put4<T>(a, out + d * a.out_channel, v);
    }
  }
}

// ---- Many rows: the wavefronts share the keys
//
// A workgroup has 64 NT rows of one head of keys, 16 NT a wavefront, and walks its piece of the context in tiles of KT
// keys, which it copies from the pages to LDS without passing registers, one tile ahead.  In LDS a row's
// 16-byte pieces are dealt out by an exclusive or with the row, so that the sixteen rows that a read takes
// lie in sixteen different places of 256 bytes.  NT is 2 and KT 64 up to 128 dims of 16 bits and 64 of fp32; else KT is 32, with NT 2
// for 256 dims of 16 bits and 128 of fp32 and 1 for 256 of fp32 (attend_staged_tiles, Stage).

// 16 bytes a lane, from its address or from a base that the lanes share and a byte offset of its own, to LDS byte address
// `to` + 16 * lane (to: the same in all lanes).  Written as asm so that the compiler does not wait for it
// before every LDS read; the wait is at the tile's end.  The compiler keeps no wait states of what is in here either: one between m0's
// write and the load, and five between a vector instruction that wrote a part of the base (readfirstlane, or a reload of it) and
// the load that reads it, wherever the compiler puts that instruction.
__device__ __forceinline__ void to_lds(uint32_t to, const void* from) {
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dwordx4 %1, off"
      :
      : "s"(__builtin_amdgcn_readfirstlane(to)), "v"(from)
      : "memory", "m0");
}
__device__ __forceinline__ void to_lds(uint32_t to, const void* base, uint32_t offset) {
  const uint64_t at = (uint64_t)base;
  const uint64_t shared = (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(at >> 32)) << 32 |
                          (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)at);
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 4\n\t"
      "global_load_lds_dwordx4 %1, %2"
      :
      : "s"(__builtin_amdgcn_readfirstlane(to)), "v"(offset), "s"(shared)
      : "memory", "m0");
}

template <class T, int DT>
struct Stage {
  static constexpr int KT = DT * sizeof(T) <= 256 ? 64 : 32;       // keys
  static constexpr int kKeyRow = DT * sizeof(T), kValueRow = KT * sizeof(T);  // bytes of a row: a key's dims, a dim's values
  static constexpr int kKeys = KT * kKeyRow, kBytes = 2 * kKeys;   // of a tile: its keys, then its values
  static constexpr int CK = kKeyRow / 16, CV = kValueRow / 16;     // pieces of a row
  // where piece c of a row lies
  static __device__ __forceinline__ int key_piece(int key, int c) {
    const int m = sizeof(T) == 4 ? key & 15 : (key >> 3 & 3) << 2 | (key & 3);  // the row of a product's tile
    return c ^ (CK >= 16 ? m : m >> 1);
  }
  static __device__ __forceinline__ int value_piece(int d, int c) { return c ^ (CV >= 16 ? d & 15 : CV == 8 ? d >> 1 & 7 : d >> 2 & 3); }
};

// EXACT: D is DT.  FINE: weights of 16-bit types are two operands, as in the kernel above: taken for fp32 outputs, whose caller asked for more than 16
// bits (2 x 4096 positions, bf16: 396 us, to bf16 292).  LARGE: the cap may be large.
template <class T, int DT, int NT, bool EXACT, bool FINE, bool LARGE>
__global__ __launch_bounds__(256, (2 + NT) * DT * (int)sizeof(T) > 1024 ? 1 : 2) void attend_staged(const sc_paged_attention a, const Cut cut) {
  typedef Rows<T, DT, NT> R;
  typedef Stage<T, DT> S;
  typedef typename R::V V;
  constexpr int N = R::N, KF = R::KF, VF = R::VF, DM = R::DM, KT = S::KT;
  constexpr int NB = KT / kBlock, kEarly = 4;
  constexpr int KI = S::kKeys / 4096;                      // copies of a wavefront's for the keys, and as many for the values
  constexpr int RK = 64 / S::CK, RV = 64 / S::CV;          // rows of one copy
  __shared__ __align__(256) char lds[2 * S::kBytes];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), col = lane & 15, part = lane >> 4;
  // the rows that see most come first, and a head of keys stays on its XCDs
  const int heads = a.B * a.G, share = a.H / a.G;
  int id = blockIdx.x;
  const int bg = id % heads;
  id /= heads;
  const int split = id % cut.splits;
  id /= cut.splits;
  const int each = cut.pitch / (64 * NT);  // tiles of a head, or 0 where a tile has several
  const int tile = each ? id % share * each + (each - 1 - id / share) : id;
  const int g = bg % a.G, b = bg / a.G;
  const Reach reach = reach_of(a, b, tile * 64 * NT, 64 * NT, cut.pitch);
  const int row0 = tile * 64 * NT + wave * 16 * NT;
  const Reach r = reach_of(a, b, row0, 16 * NT, cut.pitch);
  const Blocks tiles(a, reach, KT);
  const int per = (tiles.count + cut.splits - 1) / cut.splits, stop = min(tiles.count, (split + 1) * per);
  const int shift = 31 - __builtin_clz(a.P);
  const int32_t* table = a.table + b * a.table_batch;
  const uint32_t base = (uint32_t)(size_t)lds;

  // this wavefront's copies: rows of keys RK (4 i + wave) .., rows of values RV (4 i + wave) ..
  const int kc = lane % S::CK, kr = lane / S::CK, vr = lane / S::CV;
  const int vc = S::value_piece(RV * wave + vr, lane % S::CV) * N;  // the same for every i
  const T* k_head = static_cast<const T*>(a.k_pages) + (int64_t)g * a.P * a.D;
  const T* v_head = static_cast<const T*>(a.v_pages) + (int64_t)g * a.P * a.D;
  // copies a tile; returns which sixteens of its keys are on no page
  auto copy = [&](int k0, int buffer) __attribute__((always_inline)) {
    const uint32_t to = base + buffer * S::kBytes + wave * 1024;
    if (a.P >= KT) {  // one page holds the tile
      const int at = page_of(a, table, k0 >> shift), page = max(at, 0), in = k0 & (a.P - 1);
      const T* keys = k_head + page * a.k_page + in * a.D;
      const T* values = v_head + page * a.v_page + in;
#pragma unroll
      for (int i = 0; i < KI; i++) {
        const int key = RK * (4 * i + wave) + kr, c = S::key_piece(key, kc) * N;
        if (EXACT || c < a.D) to_lds(to + i * 4096, keys, (key * a.D + c) * (int)sizeof(T));
      }
#pragma unroll
      for (int i = 0; i < KI; i++) {
        const int d = RV * (4 * i + wave) + vr;
        if (EXACT || d < a.D) to_lds(to + S::kKeys + i * 4096, values, (d * a.P + vc) * (int)sizeof(T));
      }
      return at < 0 ? (1 << KT / 16) - 1 : 0;
    }
    int page[KT / 16], miss = 0;
#pragma unroll
    for (int h = 0; h < KT / 16; h++) {
      page[h] = page_of(a, table, (k0 + 16 * h) >> shift);
      if (page[h] < 0) page[h] = 0, miss |= 1 << h;
    }
#pragma unroll
    for (int i = 0; i < KI; i++) {
      const int first = RK * (4 * i + wave), c = S::key_piece(first + kr, kc) * N;
      int pg = page[0];
#pragma unroll
      for (int h = 1; h < KT / 16; h++) pg = first >> 4 == h ? page[h] : pg;
      const T* from = k_head + pg * a.k_page + ((k0 + first) & (a.P - 1)) * a.D;  // its RK keys are one page's
      if (EXACT || c < a.D) to_lds(to + i * 4096, from, (kr * a.D + c) * (int)sizeof(T));
    }
    int pg = page[0];
#pragma unroll
    for (int h = 1; h < KT / 16; h++) pg = vc >> 4 == h ? page[h] : pg;
    const T* from = v_head + pg * a.v_page + ((k0 + vc) & (a.P - 1)) + vr * a.P;
#pragma unroll
    for (int i = 0; i < KI; i++) {
      const int first = RV * (4 * i + wave);
      if (EXACT || first + vr < a.D) to_lds(to + S::kKeys + i * 4096, from + first * a.P);
    }
    return miss;
  };
  if (!EXACT) {  // dims past D are never copied: both products take them as 0
    for (int e = threadIdx.x; e < 2 * S::kBytes / 16; e += 256) reinterpret_cast<W4*>(lds)[e] = W4{0, 0, 0, 0};
    __syncthreads();
  }
  R rows(a, r, b, g, row0, cut.pitch, lane);
  auto walk = [&](auto odd) __attribute__((always_inline)) {
    int n = split * per, miss = 0, k0 = tiles.at(n) * KT, buffer = 0;
    if (n < stop) miss = copy(k0, 0);
    for (; n < stop; n++, buffer ^= 1) {
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");  // this tile is there, and nobody reads the one before
      const int here = k0, gone = miss;
      if (n + 1 < stop) {
        k0 = tiles.at(n + 1) * KT;
        miss = copy(k0, buffer ^ 1);
      }
      char* keys = lds + buffer * S::kBytes;
      char* values = keys + S::kKeys;
      if (here + KT > r.end || gone) {  // nothing that is not there reaches the product
        for (int e = threadIdx.x; e < S::kKeys / 16; e += 256) {
          const int d = e / S::CV, key = S::value_piece(d, e % S::CV) * N, left = gone >> (key >> 4) & 1 ? 0 : r.end - here - key;
          if (left >= N) continue;
          W4 v = reinterpret_cast<W4*>(values)[e];
#pragma unroll
          for (int j = 0; j < 4; j++) v[j] &= R::kWide ? (j < left ? ~0u : 0u) : (2 * j + 1 < left ? ~0u : 2 * j < left ? 0xffffu : 0u);
          reinterpret_cast<W4*>(values)[e] = v;
        }
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
      }
      // (A wavefront whose rows see nothing of the tile makes it all the same: with a way past it the compiler copied the sums of
      // every tile to other registers, 310 instead of 290 us for 2 x 4096 positions.)
      // The products go before another wavefront's weights: the matrix cores then have work while those are made (2 x 2048
      // positions of 64 dims: 112 -> 99 us, of 256 dims: 155 -> 147 us).
      __builtin_amdgcn_s_setprio(1);
      F4 s[2 * NB][NT];
#pragma unroll
      for (int u = 0; u < 2 * NB; u++) {
        const int key = (u / 2) * kBlock + R::key_row(u & 1, col);
        V kf[KF];
#pragma unroll
        for (int f = 0; f < KF; f++) kf[f] = *reinterpret_cast<const V*>(keys + key * S::kKeyRow + S::key_piece(key, 4 * f + part) * 16);
#pragma unroll
        for (int t = 0; t < NT; t++) {
          s[u][t] = F4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int f = 0; f < KF; f++) s[u][t] = mma(kf[f], rows.q[t][f], s[u][t]);
        }
      }
      auto value = [&](int d, int f) __attribute__((always_inline)) {
        return *reinterpret_cast<const V*>(values + (d * 16 + col) * S::kValueRow + S::value_piece(d * 16 + col, f * 4 + part) * 16);
      };
      // the first values are on their way while the weights are made
      V early[kEarly];
#pragma unroll
      for (int d = 0; d < kEarly; d++) early[d] = value(d, 0);
      __builtin_amdgcn_s_setprio(0);
      const bool whole = rows.whole(here, gone, KT);
      V p[NT][NB * VF], rest[NT][FINE ? NB * VF : 1];
      rows.template weigh<NB, FINE, LARGE>(s, p, rest, here, gone, whole);
      if (odd && !whole) {
#pragma unroll
        for (int kb = 0; kb < NB; kb++)
          rows.template add_odd<FINE>(p, rest, kb * VF, here + kb * kBlock, gone >> (2 * kb), [&](int d, int f) { return value(d, kb * VF + f); });
      } else {
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int f = 0; f < NB * VF; f++)
#pragma unroll
          for (int d = 0; d < DM; d++) {
            const V v = f == 0 && d < kEarly ? early[d & (kEarly - 1)] : value(d, f);
#pragma unroll
            for (int t = 0; t < NT; t++) {
              rows.o[d][t] = mma(v, p[t][f], rows.o[d][t]);
              if constexpr (FINE) rows.o[d][t] = mma(v, rest[t][f], rows.o[d][t]);
            }
          }
      }
    }
  };
  walk(std::false_type());
  if (__builtin_expect(__builtin_amdgcn_readfirstlane(__syncthreads_or(rows.spoilt())), false)) {
    rows.start();
    walk(std::true_type());
  }

#pragma unroll
  for (int t = 0; t < NT; t++) {
    const int row = row0 + t * 16 + col, h = row / cut.pitch, i = row - h * cut.pitch;
    const float total = rows.sum_of(t);
    if (h >= share || i >= a.L) continue;
    const bool none = (total == 0.0f) | (i >= r.len);
    if (cut.splits > 1) {
      const int64_t at = ((int64_t)bg * cut.tiles * (64 * NT) + row) * cut.splits + split;
      if (part == 0) cut.tops[at] = make_float2(none ? -kInf : rows.top[t], none ? 0.0f : total);
#pragma unroll
      for (int d = 0; d < DM; d++)
        if (EXACT || d * 16 + part * 4 < a.D) *reinterpret_cast<F4*>(cut.sums + at * a.D + d * 16 + part * 4) = rows.o[d][t];
    } else {
      const float by = none ? 0.0f : 1.0f / total;
      const int64_t out = b * a.out_batch + (int64_t)(g * share + h) * a.D * a.out_channel + i;
#pragma unroll
      for (int d = 0; d < DM; d++)
#pragma unroll
        for (int j = 0; j < 4; j++) {
          const int dim = d * 16 + part * 4 + j;
          if (!EXACT && dim >= a.D) continue;
          const float v = none ? 0.0f : rows.o[d][t][j] * by;
          if (a.flags & SC_ATT_OUT_F32)
            static_cast<float*>(a.out)[out + dim * a.out_channel] = v;
          else
            static_cast<T*>(a.out)[out + dim * a.out_channel] = T(v);
        }
    }
  }
}

// The pieces of the context, joined.  A workgroup has R rows, 16 threads a row with four dims each, and 16 / R threads for
// every R-th of the pieces: with 16 rows what neighbours store lies side by side, positions in prompts and dims of single
// positions; many pieces of few rows take the other form.  Four pieces' loads are in flight, none behind a
// branch (a piece that saw nothing has no sums: what is read there is dropped).
template <class T, int R>
__global__ __launch_bounds__(256) void attend_join(const sc_paged_attention a, const Cut cut, int rows) {
  constexpr int SG = 16 / R;
  __shared__ F4 part[SG > 1 ? SG : 1][R][16];
  __shared__ float totals[SG > 1 ? SG : 1][R][16];
  const int mine = threadIdx.x % R, piece = threadIdx.x / R & 15, sg = threadIdx.x / (16 * R);
  const int64_t row = (int64_t)blockIdx.x * R + mine, per = (int64_t)cut.tiles * rows;  // rows of a head of keys
  const int bg = row / per, b = bg / a.G, g = bg % a.G, share = a.H / a.G;
  const int at = (int)(row % per), h = at / cut.pitch, i = at - h * cut.pitch;
  const bool there = h < share && i < a.L;
  const float2* tops = cut.tops + row * cut.splits;
  float m = -kInf;
  if (there)
#pragma unroll 4
    for (int s = 0; s < cut.splits; s++) m = fmaxf(m, tops[s].x);
  const int64_t out = b * a.out_batch + (int64_t)(g * share + h) * a.D * a.out_channel + i;
  for (int d0 = 0; d0 < a.D; d0 += 64) {
    const int d = d0 + piece * 4;
    F4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    float l = 0.0f;
    if (there && d < a.D) {
      const float* sums = cut.sums + row * cut.splits * a.D + d;
#pragma unroll 4
      for (int s = sg; s < cut.splits; s += SG) {
        const float2 e = tops[s];
        const F4 p = *reinterpret_cast<const F4*>(sums + (int64_t)s * a.D);
        const bool none = e.y == 0.0f;
        const float f = none ? 0.0f : e.x == -kInf ? 1.0f : exp2_fast(e.x - m);  // without a maximum: NaN
        l += f * e.y;
        const F4 w = p * f;
        v += none ? F4{0.0f, 0.0f, 0.0f, 0.0f} : w;
      }
    }
    if (SG > 1) {
      if (d0) __syncthreads();
      part[sg][mine][piece] = v;
      totals[sg][mine][piece] = l;
      __syncthreads();
      if (sg) continue;
#pragma unroll
      for (int k = 1; k < SG; k++) v += part[k][mine][piece], l += totals[k][mine][piece];
    }
    if (there && d < a.D) put4<T>(a, out + d * a.out_channel, l == 0.0f ? F4{0.0f, 0.0f, 0.0f, 0.0f} : v * (1.0f / l));
  }
}

// Caps above kCap.
template <class T>
bool large_cap(const sc_paged_attention& a) { return sizeof(T) == 2 && a.cap > kCap; }

template <class T, int DT, int NT>
int launch_direct(const sc_paged_attention& a, const AttendPlan& p, const Cut& cut, hipStream_t st) {
  const dim3 grid((unsigned)((int64_t)a.B * a.G * p.groups()));
  if (large_cap<T>(a))
    hipLaunchKernelGGL((attend_direct<T, DT, NT, sizeof(T) == 2>), grid, dim3(256), 0, st, a, cut);
  else
    hipLaunchKernelGGL((attend_direct<T, DT, NT, false>), grid, dim3(256), 0, st, a, cut);
  return (int)hipGetLastError();
}

// 16-bit types have forms with twice the weights' bits for fp32 outputs; under a large cap there is one for all.
template <class T, int DT, int NT>
int launch_staged(const sc_paged_attention& a, const AttendPlan& p, const Cut& cut, hipStream_t st) {
  constexpr bool k16 = sizeof(T) == 2;
  const dim3 grid((unsigned)((int64_t)a.B * a.G * p.groups()));
  const bool fine = k16 && (a.flags & SC_ATT_OUT_F32);
  if (large_cap<T>(a))
    hipLaunchKernelGGL((attend_staged<T, DT, NT, false, k16, k16>), grid, dim3(256), 0, st, a, cut);
  else if (a.D == DT && fine)
    hipLaunchKernelGGL((attend_staged<T, DT, NT, true, k16, false>), grid, dim3(256), 0, st, a, cut);
  else if (a.D == DT)
    hipLaunchKernelGGL((attend_staged<T, DT, NT, true, false, false>), grid, dim3(256), 0, st, a, cut);
  else if (fine)
    hipLaunchKernelGGL((attend_staged<T, DT, NT, false, k16, false>), grid, dim3(256), 0, st, a, cut);
  else
    hipLaunchKernelGGL((attend_staged<T, DT, NT, false, false, false>), grid, dim3(256), 0, st, a, cut);
  return (int)hipGetLastError();
}

template <class T, int DT>
int launch_dims(const sc_paged_attention& a, const AttendPlan& p, const Cut& cut, hipStream_t st) {
  if (p.staged) return launch_staged<T, DT, attend_staged_tiles(sizeof(T), DT)>(a, p, cut, st);
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
  if (p.splits > 8 && rows < 64 * cus)
    hipLaunchKernelGGL((attend_join<T, 2>), dim3((unsigned)(rows / 2)), dim3(256), 0, st, a, cut, p.rows());
  else
    hipLaunchKernelGGL((attend_join<T, 16>), dim3((unsigned)(rows / 16)), dim3(256), 0, st, a, cut, p.rows());
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
