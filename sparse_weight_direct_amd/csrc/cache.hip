// The paged cache's update with rotary positions (sparseconv_cache_append) and copies of its pages
// (sparseconv_cache_copy).  Both are bound by memory: 2 x 4096 positions of 32 + 2 x 8 heads of 128 dims, three coordinates, bf16,
// 50.6 us in a row of calls, 4.0 TB/s read and written (the kernel alone 43.9; a copy: 5.1); 16 x 200 pages of 64 KB 83 us, 5.1 TB/s.
#include <hip/hip_runtime.h>

#include "attention.h"
#include "attention_plan.h"
#include "sequence_device.h"

namespace sc {

namespace {

// ---- Append
//
// A pair turns by theta = freq * position.  theta / 2 pi is made and reduced to one turn in fp64 (positions of
// 10^6 keep 2^-33 of a turn); its sine and cosine are the hardware's, which take turns and are off by 2^-22.9 at
// most over a whole turn (4 million places; the math library's sincospi is five times the instructions).

constexpr int kTile = kAppendTile;

struct Sequence {
  int past, len;
  bool idle;
};

__device__ __forceinline__ Sequence sequence_of(const sc_cache_append& a, int b) {
  Sequence s;
  s.past = a.past[b];
  s.idle = s.past < 0 || s.past > a.width * a.P;
  s.len = s.idle ? 0 : length_of(a.lengths, a.L, b);
  if (s.idle) s.past = 0;
  return s;
}

// Page of position t, negative where there is none.
__device__ __forceinline__ int page_at(const sc_cache_append& a, int b, int t) {
  const int at = t / a.P;
  const int p = at < a.width ? a.table[b * a.table_batch + at] : -1;
  return p < a.pages ? p : -1;
}

__device__ __forceinline__ void turn(double freq, int position, float& c, float& s) {
  const double turns = (double)position * (freq * 0.15915494309189535);
  const float part = (float)(turns - rint(turns));
  s = __builtin_amdgcn_sinf(part);
  c = __builtin_amdgcn_cosf(part);
}

// Dims of pair j.
__device__ __forceinline__ int first_of(const sc_cache_append& a, int j) { return a.flags & SC_ROT_INTERLEAVED ? 2 * j : j; }
__device__ __forceinline__ int second_of(const sc_cache_append& a, int j) { return a.flags & SC_ROT_INTERLEAVED ? 2 * j + 1 : j + a.pairs; }

__device__ __forceinline__ int axis_of(const sc_cache_append& a, int j) {
  const int x = a.axes ? a.axes[j] : 0;
  return x < a.num_axes ? x : -1;
}

// A few positions: a thread has a pair (or a dim that does not turn) of one head and position.  Its sine and cosine are
// made again for every head, which is nothing beside the launch (64 positions of 32 + 2 x 8 heads: 5.9 us, 4.4 of them
// a launch after another).
template <class T, class K>
__global__ __launch_bounds__(256) void append_few(const sc_cache_append a, int64_t total) {
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (at >= total) return;
  const int heads = a.q ? a.H : 0, turning = a.D - a.pairs, units = (heads + a.G) * turning + a.G * a.D;
  const int unit = at % units, i = at / units % a.L, b = at / units / a.L;
  const Sequence s = sequence_of(a, b);
  const bool live = i < s.len;
  const int t = s.past + i;
  const bool value = unit >= (heads + a.G) * turning;
  const int rest = value ? unit - (heads + a.G) * turning : unit;
  const int head = value ? rest / a.D : rest / turning, u = value ? rest % a.D : rest % turning;
  const bool query = !value && head < heads;
  if (!live && !query) return;
  const int g = query || value ? head : head - heads;
  const T* x = query ? static_cast<const T*>(a.q) + b * a.q_batch + (int64_t)head * a.D * a.q_channel + i
               : value ? static_cast<const T*>(a.v) + b * a.v_batch + (int64_t)g * a.D * a.v_channel + i
                       : static_cast<const T*>(a.k) + b * a.k_batch + (int64_t)g * a.D * a.k_channel + i;
  const int64_t xs = query ? a.q_channel : value ? a.v_channel : a.k_channel;
  K* to;
  int64_t ts;
  if (query) {
    to = static_cast<K*>(a.q_out) + b * a.q_out_batch + (int64_t)head * a.D * a.q_out_channel + i;
    ts = a.q_out_channel;
  } else {
    const int page = page_at(a, b, t), in = t % a.P;
    if (page < 0) return;
    to = value ? static_cast<K*>(a.v_pages) + page * a.v_page + (int64_t)g * a.D * a.P + in
               : static_cast<K*>(a.k_pages) + page * a.k_page + ((int64_t)g * a.P + in) * a.D;
    ts = value ? a.P : 1;
  }
  if (value || u >= a.pairs) {
    const int d = value ? u : u + a.pairs;
    to[d * ts] = live ? K((float)x[d * xs]) : K(0.0f);
    return;
  }
  const int d0 = first_of(a, u), d1 = second_of(a, u), axis = axis_of(a, u);
  float v0 = 0.0f, v1 = 0.0f;
  if (live) {
    v0 = (float)x[d0 * xs], v1 = (float)x[d1 * xs];
    if (axis >= 0) {
      float c, sn;
      turn(a.freqs[u], a.positions ? a.positions[b * a.positions_batch + axis * a.positions_axis + i] : t, c, sn);
      const float w = v0;
      v0 = v0 * c - v1 * sn;
      v1 = v1 * c + w * sn;
    }
  }
  to[d0 * ts] = K(v0);
  to[d1 * ts] = K(v1);
}

// 8 values of a row from position i on; those outside 0 .. len-1 are 0.
template <class T>
__device__ __forceinline__ typename Pack<T, 8>::type load8(const T* p, int i, int len) {
  typedef typename Pack<T, 8>::type V;
  if (i >= 0 && i + 8 <= len) return *reinterpret_cast<const V*>(p + i);
  V v;
#pragma unroll
  for (int j = 0; j < 8; j++) {
    const int at = i + j;
    T x = T(0);
    if (at >= 0 && at < len) x = p[at];
    v[j] = x;
  }
  return v;
}

// To positions i .. i+7 of a row of `len`.
template <class K>
__device__ __forceinline__ void store8(K* p, int i, int len, const float (&v)[8]) {
  typedef typename Pack<K, 8>::type V;
  if (i >= 0 && i + 8 <= len) {
    V w;
#pragma unroll
    for (int j = 0; j < 8; j++) w[j] = K(v[j]);
    *reinterpret_cast<V*>(p + i) = w;
  } else {
#pragma unroll
    for (int j = 0; j < 8; j++)
      if (i + j >= 0 && i + j < len) p[i + j] = K(v[j]);
  }
}

// A position's dims in LDS: 16 bytes apart from a power of two, where 64 KB hold them.
template <class K>
__host__ __device__ constexpr int key_pitch(int D) {
  return D * (int)sizeof(K) < 1024 ? D + 16 / (int)sizeof(K) : D;
}

// Prompts.  A workgroup has 64 positions and `chunk` heads of q and k, or of v: eight lanes along the positions, 32 rows
// of dims side by side.  A thread's sines and cosines serve all its heads; keys go through LDS, where a
// position's dims come together.
template <class T, class K, int JP>
__global__ __launch_bounds__(256) void append_prompt(const sc_cache_append a, int tiles, int turners, int sharers, int chunk) {
  extern __shared__ __align__(16) char lds_bytes[];
  K* keys = reinterpret_cast<K*>(lds_bytes);  // [kTile][pitch]
  const int pitch = key_pitch<K>(a.D);
  const int tid = threadIdx.x, at8 = (tid & 7) * 8, row = tid >> 3;
  int id = blockIdx.x;
  const int part = id % (turners + sharers);
  id /= turners + sharers;
  const int tile = id % tiles, b = id / tiles;
  const Sequence s = sequence_of(a, b);
  const int heads = a.q ? a.H : 0;
  // the tile's first position in the cache, and among the new ones (negative in the first tile where the past ends inside it)
  const int t0 = (s.past / kTile + tile) * kTile, i = t0 - s.past + at8;
  if (t0 - s.past >= a.L) return;
  const int page = page_at(a, b, t0 + at8), in = (t0 + at8) % a.P;
  if (part >= turners) {  // values: positions stay contiguous
    if (page < 0 || i + 8 <= 0 || i >= s.len) return;
    const int h1 = min((part - turners + 1) * chunk, a.G);
    for (int g = (part - turners) * chunk; g < h1; g++) {
      const T* x = static_cast<const T*>(a.v) + b * a.v_batch + (int64_t)g * a.D * a.v_channel;
      K* to = static_cast<K*>(a.v_pages) + page * a.v_page + (int64_t)g * a.D * a.P + in;
      for (int d = row; d < a.D; d += 32) {
        const auto r = load8(x + d * a.v_channel, i, s.len);
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; k++) v[k] = (float)r[k];
        store8(to + d * a.P - i, i, s.len, v);
      }
    }
    return;
  }
  float c[JP][8], sn[JP][8];
#pragma unroll
  for (int p = 0; p < JP; p++) {
    const int j = row + 32 * p, axis = j < a.pairs ? axis_of(a, j) : -1;
    const double freq = axis >= 0 ? a.freqs[j] : 0.0;
    const int32_t* where = a.positions && axis >= 0 ? a.positions + b * a.positions_batch + axis * a.positions_axis : nullptr;
    typename Pack<int32_t, 8>::type at;
    if (where) at = load8(where, i, s.len);
#pragma unroll
    for (int k = 0; k < 8; k++) {
      c[p][k] = 1.0f, sn[p][k] = 0.0f;
      if (axis >= 0) turn(freq, where ? at[k] : t0 + at8 + k, c[p][k], sn[p][k]);
    }
  }
  typedef typename Pack<T, 8>::type V8;
  int pages[kTile / 16];  // of the tile's sixteens
#pragma unroll
  for (int n = 0; n < kTile / 16; n++) pages[n] = page_at(a, b, t0 + 16 * n);
  for (int h = part; h < heads + a.G; h += turners) {  // some of q's and some of k's
    const bool query = h < heads;
    const T* x = query ? static_cast<const T*>(a.q) + b * a.q_batch + (int64_t)h * a.D * a.q_channel
                       : static_cast<const T*>(a.k) + b * a.k_batch + (int64_t)(h - heads) * a.D * a.k_channel;
    const int64_t xs = query ? a.q_channel : a.k_channel;
    K* to = query ? static_cast<K*>(a.q_out) + b * a.q_out_batch + (int64_t)h * a.D * a.q_out_channel : nullptr;
    auto put = [&](int d, const float(&v)[8]) {
      if (query) {
        store8(to + d * a.q_out_channel, i, a.L, v);
      } else {
#pragma unroll
        for (int k = 0; k < 8; k++) keys[(at8 + k) * pitch + d] = K(v[k]);
      }
    };
    if (!query) __syncthreads();  // the head before has been stored
#pragma unroll
    for (int p = 0; p < JP; p++) {
      const int j = row + 32 * p;
      if (j >= a.pairs) continue;
      const int d0 = first_of(a, j), d1 = second_of(a, j), axis = axis_of(a, j);
      const V8 r0 = load8(x + d0 * xs, i, s.len), r1 = load8(x + d1 * xs, i, s.len);
      float v0[8], v1[8];
#pragma unroll
      for (int k = 0; k < 8; k++) {
        const float u = (float)r0[k], w = (float)r1[k];
        v0[k] = axis >= 0 ? u * c[p][k] - w * sn[p][k] : u;
        v1[k] = axis >= 0 ? w * c[p][k] + u * sn[p][k] : w;
      }
      put(d0, v0);
      put(d1, v1);
    }
    for (int d = 2 * a.pairs + row; d < a.D; d += 32) {
      const V8 r = load8(x + d * xs, i, s.len);
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; k++) v[k] = (float)r[k];
      put(d, v);
    }
    if (!query) {
      __syncthreads();
      typedef typename Pack<K, 8>::type V;
      const int pieces = a.D / 8;
      for (int e = tid; e < kTile * pieces; e += 256) {
        const int n = e / pieces, d = e % pieces * 8, t = t0 + n;
        if (t < s.past || t >= s.past + s.len) continue;
        const int pg = n < 32 ? n < 16 ? pages[0] : pages[1] : n < 48 ? pages[2] : pages[3];
        if (pg < 0) continue;
        *reinterpret_cast<V*>(static_cast<K*>(a.k_pages) + pg * a.k_page + ((int64_t)(h - heads) * a.P + t % a.P) * a.D + d) =
            *reinterpret_cast<const V*>(keys + n * pitch + d);
      }
    }
  }
}

template <class T, class K>
int launch_append(const sc_cache_append& a, int cus, hipStream_t st) {
  const int heads = a.q ? a.H : 0;
  const AppendPlan p = append_plan(a, cus);
  const dim3 grid((unsigned)p.groups);
  if (p.few) {
    const int64_t total = (int64_t)a.B * a.L * ((int64_t)(heads + a.G) * (a.D - a.pairs) + (int64_t)a.G * a.D);
    hipLaunchKernelGGL((append_few<T, K>), dim3((unsigned)ceil_div(total, 256)), dim3(256), 0, st, a, total);
    return (int)hipGetLastError();
  }
  const int tiles = p.tiles, chunk = p.chunk, turners = p.turners, sharers = p.sharers;
  const int lds = kTile * key_pitch<K>(a.D) * (int)sizeof(K);
  if (a.pairs <= 32)
    hipLaunchKernelGGL((append_prompt<T, K, 1>), grid, dim3(256), lds, st, a, tiles, turners, sharers, chunk);
  else if (a.pairs <= 64)
    hipLaunchKernelGGL((append_prompt<T, K, 2>), grid, dim3(256), lds, st, a, tiles, turners, sharers, chunk);
  else
    hipLaunchKernelGGL((append_prompt<T, K, 4>), grid, dim3(256), lds, st, a, tiles, turners, sharers, chunk);
  return (int)hipGetLastError();
}

// ---- Copy: a workgroup has 16 KB of one page
typedef uint32_t W4 __attribute__((ext_vector_type(4)));

template <class V>
__global__ __launch_bounds__(256) void copy_pages(const sc_cache_copy a, int pieces) {
  constexpr int64_t kPiece = kCopyBytes / sizeof(V);
  int id = blockIdx.x;
  const int64_t at = id % pieces * kPiece;
  id /= pieces;
  const int i = id % a.count, o = id / a.count;
  const int from = a.source[i], to = a.target[i];
  if (from < 0 || from >= a.pages || to < 0 || to >= a.pages || from == to) return;
  char* block = static_cast<char*>(a.pool) + o * a.outer_stride;
  const V* src = reinterpret_cast<const V*>(block + from * a.page_stride) + at;
  V* dst = reinterpret_cast<V*>(block + to * a.page_stride) + at;
  const int64_t left = a.page_bytes / (int64_t)sizeof(V) - at;
  if (left >= kPiece && sizeof(V) == 16) {
    V v[4];
#pragma unroll
    for (int k = 0; k < 4; k++) v[k] = src[threadIdx.x + 256 * k];
#pragma unroll
    for (int k = 0; k < 4; k++) dst[threadIdx.x + 256 * k] = v[k];
  } else {
    for (int64_t k = threadIdx.x; k < (left < kPiece ? left : kPiece); k += 256) dst[k] = src[k];
  }
}

}  // namespace

int launch_cache_append(const sc_cache_append& a, int cus, void* stream) {
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if (a.dtype == SC_BF16) return launch_append<__bf16, __bf16>(a, cus, st);
  if (a.dtype == SC_F16) return launch_append<_Float16, _Float16>(a, cus, st);
  if (a.cache_dtype == SC_BF16) return launch_append<float, __bf16>(a, cus, st);
  if (a.cache_dtype == SC_F16) return launch_append<float, _Float16>(a, cus, st);
  return launch_append<float, float>(a, cus, st);
}

int launch_cache_copy(const sc_cache_copy& a, void* stream) {
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  const int pieces = (int)ceil_div(a.page_bytes, kCopyBytes);
  const dim3 grid((unsigned)((int64_t)a.outer * a.count * pieces));
  const bool wide = ((reinterpret_cast<uintptr_t>(a.pool) | (uintptr_t)a.outer_stride | (uintptr_t)a.page_stride | (uintptr_t)a.page_bytes) & 15) == 0;
  if (wide)
    hipLaunchKernelGGL(copy_pages<W4>, grid, dim3(256), 0, st, a, pieces);
  else
    hipLaunchKernelGGL(copy_pages<uint8_t>, grid, dim3(256), 0, st, a, pieces);
  return (int)hipGetLastError();
}

}  // namespace sc
