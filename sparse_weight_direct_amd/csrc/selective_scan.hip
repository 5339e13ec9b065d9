// Selective state space scan (sparseconv_selective_scan).
//
//   h_t[n] = exp(s_t A[d,n]) h_{t-1}[n] + s_t b_t[n] x_t,   out_t = (sum_n c_t[n] h_t[n] + skip[d] x_t) silu(z_t)
//
// Prompts are bound by vector issue: a state and position costs 1 exp2 (8 cycles a wavefront), 2 products
// and 3 FMAs (4 each), 28 cycles, and there is nothing here that the matrix cores could take: the decay
// differs per channel, state and position.  4 x 4096 channels x 2048 positions x 16 states (bf16): 96 us
// of that alone at 2.4 GHz, 50 us of memory traffic, measured 166 us with the vector units busy 88% of
// the time; the rest of the instructions are softplus, gate and conversions (36 a position, shared by 16 states),
// the lanes' scan (22 a state, shared by 16 positions) and the staging of b and c.
// Single positions are bound by the states' bytes: 128 x 4096 channels x 16 states 15.4 us, 4.6 TB/s.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "sequence_device.h"
#include "sequence_plan.h"

namespace sc {

namespace {

// ---- Prompts
//
// The steps h -> a h + v of one state compose: two segments (P1, S1), (P2, S2), each its product
// of a's and its end state from 0, make (P1 P2, P2 S1 + S2).  Sixteen lanes (a DPP row) hold TI
// consecutive positions each of one channel; a lane walks its positions once for (P, S), the
// sixteen are scanned by row shifts, and the lane walks again from the state it now knows, adding
// c h to its outputs, which stay in registers over all states n.  P needs no product over the
// positions: it is exp(A sum s).  Per (position, channel, state): 1 exp2, 2 products and 3 FMAs.
//
// A workgroup takes 16 channels of one group (4 a wavefront) and walks its positions, 16 TI at a
// time, with one copy of b and c in LDS (fp32, kStates states at a time): the four channels of a
// wavefront read the same addresses.  (One channel a wavefront with its states over four rows of lanes:
// 17 instead of 4 cycles an LDS read, 280 us instead of 165.  One position after another, four lanes a
// channel, needs no second walk and no scan, 6 units instead of 7, but has one wavefront a SIMD at the same
// size: 227 us.  Two states at once take 2 wavefronts a SIMD's registers: 181 us.)  Where there are few
// channels the axis is cut in segments: a first pass makes each segment's end state from 0 (no outputs,
// no c), the second composes the ends before its segment and walks it.

constexpr int kRows = kScanRows;  // channels per workgroup
constexpr int kStates = 16;  // states of b and c in LDS at a time

// Pitch of a channel's {A, h} in LDS: one past N, so that the four channels of a wavefront read other banks.
__host__ __device__ constexpr int ah_pitch(int N) { return N + 1; }

struct Split {
  int segments, chunks;  // segments of so many chunks of 16 TI positions
  float* state;  // [B][segments][D][N]: entry 0 the initial state, entry s the end of segment s-1 from 0
  float* sum;    // [B][segments][D]: entry s the sum of segment s-1's steps
};

template <int SHIFT>
__device__ __forceinline__ float row_shr(float old, float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(__builtin_bit_cast(int, old), __builtin_bit_cast(int, v),
                                                               0x110 + SHIFT, 0xf, 0xf, false));
}

// Inclusive scan of (P, S) over the sixteen lanes of a DPP row.  A lane without a source 1, 2, 4 or 8
// lanes below keeps its values (its write is disabled), which is the identity step, so the shifts
// need no constants: 8 instructions, and the two wait states between a write and its DPP read.
__device__ __forceinline__ void compose16(float& P, float& S) {
#define SCAN_STEP(d)                                                       \
  "s_nop 1\n\t"                                                            \
  "v_fmac_f32_dpp %1, %1, %0 row_shr:" d " row_mask:0xf bank_mask:0xf\n\t" \
  "v_mul_f32_dpp %0, %0, %0 row_shr:" d " row_mask:0xf bank_mask:0xf\n\t"
  asm(SCAN_STEP("1") SCAN_STEP("2") SCAN_STEP("4") SCAN_STEP("8") "s_nop 1" : "+v"(P), "+v"(S));
#undef SCAN_STEP
}

// TI values of a row from position t0 on, as fp32; those at or past `end` are 0 and not read.
template <class T, int TI>
__device__ __forceinline__ void load_row(const T* p, int t0, int end, float (&v)[TI]) {
  constexpr int V = TI * sizeof(T) >= 16 ? 16 / sizeof(T) : TI;
  typedef typename Pack<T, V>::type Vec;
  if (t0 + TI <= end) {
#pragma unroll
    for (int i = 0; i < TI; i += V) {
      const Vec w = *reinterpret_cast<const Vec*>(p + t0 + i);
#pragma unroll
      for (int j = 0; j < V; j++) v[i + j] = (float)w[j];
    }
  } else {
#pragma unroll
    for (int i = 0; i < TI; i++) v[i] = t0 + i < end ? (float)p[t0 + i] : 0.0f;
  }
}

template <class T, int TI>
__device__ __forceinline__ void store_row(T* p, int t0, int end, const float (&v)[TI]) {
  constexpr int V = TI * sizeof(T) >= 16 ? 16 / sizeof(T) : TI;
  typedef typename Pack<T, V>::type Vec;
#pragma unroll
  for (int i = 0; i < TI; i += V) {
    Vec w;
#pragma unroll
    for (int j = 0; j < V; j++) w[j] = T(v[i + j]);
    store_some<T, V>(p + t0 + i, end - t0 - i, w);
  }
}

template <class T, int TI, bool ENDS, bool AHEAD>
__global__ __launch_bounds__(256, AHEAD ? 2 : 4) void scan_prompt(const sc_selective_scan a, const Split sp) {
  constexpr int CH = 16 * TI;         // positions per chunk
  constexpr int MATS = ENDS ? 1 : 2;  // b, and c where outputs are wanted
  constexpr int PIECES = MATS * kStates * CH / 8;  // of 8 positions of one state
  extern __shared__ float lds[];
  // A chunk's positions lie in LDS as [TI/4][16 lanes][4]: a lane's quads are 16 bytes and neighbouring
  // lanes' quads adjacent.
  float4* bc = reinterpret_cast<float4*>(lds);                        // [MATS][kStates][CH/4]
  float2* ah = reinterpret_cast<float2*>(lds + MATS * kStates * CH);  // [kRows + 1][ah_pitch(N)]: {A log2(e), h}
  const int tid = threadIdx.x, lane = tid & 15, row = tid >> 4;
  const int share = a.D / a.G, tiles = (share + kRows - 1) / kRows;
  const int segments = ENDS ? sp.segments - 1 : sp.segments;
  // neighbouring workgroups stay on different XCDs: sequences differ in length, and b and c are small
  int id = blockIdx.x;
  const int tile = id % tiles;
  id /= tiles;
  const int seg = id % segments;
  id /= segments;
  const int g = id % a.G, b = id / a.G;
  const bool live = tile * kRows + row < share;
  const int d = g * share + min(tile * kRows + row, share - 1);
  const int slot = slot_of(a.slots, a.num_slots, b);
  const int len = slot < 0 ? 0 : length_of(a.lengths, a.L, b);
  const int N = a.N, AH = ah_pitch(N);
  const T* x = static_cast<const T*>(a.x) + b * a.x_batch + d * a.x_channel;
  const T* dt = static_cast<const T*>(a.dt) + b * a.dt_batch + d * a.dt_channel;
  const T* z = !ENDS && a.z ? static_cast<const T*>(a.z) + b * a.z_batch + d * a.z_channel : nullptr;
  const T* bm = static_cast<const T*>(a.b) + b * a.b_batch + g * a.b_group;
  const T* cm = static_cast<const T*>(a.c) + b * a.c_batch + g * a.c_group;
  T* out = static_cast<T*>(a.out) + b * a.out_batch + d * a.out_channel;
  const float skip = a.skip ? a.skip[d] : 0.0f, bias = a.dt_bias ? a.dt_bias[d] : 0.0f;
  const bool soft = a.flags & SC_SEQ_SOFTPLUS;

  // the starting states: sixteen lanes over the states of their channel
  for (int n = lane; n < N; n += 16) {
    const float A = a.A[(int64_t)d * N + n] * kLog2e;
    float h = 0.0f;
    if (!ENDS && sp.segments > 1) {
      const float* st = sp.state + (((int64_t)b * sp.segments) * a.D + d) * N + n;
      const float* sm = sp.sum + (int64_t)b * sp.segments * a.D + d;
      h = st[0];
      for (int s = 1; s <= seg; s++) h = fmaf(exp2_fast(A * sm[(int64_t)s * a.D]), h, st[(int64_t)s * a.D * N]);
    } else if (a.initial_state && slot >= 0 && seg == 0) {
      h = a.initial_state[slot * a.initial_stride + (int64_t)d * N + n];
    }
    if (ENDS) {
      // the initial state goes to the workspace first: the second pass may overwrite it in place
      if (seg == 0 && live) sp.state[(((int64_t)b * sp.segments) * a.D + d) * N + n] = h;
      h = 0.0f;
    }
    ah[row * AH + n] = make_float2(A, h);
  }
  // a DPP row's last lane has a chunk's end state; the others write theirs to a spare row
  float* const carry = &ah[(lane == 15 ? row : kRows) * AH].y;

  const int first = seg * sp.chunks * CH;
  const int last = sp.segments == 1 ? a.L : min(a.L, first + sp.chunks * CH);
  const int walk = min(last, len);  // nothing of the sequence lies past it

  // AHEAD: the next pass's b and c and the next chunk's rows are on their way during the state loop,
  // in registers and without a branch; only whole chunks are.
  static_assert(!AHEAD || TI == 16, "");
  typedef typename Pack<T, 8>::type Vec8;
  constexpr int AR = AHEAD ? TI / 8 : 1, AP = AHEAD ? PIECES / 256 : 1;
  Vec8 xr[AR], dr[AR], zr[AR], stage[AP];
  auto take = [&](const T* p, Vec8(&r)[AR]) {
#pragma unroll
    for (int i = 0; i < AR; i++) r[i] = *reinterpret_cast<const Vec8*>(p + 8 * i);
  };
  auto fetch_rows = [&](int c0) {
    if (c0 + CH > len) return;
    take(x + c0 + lane * TI, xr);
    take(dt + c0 + lane * TI, dr);
  };
  auto piece = [&](int i, int n0) {  // piece i of the states from n0 on: its first position's address
    const int q = i % (CH / 8), m = i / (CH / 8), n = min(n0 + m % kStates, N - 1);
    return (MATS == 2 && m >= kStates ? cm + n * a.c_state : bm + n * a.b_state) + q * 8;
  };
  auto fetch_bc = [&](int n0, int c0) {
    if (c0 + CH > len) return;
#pragma unroll
    for (int k = 0; k < AP; k++) stage[k] = *reinterpret_cast<const Vec8*>(piece(tid + 256 * k, n0) + c0);
  };
  if (AHEAD && first < walk) {
    fetch_rows(first);
    fetch_bc(0, first);
  }
  float total = 0.0f;
  for (int c0 = first; c0 < walk; c0 += CH) {
    const int t0 = c0 + lane * TI;
    const bool whole = c0 + CH <= len;
    float s[TI], sx[TI], y[TI], sum = 0.0f;
    if (AHEAD && whole) {
#pragma unroll
      for (int i = 0; i < TI; i++) y[i] = (float)xr[i / 8 % AR][i % 8], s[i] = (float)dr[i / 8 % AR][i % 8];
      if (z) take(z + t0, zr);
      if (c0 + CH < walk) fetch_rows(c0 + CH);
    } else {
      load_row<T, TI>(x, t0, len, y);
      load_row<T, TI>(dt, t0, len, s);
    }
#pragma unroll
    for (int i = 0; i < TI; i++) {
      const float raw = s[i] + bias;
      s[i] = soft ? softplus(raw) : raw;
    }
    if (!whole)
#pragma unroll
      for (int i = 0; i < TI; i++) s[i] = t0 + i < len ? s[i] : 0.0f;
#pragma unroll
    for (int i = 0; i < TI; i++) {
      sx[i] = s[i] * y[i];
      y[i] *= skip;
      sum += s[i];
    }
    if (!a.skip)  // no term in x at all: 0 times an infinite x is no 0
#pragma unroll
      for (int i = 0; i < TI; i++) y[i] = 0.0f;
    total += sum;
    for (int n0 = 0; n0 < N; n0 += kStates) {
      const int ns = min(kStates, N - n0);
      __syncthreads();
      auto put = [&](int i, const float(&v)[8]) {
        const int q = i % (CH / 8), m = i / (CH / 8);
#pragma unroll
        for (int j = 0; j < 2; j++) {
          const int w = q * 2 + j;  // quad of the chunk, of lane w / (TI/4)
          bc[m * (CH / 4) + w % (TI / 4) * 16 + w / (TI / 4)] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
        }
      };
      float v[8];
      if (AHEAD && whole) {
#pragma unroll
        for (int k = 0; k < AP; k++) {
#pragma unroll
          for (int j = 0; j < 8; j++) v[j] = (float)stage[k][j];
          put(tid + 256 * k, v);
        }
      } else {
#pragma unroll(AHEAD ? 1 : (PIECES + 255) / 256)
        for (int k = 0; k < (PIECES + 255) / 256; k++) {
          const int i = tid + 256 * k, q = i % (CH / 8), m = i / (CH / 8), n = m % kStates;
          if (n >= ns || (PIECES % 256 && i >= PIECES)) continue;
          load_row<T, 8>(piece(i, n0) - q * 8, c0 + q * 8, len, v);
          put(i, v);
        }
      }
      __syncthreads();
      if (AHEAD && n0 + kStates < N)
        fetch_bc(n0 + kStates, c0);
      else if (AHEAD && c0 + CH < walk)
        fetch_bc(0, c0 + CH);
      for (int n = 0; n < ns; n++) {
        const float2 Ah = ah[row * AH + n0 + n];
        float av[TI], bv[TI];
        float P = exp2_fast(Ah.x * sum), S = 0.0f;
#pragma unroll
        for (int k = 0; k < TI / 4; k++) {
          const float4 q = bc[n * (CH / 4) + k * 16 + lane];
          const float w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
          for (int j = 0; j < 4; j++) {
            const int i = 4 * k + j;
            av[i] = exp2_fast(s[i] * Ah.x);
            bv[i] = sx[i] * w[j];
            S = i ? fmaf(av[i], S, bv[i]) : bv[i];
          }
        }
        compose16(P, S);
        if (!ENDS) {
          float h = fmaf(row_shr<1>(1.0f, P), Ah.y, row_shr<1>(0.0f, S));
#pragma unroll
          for (int k = 0; k < TI / 4; k++) {
            const float4 q = bc[(kStates + n) * (CH / 4) + k * 16 + lane];
            const float w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int j = 0; j < 4; j++) {
              const int i = 4 * k + j;
              h = fmaf(av[i], h, bv[i]);
              y[i] = fmaf(w[j], h, y[i]);
            }
          }
        }
        carry[2 * (n0 + n)] = fmaf(P, Ah.y, S);
      }
    }
    if (!ENDS && live) {
      if (z) {
        float gate[TI];
        if (AHEAD && whole)
#pragma unroll
          for (int i = 0; i < TI; i++) gate[i] = (float)zr[i / 8 % AR][i % 8];
        else
          load_row<T, TI>(z, t0, len, gate);
#pragma unroll
        for (int i = 0; i < TI; i++) y[i] *= silu(gate[i]);
      }
      if (!whole)
#pragma unroll
        for (int i = 0; i < TI; i++) y[i] = t0 + i < len ? y[i] : 0.0f;
      store_row<T, TI>(out, t0, a.L, y);
    }
  }
  __syncthreads();
  if (!live) return;
  if (ENDS) {
    float* st = sp.state + (((int64_t)b * sp.segments + seg + 1) * a.D + d) * N;
    for (int n = lane; n < N; n += 16) st[n] = ah[row * AH + n].y;
#pragma unroll
    for (int m = 8; m; m >>= 1) total += __shfl_xor(total, m);
    if (lane == 0) sp.sum[((int64_t)b * sp.segments + seg + 1) * a.D + d] = total;
    return;
  }
  // the rest of the row: 0
  const float zero[TI] = {};
  for (int t0 = (walk > first ? first + (walk - first + CH - 1) / CH * CH : first) + lane * TI; t0 < last; t0 += CH)
    store_row<T, TI>(out, t0, a.L, zero);
  if (a.final_state && slot >= 0 && seg == segments - 1)
    for (int n = lane; n < N; n += 16) a.final_state[slot * a.final_stride + (int64_t)d * N + n] = ah[row * AH + n].y;
}

// ---- Single positions
//
// The states are all that counts: 8 N bytes a channel, read and written once.  Q lanes share a
// channel, four states a lane and pass (one 16-byte load), and a thread has four channels' loads in
// flight; b and c of its states serve all four.  Lane k of a quad makes channel k's step and gate,
// which its quad reads by DPP, and stores its output.
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  const int w = __builtin_bit_cast(int, v);
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(w, w, CTRL, 0xf, 0xf, false));
}

// Four values of which the first n exist, `stride` apart.
template <class T>
__device__ __forceinline__ void load_states(const T* p, int64_t stride, int n, float (&v)[4]) {
  if (stride == 1) {
    const auto w = load_some<T, 4>(p, n);
#pragma unroll
    for (int j = 0; j < 4; j++) v[j] = (float)w[j];
  } else {
#pragma unroll
    for (int j = 0; j < 4; j++) v[j] = j < n ? (float)p[j * stride] : 0.0f;
  }
}

// PLAIN: whole quads of states, and b and c contiguous over them: no branch between the loads.
template <class T, int Q, bool PLAIN>
__global__ __launch_bounds__(256) void scan_token(const sc_selective_scan a, int blocks) {
  constexpr int U = 4, CPP = 256 / Q;  // channels per thread; per workgroup and u
  typedef typename Pack<float, 4>::type F4;
  const int q = threadIdx.x % Q, k = threadIdx.x & 3, p = threadIdx.x / Q;
  const int share = a.D / a.G;
  const int base = blockIdx.x % blocks * (U * CPP) + p, g = blockIdx.x / blocks % a.G, b = blockIdx.x / blocks / a.G;
  const int slot = slot_of(a.slots, a.num_slots, b);
  const bool on = slot >= 0 && length_of(a.lengths, 1, b) == 1;
  const T* bm = static_cast<const T*>(a.b) + b * a.b_batch + g * a.b_group;
  const T* cm = static_cast<const T*>(a.c) + b * a.c_batch + g * a.c_group;
  const int64_t c0 = (int64_t)(g * share) * a.N;
  const float* from = a.initial_state && slot >= 0 ? a.initial_state + slot * a.initial_stride + c0 : nullptr;
  float* to = a.final_state && slot >= 0 ? a.final_state + slot * a.final_stride + c0 : nullptr;
  F4 h[U], A[U];
  float bv[4], cv[4];
  auto fetch = [&](int n0) {
    const int ns = PLAIN ? 4 : a.N - n0;
#pragma unroll
    for (int u = 0; u < U; u++) {
      const int64_t at = (int64_t)min(base + u * CPP, share - 1) * a.N + n0;
      h[u] = from ? load_some<float, 4>(from + at, ns) : F4{0.0f, 0.0f, 0.0f, 0.0f};
      A[u] = load_some<float, 4>(a.A + c0 + at, ns);
    }
    load_states(bm + n0 * a.b_state, PLAIN ? 1 : a.b_state, ns, bv);
    load_states(cm + n0 * a.c_state, PLAIN ? 1 : a.c_state, ns, cv);
  };
  int n0 = q * 4;
  if (n0 < a.N) fetch(n0);  // the states first: the longest way
  const int own = min(base + k * CPP, share - 1), d = g * share + own;
  const float x = (float)static_cast<const T*>(a.x)[b * a.x_batch + d * a.x_channel];
  const float raw = (float)static_cast<const T*>(a.dt)[b * a.dt_batch + d * a.dt_channel] + (a.dt_bias ? a.dt_bias[d] : 0.0f);
  const float gate = a.z ? (float)static_cast<const T*>(a.z)[b * a.z_batch + d * a.z_channel] : 0.0f;
  const float skip = a.skip ? a.skip[d] : 0.0f, x_skip = a.skip ? x : 0.0f;  // x may be infinite
  const float s_own = a.flags & SC_SEQ_SOFTPLUS ? softplus(raw) : raw, sx_own = s_own * x;
  const float s[U] = {dpp<0x00>(s_own), dpp<0x55>(s_own), dpp<0xaa>(s_own), dpp<0xff>(s_own)};
  const float sx[U] = {dpp<0x00>(sx_own), dpp<0x55>(sx_own), dpp<0xaa>(sx_own), dpp<0xff>(sx_own)};
  float y[U] = {};
  while (n0 < a.N) {
    const int ns = PLAIN ? 4 : a.N - n0;
#pragma unroll
    for (int u = 0; u < U; u++) {
      if (on)
#pragma unroll
        for (int j = 0; j < 4; j++) {
          h[u][j] = fmaf(exp2_fast(s[u] * (A[u][j] * kLog2e)), h[u][j], sx[u] * bv[j]);
          // states past N are not added: 0 times an infinite step or input is no 0
          if (PLAIN || j < ns) y[u] = fmaf(cv[j], h[u][j], y[u]);
        }
      if (to && base + u * CPP < share) store_some<float, 4>(to + (int64_t)(base + u * CPP) * a.N + n0, ns, h[u]);
    }
    n0 += 4 * Q;
    if (n0 < a.N) fetch(n0);
  }
  // the sum over the channel's lanes, in every lane: neighbours in a quad, then quads, then halves of a row
#pragma unroll
  for (int u = 0; u < U; u++) {
    y[u] += dpp<0xb1>(y[u]);
    y[u] += dpp<0x4e>(y[u]);
    if (Q >= 8) y[u] += dpp<0x141>(y[u]);
    if (Q >= 16) y[u] += dpp<0x140>(y[u]);
  }
  if (q < U && base + k * CPP < share) {
    float o = fmaf(skip, x_skip, k == 0 ? y[0] : k == 1 ? y[1] : k == 2 ? y[2] : y[3]);
    if (a.z) o *= silu(gate);
    static_cast<T*>(a.out)[b * a.out_batch + d * a.out_channel] = T(on ? o : 0.0f);
  }
}

template <class T, int Q>
int launch_token(const sc_selective_scan& a, hipStream_t st) {
  const int blocks = (int)ceil_div(a.D / a.G, 4 * (256 / Q));
  const dim3 grid((unsigned)((int64_t)a.B * a.G * blocks));
  if (a.N % 4 == 0 && a.b_state == 1 && a.c_state == 1)
    hipLaunchKernelGGL((scan_token<T, Q, true>), grid, dim3(256), 0, st, a, blocks);
  else
    hipLaunchKernelGGL((scan_token<T, Q, false>), grid, dim3(256), 0, st, a, blocks);
  return (int)hipGetLastError();
}

template <class T, int TI, bool ENDS, bool AHEAD>
int launch_part(const sc_selective_scan& a, const ScanPlan& p, const Split& sp, hipStream_t st) {
  const int lds = ((ENDS ? 1 : 2) * kStates * 16 * TI + (kRows + 1) * ah_pitch(a.N) * 2) * 4;
  const int64_t blocks = p.groups * (ENDS ? p.segments - 1 : p.segments);
  hipLaunchKernelGGL((scan_prompt<T, TI, ENDS, AHEAD>), dim3((unsigned)blocks), dim3(256), lds, st, a, sp);
  return (int)hipGetLastError();
}

template <class T>
int launch_prompt(const sc_selective_scan& a, const ScanPlan& p, hipStream_t st) {
  Split sp{p.segments, p.chunks, nullptr, nullptr};
  if (p.ti == 4) return launch_part<T, 4, false, false>(a, p, sp, st);
  if (p.ti == 8) return launch_part<T, 8, false, false>(a, p, sp, st);
  if (p.segments > 1) {
    sp.state = static_cast<float*>(a.workspace);
    sp.sum = sp.state + (int64_t)a.B * p.segments * a.D * a.N;
    if (const int e = p.ahead ? launch_part<T, 16, true, true>(a, p, sp, st) : launch_part<T, 16, true, false>(a, p, sp, st)) return e;
  }
  return p.ahead ? launch_part<T, 16, false, true>(a, p, sp, st) : launch_part<T, 16, false, false>(a, p, sp, st);
}

template <class T>
int launch_type(const sc_selective_scan& a, int cus, hipStream_t st) {
  if (a.L == 1) {
    switch (scan_token_lanes(a.N)) {
      case 4: return launch_token<T, 4>(a, st);
      case 8: return launch_token<T, 8>(a, st);
      default: return launch_token<T, 16>(a, st);
    }
  }
  return launch_prompt<T>(a, scan_plan(a, cus), st);
}

}  // namespace

int64_t scan_workspace(const sc_selective_scan& a, int cus) {
  if (a.L <= 1) return 0;
  const ScanPlan p = scan_plan(a, cus);
  return p.segments == 1 ? 0 : (int64_t)a.B * p.segments * a.D * (a.N + 1) * 4;
}

int launch_selective_scan(const sc_selective_scan& a, int cus, void* stream) {
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if (a.dtype == SC_F32) return launch_type<float>(a, cus, st);
  if (a.dtype == SC_BF16) return launch_type<__bf16>(a, cus, st);
  return launch_type<_Float16>(a, cus, st);
}

}  // namespace sc
