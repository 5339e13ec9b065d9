// What the sequence operators' launches are cut into, from their sizes alone: used by the launchers, by the
// checks in sequence.cpp (a launch must fit the device's grid) and by host tests.  Host code; sizes reach
// 2^31 - 1, so every sum here is made in 64 bits or cannot pass.
#pragma once
#include <algorithm>
#include <cstdint>

#include "../../include/sparseconv.h"

namespace sc {

// Threads of a launch: the device counts them in 32 bits.
constexpr int64_t kGridThreads = 1LL << 32;

constexpr int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// ---- Causal convolution: a thread makes kConvV positions of a row, or kConvC channels of a single position.
constexpr int kConvV = 8;  // at least K - 1, so only a row's first thread meets the state
constexpr int kConvC = 4;

// Threads' worth of a row; a row without positions has one for its state.
inline int64_t conv_places(const sc_causal_conv& a) { return std::max<int64_t>(1, ceil_div(a.L, kConvV)); }

// The limit on its sizes: fewer than 2^31 of them (workgroups that stay in a row add less than half).
inline bool conv_fits(const sc_causal_conv& a) { return (int64_t)a.B * a.D < (1LL << 31) && (int64_t)a.B * a.D * conv_places(a) < (1LL << 31); }

// Whether rows get workgroups of their own.  Measured, us, own workgroups / all places in one line, by the share of the
// threads that own workgroups keep busy (six inputs in rotation, K = 4):
//
//   8 x 2048 rows     0.59        0.75        0.83        0.93        0.98        1.0
//   bf16, 1 a row     21.3/18.6   30.5/25.4   28.0/25.7   28.4/27.9   26.2/26.0   26.0/26.2
//   bf16, 2 a row     45.8/34.5   46.2/39.1   47.2/42.2   51.8/49.1   47.5/49.8   48.3/50.2
//   fp32, 1 a row     38.3/38.9   42.7/45.4   49.0/48.9   53.5/53.8   53.3/52.3   53.3/52.4
//   fp32, 2 a row                            102.2/83.9  101.3/99.2  100.8/97.2   99.1/98.7
//
// (nearest sizes: 0.61 and 0.71 for bf16 with 2 a row, 0.64 for fp32; 5 x 1000 rows in fp32: 13.1/13.8, 16.8/17.8,
// 18.6/18.9, 20.4/21.0; 31.0/25.2 with 2 a row at 0.61.)  So 16-bit rows have to fill them, and fp32 gains where one
// workgroup takes a row.
inline bool conv_own_rows(const sc_causal_conv& a) {
  const int64_t places = conv_places(a), threads = ceil_div(places, 256) * 256;
  return a.dtype == SC_F32 ? threads == 256 && 3 * places >= 2 * threads : 32 * places >= 31 * threads;
}

// ---- Selective scan
constexpr int kScanRows = 16;     // channels per workgroup of a prompt
constexpr int kScanThreads = 256;

// Lanes that share a channel's states at a single position, and its channels per workgroup (four a thread).
inline int scan_token_lanes(int N) { return N <= 16 ? 4 : N <= 32 ? 8 : 16; }
inline int64_t scan_token_channels(int N) { return 4 * (kScanThreads / scan_token_lanes(N)); }

// How a prompt's scan is cut.  Measured with 16 states, bf16, us, one sequence of D channels and L positions:
//
//   segments   D 512, L 8192   D 1024, L 1024   D 2048, L 8192   D 4096, L 2048
//      1            256             34.5             268              70.8
//      4            121             20.8             163              71.7
//     16             50                              139
//
// so the axis is cut where fewer than 5/8 of the CUs have a workgroup, into 4 workgroups a CU or single
// chunks; two segments cost what they save (two chunks: 18.4 and 19.5 us).  Reading ahead takes registers
// that a fourth wavefront a SIMD could use: with up to 2 workgroups a CU it gains (D 4096, L 1024: 46.7 ->
// 37.9 us), with 4 it loses (4 x 4096 x 2048: 166 -> 181 us).
//
// Positions a lane (a chunk is 16 lanes of them); a chunk that is not whole is padded and takes the guarded loads:
//
//   B x D       a lane   L 160   L 256   L 300   L 384   L 520
//   8 x 4096      16      46.4    43.4    87.1    84.5   125.7
//                  8      45.2    43.8    67.8    65.2   107.5
//   1 x 4096      16      14.6    11.1    25.5    23.7    32.8
//                  8      13.7    12.6    20.8    19.7    32.1
//   1 x 1024      16      14.3    10.8    24.6    22.0    24.3
//                  8      13.4    12.4    19.4    17.2    27.9
//
// so eight up to 384 positions unless they fill a chunk of sixteens; above, the two change places with every chunk, and
// sixteen is taken throughout (at 520, where two of three chunks are full, that costs 17% in the largest of these).
struct ScanPlan {
  int ti, chunks, segments;  // positions per lane; chunks of 16 of them per segment
  int64_t groups;            // workgroups of a segment
  bool ahead;
};

inline ScanPlan scan_plan(const sc_selective_scan& a, int cus) {
  ScanPlan p;
  const bool eight = a.L <= 384 && a.L != 256;
  p.ti = a.L <= 64 ? 4 : eight || a.N > 239 ? 8 : 16;  // beyond 239 states 16 would pass 64 KB of LDS
  p.groups = (int64_t)a.B * a.G * ceil_div(a.D / a.G, kScanRows);
  const int chunks = std::max(1, (a.L + 16 * p.ti - 1) / (16 * p.ti));
  int segments = 1;
  if (p.ti == 16 && 8 * p.groups <= 5 * cus) segments = (int)std::min<int64_t>(std::min(chunks, 64), (4 * cus + p.groups - 1) / p.groups);
  if (segments < 3) segments = 1;
  p.chunks = (chunks + segments - 1) / segments;
  p.segments = (chunks + p.chunks - 1) / p.chunks;
  p.ahead = p.ti == 16 && p.groups * p.segments <= 2 * cus;
  return p;
}

// Whether a launch holds its threads (cutting the axis makes no more of them than a few a CU) and a channel's
// number, counted up to the workgroup's end, stays in 32 bits.
inline bool scan_fits(const sc_selective_scan& a) {
  const int64_t share = a.D / a.G, per = a.L == 1 ? scan_token_channels(a.N) : kScanRows;
  return share + per < (1LL << 31) && (int64_t)a.B * a.G * ceil_div(share, per) * kScanThreads < kGridThreads;
}

// ---- Low-rank adapters
constexpr int kAdapterToken = 512;   // threads of a workgroup of single positions
constexpr int kAdapterTokenRows = 2;  // output channels per thread
constexpr int kAdapterMost = 2147483647 - 1023;  // channels: counted up to a workgroup's end in 32 bits

struct AdapterPlan {
  bool token;
  int ltiles, segments, rpieces;  // positions' tiles; pieces of C and of R
  int mtiles, mrows;              // output channels' pieces
  bool wide;                      // second product: four tiles of positions side by side
  int64_t down_blocks, up_blocks;  // workgroups of the two products (single positions: the second's alone)
  int down_threads, up_threads;
};

// The sizes have been checked (C, M <= kAdapterMost, R <= 128, L < 2^30).
inline AdapterPlan adapter_plan(const sc_adapter& a, int cus) {
  AdapterPlan p{};
  const bool wide = a.dtype == SC_F32;
  p.token = a.L < (wide ? 4 : 8);  // a tile's lane holds so many positions
  if (p.token) {
    p.mrows = kAdapterTokenRows * kAdapterToken;
    p.mtiles = (int)ceil_div(a.M, p.mrows);
    p.up_blocks = (int64_t)a.B * a.L * p.mtiles, p.up_threads = kAdapterToken;
    return p;
  }
  p.ltiles = (int)ceil_div(a.L, wide ? 64 : 128);
  const int64_t tiles = (int64_t)a.B * p.ltiles;
  const int blocks = (int)ceil_div(a.C, wide ? 16 : 32);
  p.rpieces = (a.R + 63) / 64;
  const int nw = a.R <= 32 ? 8 : 4;
  // 1, 2 or 4 pieces of C, so that every CU has a workgroup or two (an empty piece's sums are 0)
  const int64_t want = 2 * cus / (tiles * p.rpieces);
  p.segments = want >= 4 && blocks >= 4 * nw ? 4 : want >= 2 && blocks >= 2 * nw ? 2 : 1;
  p.down_blocks = tiles * p.segments * p.rpieces, p.down_threads = 64 * nw;
  // Four wavefronts side by side read and write 1 KB of a row together instead of 256 bytes (fp32,
  // 8 x 2048 -> 4096 x 1024: 78 -> 73 us), where that leaves few of them idle, LDS holds four tiles and
  // there is a workgroup for every CU and more (bf16, 8 x 2048 -> 2048 x 512, 128 of them: 24.9 us against 16.4).
  const int64_t mmost = ceil_div(a.M, 128);
  p.wide = a.R <= 16 && (p.ltiles % 4 == 0 || p.ltiles >= 12) && (int64_t)a.B * ceil_div(p.ltiles, 4) * mmost >= 3 * cus;
  const int64_t sets = (int64_t)a.B * (p.wide ? ceil_div(p.ltiles, 4) : p.ltiles);
  p.mtiles = (int)std::clamp<int64_t>((4 * cus + sets - 1) / sets, 1, mmost);
  p.mrows = (int)ceil_div(ceil_div(a.M, p.mtiles), 64) * 64;
  p.mtiles = (int)ceil_div(a.M, p.mrows);
  p.up_blocks = sets * p.mtiles, p.up_threads = 256;
  return p;
}

// Whether both launches hold their threads.  (How many CUs there are decides about launches of a few workgroups
// for each, far from this.)
inline bool adapter_fits(const sc_adapter& a) {
  if (a.B == 0 || a.L == 0) return true;
  const AdapterPlan p = adapter_plan(a, 256);
  return p.down_blocks * p.down_threads < kGridThreads && p.up_blocks * p.up_threads < kGridThreads;
}

}  // namespace sc
