// What the attention operators' launches are cut into, from their sizes alone: used by the launchers and by the
// checks in attention.cpp (a launch must fit the device's grid), and by host tests.  Host code.
#pragma once
#include <algorithm>
#include <cstdint>

#include "../../include/sparseconv.h"
#include "sequence_plan.h"

namespace sc {

constexpr int64_t kMostGroups = 1LL << 24;  // workgroups of 256 threads that a launch holds

// ---- Attention.  The rows of a head of keys are its H/G heads' positions, `pitch` apart from head to head; a
// workgroup takes 16 * nt of them, or 64 * nt where its wavefronts share the keys.
struct AttendPlan {
  bool staged;
  int nt;            // tiles of 16 rows of a wavefront
  int pitch;         // rows a head: L, or L rounded up so that no workgroup has two heads
  int64_t tiles;     // workgroups of one head of keys
  int splits;        // pieces of the context
  int rows() const { return (staged ? 64 : 16) * nt; }
  int64_t groups() const { return tiles * splits; }
};

// Tiles of rows of a wavefront: as many as leave its registers room for a block's keys and values, and as there is use for.
constexpr int attend_most_tiles(int64_t size, int dims) { return dims > 128 ? 1 : size == 4 && dims <= 64 ? 4 : 2; }
constexpr int attend_staged_tiles(int64_t size, int dims) { return size * dims <= 512 ? 2 : 1; }

// How the context is cut.  Single positions, 8 heads of keys of 128 dims with 4 of queries each, bf16, us:
//
//   pieces                       1      2      3      4      8      16     32     64
//   1 sequence of 250           8.9   11.7          11.6
//   1 of 777                   16.5   15.3          13.3   14.1
//   1 of 8000                                       39.4   29.7   18.2   17.7   22.0
//   1 of 32000                                             77.3   44.3   35.2   38.8
//   16 of 0 to 8191             130   79.5          83.0   78.3
//   64 of 0 to 8191             267    248   232     227    237
//   64 of 8191 each             357    366   370     372    390
//   fp32, 24 x 16 heads of 64 dims, 0 to 3000: 98.2, 81.9, -, 74.9, 75.4; with a window of 1024: 47.3, 43.8, -, 46.4, 53.0
//   512 positions after 30000 (keys shared by wavefronts): 715, 377, -, 271, 286
//   333 positions, fp16, 5 x 6 heads of 80 dims (likewise): 69.9, 47.6, -, 38.9, 45.3, with six 39.5
//
// so enough pieces for two workgroups a CU, of six blocks of 32 keys at least, at most 32; and where there are enough without
// cutting, four of 64 blocks at least: sequences' lengths differ as a rule, and evenly long ones lose less than that gains.
// Single positions take a power of two of them (1 of 8000 in 31: 20.1).  The six blocks rest on the sequences of 250 and 777; between
// those, and for more than the two chunks of many rows above (333 positions lose 2% by it), nothing is measured.  The table's width is
// what is counted, whatever a window leaves of it.
//
// From how many rows on the wavefronts share the keys, us, shared / each its own (16 heads over 4, contexts 1 x 30000,
// 8 x 4000, 64 x 500):
//
//   rows        16                   32                   48                   64                   96
//   bf16, 64    29/19 23/15 24/15    29/21 23/18 25/18    29/39 24/31 25/30    29/40 24/31 27/32    30/41 25/39 28/35
//   bf16, 128   38/28 31/22 35/22    39/39 32/30 37/31    39/42 33/42 37/30    39/41 34/41 38/33    40/52 36/52 40/62
//   bf16, 256   74/47 69/45 79/46    75/89 72/91 82/93    75/100 72/127 84/119 76/102 74/130 88/132 78/163 78/166 92/192
//   fp32, 64    79/26 52/21 54/21    78/33 53/28 54/27    78/53 53/46 54/46    78/53 54/49 58/51    78/56 53/65 59/68
//   fp32, 128   146/43 99/40 103/41  147/58 101/53 103/55 148/62 99/75 104/66  147/63 102/76 110/77 149/106 104/107 115/112
//
// so above 32 rows for 16-bit types (above 16 for more than 128 dims), else from 96 on.
inline AttendPlan attend_plan(const sc_paged_attention& a, int cus) {
  AttendPlan p;
  const int64_t share = a.H / a.G, rows = share * a.L, size = a.dtype == SC_F32 ? 4 : 2;
  const int dims = a.D <= 64 ? 64 : a.D <= 128 ? 128 : 256;
  p.staged = size == 4 ? rows >= 96 : rows > (dims > 128 ? 16 : 32);
  p.nt = p.staged ? attend_staged_tiles(size, dims) : std::min(attend_most_tiles(size, dims), rows <= 16 ? 1 : rows <= 32 ? 2 : 4);
  const int tile = p.rows();
  p.pitch = a.L < tile ? a.L : (int)(ceil_div(a.L, tile) * tile);
  p.tiles = ceil_div(share * p.pitch, tile);
  const int64_t base = (int64_t)a.B * a.G * p.tiles, blocks = ceil_div((int64_t)a.width * a.P, 32);
  int64_t pieces = std::min<int64_t>({ceil_div(2 * cus, base), blocks / 6, 32});
  if (!p.staged && base >= 2 * cus && base < 8 * cus) pieces = std::min<int64_t>(4, blocks / 64);
  if (!p.staged)
    while (pieces & (pieces - 1)) pieces &= pieces - 1;
  p.splits = (int)std::max<int64_t>(1, pieces);
  return p;
}

inline int64_t attend_rows(const sc_paged_attention& a, const AttendPlan& p) { return (int64_t)a.B * a.G * p.tiles * p.rows(); }

inline int64_t attend_workspace(const sc_paged_attention& a, int cus) {
  if (a.B == 0 || a.L == 0) return 0;
  const AttendPlan p = attend_plan(a, cus);
  return p.splits == 1 ? 0 : attend_rows(a, p) * p.splits * (a.D + 2) * 4;
}

// The documented limit, whatever the launch takes, and what the launch takes where that is more (tiles of 16 rows whose heads lie apart:
// fp32 of more than 128 dims).  The factors are looked at one by one: together they pass 64 bits.
inline bool attend_fits(const sc_paged_attention& a) {
  if (a.B == 0 || a.L == 0) return true;
  const int64_t L = a.L < 128 ? a.L : ceil_div(a.L, 128) * 128, heads = (int64_t)a.B * a.G, most = ceil_div((int64_t)(a.H / a.G) * L, 16);
  return heads < kMostGroups && most < kMostGroups && heads * most < kMostGroups && heads * attend_plan(a, 256).tiles < kMostGroups;
}

// ---- Append
constexpr int kAppendTile = 64;  // positions of a prompt's tile, whole in the cache: a thread's 8 lie in one page

// Heads of a workgroup: their sines and cosines are made once.  Measured with 1, 2, 4, 8 of them, us, 32 heads of q over 8 of
// 128 dims, bf16: 2 x 4096 positions 63.8, 51.2, 44.8, 44.1; 1 x 512: 9.2, 10.1, 11.1, 16.8; 1 x 17: 7.2, 9.4, 14.2, 23.8;
// 16 over 16 of 64 dims, 4 x 1000: 20.4, 15.8, 16.8, 21.8.  So as many, up to 8, as leave three workgroups a CU.
struct AppendPlan {
  int chunk;
  bool few;                        // a thread for every pair of every position
  int tiles, turners, sharers;     // else: tiles of a sequence (one more than its length needs, where the past ends
                                   // inside one); workgroups of a tile that turn q and k, and that move v
  int64_t groups;
};

inline AppendPlan append_plan(const sc_cache_append& a, int cus) {
  AppendPlan p{};
  const int64_t heads = a.q ? a.H : 0;
  p.few = a.L < 16;
  if (p.few) {
    p.groups = ceil_div((int64_t)a.B * a.L * ((heads + a.G) * (a.D - a.pairs) + (int64_t)a.G * a.D), 256);
  } else {
    p.tiles = (int)(ceil_div(a.L, kAppendTile) + 1);
    for (p.chunk = 8; p.chunk >= 1; p.chunk /= 2) {
      p.turners = (int)ceil_div(heads + a.G, p.chunk), p.sharers = (int)ceil_div(a.G, p.chunk);
      p.groups = (int64_t)a.B * p.tiles * (p.turners + p.sharers);
      if (p.chunk == 1 || p.groups >= 3 * cus) break;
    }
  }
  return p;
}

// The documented limit; the launch makes no more workgroups than that.  (B, H, G, D and L are at most 2^31, 2^16, 2^16,
// 2^8 and 2^30, so B*L is looked at first.)
inline bool append_fits(const sc_cache_append& a) {
  const int64_t heads = (a.q ? a.H : 0) + 2LL * a.G;
  if (a.L < 16) return (int64_t)a.B * a.L < (1LL << 32) && (int64_t)a.B * a.L * heads * a.D < (kMostGroups << 8);
  const int64_t tiles = a.B * (ceil_div(a.L, kAppendTile) + 1);
  return tiles < kMostGroups && tiles * (ceil_div(heads, 8) + 1) < kMostGroups;  // (smaller chunks make few workgroups)
}

constexpr int kCopyBytes = 16384;  // of a page, by one workgroup

inline bool copy_fits(const sc_cache_copy& a) {
  const int64_t pieces = ceil_div(a.page_bytes, kCopyBytes);
  return pieces < kMostGroups && (int64_t)a.outer * a.count < kMostGroups && a.outer * pieces * a.count < kMostGroups;
}

// ---- Norm
enum NormForm { kNormAny, kNormPrompt, kNormToken };

// Prompts.  Measured, us (16-bit, or fp32 where it says so; lanes side by side, channels a thread, threads):
//
//   8 x 2048 x 2048       4,16,512: 79.7   2,8,512: 129    1,4,512: 124    2,16,256: 115   4,8,1024: 97
//   8 x 1024 x 2048       4,8,512: 44.7    2,4,512: 37.4   4,16,256: 34.5  2,8,256: 57.9
//   4 x 4096 x 2048       2,16,512: 107    1,8,512: 135    1,16,256: 127   2,8,1024: 111
//   1 x 1024 x 512        4,8,512: 17.2    2,4,512: 11.1   4,16,256: 19.6  2,8,256: 15.3
//   4 x 1024 x 512, fp32  4,8,512: 15.1    2,4,512: 13.6   4,16,256: 18.0
//
// so four lanes (64 bytes of a row) and as few threads as hold the channels, where every CU has two tiles, else two lanes.
struct NormPlan {
  NormForm form;
  int tiles;     // of a sequence's positions
  int lp_shift;  // prompts: log2 of the lanes side by side along the positions, 16 bytes each
  int pass;      // prompts: channels of a thread
  int threads;
};

inline NormPlan norm_plan(const sc_residual_norm& a, int cus) {
  NormPlan p{kNormAny, (int)ceil_div(a.L, 16), 0, 0, 256};
  const bool rows = (!a.y || a.y_channel == 1) && (!a.sum || a.sum_channel == 1) && (!a.out || a.out_channel == 1) && a.x_channel == 1;
  if (a.L == 1 && rows && a.C <= 8192) {
    p.form = kNormToken;
    p.threads = a.C <= 2048 ? 256 : a.C <= 4096 ? 512 : 1024;
    return p;
  }
  const int V = a.dtype == SC_F32 ? 4 : 8;
  const bool many = a.B * ceil_div(a.L, 4 * V) >= 2 * cus;
  for (int shift = many ? 2 : 1; shift >= 0; shift--)
    for (int threads = many ? 256 : 512; threads <= 512; threads *= 2) {
      const int64_t need = ceil_div(a.C, threads >> shift);
      if (need > 16) continue;
      p.form = kNormPrompt;
      p.lp_shift = shift, p.threads = threads;
      p.tiles = (int)ceil_div(a.L, V << shift);
      p.pass = need <= 4 ? 4 : need <= 8 ? 8 : 16;
      return p;
    }
  return p;
}

// Tiles of at least 4 positions, of at most 1024 threads.
inline bool norm_fits(const sc_residual_norm& a) { return a.B * ceil_div(a.L, 4) < (1LL << 22); }

}  // namespace sc
