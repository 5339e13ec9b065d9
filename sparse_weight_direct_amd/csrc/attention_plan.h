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

// Tiles of rows whose queries and sums leave a wavefront's registers room for a block's keys and values.
constexpr int attend_most_tiles(int64_t size, int dims) { return size * dims <= 256 ? 4 : size * dims <= 512 ? 2 : 1; }
constexpr int attend_staged_tiles(int64_t size, int dims) { return size * dims <= 512 ? 2 : 1; }

inline AttendPlan attend_plan(const sc_paged_attention& a, int cus) {
  AttendPlan p;
  const int64_t share = a.H / a.G, rows = share * a.L, size = a.dtype == SC_F32 ? 4 : 2;
  const int dims = a.D <= 64 ? 64 : a.D <= 128 ? 128 : 256;
  p.staged = rows >= 128;
  p.nt = p.staged ? attend_staged_tiles(size, dims) : std::min(attend_most_tiles(size, dims), rows <= 16 ? 1 : rows <= 32 ? 2 : 4);
  const int tile = p.rows();
  p.pitch = a.L < tile ? a.L : (int)(ceil_div(a.L, tile) * tile);
  p.tiles = ceil_div(share * p.pitch, tile);
  const int64_t base = (int64_t)a.B * a.G * p.tiles, blocks = ceil_div((int64_t)a.width * a.P, 32);
  p.splits = (int)std::max<int64_t>(1, std::min<int64_t>({(2 * cus + base - 1) / base, ceil_div(blocks, 4), 64}));
  return p;
}

inline int64_t attend_rows(const sc_paged_attention& a, const AttendPlan& p) { return (int64_t)a.B * a.G * p.tiles * p.rows(); }

inline int64_t attend_workspace(const sc_paged_attention& a, int cus) {
  if (a.B == 0 || a.L == 0) return 0;
  const AttendPlan p = attend_plan(a, cus);
  return p.splits == 1 ? 0 : attend_rows(a, p) * p.splits * (a.D + 2) * 4;
}

// The documented limit, whatever the launch takes; the launch makes no more workgroups than that.
inline bool attend_fits(const sc_paged_attention& a) {
  const int64_t L = a.L < 128 ? a.L : ceil_div(a.L, 128) * 128;
  return (int64_t)a.B * a.G * ceil_div((int64_t)(a.H / a.G) * L, 16) < kMostGroups;
}

// ---- Append
constexpr int kAppendTile = 64;  // positions of a prompt's tile, whole in the cache: a thread's 8 lie in one page
constexpr int kAppendHeads = 8;  // heads of a workgroup

struct AppendPlan {
  bool few;                        // a thread for every pair of every position
  int tiles, turners, sharers;     // else: tiles of a sequence (one more than its length needs, where the past ends
                                   // inside one); workgroups of a tile that turn q and k, and that move v
  int64_t groups;
};

inline AppendPlan append_plan(const sc_cache_append& a) {
  AppendPlan p{};
  const int64_t heads = a.q ? a.H : 0;
  p.few = a.L < 16;
  if (p.few) {
    p.groups = ceil_div((int64_t)a.B * a.L * ((heads + a.G) * (a.D - a.pairs) + (int64_t)a.G * a.D), 256);
  } else {
    p.tiles = (int)(ceil_div(a.L, kAppendTile) + 1);
    p.turners = (int)ceil_div(heads + a.G, kAppendHeads), p.sharers = (int)ceil_div(a.G, kAppendHeads);
    p.groups = (int64_t)a.B * p.tiles * (p.turners + p.sharers);
  }
  return p;
}

// The documented limit; the launch makes no more workgroups than that.  (B, H, G, D and L are at most 2^31, 2^16, 2^16,
// 2^8 and 2^30, so B*L is looked at first.)
inline bool append_fits(const sc_cache_append& a) {
  const int64_t heads = (a.q ? a.H : 0) + 2LL * a.G;
  if (a.L < 16) return (int64_t)a.B * a.L < (1LL << 32) && (int64_t)a.B * a.L * heads * a.D < (kMostGroups << 8);
  const int64_t tiles = a.B * (ceil_div(a.L, kAppendTile) + 1);
  return tiles < kMostGroups && tiles * (ceil_div(heads, kAppendHeads) + 1) < kMostGroups;
}

constexpr int kCopyBytes = 16384;  // of a page, by one workgroup

inline bool copy_fits(const sc_cache_copy& a) {
  const int64_t pieces = ceil_div(a.page_bytes, kCopyBytes);
  return pieces < kMostGroups && (int64_t)a.outer * a.count < kMostGroups && a.outer * pieces * a.count < kMostGroups;
}

// ---- Norm: tiles of at least 8 positions
inline bool norm_fits(const sc_residual_norm& a) { return a.B * ceil_div(a.L, 8) < (1LL << 22); }

}  // namespace sc
