// What the sequence operators' launches are cut into, from their sizes alone: used by the launchers, by the
// checks in sequence.cpp (a launch must fit the device's grid) and by host tests.  Host code; sizes reach
// 2^31 - 1, so every sum here is made in 64 bits or cannot pass.
#pragma once
#include <algorithm>
#include <cstdint>

#include "../../include/sparseconv.h"

namespace sc {

constexpr int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// ---- Causal convolution: a thread makes kConvV positions of a row, or kConvC channels of a single position.
constexpr int kConvV = 8;  // at least K - 1, so only a row's first thread meets the state
constexpr int kConvC = 4;

// Threads' worth of a row; a row without positions has one for its state.
inline int64_t conv_places(const sc_causal_conv& a) { return std::max<int64_t>(1, ceil_div(a.L, kConvV)); }

// The limit on its sizes: fewer than 2^31 of them (workgroups that stay in a row add less than half).
inline bool conv_fits(const sc_causal_conv& a) { return (int64_t)a.B * a.D < (1LL << 31) && (int64_t)a.B * a.D * conv_places(a) < (1LL << 31); }

}  // namespace sc
