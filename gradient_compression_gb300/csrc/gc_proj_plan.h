// How the gated projection cuts a call (host code without CUDA).
#pragma once

#include <stdint.h>

#include <algorithm>

namespace gc {

constexpr int GP_M = 128, GP_K = 64;  // rows of a tile, summed index of a part of a stage
constexpr int GP_RING = 192 * 1024;
constexpr int GP_SMS = 152;     // of a GB300
constexpr int GP_CLUSTER = 8;   // CTAs of a cluster, at most

// How a call is cut: pairs of CTAs or single ones, the tile's width, and the
// splits of its sum, the CTAs of a cluster, where there are fewer tiles than SMs.
struct GpPlan {
  bool pair, apart;  // apart: the splits are CTAs of their own, joined by another kernel
  int bn, parts, tiles_m, tiles_n, splits, span;
};
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
// Two parts to a stage where four such stages fit the ring: waiting for a stage
// and saying that it is done take 250 clocks whatever its size.
inline int gp_parts_of(int part) { return 8 * part <= GP_RING ? 2 : 1; }
// Room of a part: its rows, its columns.
inline int gp_room(int64_t rows) { return ((rows < GP_M ? (int)rows : GP_M) * GP_K * 2 + 1023) / 1024 * 1024; }
inline int gp_columns(int bn, bool pair, bool back) {
  const int wide = back ? bn : 2 * bn, mine = pair ? wide / 2 : wide;
  return (back ? (mine + 63) / 64 * 64 : mine) * GP_K * 2;
}
// Whether what a cluster's splits send and receive of a tile's groups fits the ring.
inline bool gp_fits(int groups, int s, bool back) {
  return ((groups + s - 1) / s * (s - 1) + groups - groups / s) * (back ? 1 : 2) * GP_M * 128 <= GP_RING;
}
// A part takes the SMs 2 N clocks to multiply, its bytes once in and once out of
// shared memory at 128 a clock, and not less than 400 to issue (250 of two); a
// tile's fixed part is 3000 clocks.  Joining splits takes a cluster 10400 (of two) to
// 14600 (of eight), or less for few rows; the gradient, whose sum may be long and
// whose tiles few, may also be cut into more splits, whose sums go through the
// workspace and cost another kernel.  Operands that half of L2 does not hold come
// from memory, at 27 bytes a clock and SM and 3500 in all.  fine: tiles may end
// inside a group of 32 columns (those without checkpoints): 64 x 5632 x 4096 takes 19.8 us
// in tiles of 48 columns and 22.8 in ones of 96, 17 x 11136 x 3840 29.5 in ones of 80 and
// 30.7 in ones of 96.  Of plans that cost the same the narrower tiles are taken, which
// copy on more SMs: 4 x 4096 x 1024 takes 6.1 us in tiles of 32 and 6.6 in ones of 48.
// clusters(n): how many clusters of n CTAs the GPU holds.
template <typename Clusters>
GpPlan gp_plan(int64_t rows, int64_t cols, int64_t summed, bool back, bool fine, Clusters&& clusters) {
  GpPlan best = {};
  double least = 0.0;
  const double bytes_in = (4.0 * (double)cols + (back ? 4.0 : 2.0) * (double)rows) * (double)summed;
  const bool memory = bytes_in > 64e6;
  const double quads = rows < GP_M ? (double)ceil_div(rows, 32) : 4.0;
  const int blocks = (int)ceil_div(summed, GP_K);
  for (int pair = 0; pair < (rows > GP_M ? 2 : 1); ++pair) {
    const int tm = (int)ceil_div(rows, pair ? 2 * GP_M : GP_M), workers = pair ? GP_SMS / 2 : GP_SMS, of = pair ? 2 : 1;
    for (int bn = back ? 256 : 128; bn >= 32; bn -= fine ? 16 : 32) {
      const int tn = (int)ceil_div(cols, bn), tiles = tm * tn, groups = (bn + 31) / 32, wide = back ? bn : 2 * bn;
      const int parts = gp_parts_of(gp_room(rows) + gp_columns(bn, pair != 0, back));
      const int steps = (back ? 2 : 1) * ((blocks + parts - 1) / parts);
      const int bytes = 2 * (gp_room(rows) + 128 * wide / of) / 128, work = bytes > 2 * wide ? bytes : 2 * wide, issue = parts == 2 ? 250 : 400;
      const double stage = parts * (work > issue ? work : issue);  // clocks
      const auto feed = [&](int rounds, int items, int ctas) {  // clocks for the operands: of all SMs, of the one with most
        const double most = back ? bytes_in / ((items < workers ? items : workers) * of) : rounds * 4.0 * bn * (double)summed / (tm * ctas);
        return std::max(bytes_in / 3500.0, most / 27.0);
      };
      for (int s = 1; s * of <= GP_CLUSTER && (s == 1 || tiles <= workers / s); ++s) {
        const int span = (steps + s - 1) / s;
        if (s > 1 && (span < 2 || (steps + span - 1) / span != s || !gp_fits(groups, s, back) || tiles > clusters(s * of)))
          continue;
        const int rounds = (tiles * s + workers - 1) / workers;
        const double product = (double)rounds * span * stage, fed = memory ? feed(rounds, tiles * s, s * of) : 0.0;
        const double clocks = (product > fed ? product : fed) + rounds * 3000.0 + (s > 1 ? 3500.0 + (1400.0 + 175.0 * s) * quads : 0.0);
        if (best.bn == 0 || clocks <= least) best = {pair != 0, false, bn, parts, tm, tn, s, span}, least = clocks;
      }
      if (!back || tiles > workers / 2) continue;
      for (int span = 2; span < steps; span = span < 8 ? span + 1 : span * 5 / 4) {
        const int s = (steps + span - 1) / span;
        if (s < 2 || s > workers / tiles) continue;
        const double product = span * stage, fed = memory ? feed(1, tiles * s, s * of) : 0.0;
        const double clocks = (product > fed ? product : fed) + 3000.0 + 8000.0 + s * (30.0 + (double)rows * (double)cols * 0.0023);
        if (clocks < least) best = {pair != 0, true, bn, parts, tm, tn, s, span}, least = clocks;
      }
    }
  }
  return best;
}
// Whether a call without checkpoints goes by the FMA units, by its sizes alone: the same bits wherever
// rows start.  (k_gated_proj_row says what both ways were measured to take, one row's included.)
inline bool gp_few(int64_t rows, int64_t n, int64_t k) {
  const double steps = (double)ceil_div(rows, 2) * (double)(n < 16 ? 16 : n) * ((double)ceil_div(k, 256) + 1.25);
  return rows == 1 || steps <= 24000.0 + 3.5 * (double)k;
}

}  // namespace gc
