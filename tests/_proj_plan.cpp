// How the gated projection cuts calls, for tests without a GPU.
#include "../gradient_compression_gb300/csrc/gc_proj_plan.h"

// calls: rows, columns, summed index, 1 for the gradient, 1 for tiles of any multiple of 16
// columns, of each; cuts: pair, apart, bn, parts, tiles_m, tiles_n, splits, span; held[c]:
// clusters of c CTAs.
extern "C" void proj_plans(const int64_t* calls, int64_t count, const int* held, int64_t* cuts) {
  for (int64_t i = 0; i < count; ++i, calls += 5, cuts += 8) {
    const gc::GpPlan p = gc::gp_plan(calls[0], calls[1], calls[2], calls[3] != 0, calls[4] != 0, [=](int ctas) { return held[ctas]; });
    const int64_t x[8] = {p.pair, p.apart, p.bn, p.parts, p.tiles_m, p.tiles_n, p.splits, p.span};
    for (int j = 0; j < 8; ++j) cuts[j] = x[j];
  }
}
extern "C" int proj_few(int64_t rows, int64_t n, int64_t k) { return gc::gp_few(rows, n, k); }
extern "C" int proj_fits(int groups, int splits, int back) { return gc::gp_fits(groups, splits, back != 0); }
extern "C" int64_t proj_stage(int64_t rows, int bn, int pair, int back) {
  return gc::gp_room(rows) + gc::gp_columns(bn, pair != 0, back != 0);
}
