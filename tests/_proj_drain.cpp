// How a pair of CTAs of the gated projection ends after a wait that ran out: the
// kernel's own gp_feed and gp_drain (taken from its source, on a host that
// only notes down what they do) from every place where either CTA may have given up.
#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <random>
#include <tuple>
#include <vector>

#include "gc_proj_plan.h"

namespace gc {
using std::max;
using std::min;
struct CUtensorMap {
  int id;
};
constexpr uint32_t FULL = 0xffffffffu;
struct Dim {
  unsigned x;
};
static Dim blockIdx, gridDim, threadIdx;
static int __shfl_sync(uint32_t, int v, int) { return v; }
static void __syncwarp() {}
static bool elected() { return true; }

// What happened: copies (to, map, x, y), expected bytes by barrier, waits (barrier, parity).
typedef std::tuple<uint32_t, int, int, int, uint32_t> Copy;
static std::vector<Copy> copies;
static std::vector<std::pair<uint32_t, uint32_t>> expected, waits;
static int commits, there_i, there_s;
static int cluster_rank() { return (int)(blockIdx.x & 1u); }
static uint32_t of_cta(uint32_t addr, int cta) { return addr | (uint32_t)cta << 28; }
static uint32_t smem_u32(const void*) { return 0; }
static void mbar_expect(uint32_t bar, uint32_t bytes) { expected.push_back({bar, bytes}); }
template <bool PAIR>
static void gp_commit(uint32_t, int) {
  ++commits;
}
static bool gp_wait_warp(uint32_t bar, uint32_t parity) {
  waits.push_back({bar, parity});
  return true;
}
template <bool PAIR>
static void tma_load_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  copies.push_back(Copy(dst, map->id, x, y, bar));
}

#include "extracted.h"

static void check(bool ok, const char* what) {
  if (ok) return;
  std::printf("%s\n", what);
  std::exit(1);
}

template <bool BACK, bool PAIR, int PARTS>
static void run(std::mt19937& rng) {
  const auto any = [&](int low, int high) { return low + (int)(rng() % (unsigned)(high - low + 1)); };
  GpMaps maps = {{0}, {1}, {2}, {3}};
  GpArgs a = {};
  a.tiles_m = any(1, 5), a.tiles_n = any(1, 7), a.band = any(1, 4);
  a.half = any(1, 6), a.steps = BACK ? 2 * a.half : a.half, a.last = any(1, PARTS);
  a.splits = any(1, std::min(3, a.steps)), a.span = (a.steps + a.splits - 1) / a.splits;
  if ((a.splits - 1) * a.span >= a.steps) a.splits = 1, a.span = a.steps;
  a.items = a.tiles_m * a.tiles_n * a.splits;
  a.bn = 64, a.room = 16384, a.part = a.room + 8192, a.bytes = a.part, a.slots = any(1, 8);
  const int stride = any(1, a.items), first = any(0, stride - 1);
  const uint32_t base = 1024, bar0 = 256;
  gridDim.x = (unsigned)(stride * (PAIR ? 2 : 1));

  // all stages of this CTA, or pair, and where each leaves its CTA
  struct Stage {
    GpItem t;
    int i, s;
  };
  std::vector<Stage> all;
  int end = first;
  for (; end < a.items; end += stride) {
    const GpItem t = gp_item(a, end);
    for (int s = t.s0; s < t.s1; ++s) all.push_back({t, end, s});
  }
  const int stages = (int)all.size();
  const auto place = [&](int n) {  // of a CTA that has issued n of them
    GpFed f;
    f.i = n < stages ? all[n].i : end, f.s = n < stages ? all[n].s : 0;
    f.slot = n % a.slots, f.turn = (uint32_t)(n / a.slots), f.used = std::min(n, a.slots);
    return f;
  };
  // neither is further ahead than the ring
  const int issued0 = any(0, stages), issued1 = PAIR ? std::min(stages, std::max(0, issued0 + any(-a.slots, a.slots))) : issued0;
  const int issued[2] = {issued0, issued1}, most = std::max(issued0, issued1);
  for (int rank = 0; rank < (PAIR ? 2 : 1); ++rank) {
    blockIdx.x = (unsigned)((PAIR ? 2 : 1) * first + rank);
    // the stages that the CTA is behind by, as its copying warp would have issued them
    copies.clear(), expected.clear();
    for (int n = issued[rank]; n < most; ++n) gp_feed<BACK, PAIR, PARTS>(maps, a, all[n].t, all[n].s, n % a.slots, base, bar0, rank, 0);
    const auto want = copies;
    const auto bytes = expected;
    check((rank == 0 ? (int)bytes.size() : 0) == (rank == 0 ? most - issued[0] : 0) && (rank == 0 || bytes.empty()), "expected bytes");
    copies.clear(), expected.clear(), waits.clear(), commits = 0;
    const GpFed mine = place(issued[rank]), other = place(issued[PAIR ? rank ^ 1 : rank]);
    there_i = other.i, there_s = other.s;
    threadIdx.x = 0;
    gp_drain<BACK, PAIR, PARTS>(maps, a, mine, base, bar0);
    check(copies == want && expected == bytes && commits == 0, "copies");
    // the first CTA waits for every stage that may be in flight, by the parity of its turn
    check((int)waits.size() == (rank == 0 ? std::min(most, a.slots) : 0), "waits");
    for (int j = 0; j < (int)waits.size(); ++j) {
      const int n = most - 1 - j;
      check(waits[j] == std::make_pair(bar0 + 8u * (uint32_t)(n % a.slots), (uint32_t)(n / a.slots) & 1u), "a wait's stage");
    }
    // the MMAs: the first CTA says when, both wait
    copies.clear(), waits.clear(), threadIdx.x = 32;
    gp_drain<BACK, PAIR, PARTS>(maps, a, mine, base, bar0);
    check(copies.empty() && commits == (rank == 0) && waits.size() == 1 && waits[0] == std::make_pair(bar0 + GP_DRAINED, 0u), "MMAs");
    for (int warp = 2; warp < 12; ++warp) {
      copies.clear(), waits.clear(), threadIdx.x = 32u * (unsigned)warp;
      gp_drain<BACK, PAIR, PARTS>(maps, a, mine, base, bar0);
      check(copies.empty() && waits.empty(), "another warp");
    }
  }
}
}  // namespace gc

int main() {
  std::mt19937 rng(5);
  for (int i = 0; i < 20000; ++i) {
    gc::run<true, true, 1>(rng), gc::run<true, true, 2>(rng), gc::run<false, true, 1>(rng), gc::run<false, true, 2>(rng);
    gc::run<true, false, 1>(rng), gc::run<true, false, 2>(rng), gc::run<false, false, 1>(rng), gc::run<false, false, 2>(rng);
  }
  std::printf("done\n");
}
