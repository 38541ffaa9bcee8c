// Gated projection on the fifth-generation tensor cores, out = act(x Wg^T) *
// (x Wu^T), and its input's gradient dx = dgate Wg + dup Wu.
#include <algorithm>
#include <type_traits>

#include "gc_act.cuh"
#include "gc_gate.cuh"
#include "gc_host.h"
#include "gc_mma.cuh"
#include "gc_proj_plan.h"

namespace gc {

// Mathematics and precision.  The operands are of 16 bits, so every product is
// exact in the tensor cores' fp32; their sums truncate.  A step of 16 products cuts each
// of them two bits below the last one of the sum, or of a larger product (measured: 16
// of 2^-2 of it are added, of 2^-3 not), and then the sum: less than 16 / 4 + 1 last bits,
// 5 2^-23 of the sum that is reached, and half of that on average.  Of terms of one
// sign, where nothing cancels, 6e-9 of the result per term of a chain was measured: 1.7e-4
// for the 28672 of a gradient, a third of the output's own half step in fp16 (2^-11) and
// a 23rd in bf16 (2^-8), so that chains are not cut.  G and U stay in fp32 from
// tensor memory to the activation, and the checkpoints are taken of that.
// The gradient's product has dgate and dup as they are rounded to 16 bits: operands in fp32
// would be two or three terms, and as many times the MMAs.  That is what the weight
// gradient reads, too, and what a product after gc_gated_act_backward would have; dx's error
// against 64 bits is 1.4 times that of a sum of the fp32 values (2.4e-3 of it in bf16
// where that is 1.7e-3, 2.9e-4 in fp16 where that is 2.1e-4).
//
// Tile.  128 rows of x by `bn` columns of out, one MMA of N = 2 bn for both
// projections: the rows of Wg and of Wu lie one after another in shared memory, so
// G is in the first bn columns of the accumulator and U in the next, and a
// thread that reads out a row has both.  The gradient's tile is 128 rows by bn
// columns of dx, its sum the concatenation of (dgate, Wg) and (dup, Wu).  Two
// accumulators of up to 256 columns: one is read out while the next is summed.
//
// x, dgate and dup are "K-major" (the summed index is consecutive), and so are
// the weights of the projection; the gradient sums over the weights' rows, which makes
// them "MN-major".  Everything comes by bulk tensor copies under the 128-byte
// swizzle, with zeros for what is outside a matrix.
//
// Pairs.  Of more than 128 rows two CTAs share a tile of 256: each stages its own
// rows and half of the columns' operand, 32 KB a stage instead of 48 for the same
// MMAs, which shared memory would bound otherwise (8192 x 14336 x 4096: 1071 us
// instead of 1218).  A stage of 64 takes 525 clocks where the MMAs alone take 512.
//
// Measured in bf16, back to back: 8192 x 14336 x 4096 1.04-1.11 ms (1.73-1.85
// PFLOP/s under the power cap; a library's product of the same size, without the
// activation, 1.06-1.11), with checkpoints 1.08-1.13, its gradient 1.09-1.14 behind
// dgate and dup (a library's product 1.08-1.13); on its own 2048 x 14336 x 4096's
// gradient takes 249 us, tensor pipe active 93%.  2048 x 4096 x 1024: 23 and, with
// checkpoints, 25 us, the gradient 27: four rounds of tiles where 3.4 would do, and
// the splits' join.  48 x 14336 x 4096: 39 us, 6.0 TB/s of weights.
constexpr int GP_SLOTS = 12;  // stages in the ring, at most
// An MMA reads 128 rows also where there are fewer, whose room is smaller: past
// the last one's there has to be shared memory, too (whatever it holds, it only
// reaches rows of the accumulator that are not there: it is the warps' stages for
// what they write).
constexpr int GP_SHARED = GP_RING + GP_M * GP_K * 2;
constexpr int GP_OUT = 8, GP_FIRST = 4;      // warps that read out, the first of them
constexpr int GP_THREADS = (GP_FIRST + GP_OUT) * 32;
constexpr int GP_POLLS = 1 << 22;            // limit of every wait

// All lanes of a warp, which go on or give up together.  (Asked first without
// being suspended, which costs 40 clocks where the phase is complete already.)
__device__ __forceinline__ bool gp_wait_warp(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n.reg .pred p;\nmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.b32 %0, 1, 0, p;\n}\n"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  if (__all_sync(FULL, done != 0u)) return true;
  for (int i = 0; i < GP_POLLS; ++i)
    if (__all_sync(FULL, mbar_poll(bar, parity))) return true;
  return false;
}
// One lane of a warp that is all there, always the same.  What a whole warp goes
// through, and one lane of it issues, is issued from uniform registers: with a
// branch for lane 0 a stage's four MMAs took 561 clocks to issue, now 380.
__device__ __forceinline__ bool elected() {
  uint32_t p;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.b32 %0, 1, 0, p;\n}\n" : "=r"(p)::"memory");
  return p != 0u;
}
// (The barrier may be the other CTA's of a pair.)
template <bool PAIR>
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  if (PAIR)
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%3, %4}], "
        "[%2];" ::"r"(dst),
        "l"(map), "r"(bar), "r"(x), "r"(y)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(map), "r"(bar), "r"(x), "r"(y)
        : "memory");
}
// MMAs, and arrivals when the ones before are done, of a CTA or of a pair (there
// on the barriers of both).
template <bool PAIR>
__device__ __forceinline__ void gp_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  if (PAIR)
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\ntcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
        : "memory");
  else
    mma_f16(d, a, b, idesc, add);
}
template <bool PAIR>
__device__ __forceinline__ void gp_commit(uint32_t bar, int leader) {
  if (PAIR)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((uint16_t)(3 << leader))
        : "memory");
  else
    mma_commit(bar);
}
// The same shared memory of another CTA of the cluster.
__device__ __forceinline__ uint32_t of_cta(uint32_t addr, int cta) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(cta));
  return r;
}
__device__ __forceinline__ int cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return (int)r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Shared-memory operand descriptor of a K-major tile under the 128-byte
// swizzle: rows of 128 bytes, groups of 8 rows 1024 bytes apart.
__device__ __forceinline__ uint64_t k_desc(uint32_t addr) { return mn_desc(addr, 16); }

struct GpMaps {
  CUtensorMap a0, a1, b0, b1;  // x, -, Wg, Wu; or dgate, dup, Wg, Wu
};
struct GpArgs {
  int64_t rows, cols;          // of the result
  int half, steps;             // stages of the first pair of operands, of both
  int last;                    // parts of the last stage of a pair of operands
  int bn, slots;               // columns of a tile, stages in the ring
  int part, room, bytes;       // room of a part, of its rows (a multiple of 1024), bytes that arrive
  int tiles_m, tiles_n, splits, items, span;  // span: stages of a split
  int band;                    // tiles of a band of rows, which goes along all columns before the next one
  void* out;
  int64_t ldo;
  int vec;                     // what rows of `out` start on, as gp_put takes it
  bool whole, even;            // codes start on a 32-byte boundary; rows of steps on even addresses
  int8_t *gcodes, *ucodes;
  uint8_t *gsteps, *usteps;
  float* sums;                 // of splits that a kernel of its own joins, one [rows, lds] after another
  int64_t lds;
  uint32_t* diag;
};
struct GpItem {
  int m, n, split, s0, s1;
};
__device__ __forceinline__ GpItem gp_item(const GpArgs& a, int i) {
  GpItem t;
  t.split = i % a.splits;
  const int tile = i / a.splits, band = tile / (a.band * a.tiles_n), r = tile % (a.band * a.tiles_n);
  const int high = min(a.band, a.tiles_m - band * a.band);
  t.m = band * a.band + r % high, t.n = r / high;
  t.s0 = t.split * a.span, t.s1 = min(t.s0 + a.span, a.steps);
  return t;
}

// 32 bytes, which a thread has of its row, in as few stores as their address
// allows: every thread's store is a request of its own to L2, which takes the SM 1.5
// clocks whatever its size.
__device__ __forceinline__ void gp_put32(void* to, const uint32_t (&w)[8], bool whole) {
  if (whole) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                 "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    static_cast<uint4*>(to)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    static_cast<uint4*>(to)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}
// The codes of the 32 values of a group that one thread holds; returns their step.
__device__ __forceinline__ uint32_t gp_hold(const float (&v)[32], int8_t* codes, bool whole) {
  float top = max_nan(fabsf(v[0]), fabsf(v[1]));
#pragma unroll
  for (int i = 2; i < 32; i += 2) top = max_nan(top, fabsf(v[i]), fabsf(v[i + 1]));
  const uint32_t b = act_step(__float_as_uint(top));
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float x[CHUNK];
#pragma unroll
    for (int e = 0; e < CHUNK; ++e) x[e] = v[8 * i + e];
    const uint2 q = chunk_codes(x, b);
    w[2 * i] = q.x, w[2 * i + 1] = q.y;
  }
  gp_put32(codes, w, whole);
  return b;
}
// n of the 32 values of each lane's row, a warp's rows one after another from the
// one at `to` on; there: this lane's row is.  vec: 0 where rows start anywhere, 1 on
// 16-byte boundaries, 2 on 32-byte ones.  Rows that start anywhere, and the last
// columns, go through `stage` (the warp's own 2 KB) and a lane per column: stored by
// the lanes of their rows 138 x 7785 took 23 us instead of 8.
template <typename T>
__device__ __forceinline__ void gp_put(const float (&v)[32], T* to, int64_t ld, bool there, int n, int vec, uint32_t stage) {
  const int lane = threadIdx.x & 31;
  uint32_t w[2][8];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    alignas(16) T r[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) r[e] = from_f32<T>(v[16 * i + e]);
#pragma unroll
    for (int e = 0; e < 8; ++e) w[i][e] = reinterpret_cast<const uint32_t*>(r)[e];
  }
  if (vec && (n & 15) == 0) {
    T* const row = to + lane * ld;
    if (there) gp_put32(row, w[0], vec == 2);
    if (there && n == 32) gp_put32(row + 16, w[1], vec == 2);
    return;
  }
  // 16-byte chunk c of row r at chunk c ^ (r / 2 & 3)
  const int rows = __popc(__ballot_sync(FULL, there));
  __syncwarp();
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const uint32_t* const x = &w[c >> 1][4 * (c & 1)];
    st_shared16(stage + (uint32_t)lane * 64u + (uint32_t)((c ^ ((lane >> 1) & 3)) << 4), x[0], x[1], x[2], x[3]);
  }
  __syncwarp();
  if (lane < n) {
    uint16_t* o = reinterpret_cast<uint16_t*>(to + lane);
#pragma unroll 4
    for (int r = 0; r < rows; ++r, o += ld) {
      uint16_t x;
      asm volatile("ld.shared.u16 %0, [%1];"
                   : "=h"(x)
                   : "r"(stage + (uint32_t)r * 64u + (uint32_t)(((lane >> 3) ^ ((r >> 1) & 3)) << 4) + (uint32_t)(lane & 7) * 2u)
                   : "memory");
      *o = x;
    }
  }
}
// fp32 sums of a split: rows on 32-byte boundaries.
__device__ __forceinline__ void gp_put_sums(const float (&v)[32], float* to, int n) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = __float_as_uint(v[8 * i + e]);
    if (8 * i < n) gp_put32(to + 8 * i, w, true);  // rows have room for whole eights
  }
}
// How far a CTA's copies have come: the stage that is next (past the last one: an
// item that is not there, stage 0), its place in the ring, how many before it may not
// have been multiplied yet.
struct alignas(8) GpFed {
  int i, s, slot, used;
  uint32_t turn;
};
// The columns of a tile that are there; its groups of 32 of them.
__device__ __forceinline__ int gp_width(const GpArgs& a, int n) { return (int)min((int64_t)a.bn, a.cols - (int64_t)n * a.bn); }
__device__ __forceinline__ int gp_groups(const GpArgs& a, int n) { return (gp_width(a, n) + 31) / 32; }
constexpr int GP_BACK = -1;
// What a warp does with the sums of n of 32 columns, from `col` on, of its rows, row0 + lane: the
// gradient's as they are; the projections' through the checkpoints and the activation.  held: the
// steps of the group before, where this warp had that one (after) and two groups' steps
// are written at a time; next: it has the next one, too.
template <typename T, int KIND, int U>
__device__ __forceinline__ void gp_finish(const GpArgs& a, int64_t row0, int64_t col, int n, float (&g)[32], float (&u)[U],
                                          uint32_t* held, bool after, bool next, uint32_t stage) {
  const int64_t row = row0 + (threadIdx.x & 31);
  const bool there = row < a.rows;
  if constexpr (KIND != GP_BACK) {
    if (n < 32) {
#pragma unroll
      for (int e = 0; e < 32; ++e)
        if (e >= n) g[e] = u[e] = 0.0f;
    }
    if (a.gcodes && there) {
      const int64_t at = row * (act_ldc(a.cols) >> 5) + (col >> 5);  // the group
      const bool odd = ((col >> 5) & 1) != 0;
      const uint32_t bg = gp_hold(g, a.gcodes + 32 * at, a.whole), bu = gp_hold(u, a.ucodes + 32 * at, a.whole);
      if (a.even && !odd && next) {
        *held = bg | bu << 16;
      } else if (a.even && odd && after) {
        *reinterpret_cast<uint16_t*>(a.gsteps + at - 1) = (uint16_t)((*held & 255u) | bg << 8);
        *reinterpret_cast<uint16_t*>(a.usteps + at - 1) = (uint16_t)(*held >> 16 | bu << 8);
      } else {
        a.gsteps[at] = (uint8_t)bg, a.usteps[at] = (uint8_t)bu;
      }
    }
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
      F2 dp;
      put2(g + e, mul2(mul2(get2(g + e), gate_sigmoid2<KIND>(g + e, &dp)), get2(u + e)));
    }
  }
  gp_put(g, static_cast<T*>(a.out) + row0 * a.ldo + col, a.ldo, there, n, a.vec, stage);
}

// The barriers of a CTA, one after another: of a stage's copies (the first CTA's of a
// pair: both CTAs' are there) and of its MMAs, of an accumulator's MMAs and (the first
// CTA's) of its having been read out, of all MMAs after a wait that ran out, of the other
// splits' sums.
constexpr uint32_t GP_EMPTY = 8u * GP_SLOTS, GP_ACC_FULL = 16u * GP_SLOTS, GP_ACC_EMPTY = GP_ACC_FULL + 16u,
                   GP_DRAINED = GP_ACC_EMPTY + 16u, GP_JOINED = GP_DRAINED + 8u;
// The copies of a stage into its place in the ring, by a whole warp.
template <bool BACK, bool PAIR, int PARTS>
__device__ __forceinline__ void gp_feed(const GpMaps& maps, const GpArgs& a, const GpItem& t, int s, int slot, uint32_t base,
                                        uint32_t bar0, int rank, int leader) {
  const int row = t.m * (PAIR ? 2 * GP_M : GP_M) + rank * GP_M, cols = PAIR ? a.bn / 2 : a.bn;
  const uint32_t full = bar0 + 8u * slot, bar = PAIR ? of_cta(full, leader) : full;
  const int parts = PARTS > 1 && (s + 1 == a.half || s + 1 == a.steps) ? a.last : PARTS;
  uint32_t st = base + (uint32_t)(slot * PARTS * a.part);
  if (elected()) {
    if (rank == 0) mbar_expect(full, (uint32_t)((PAIR ? 2 : 1) * parts * a.bytes));
    const bool second = BACK && s >= a.half;
    int x = (second ? s - a.half : s) * (PARTS * GP_K);
#pragma unroll
    for (int h = 0; h < PARTS; ++h, x += GP_K, st += (uint32_t)a.part) {
      if (h >= parts) break;
      if (BACK) {
        tma_load_2d<PAIR>(st, second ? &maps.a1 : &maps.a0, x, row, bar);
        for (int b = 0; b < cols; b += 64)
          tma_load_2d<PAIR>(st + a.room + b * (GP_K * 2), second ? &maps.b1 : &maps.b0, t.n * a.bn + rank * cols + b, x, bar);
      } else {
        tma_load_2d<PAIR>(st, &maps.a0, x, row, bar);
        if (PAIR) {  // the first CTA has Wg's rows, the second Wu's
          tma_load_2d<PAIR>(st + a.room, rank ? &maps.b1 : &maps.b0, x, t.n * a.bn, bar);
        } else {
          tma_load_2d<PAIR>(st + a.room, &maps.b0, x, t.n * a.bn, bar);
          tma_load_2d<PAIR>(st + a.room + a.bn * (GP_K * 2), &maps.b1, x, t.n * a.bn, bar);
        }
      }
    }
  }
  __syncwarp();
}
// Says that a wait ran out to all CTAs of the cluster, before it ends its role (and so
// before the cluster's next barrier).  Out of line, as the next one, so that the common
// path stays as short as it is.
__device__ __noinline__ void gp_tell(const uint32_t* lost, int ctas) {
  if ((threadIdx.x & 31) == 0)
    for (int c = 0; c < ctas; ++c) asm volatile("st.shared::cluster.u32 [%0], 1;" ::"r"(of_cta(smem_u32(lost), c)) : "memory");
}
// The end of a CTA of whose cluster a wait ran out: until what is on its way to its
// shared memory is there.
template <bool BACK, bool PAIR, int PARTS>
__device__ __noinline__ void gp_drain(const GpMaps& maps, const GpArgs& a, const GpFed& fed, uint32_t base, uint32_t bar0) {
  const int warp = __shfl_sync(FULL, (int)(threadIdx.x >> 5), 0);
  const int rank = PAIR ? (int)(blockIdx.x & 1u) : 0, leader = PAIR ? cluster_rank() & ~1 : 0;
  // MMAs in flight read the CTAs' memory, and say so on their barriers when they are
  // done: by a barrier that nothing else completes.
  if (warp == 1) {
    if (rank == 0 && elected()) gp_commit<PAIR>(bar0 + GP_DRAINED, leader);
    __syncwarp();
    gp_wait_warp(bar0 + GP_DRAINED, 0u);
  }
  // Copies land on the first CTA's barriers, which are complete when both CTAs' have.  The
  // one that gave up first issues what the other one has beyond it (whose room is free: the
  // other one has waited for that), and every stage in flight is one that ends.
  if (warp == 0) {
    GpFed f = fed;
    if (PAIR) {
      const int stride = (int)(gridDim.x >> 1);
      const uint32_t there = of_cta(smem_u32(&fed), leader + (rank ^ 1));
      int i, s;
      asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(i), "=r"(s) : "r"(there) : "memory");
      while (f.i < i || (f.i == i && f.s < s)) {
        const GpItem t = gp_item(a, f.i);
        gp_feed<BACK, PAIR, PARTS>(maps, a, t, f.s, f.slot, base, bar0, rank, leader);
        if (++f.slot == a.slots) f.slot = 0, ++f.turn;
        f.used = min(f.used + 1, a.slots);
        if (++f.s == t.s1) f.i += stride, f.s = f.i < a.items ? gp_item(a, f.i).s0 : 0;
      }
    }
    for (int j = 0; rank == 0 && j < f.used; ++j) {
      if (--f.slot < 0) f.slot = a.slots - 1, --f.turn;
      gp_wait_warp(bar0 + 8u * f.slot, f.turn & 1u);
    }
  }
}

// KIND: the activation; GP_BACK: the gradient.  PAIR: a cluster of two CTAs
// computes a tile of 256 rows, half of them each; the first one's thread issues
// the MMAs of both, which read each CTA's rows and half of the columns' operand out
// of its own memory.  PARTS: of GP_K in a stage.
// A role whose wait runs out says so to the whole cluster, whose CTAs then end
// together: none joins its sums, and each awaits what is on its way to it, below.
template <typename T, int KIND, bool PAIR, int PARTS>
__global__ void __launch_bounds__(GP_THREADS, 1)
    k_gated_proj(const __grid_constant__ GpMaps maps, const __grid_constant__ GpArgs a) {
  constexpr bool BACK = KIND == GP_BACK;
  extern __shared__ __align__(1024) unsigned char smem[];
  __shared__ __align__(8) uint64_t bars[2 * GP_SLOTS + 6];
  __shared__ uint32_t tmem_base, lost;
  __shared__ GpFed fed;
  const int warp = __shfl_sync(FULL, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;  // (a uniform register)
  const int rank = PAIR ? (int)(blockIdx.x & 1u) : 0, leader = PAIR ? cluster_rank() & ~1 : 0;
  const int first = PAIR ? (int)(blockIdx.x >> 1) : (int)blockIdx.x, stride = PAIR ? (int)(gridDim.x >> 1) : (int)gridDim.x;
  const uint32_t base = smem_u32(smem), bar0 = smem_u32(bars);
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + GP_EMPTY + 8u * s; };
  auto acc_full = [&](int h) { return bar0 + GP_ACC_FULL + 8u * h; };
  auto acc_empty = [&](int h) { return bar0 + GP_ACC_EMPTY + 8u * h; };
  const uint32_t drained = bar0 + GP_DRAINED, joined = bar0 + GP_JOINED;

  if (warp == 2 && elected()) {
    for (const CUtensorMap* m : {&maps.a0, &maps.a1, &maps.b0, &maps.b1}) asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < GP_SLOTS; ++s) mbar_init(full(s), 1), mbar_init(empty(s), 1);
    for (int h = 0; h < 2; ++h) mbar_init(acc_full(h), 1), mbar_init(acc_empty(h), PAIR ? 2 * GP_OUT : GP_OUT);
    mbar_init(drained, 1), mbar_init(joined, 1);
    lost = 0u;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    if (PAIR) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&tmem_base)) : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&tmem_base)) : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  const bool joint = a.splits > 1 && !a.sums;  // a cluster's splits
  const int ctas = (PAIR ? 2 : 1) * (joint ? a.splits : 1);
  if (PAIR || joint) cluster_sync();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = __shfl_sync(FULL, tmem_base, 0);
  chain_wait();
  if (blockIdx.x == 0 && threadIdx.x <= DIAG_PATH) a.diag[threadIdx.x] = 0u;  // all that the status call reads

  bool ok = true;
  if (warp == 0) {
    // ------------------------------------------------ operands
    int i = first, at = 0, slot = 0, used = 0;  // used: the stages whose copies were issued, up to a ring's
    uint32_t turn = 0u;
    for (; i < a.items; i += stride) {
      const GpItem t = gp_item(a, i);
      for (int s = t.s0; s < t.s1; ++s) {
        if (!(ok = gp_wait_warp(empty(slot), (turn & 1u) ^ 1u))) {
          at = s;
          break;
        }
        gp_feed<BACK, PAIR, PARTS>(maps, a, t, s, slot, base, bar0, rank, leader);
        if (++slot == a.slots) slot = 0, ++turn;
        used = min(used + 1, a.slots);
      }
      if (!ok) break;
    }
    if (lane == 0) fed = {i, at, slot, used, turn};
    // before this CTA may end: the last stages have been multiplied, and said so on its barriers
    for (int j = 0; ok && j < used; ++j) {
      if (--slot < 0) slot = a.slots - 1, --turn;
      ok = gp_wait_warp(empty(slot), turn & 1u);
    }
    if (!ok) gp_tell(&lost, ctas);
  } else if (warp == 1) {
    // ------------------------------------------------ MMA
    if (rank == 0) {
      // fp32 accumulator, the operands' type, N, M = 128 or 256
      constexpr uint32_t type = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
      const uint32_t idesc = (1u << 4) | (type << 7) | (type << 10) | (BACK ? 1u << 16 : 0u) |
                             ((uint32_t)((BACK ? a.bn : 2 * a.bn) >> 3) << 17) | (PAIR ? 16u << 24 : 8u << 24);
      int slot = 0;
      uint32_t turn = 0u, count = 0u;
      for (int i = first; ok && i < a.items; i += stride, ++count) {
        const GpItem t = gp_item(a, i);
        const uint32_t acc = count & 1u;
        if (!(ok = gp_wait_warp(acc_empty(acc), ((count >> 1) & 1u) ^ 1u))) break;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        for (int s = t.s0; s < t.s1; ++s) {
          // (what was copied is ordered by the barrier alone)
          if (!(ok = gp_wait_warp(full(slot), turn & 1u))) break;
          const uint32_t d = tmem + 256u * acc;
          const int parts = PARTS > 1 && (s + 1 == a.half || s + 1 == a.steps) ? a.last : PARTS;
          uint32_t st = base + (uint32_t)(slot * PARTS * a.part);
          if (elected()) {
#pragma unroll
            for (int h = 0; h < PARTS; ++h, st += (uint32_t)a.part) {
              if (h >= parts) break;
              const uint64_t da = k_desc(st), db = BACK ? mn_desc(st + a.room, GP_K * 128) : k_desc(st + a.room);
              gp_mma<PAIR>(d, da, db, idesc, h > 0 || s > t.s0);
#pragma unroll
              for (int j = 1; j < GP_K / 16; ++j) gp_mma<PAIR>(d, da + 2u * j, db + (BACK ? 128u : 2u) * j, idesc, true);
            }
            gp_commit<PAIR>(empty(slot), leader);
            if (s + 1 == t.s1) gp_commit<PAIR>(acc_full(acc), leader);
          }
          __syncwarp();
          if (++slot == a.slots) slot = 0, ++turn;
        }
      }
      if (!ok) gp_tell(&lost, ctas);
    }
  } else if (warp >= GP_FIRST) {
    // ------------------------------------------------ result
    const int quad = warp & 3, side = (warp - GP_FIRST) >> 2;
    uint32_t count = 0u;
    for (int i = first; ok && i < a.items; i += stride, ++count) {
      const GpItem t = gp_item(a, i);
      const uint32_t acc = count & 1u;
      if (!(ok = gp_wait_warp(acc_full(acc), (count >> 1) & 1u))) {
        gp_tell(&lost, ctas);
        break;
      }
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const uint32_t from = tmem + 256u * acc + ((uint32_t)(32 * quad) << 16);
      if (joint) break;  // the tile's only one: below
      const int64_t row0 = (int64_t)t.m * (PAIR ? 2 * GP_M : GP_M) + rank * GP_M + 32 * quad, c0 = (int64_t)t.n * a.bn;
      const uint32_t stage = base + GP_RING + (uint32_t)(warp - GP_FIRST) * 2048u;
      // the groups of 32 columns of this warp, next to each other
      const int width = gp_width(a, t.n), groups = gp_groups(a, t.n), half = (groups + 1) / 2;
      const int begin = side ? half : 0, end = side ? groups : half;
      uint32_t held = 0u;  // the steps of the group before
      auto read_out = [&] {  // the accumulator may be written again
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          // (at the scope of the CTA: what is to be ordered is in tensor memory, by the
          // fence above; a release to the cluster waits 2000 clocks for this thread's stores)
          if (PAIR)
            asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(of_cta(acc_empty(acc), leader)) : "memory");
          else
            mbar_arrive(acc_empty(acc));
        }
      };
      if (begin == end) read_out();
      for (int q = begin; q < end; ++q) {
        float g[32], u[BACK ? 1 : 32];
        tmem_load32(g, from + 32 * q);
        if constexpr (!BACK) tmem_load32(u, from + a.bn + 32 * q);
        if (q + 1 == end) read_out();
        const int n = min(32, width - 32 * q);
        if (row0 < a.rows) {
          if (BACK && a.sums) {
            if (row0 + lane < a.rows) gp_put_sums(g, a.sums + ((int64_t)t.split * a.rows + row0 + lane) * a.lds + c0 + 32 * q, n);
          } else {
            gp_finish<T, KIND>(a, row0, c0 + 32 * q, n, g, u, &held, q > begin, q + 1 < end, stage);
          }
        }
        __syncwarp();
      }
    }
  }
  if (joint) {
    // The cluster's CTAs (pairs) have summed a part of the tile each, and end together
    // here.  Group q of its columns is finished by split q % splits: the others
    // send it their sums, and it adds them in the splits' order.  They go by bulk
    // copies from ring to ring, which nothing else reads or writes any more when all are
    // here: what arrives first, what leaves behind it, 4 KB (32 rows) of a block by
    // each warp.  (Stored by the threads themselves, a row each, 64 KB took 9500 clocks.)
    const GpItem t = gp_item(a, first);
    const int quad = warp & 3, side = (warp - GP_FIRST) >> 2, groups = gp_groups(a, t.n), most = (groups + a.splits - 1) / a.splits;
    constexpr uint32_t BLOCK = GP_M * 128;  // 32 columns of a CTA's rows
    constexpr int BLOCKS = BACK ? 1 : 2;
    const uint32_t here = (uint32_t)(32 * quad) * 128u;  // of a warp's part of a block
    const uint32_t row128 = here + (uint32_t)lane * 128u;
    const int64_t row0 = (int64_t)t.m * (PAIR ? 2 * GP_M : GP_M) + rank * GP_M;
    const int quads = (int)min((int64_t)4, max((int64_t)0, (a.rows - row0 + 31) / 32));  // that have rows
    if (threadIdx.x == 0)
      mbar_expect(joined, (uint32_t)((groups - t.split + a.splits - 1) / a.splits * (a.splits - 1) * BLOCKS * quads) * 4096u);
    __syncwarp();
    cluster_sync();
    const bool mine = warp >= GP_FIRST && quad < quads && lost == 0u;  // (all CTAs see the same here: all send, or none)
    const uint32_t from = tmem + ((uint32_t)(32 * quad) << 16);
    // where split `of` puts its sums of the owner's group q
    auto block = [&](int q, int owner, int of) { return (uint32_t)((q / a.splits) * (a.splits - 1) + of - (of > owner)) * (BLOCKS * BLOCK); };
    if (mine) {
      for (int q = side; q < groups; q += 2) {
        const int owner = q % a.splits, cta = PAIR ? 2 * owner + rank : owner;
        if (owner == t.split) continue;
        const int sent = q - (q + a.splits - 1 - t.split) / a.splits;  // of the groups of others
        const uint32_t src = base + (uint32_t)(most * (a.splits - 1) + sent) * (BLOCKS * BLOCK), dst = base + block(q, owner, t.split);
#pragma unroll
        for (int b = 0; b < BLOCKS; ++b) {
          float v[32];
          tmem_load32(v, from + 32 * q + (b ? a.bn : 0));
#pragma unroll
          for (int c = 0; c < 8; ++c)
            st_shared16(src + b * BLOCK + row128 + (uint32_t)((c ^ (lane & 7)) << 4), __float_as_uint(v[4 * c]),
                        __float_as_uint(v[4 * c + 1]), __float_as_uint(v[4 * c + 2]), __float_as_uint(v[4 * c + 3]));
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (elected())
            asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], 4096, [%2];" ::"r"(
                             of_cta(dst + b * BLOCK + here, cta)),
                         "r"(src + b * BLOCK + here), "r"(of_cta(joined, cta))
                         : "memory");
          __syncwarp();
        }
      }
      ok = gp_wait_warp(joined, 0u);  // what is on its way here lands before this CTA ends
    }
    if (mine && ok) {
      const uint32_t at = base + row128;
      const uint32_t stage = base + GP_RING + (uint32_t)(warp - GP_FIRST) * 2048u;
      for (int q = t.split + side * a.splits; q < groups; q += 2 * a.splits) {
        float sum[BLOCKS][32];
#pragma unroll
        for (int b = 0; b < BLOCKS; ++b) {
          float own[32];
          tmem_load32(own, from + 32 * q + (b ? a.bn : 0));
#pragma unroll
          for (int e = 0; e < 32; ++e) sum[b][e] = t.split == 0 ? own[e] : 0.0f;
          for (int p = 0; p < a.splits; ++p) {
            if (p == t.split) {
              if (p > 0) {
#pragma unroll
                for (int e = 0; e < 32; ++e) sum[b][e] = __fadd_rn(sum[b][e], own[e]);
              }
              continue;
            }
            const uint32_t src = at + block(q, t.split, p) + b * BLOCK;
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              const uint4 x = shared16(src + (uint32_t)((c ^ (lane & 7)) << 4));
              sum[b][4 * c] = __fadd_rn(sum[b][4 * c], __uint_as_float(x.x)), sum[b][4 * c + 1] = __fadd_rn(sum[b][4 * c + 1], __uint_as_float(x.y));
              sum[b][4 * c + 2] = __fadd_rn(sum[b][4 * c + 2], __uint_as_float(x.z)), sum[b][4 * c + 3] = __fadd_rn(sum[b][4 * c + 3], __uint_as_float(x.w));
            }
          }
        }
        uint32_t held = 0u;
        gp_finish<T, KIND>(a, row0 + 32 * quad, (int64_t)t.n * a.bn + 32 * q, min(32, gp_width(a, t.n) - 32 * q), sum[0],
                           sum[BLOCKS - 1], &held, false, false, stage);
        __syncwarp();
      }
    }
  }
  if (!ok) atomicOr(a.diag + DIAG_ERR, GC_DIAG_TIMEOUT);
  __syncwarp();
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (PAIR || joint) cluster_sync();  // none ends, or gives its tensor memory back, while another may reach it
  if (lost != 0u) {
    gp_drain<BACK, PAIR, PARTS>(maps, a, fed, base, bar0);
    __syncthreads();
    if (PAIR || joint) cluster_sync();
  }
  if (warp == 1) {
    if (PAIR)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    else
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}
// dx = the splits' sums in their order, a column per thread and eight sums' loads
// at a time.
template <typename T>
__global__ void __launch_bounds__(256) k_gated_proj_join(const float* sums, int splits, int64_t rows, int cols, int64_t lds, T* out,
                                                         int64_t ldo) {
  chain_wait();
  const int64_t r = blockIdx.y, plane = rows * lds;
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= cols) return;
  const float* const from = sums + r * lds + c;
  float sum = 0.0f;
  for (int p = 0; p < splits; p += 8) {
    float v[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] = p + q < splits ? __ldg(from + (p + q) * plane) : 0.0f;
#pragma unroll
    for (int q = 0; q < 8; ++q) sum = __fadd_rn(sum, v[q]);
  }
  out[r * ldo + c] = from_f32<T>(sum);
}

// 8 elements of a row from column c on, wherever it starts; zeros past its end k.
// The granules of memory that hold them are read whole and the elements shifted out.
template <typename T, bool SPAN>
struct Eight {
  static constexpr int N = SPAN ? 2 : 1;
  uint4 w[N];
  __device__ __forceinline__ void load(const T* row, int64_t c, int64_t k, bool stream) {
    const T* const at = row + c;
    const int skip = SPAN ? (int)((uintptr_t)at & 15u) : 0;
    const int64_t bytes = skip + 2 * min((int64_t)CHUNK, k - c);  // of granules, from the first one on
    const uint4* const from = reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(at) - skip);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      w[i] = make_uint4(0u, 0u, 0u, 0u);
      if (k - c > 0 && bytes > 16 * i) w[i] = stream ? __ldcs(from + i) : __ldg(from + i);
    }
  }
  __device__ __forceinline__ uint4 words(const T* row, int64_t c) const {
    uint32_t x[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[N - 1].x, w[N - 1].y, w[N - 1].z, w[N - 1].w};
    if (SPAN) shift_words<4>(x, (int)((uintptr_t)(row + c) & 15u));
    return make_uint4(x[0], x[1], x[2], x[3]);
  }
  __device__ __forceinline__ void take(const T* row, int64_t c, int64_t k, float (&v)[CHUNK]) const {
    Raw8<T> r;
    *reinterpret_cast<uint4*>(&r) = words(row, c);
    unpack(r, v);
    if (k - c < CHUNK) {
#pragma unroll
      for (int e = 0; e < CHUNK; ++e)
        if (e >= k - c) v[e] = 0.0f;
    }
  }
};

// Copies whose rows start on 16-byte boundaries, of up to three matrices of
// 16-bit elements with as many columns each, which have blocks in turn.  A thread
// copies 8 elements, and 8 more half the matrix later: a call of 400 x 4097 x 1001
// takes 16.9 us with these two, 21.0 with one and 17.7 with four; up to 16 CTAs an
// SM, which then go round again.  The elements past a row's end are whatever follows
// it (what reads the copies does not).
struct GpAlign {
  const void* from[3];
  void* to[3];
  int64_t ld[3], rows[3];
  unsigned first[4];  // block of each
  int count;
};
__global__ void __launch_bounds__(256) k_align_rows(const __grid_constant__ GpAlign a, int64_t cols, uint32_t chunks) {
  using B = __nv_bfloat16;  // any 16 bits
  chain_wait();
  const int z = (blockIdx.x >= a.first[1]) + (blockIdx.x >= a.first[2]);
  const B* const x = static_cast<const B*>(a.from[z]);
  uint4* const to = static_cast<uint4*>(a.to[z]);
  const int64_t ld = a.ld[z], total = a.rows[z] * chunks, stride = (int64_t)(a.first[z + 1] - a.first[z]) * 256;
  for (int64_t q0 = (int64_t)(blockIdx.x - a.first[z]) * 256 + threadIdx.x; q0 < total; q0 += 2 * stride) {
    Eight<B, true> v[2];
    const B* row[2];
    int64_t c[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t q = q0 + i * stride;
      if (q >= total) break;
      const int64_t r = total < (int64_t(1) << 32) ? (int64_t)((uint32_t)q / chunks) : q / chunks;
      row[i] = x + r * ld, c[i] = (q - r * chunks) * CHUNK;
      v[i].load(row[i], c[i], cols, false);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (q0 + i * stride < total) to[q0 + i * stride] = v[i].words(row[i], c[i]);
  }
}

// ---------------------------------------------------------------- few rows
// The projection of one row reads its weights once and does little else: a warp
// per two columns of out streams their four rows of weights, 8 elements a lane,
// through the FMA units.  Sums are fp32, a lane's share of a row in two chains,
// then over the lanes, then over the warps that share the row (up to eight, where n is
// small: 300 x 8192 takes 5.0 us, by one warp each 18.0).  14336 x 4096 in bf16 takes
// 34.8 us from memory (6.7 TB/s) and 4096 x 1024 5.3; the tensor cores' kernel, whose copies
// take longer to get going, 37.5 and 7.4.
// One row always goes this way.  From memory, where a token's weights come from, it is
// faster or within 3% at 37 of 41 sizes measured, and 6 to 23% slower at four whose last wave
// of CTAs (16 columns each, 456 at a time) is mostly empty: 7448 x 4352 29.2 us, by the
// tensor cores 23.9; 9728 x 7992 54.6 and 50.5.  Weights of 60 to 100 MB that L2 still
// holds from the call before are read faster by the tensor cores' copies (11128 x 1664
// 15.6 us and 11.8, 14200 x 1696 19.1 and 14.8), smaller ones slower.
// Of more rows a warp has R = 2 at a time (one: 9.7 us for 8 x 1000 x 777, two 6.7, four, whose
// registers leave half the loads in flight, 7.0) and what they cost is instructions: some
// 1.25 steps of 256 k to begin and end a pair of rows by two columns, and one for each.  Two
// rows of 4096 x 1024 take 5.4 us and four 8.2, there 7.4; 16 of 333 x 1001 6.3 and
// 40 9.5, there 7.9; 40 of 512 x 64 6.2, there 5.5; there, too, k costs latency.
// SPAN: rows of weights or of x off 16-byte boundaries.
template <typename T, int KIND, bool SPAN, int R, bool JOIN>
__global__ void __launch_bounds__(256, R > 1 ? 2 : 3)
    k_gated_proj_row(const T* x, int64_t ldx, const T* wg, int64_t ldwg, const T* wu, int64_t ldwu, int64_t n, int64_t k, T* out,
                     int64_t ldo, int rows, int shared, uint32_t* diag) {
  __shared__ __align__(16) float sums[JOIN ? 8 : 1][R][4];
  chain_wait();
  if (blockIdx.x == 0 && threadIdx.x <= DIAG_PATH) diag[threadIdx.x] = 0u;
  const unsigned groups = (unsigned)(rows + R - 1) / R;
  const int split = JOIN ? shared : 0, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, parts = 1 << split, part = warp & (parts - 1);
  const int row0 = R * (int)(blockIdx.x % groups);
  const int64_t j = 2 * (((int64_t)(blockIdx.x / groups) * 8 + warp) >> split);
  const int64_t j0 = min(j, n - 1), j1 = min(j + 1, n - 1);
  const T* const w[4] = {wg + j0 * ldwg, wg + j1 * ldwg, wu + j0 * ldwu, wu + j1 * ldwu};
  const T* xr[R];
#pragma unroll
  for (int r = 0; r < R; ++r) xr[r] = x + min(row0 + r, rows - 1) * ldx;
  F2 sum[R][4];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int i = 0; i < 4; ++i) sum[r][i] = f2(0.0f);
  constexpr int STEPS = SPAN ? 1 : 2;  // steps whose loads are in flight together
  const int64_t step = 256 << split;     // (the same steps for each warp wherever rows start: the same bits)
  for (int64_t c0 = 8 * lane + 256 * part; c0 < k; c0 += step * STEPS) {
    Eight<T, SPAN> ws[STEPS][4], xs[STEPS][R];
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i) ws[s][i].load(w[i], c0 + step * s, k, true);
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
#pragma unroll
      for (int r = 0; r < R; ++r) xs[s][r].load(xr[r], c0 + step * s, k, false);
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const int64_t c = c0 + step * s;
      float xv[R][CHUNK];
#pragma unroll
      for (int r = 0; r < R; ++r) xs[s][r].take(xr[r], c, k, xv[r]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float wv[CHUNK];
        ws[s][i].take(w[i], c, k, wv);
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int e = 0; e < CHUNK; e += 2) sum[r][i] = fma2(get2(wv + e), get2(xv[r] + e), sum[r][i]);
      }
    }
  }
  float v[4];  // of row row0 + lane
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float two[2];
      put2(two, sum[r][i]);
      float all = __fadd_rn(two[0], two[1]);
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) all = __fadd_rn(all, __shfl_xor_sync(FULL, all, d));
      if (r == 0 || lane == r) v[i] = all;
    }
  if constexpr (JOIN) {
    if (part != 0 && lane < R) *reinterpret_cast<float4*>(sums[warp][lane]) = make_float4(v[0], v[1], v[2], v[3]);
    __syncthreads();
  }
  if (part != 0 || lane >= R || row0 + lane >= rows || j >= n) return;
  if constexpr (JOIN) {
    for (int p = 1; p < parts; ++p)
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = __fadd_rn(v[i], sums[warp + p][lane][i]);
  }
  F2 dp;
  put2(v, mul2(mul2(get2(v), gate_sigmoid2<KIND>(v, &dp)), get2(v + 2)));
  T* const o = out + (row0 + lane) * ldo;
  o[j] = from_f32<T>(v[0]);
  if (j + 1 < n) o[j + 1] = from_f32<T>(v[1]);
}

// ---------------------------------------------------------------- host
static bool make_map(CUtensorMap* m, int32_t dtype, const void* p, int64_t ld, int64_t rows, int64_t cols, int box_rows) {
  const TensorMapEncode encode = tensor_map_encode();
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)ld * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)box_rows}, step[2] = {1, 1};
  return encode && encode(m, dtype == GC_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
                          const_cast<void*>(p), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Clusters of so many CTAs (of any of the kernels, which take an SM each) that the GPU holds.
static int gp_clusters(int device, int ctas) {
  static PerDevice held[GP_CLUSTER + 1];
  return held[ctas].get(device, [=] {
    const auto kern = &k_gated_proj<__nv_bfloat16, GP_BACK, false, 1>;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)ctas, at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas), cfg.blockDim = dim3(GP_THREADS), cfg.dynamicSmemBytes = GP_SHARED, cfg.attrs = &at, cfg.numAttrs = 1;
    int n = 0;
    if (grant_shared(kern, GP_SHARED) && cudaOccupancyMaxActiveClusters(&n, kern, &cfg) == cudaSuccess) return n;
    (void)cudaGetLastError();
    return 0;
  });
}
static GpPlan plan_here(int64_t rows, int64_t cols, int64_t summed, bool back, bool fine) {
  const int device = current_device();
  return gp_plan(rows, cols, summed, back, fine, [=](int ctas) { return gp_clusters(device, ctas); });
}
static int64_t gp_ld(int64_t cols) { return (cols + 7) / 8 * 8; }

// Workspace: the diagnostic words, the aligned copies, the sums of the splits that go
// through it (whose tiles all fit the SMs: 20 MB at most).
struct GpSpace {
  size_t rows, weights[2], sums, bytes;
};
static int64_t gp_lds(int64_t cols) { return (cols + 7) / 8 * 8; }
static GpSpace gp_space(int64_t rows, int64_t n, int64_t k, uint32_t copied, bool back) {
  GpSpace w = {};
  size_t at = DIAG_BYTES;
  const auto room = [&](int64_t r, int64_t c) {
    const size_t here = at;
    at += align_up((size_t)r * gp_ld(c) * 2, 256);
    return here;
  };
  if (copied & GC_COPY_WEIGHTS) w.weights[0] = room(n, k), w.weights[1] = room(n, k);
  if (copied & GC_COPY_ROWS) {
    w.rows = room(back ? 2 * rows : rows, back ? n : k);
  }
  w.sums = at;
  if (back) {
    const double sums = (double)GP_SMS * (double)rows * (double)gp_lds(k) * 4.0;
    constexpr double MOST = (double)GP_SMS * GP_M * 256 * 4;
    at += align_up((size_t)(sums < MOST ? sums : MOST), 256);
  }
  w.bytes = at;
  return w;
}
static int put_width(const void* p, int64_t ld) {
  return !(aligned16(p) && ld % 8 == 0) ? 0 : ((uintptr_t)p & 31u) == 0u && ld % 16 == 0 ? 2 : 1;
}
static bool bulk_rows(const void* p, int64_t ld) { return aligned16(p) && ld % 8 == 0; }

// Adds a matrix to those that are copied, and takes its copy in its place.
static void add_copy(GpAlign* l, const void** x, int64_t* ld, int64_t rows, int64_t cols, unsigned char* to) {
  l->from[l->count] = *x, l->to[l->count] = to, l->ld[l->count] = *ld, l->rows[l->count] = rows, ++l->count;
  *x = to, *ld = gp_ld(cols);
}
static void align_rows(GpAlign& l, int64_t cols, cudaStream_t s) {
  if (l.count == 0) return;
  const int64_t chunks = gp_ld(cols) / CHUNK;
  for (int i = 0; i < 3; ++i) {
    const int64_t blocks = i < l.count ? ceil_div(l.rows[i] * chunks, 2 * 256) : 0;
    l.first[i + 1] = l.first[i] + (unsigned)(blocks < GP_SMS * 16 ? blocks : GP_SMS * 16);
  }
  launch_chained(k_align_rows, l.first[3], 256, 0, s, l, cols, (uint32_t)chunks);
}

template <typename T, int KIND, int R>
static void launch_rows(const void* x, int64_t ldx, int64_t rows, const void* wg, int64_t ldwg, const void* wu, int64_t ldwu, int64_t n,
                        int64_t k, void* out, int64_t ldo, bool span, uint32_t* diag, cudaStream_t s) {
  const int64_t groups = ceil_div(rows, R);
  int split = 0;  // warps that share a row's sum, as a power of 2: while no more than two CTAs an SM come of it
  while (split < 3 && groups * ceil_div(n, 8 >> split) <= GP_SMS * 2 && (256 << split) < k) ++split;
  const auto kern = split ? (span ? &k_gated_proj_row<T, KIND, true, R, true> : &k_gated_proj_row<T, KIND, false, R, true>)
                          : (span ? &k_gated_proj_row<T, KIND, true, R, false> : &k_gated_proj_row<T, KIND, false, R, false>);
  launch_chained(kern, (unsigned)(groups * ceil_div(n, 16 >> split)), 256, 0, s, static_cast<const T*>(x), ldx, static_cast<const T*>(wg), ldwg,
                 static_cast<const T*>(wu), ldwu, n, k, static_cast<T*>(out), ldo, (int)rows, split, diag);
}
template <typename T, int KIND>
static void launch_row(const void* x, int64_t ldx, int64_t rows, const void* wg, int64_t ldwg, const void* wu, int64_t ldwu, int64_t n,
                       int64_t k, void* out, int64_t ldo, bool span, uint32_t* diag, cudaStream_t s) {
  const auto launch = rows > 1 ? &launch_rows<T, KIND, 2> : &launch_rows<T, KIND, 1>;
  launch(x, ldx, rows, wg, ldwg, wu, ldwu, n, k, out, ldo, span, diag, s);
}

template <typename T, int KIND, bool PAIR, int PARTS>
static bool launch_gp(const GpMaps& maps, const GpArgs& a, cudaStream_t s) {
  auto kern = k_gated_proj<T, KIND, PAIR, PARTS>;
  static PerDevice ready;
  if (!ready.get(current_device(), [=] { return grant_shared(kern, GP_SHARED) ? 1 : 0; })) return false;
  constexpr int WORKERS = PAIR ? GP_SMS / 2 : GP_SMS;
  const bool joint = a.splits > 1 && !a.sums;
  if (joint && !gp_fits((a.bn + 31) / 32, a.splits, KIND == GP_BACK)) return false;
  const unsigned workers = (unsigned)(joint || a.items < WORKERS ? a.items : WORKERS);
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)((PAIR ? 2 : 1) * (joint ? a.splits : 1)), at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((PAIR ? 2 : 1) * workers), cfg.blockDim = dim3(GP_THREADS), cfg.dynamicSmemBytes = GP_SHARED, cfg.stream = s;
  cfg.attrs = at, cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, kern, maps, a) == cudaSuccess) return true;
  (void)cudaGetLastError();
  cfg.numAttrs = 1;  // not as a dependent launch, then
  if (cudaLaunchKernelEx(&cfg, kern, maps, a) == cudaSuccess) return true;
  (void)cudaGetLastError();  // this call's, not the next one's
  return false;
}
template <typename T, int KIND>
static bool launch_gp(const GpMaps& maps, const GpArgs& a, const GpPlan& p, cudaStream_t s) {
  if (p.parts == 2) return p.pair ? launch_gp<T, KIND, true, 2>(maps, a, s) : launch_gp<T, KIND, false, 2>(maps, a, s);
  return p.pair ? launch_gp<T, KIND, true, 1>(maps, a, s) : launch_gp<T, KIND, false, 1>(maps, a, s);
}
// Rows of the copies of x, dgate and dup: no more than there are (copies of rows
// that are not there cost as much as others).
static int gp_box(int64_t rows) { return rows < GP_M ? (int)rows : GP_M; }
static void set_plan(GpArgs* a, const GpPlan& p, int64_t summed, bool back) {
  a->bn = p.bn, a->tiles_m = p.tiles_m, a->tiles_n = p.tiles_n, a->splits = p.splits, a->span = p.span;
  a->items = p.tiles_m * p.tiles_n * p.splits;
  // Tiles of a band of rows, which are computed column by column: 8192 x 14336 x 4096 takes
  // 1119 us in bands of 8, 1091 of 16 and 1170 of 32 (with checkpoints), its gradient
  // 1093, 1107 and 1155 (the rows that a band keeps in L2 are seven times as long there).
  a->band = back ? 8 : 16;
  const int blocks = (int)ceil_div(summed, GP_K), stages = (blocks + p.parts - 1) / p.parts, columns = gp_columns(p.bn, p.pair, back);
  a->half = stages, a->steps = back ? 2 * stages : stages;
  a->last = blocks - (stages - 1) * p.parts;
  a->bytes = gp_box(a->rows) * GP_K * 2 + columns;
  a->room = gp_room(a->rows), a->part = a->room + columns;
  a->slots = GP_RING / (p.parts * a->part) < GP_SLOTS ? GP_RING / (p.parts * a->part) : GP_SLOTS;
}
static gc_status check_sizes(int64_t rows, int64_t n, int64_t k) {
  gc_status st = validate_matrix(rows, n, GC_BF16);
  if (st == GC_OK) st = validate_matrix(rows, k, GC_BF16);
  // tiles are counted in 32 bits
  return st != GC_OK ? st : ceil_div(rows, GP_M) * ceil_div(n > k ? n : k, 32) > INT64_C(1073741823) ? GC_ERR_LAYOUT : GC_OK;
}
static bool valid_kind(int32_t kind) { return kind == GC_GATE_SILU || kind == GC_GATE_GELU_TANH; }

}  // namespace gc

using namespace gc;

extern "C" gc_status gc_gated_proj_workspace_size(int64_t rows, int64_t n, int64_t k, uint32_t copied, size_t* bytes) {
  const gc_status st = check_sizes(rows, n, k);
  if (st != GC_OK) return st;
  if (!bytes || (copied & ~(GC_COPY_ROWS | GC_COPY_WEIGHTS))) return GC_ERR_INVALID_ARG;
  *bytes = gp_space(rows, n, k, copied, false).bytes;
  return GC_OK;
}
extern "C" gc_status gc_gated_proj_backward_workspace_size(int64_t rows, int64_t n, int64_t k, uint32_t copied, size_t* bytes) {
  const gc_status st = check_sizes(rows, n, k);
  if (st != GC_OK) return st;
  if (!bytes || (copied & ~(GC_COPY_ROWS | GC_COPY_WEIGHTS))) return GC_ERR_INVALID_ARG;
  *bytes = gp_space(rows, n, k, copied, true).bytes;
  return GC_OK;
}

extern "C" gc_status gc_gated_proj(int32_t kind, const void* x, int64_t ldx, const void* w_gate, int64_t ldwg,
                                   const void* w_up, int64_t ldwu, int32_t dtype, int64_t rows, int64_t n, int64_t k,
                                   void* out, int64_t ldo, int8_t* gate_codes, uint8_t* gate_steps, int8_t* up_codes,
                                   uint8_t* up_steps, void* workspace, size_t ws_bytes, void* stream) {
  NvtxRange nvtx_range("gc_gated_proj");
  gc_status st = check_sizes(rows, n, k);
  if (st != GC_OK) return st;
  if (!valid_kind(kind) || !(dtype == GC_BF16 || dtype == GC_F16)) return GC_ERR_INVALID_ARG;
  if (rows > 0) {
    if ((st = check_matrix(x, ldx, k, dtype)) != GC_OK || (st = check_matrix(w_gate, ldwg, k, dtype)) != GC_OK ||
        (st = check_matrix(w_up, ldwu, k, dtype)) != GC_OK || (st = check_matrix(out, ldo, n, dtype)) != GC_OK)
      return st;
    if (gate_codes || gate_steps || up_codes || up_steps)
      if ((st = check_codes(gate_codes, gate_steps)) != GC_OK || (st = check_codes(up_codes, up_steps)) != GC_OK) return st;
  }
  const uint32_t copied = rows == 0 ? 0u
                                    : (bulk_rows(x, ldx) ? 0u : GC_COPY_ROWS) |
                                          (bulk_rows(w_gate, ldwg) && bulk_rows(w_up, ldwu) ? 0u : GC_COPY_WEIGHTS);
  const GpSpace w = gp_space(rows, n, k, copied, false);
  if ((st = check_workspace(workspace, ws_bytes, w.bytes)) != GC_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  unsigned char* const ws = static_cast<unsigned char*>(workspace);
  if (rows == 0) return zero_chained(ws, DIAG_BYTES, s) ? GC_OK : GC_ERR_CUDA;
  const bool silu = kind == GC_GATE_SILU;
  if (!gate_codes && gp_few(rows, n, k)) {
    const auto launch = dtype == GC_BF16 ? (silu ? &launch_row<__nv_bfloat16, GC_GATE_SILU> : &launch_row<__nv_bfloat16, GC_GATE_GELU_TANH>)
                                         : (silu ? &launch_row<__half, GC_GATE_SILU> : &launch_row<__half, GC_GATE_GELU_TANH>);
    launch(x, ldx, rows, w_gate, ldwg, w_up, ldwu, n, k, out, ldo, copied != 0, reinterpret_cast<uint32_t*>(ws), s);
    return cudaGetLastError() == cudaSuccess ? GC_OK : GC_ERR_CUDA;
  }
  GpAlign copies = {};
  if (copied & GC_COPY_ROWS) add_copy(&copies, &x, &ldx, rows, k, ws + w.rows);
  if (!bulk_rows(w_gate, ldwg)) add_copy(&copies, &w_gate, &ldwg, n, k, ws + w.weights[0]);
  if (!bulk_rows(w_up, ldwu)) add_copy(&copies, &w_up, &ldwu, n, k, ws + w.weights[1]);
  align_rows(copies, k, s);
  GpArgs a = {};
  a.rows = rows, a.cols = n;
  const GpPlan p = plan_here(rows, n, k, false, !gate_codes);
  set_plan(&a, p, k, false);
  a.out = out, a.ldo = ldo, a.vec = put_width(out, ldo);
  a.gcodes = gate_codes, a.ucodes = up_codes, a.gsteps = gate_steps, a.usteps = up_steps;
  a.whole = (((uintptr_t)gate_codes | (uintptr_t)up_codes) & 31u) == 0u;
  a.even = (((uintptr_t)gate_steps | (uintptr_t)up_steps | (uintptr_t)(act_ldc(n) >> 5)) & 1u) == 0u;
  a.diag = reinterpret_cast<uint32_t*>(ws);
  GpMaps maps;
  if (!make_map(&maps.a0, dtype, x, ldx, rows, k, gp_box(rows)) || !make_map(&maps.b0, dtype, w_gate, ldwg, n, k, a.bn) ||
      !make_map(&maps.b1, dtype, w_up, ldwu, n, k, a.bn))
    return GC_ERR_CUDA;
  maps.a1 = maps.a0;
  const bool ok = dtype == GC_BF16 ? (silu ? launch_gp<__nv_bfloat16, GC_GATE_SILU>(maps, a, p, s)
                                           : launch_gp<__nv_bfloat16, GC_GATE_GELU_TANH>(maps, a, p, s))
                                   : (silu ? launch_gp<__half, GC_GATE_SILU>(maps, a, p, s)
                                           : launch_gp<__half, GC_GATE_GELU_TANH>(maps, a, p, s));
  return ok && cudaGetLastError() == cudaSuccess ? GC_OK : GC_ERR_CUDA;
}

extern "C" gc_status gc_gated_proj_backward(int32_t kind, const void* dout, int64_t lddo, int32_t dtype,
                                            const int8_t* gate_codes, const uint8_t* gate_steps, const int8_t* up_codes,
                                            const uint8_t* up_steps, const void* w_gate, int64_t ldwg, const void* w_up,
                                            int64_t ldwu, int64_t rows, int64_t n, int64_t k, void* dgate, int64_t lddg,
                                            void* dup, int64_t lddu, void* dx, int64_t lddx, int8_t* out_codes,
                                            uint8_t* out_steps, void* workspace, size_t ws_bytes, void* stream) {
  NvtxRange nvtx_range("gc_gated_proj_backward");
  gc_status st = check_sizes(rows, n, k);
  if (st != GC_OK) return st;
  if (!valid_kind(kind) || !(dtype == GC_BF16 || dtype == GC_F16)) return GC_ERR_INVALID_ARG;
  if (rows > 0 &&
      ((st = check_matrix(w_gate, ldwg, k, dtype)) != GC_OK || (st = check_matrix(w_up, ldwu, k, dtype)) != GC_OK ||
       (st = check_matrix(dgate, lddg, n, dtype)) != GC_OK || (st = check_matrix(dup, lddu, n, dtype)) != GC_OK ||
       (st = check_matrix(dx, lddx, k, dtype)) != GC_OK))
    return st;
  const uint32_t copied = rows == 0 ? 0u
                                    : (bulk_rows(dgate, lddg) && bulk_rows(dup, lddu) ? 0u : GC_COPY_ROWS) |
                                          (bulk_rows(w_gate, ldwg) && bulk_rows(w_up, ldwu) ? 0u : GC_COPY_WEIGHTS);
  const GpSpace w = gp_space(rows, n, k, copied, true);
  if ((st = check_workspace(workspace, ws_bytes, w.bytes)) != GC_OK) return st;
  // checks the rest before anything is enqueued
  unsigned char* const ws = static_cast<unsigned char*>(workspace);
  unsigned char* const copies = (copied & GC_COPY_ROWS) ? ws + w.rows : nullptr;  // of dgate and dup
  st = gated_act_backward(kind, dout, lddo, dtype, gate_codes, gate_steps, up_codes, up_steps, rows, n, dgate, lddg, dup, lddu,
                          out_codes, out_steps, copies, stream);
  if (st != GC_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (rows == 0) return zero_chained(ws, DIAG_BYTES, s) ? GC_OK : GC_ERR_CUDA;
  const void *dg = dgate, *du = dup;
  if (copies) lddg = lddu = gp_ld(n), dg = copies, du = copies + (size_t)rows * lddg * 2;
  GpAlign weights = {};
  if (!bulk_rows(w_gate, ldwg)) add_copy(&weights, &w_gate, &ldwg, n, k, ws + w.weights[0]);
  if (!bulk_rows(w_up, ldwu)) add_copy(&weights, &w_up, &ldwu, n, k, ws + w.weights[1]);
  align_rows(weights, k, s);
  GpArgs a = {};
  a.rows = rows, a.cols = k;
  const GpPlan p = plan_here(rows, k, n, true, false);
  set_plan(&a, p, n, true);
  a.out = dx, a.ldo = lddx, a.vec = put_width(dx, lddx);
  if (p.apart) a.sums = reinterpret_cast<float*>(ws + w.sums), a.lds = gp_lds(k);
  a.diag = reinterpret_cast<uint32_t*>(ws);
  GpMaps maps;
  if (!make_map(&maps.a0, dtype, dg, lddg, rows, n, gp_box(rows)) || !make_map(&maps.a1, dtype, du, lddu, rows, n, gp_box(rows)) ||
      !make_map(&maps.b0, dtype, w_gate, ldwg, n, k, GP_K) || !make_map(&maps.b1, dtype, w_up, ldwu, n, k, GP_K))
    return GC_ERR_CUDA;
  if (!(dtype == GC_BF16 ? launch_gp<__nv_bfloat16, GP_BACK>(maps, a, p, s) : launch_gp<__half, GP_BACK>(maps, a, p, s)))
    return GC_ERR_CUDA;
  if (p.apart) {
    const dim3 grid((unsigned)ceil_div(k, 256), (unsigned)rows);  // at most 128 of each SM
    if (dtype == GC_BF16)
      launch_chained(&k_gated_proj_join<__nv_bfloat16>, grid, 256, 0, s, a.sums, p.splits, rows, (int)k, a.lds,
                     static_cast<__nv_bfloat16*>(dx), lddx);
    else
      launch_chained(&k_gated_proj_join<__half>, grid, 256, 0, s, a.sums, p.splits, rows, (int)k, a.lds, static_cast<__half*>(dx), lddx);
  }
  return cudaGetLastError() == cudaSuccess ? GC_OK : GC_ERR_CUDA;
}
