// Weight gradient from an activation checkpoint on the fifth-generation
// tensor cores: dw[n, k] = sum_t dy[t, n] * q[t, k], q = code * step.
#include <cmath>

#include "gc_act.cuh"
#include "gc_host.h"
#include "gc_mma.cuh"

namespace gc {

// Mathematics and precision.  q's code has 7 bits and its step is a power of
// two, so q is exact in bf16; a bf16 dy is too, an fp16 dy is the exact sum
// of two bf16 terms (11 bits = 8 + 3) and an fp32 dy of three (24 = 8 + 8 +
// 8, for numbers above 2^-109).  Every product is therefore exact and only the
// fp32 sums round.  The terms, and a bf16 dy whose rows cannot be copied in bulk, are written to the
// workspace first: 8192 x 1024 x 1024 in fp16 takes 40 us so, and took 52 with
// dy split beside the MMAs by the unpacking warps.
//
// Tile.  A CTA computes 256 (n) x 256 (k) of dw: two accumulators of 128 x
// 256 fp32, all 512 columns of the SM's tensor memory.  q has to be unpacked
// from codes by ordinary instructions, and the unpacked tile serves both
// accumulators: 16 codes per clock at the tensor cores' full rate.  Shared
// memory bounds the loop: per 64 t the MMAs read 96 KB and the copies of dy
// and the unpacked q write 32 KB each, 1280 clocks at 128 bytes each, where
// the MMAs alone would take 1024.  With several terms of dy the tile is 128 x
// 256: the leading terms go into one accumulator, the others, 2^-8 of their
// size, into the second, where the truncation below costs them nothing.
//
// Chains.  The tensor cores truncate what they add to an accumulator, a bias
// towards zero that grows with the number of additions: 8192 rows in one
// chain end with a relative error of 3.0e-6, 2048 rows with 4.8e-7 (fp32
// additions that round: 5e-7).  An accumulator is therefore added to the
// result, in fp32 that rounds, after at most WG_CHAIN rows, by warps of their
// own.  The two accumulators' chains end half a chain apart, so that the
// other one's MMAs go on with the stages at hand meanwhile; and CTAs end them
// at different times, so that they do not all write at once.
//
// Measured: 16384 x 14336 x 4096 in bf16 1.36 ms, 1415 TFLOP/s, back to back under
// the power cap (a call on its own 1.22 ms, one chain 1.12 ms); 8192 x 4864 x 2048 110 us, where a
// library's product of two bf16 matrices takes 92; 8192 x 1024 x 1024 25 us, in
// fp16 40 us.
//
// Both operands have the summed index t as their slow dimension in memory,
// so both are staged "MN-major": 128-byte rows of 64 consecutive n (or k) of
// one t, 16-byte chunk c of row t at chunk c ^ (t & 7) (the 128-byte
// swizzle), 64-wide column blocks one after another.
constexpr int WG_N = 256;                  // k of a CTA's tile
// The unpacking warps work in teams, each on every WG_TEAMS-th stage: a team
// has as many stages' time for its own, so the latency of its loads of codes
// is hidden without keeping several stages' codes in registers.
constexpr int WG_TEAMS = 2, WG_TEAM = 4;   // teams, warps of a team
constexpr int WG_CONV = WG_TEAMS * WG_TEAM;
constexpr int WG_OUT = 8;                  // warps that write the result
constexpr int WG_TMA = WG_CONV + WG_OUT, WG_MMA = WG_TMA + 1;  // the warps that issue loads of dy, MMAs
constexpr int WG_THREADS = (WG_CONV + WG_OUT + 4) * 32;        // two warps idle: registers go by groups of four
constexpr int WG_REGS = 96;                // registers per thread at launch
constexpr int WG_RING = 192 * 1024;        // shared memory of the stages
constexpr int WG_SMEM = WG_RING + WG_OUT * 4096;  // + a 32 x 32 tile of the result per writing warp
constexpr int WG_CHAIN = 3200;             // rows of a chain

// A bulk copy or reduction ends on a 16-byte boundary of a row, not at its last
// element: it takes rows of the result that start on one, and the tile that a row
// ends in only where it ends on one too, or where what follows is not the caller's.
constexpr int WG_NONE = 0, WG_WHOLE = 1, WG_ALL = 2;

struct WgArgs {
  const __nv_bfloat16* dy;      // the terms, one [rows, lddy] after another
  int64_t lddy, rows, n, k, ldc;
  const int8_t* codes;
  const uint8_t* steps;
  const void* cscale;           // of the result; NULL where it is a split's sums
  int ctype, accumulate;
  int bulk;                     // tiles of the result that are written in bulk: WG_NONE, WG_WHOLE, WG_ALL
  float* out;                   // dw, or the splits' sums one [n, ldo] after another
  int64_t ldo;
  int splits, tiles_n, items;   // tiles along k; tiles * splits
  int64_t span;                 // rows of a split, a multiple of 64
  uint32_t* diag;
};

constexpr int WG_POLLS = 1 << 22;  // limit of every wait
// Waits for a phase, a bounded number of polls: a thread of its own, or all lanes of
// a warp, which go on or give up together (lanes that gave up by themselves
// would leave the others waiting for them at the next vote).
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity) {
  for (int i = 0; i < WG_POLLS; ++i)
    if (mbar_poll(bar, parity)) return true;
  return false;
}
__device__ __forceinline__ bool mbar_wait_warp(uint32_t bar, uint32_t parity) {
  for (int i = 0; i < WG_POLLS; ++i)
    if (__all_sync(FULL, mbar_poll(bar, parity))) return true;
  return false;
}
// A 32 x 32 tile of the result, 128-byte rows under the 128-byte swizzle, to
// global memory: stored, or added to it.  Whoever issued it may then wait
// until its source may be written again, or until it is complete.
__device__ __forceinline__ void tma_put(const CUtensorMap* map, int x, int y, int z, uint32_t src, bool add) {
  if (add)
    asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map),
                 "r"(x), "r"(y), "r"(z), "r"(src)
                 : "memory");
  else
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map), "r"(x),
                 "r"(y), "r"(z), "r"(src)
                 : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void tma_put_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void tma_put_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// One float of the result: stored, or added to what is there, which nobody
// else changes meanwhile, without waiting for it.
__device__ __forceinline__ void put1(float* o, float v, bool add) {
  if (add)
    asm volatile("red.relaxed.gpu.global.add.f32 [%0], %1;" ::"l"(o), "f"(v) : "memory");
  else
    *o = v;
}

// Adds 16 consecutive columns of the 32 lanes of tensor memory at `addr` to v.
__device__ __forceinline__ void tmem_add16(float* v, uint32_t addr) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];\ntcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __fadd_rn(v[i], __uint_as_float(r[i]));
}

// The codes in bytes 0 and 2 of w (the low byte of each half) as bf16 times
// their step.  With s a code's sign bit and l its low 7 bits, code = l - 128 s
// = (128 + l) - 128 (1 + s); as bf16 0x4300 | l is 128 + l and 0x4300 | 128 s
// is 128 (1 + s).  `lead` is 0x4300 with the step added to its exponent,
// `minus` the step negated, so one fused multiply-add gives the value, exactly.
__device__ __forceinline__ uint32_t codes_bf16(uint32_t w, uint32_t lead, uint32_t minus) {
  const uint32_t lo = (w & 0x007F007Fu) | lead, hi = (w & 0x00800080u) | 0x43004300u;
  uint32_t v;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(v) : "r"(hi), "r"(minus), "r"(lo));
  return v;
}
// Two codes by way of fp32, for the steps whose lead would leave bf16's
// exponents (0, 248 and 255, the step of a group that is not finite).
__device__ __forceinline__ uint32_t codes_bf16_any(uint32_t w, uint32_t step) {
  const float sc = act_scale(step);
  const float a = __fmul_rn((float)(int8_t)(w & 255u), sc), b = __fmul_rn((float)(int8_t)((w >> 16) & 255u), sc);
  return (__float_as_uint(a) >> 16) | (__float_as_uint(b) & 0xFFFF0000u);
}
// The bytes of a word come out in the order 0, 2, 1, 3, so accumulator columns
// 4 q + 1 and 4 q + 2 hold columns 4 q + 2 and 4 q + 1; the result undoes it.

// 8 elements of dy from column c on; 0 outside [0, n).  The row may start
// anywhere: the 16-byte granules that hold an element of the 8 are read as
// they lie, and the elements shifted out of them.
__device__ __forceinline__ Raw8<__nv_bfloat16> load8(const __nv_bfloat16* row, int64_t c, int64_t n) {
  const int in = (int)max((int64_t)0, min((int64_t)CHUNK, n - c));
  const int skip = (int)((uintptr_t)(row + c) & 15u), total = in > 0 ? skip + 2 * in : 0;
  const uint4* from = reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(row + c) - skip);
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint4 x = 16 * i < total ? __ldg(from + i) : make_uint4(0u, 0u, 0u, 0u);
    w[4 * i] = x.x, w[4 * i + 1] = x.y, w[4 * i + 2] = x.z, w[4 * i + 3] = x.w;
  }
  shift_words<4>(w, skip);
  Raw8<__nv_bfloat16> v;
#pragma unroll
  for (int i = 0; i < 4; ++i) reinterpret_cast<uint32_t*>(&v)[i] = w[i];
  if (in < CHUNK) {
#pragma unroll
    for (int i = 0; i < CHUNK; ++i)
      if (i >= in) v.e[i] = from_f32<__nv_bfloat16>(0.0f);
  }
  return v;
}

// TMA: the terms of dy come by bulk tensor copies; else a bf16 dy whose rows
// do not start on 16-byte boundaries, by the unpacking warps' own loads.
template <int PARTS, bool TMA>
struct WgShape {
  static constexpr int M = PARTS == 1 ? 256 : 128;      // n of a tile
  static constexpr int KT = TMA ? 64 : 32;              // t of a stage
  static constexpr int BLOCK = KT * 128;                // bytes of a 64-wide column block
  static constexpr int A_BYTES = M / 64 * BLOCK, B_BYTES = WG_N / 64 * BLOCK, STAGE = PARTS * A_BYTES + B_BYTES;
  static constexpr int STAGES = WG_RING / STAGE < 6 ? WG_RING / STAGE : 6;
  static constexpr int CHAIN = WG_CHAIN / KT;           // stages of a chain
  // Registers per thread as the roles share out those of the launch, so that
  // none keeps its variables in memory (without TMA 24 bytes are): unpacking,
  // writing, the rest.
  static constexpr int REGS_CONV = TMA ? 80 : 96, REGS_OUT = TMA ? 120 : 112, REGS_REST = TMA ? 80 : 64;
  static_assert(WG_CONV * REGS_CONV + WG_OUT * REGS_OUT + 4 * REGS_REST <= WG_THREADS / 32 * WG_REGS, "registers");
};

// A tile and a split of the rows.
struct WgItem {
  int split, iters, halves;  // iters: stages; halves: accumulators with rows of their own
  int64_t n0, k0, t0, t1;
};
template <typename S>
__device__ __forceinline__ WgItem wg_item(const WgArgs& a, int i) {
  WgItem m;
  m.split = i % a.splits;
  const int tile = i / a.splits;
  m.n0 = (int64_t)(tile / a.tiles_n) * S::M, m.k0 = (int64_t)(tile % a.tiles_n) * WG_N;
  m.t0 = m.split * a.span, m.t1 = min(m.t0 + a.span, a.rows);
  m.iters = (int)((m.t1 - m.t0 + S::KT - 1) / S::KT);
  m.halves = S::M == 256 && m.n0 + 128 < a.n ? 2 : 1;
  return m;
}
// Where the chain of accumulator h that is at stage `pos` ends.
template <typename S>
__device__ __forceinline__ int wg_chain_end(int iters, int h, int pos) {
  if (iters <= S::CHAIN) return iters;
  const int off = (int)(blockIdx.x % 8u) * (S::CHAIN / 16) + h * (S::CHAIN / 2);
  return min(iters, pos + S::CHAIN - (pos + off) % S::CHAIN);
}

// The role of the writing warps.  A warp reads the 32 lanes of tensor
// memory that its number gives, and 128 of their columns in four tiles of 32.
// What it may write out at once goes at the rate of the SM's writes, 4000
// clocks for an accumulator; the accumulator is given back as soon as its
// last tile is in registers, with one tile written and one on its way.
template <typename S>
__device__ __forceinline__ bool wg_write(const WgArgs& a, const CUtensorMap* map, uint32_t tiles, uint32_t full, uint32_t empty,
                                      uint32_t tmem) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, quad = warp & 3, side = (warp - WG_CONV) >> 2;
  const uint32_t tile = tiles + (uint32_t)(side * 4 + quad) * 4096u;
  const uint32_t columns = tmem + ((uint32_t)(32 * quad) << 16) + (uint32_t)side * (WG_N / 2);
  bool ok = true;
  uint32_t used0 = 0u, used1 = 0u;
  for (int i = blockIdx.x; ok && i < a.items; i += gridDim.x) {
    const WgItem m = wg_item<S>(a, i);
    int pos0 = 0, pos1 = m.halves == 2 ? 0 : m.iters;
    while (ok && (pos0 < m.iters || pos1 < m.iters)) {
      // the chains in the order of their ends
      const int end0 = pos0 < m.iters ? wg_chain_end<S>(m.iters, 0, pos0) : m.iters + 1;
      const int end1 = pos1 < m.iters ? wg_chain_end<S>(m.iters, 1, pos1) : m.iters + 1;
      const int h = end1 < end0 ? 1 : 0;
      const bool later = (h ? pos1 : pos0) > 0, add = later || a.accumulate;
      ok = mbar_wait_warp(full + 8u * h, (h ? used1 : used0) & 1);
      if (!ok) break;
      if (h)
        ++used1, pos1 = end1;
      else
        ++used0, pos0 = end0;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const int64_t r0 = m.n0 + 128 * h + 32 * quad, k0 = m.k0 + side * (WG_N / 2);
      const int rows = (int)max((int64_t)0, min((int64_t)32, a.n - r0));
      float v[64];
      auto fetch = [&](int c, float* x) {  // tile c
        __syncwarp();
        tmem_load32(x, columns + 256u * h + 32u * c);
        if (S::M == 128) {
          tmem_add16(x, columns + 256u + 32u * c);
          tmem_add16(x + 16, columns + 256u + 32u * c + 16u);
        }
      };
      auto put = [&](int c, float* x) {
        const int64_t c0 = k0 + 32 * c;
        if (rows == 0 || c0 >= a.k) return;  // uniform in the warp
        const bool bulk = a.bulk == WG_ALL || (a.bulk == WG_WHOLE && c0 + 32 <= a.k);
        if (a.bulk && lane == 0) tma_put_read();
        if (a.cscale) {
          const float cs = c0 + lane < a.k ? load_as_f32(a.cscale, a.ctype, c0 + lane) : 0.0f;
#pragma unroll
          for (int q = 0; q < 32; ++q)
            x[q] = __fmul_rn(x[q], __shfl_sync(FULL, cs, (q & ~3) | ((q & 1) << 1) | ((q >> 1) & 1)));
        }
        __syncwarp();
#pragma unroll
        for (int q = 0; q < 8; ++q)
          st_shared16(tile + (uint32_t)lane * 128u + (uint32_t)((q ^ (lane & 7)) << 4), __float_as_uint(x[4 * q]),
                      __float_as_uint(x[4 * q + 2]), __float_as_uint(x[4 * q + 1]), __float_as_uint(x[4 * q + 3]));
        if (bulk) {
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) tma_put(map, (int)c0, (int)r0, m.split, tile, add);
        } else {
          __syncwarp();
          if (c0 + lane < a.k) {
            float* o = a.out + ((int64_t)m.split * a.n + r0) * a.ldo + c0 + lane;
#pragma unroll 4
            for (int r = 0; r < rows; ++r, o += a.ldo) {
              float y;
              asm volatile("ld.shared.f32 %0, [%1];"
                           : "=f"(y)
                           : "r"(tile + (uint32_t)r * 128u + (uint32_t)(((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4u)
                           : "memory");
              put1(o, y, add);
            }
          }
        }
      };
      if (a.bulk && later && lane == 0) tma_put_done();  // the chain before is in the result
      fetch(0, v);
      put(0, v);
      fetch(1, v);
      if (S::M == 256) fetch(2, v + 32);
      put(1, v);
      if (S::M == 128) {
        fetch(2, v + 32);
        put(2, v + 32);
      }
      fetch(3, v);
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(empty + 8u * h);
      if (S::M == 256) put(2, v + 32);
      put(3, v);
    }
  }
  if (lane == 0) tma_put_done();
  return ok;
}

// A CTA takes every gridDim.x-th item (a tile and a split of the rows); all
// roles walk the same items, and `g` counts the stages.  !TMA is reached by a
// bf16 dy off 16-byte boundaries whose n is a multiple of 8, for which no
// workspace is set aside.
template <int PARTS, bool TMA>
__global__ void __launch_bounds__(WG_THREADS, 1)
    k_weight_grad(const __grid_constant__ CUtensorMap dy_map, const __grid_constant__ CUtensorMap out_map,
                  const __grid_constant__ WgArgs a) {
  using S = WgShape<PARTS, TMA>;
  constexpr int KT = S::KT, BLOCK = S::BLOCK, A_BYTES = S::A_BYTES, STAGES = S::STAGES, CHAIN = S::CHAIN;
  constexpr int ROWS = KT / WG_TEAM;                    // t per unpacking warp and stage
  extern __shared__ __align__(1024) unsigned char smem[];
  __shared__ __align__(8) uint64_t bars[3 * 8 + 5];
  __shared__ uint32_t tmem_base;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t base = smem_u32(smem), bar0 = smem_u32(bars);
  auto full_a = [&](int s) { return bar0 + 8u * s; };
  auto full_b = [&](int s) { return bar0 + 64u + 8u * s; };
  auto empty = [&](int s) { return bar0 + 128u + 8u * s; };
  auto acc_full = [&](int h) { return bar0 + 192u + 8u * h; };   // a chain's MMAs are done
  auto acc_empty = [&](int h) { return bar0 + 208u + 8u * h; };  // its sums have been read out
  const uint32_t drained = bar0 + 224u;                          // all MMAs are done, after a wait that ran out

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) mbar_init(full_a(s), 1), mbar_init(full_b(s), WG_TEAM), mbar_init(empty(s), 1);
    for (int h = 0; h < 2; ++h) mbar_init(acc_full(h), 1), mbar_init(acc_empty(h), WG_OUT);
    mbar_init(drained, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == WG_MMA) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&tmem_base)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = tmem_base;
  chain_wait();
  if (blockIdx.x == 0 && threadIdx.x <= DIAG_PATH) a.diag[threadIdx.x] = 0u;  // all that the status call reads

  auto item_at = [&](int i) { return wg_item<S>(a, i); };
  bool ok = true;
  int g = 0;

  if (warp < WG_CONV) {
    // ------------------------------------------------ unpack q
    if (S::REGS_CONV < WG_REGS) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::REGS_CONV));
    // Lanes past q's last column read the last columns again: what they put
    // into the tile reaches only columns of the accumulators that are not
    // written out.
    const int team = warp / WG_TEAM, w = warp % WG_TEAM;  // rows w, w + 4, ... of q
    const int64_t groups = a.ldc >> 5;
    const uint32_t off0 = PARTS * A_BYTES + (uint32_t)(lane >> 3) * BLOCK + (uint32_t)w * 128u + (uint32_t)(((lane & 7) ^ w) << 4);
    const uint32_t off1 =
        PARTS * A_BYTES + (uint32_t)(lane >> 3) * BLOCK + (uint32_t)w * 128u + 512u + (uint32_t)(((lane & 7) ^ (w + 4)) << 4);
    for (int i0 = blockIdx.x; ok && i0 < a.items; i0 += gridDim.x) {
      const WgItem m = item_at(i0);
      const int64_t kc = min(m.k0 + 8 * lane, a.ldc - 8), span = m.t1 - m.t0;
      int it = (team + WG_TEAMS - g % WG_TEAMS) % WG_TEAMS;  // this team's first stage of the item
      const int8_t* cp = a.codes + (m.t0 + (int64_t)it * KT + w) * a.ldc + kc;
      const uint8_t* sp = a.steps + (m.t0 + (int64_t)it * KT + w) * groups + (kc >> 5);
      for (; it < m.iters; it += WG_TEAMS) {
        uint2 code[ROWS];
        uint32_t step[ROWS];
        {
          // row by row: with its multiples of the stride kept at hand the loop
          // would take 32 registers more
          int64_t down = WG_TEAM * a.ldc, down_steps = WG_TEAM * groups;
          asm volatile("" : "+l"(down), "+l"(down_steps));
          const int8_t* c = cp;
          const uint8_t* b = sp;
          if ((int64_t)(it + 1) * KT <= span) {
#pragma unroll
            for (int i = 0; i < ROWS; ++i, c += down, b += down_steps) {
              code[i] = __ldg(reinterpret_cast<const uint2*>(c));
              step[i] = __ldg(b);
            }
          } else {
            const int left = (int)(span - (int64_t)it * KT) - w;  // rows past the split's end: zeros
#pragma unroll
            for (int i = 0; i < ROWS; ++i, c += down, b += down_steps) {
              code[i] = WG_TEAM * i < left ? __ldg(reinterpret_cast<const uint2*>(c)) : make_uint2(0u, 0u);
              step[i] = WG_TEAM * i < left ? __ldg(b) : 1u;
            }
          }
        }
        cp += WG_TEAMS * KT * a.ldc;
        sp += WG_TEAMS * KT * groups;
        const int slot = (g + it) % STAGES;
        const uint32_t st = base + (uint32_t)slot * S::STAGE;
        if constexpr (TMA) {
          if (!(ok = mbar_wait_warp(empty(slot), (((g + it) / STAGES) & 1) ^ 1))) break;
        } else {
          // rows w, w + 4, ... of dy, 32 lanes each
          Raw8<__nv_bfloat16> d[ROWS];
#pragma unroll
          for (int i = 0; i < ROWS; ++i) {
            const int64_t t = m.t0 + (int64_t)it * KT + WG_TEAM * i + w;
            const bool in = t < m.t1;  // rows past the split's end: zeros
            d[i] = load8(a.dy + (in ? t : m.t0) * a.lddy, m.n0 + 8 * lane, in ? a.n : 0);
          }
          if (!(ok = mbar_wait_warp(empty(slot), (((g + it) / STAGES) & 1) ^ 1))) break;
#pragma unroll
          for (int i = 0; i < ROWS; ++i) {
            const uint4 x = *reinterpret_cast<const uint4*>(&d[i]);
            st_shared16(st + ((i & 1) ? off1 : off0) - A_BYTES + 1024u * (i >> 1), x.x, x.y, x.z, x.w);
          }
        }
        uint32_t odd = 0u;
#pragma unroll
        for (int i = 0; i < ROWS; ++i) odd = max(odd, step[i] - 1u);
        if (__any_sync(FULL, odd >= 247u)) {
#pragma unroll
          for (int i = 0; i < ROWS; ++i)
            st_shared16(st + ((i & 1) ? off1 : off0) + 1024u * (i >> 1), codes_bf16_any(code[i].x, step[i]),
                        codes_bf16_any(code[i].x >> 8, step[i]), codes_bf16_any(code[i].y, step[i]),
                        codes_bf16_any(code[i].y >> 8, step[i]));
        } else {
#pragma unroll
          for (int i = 0; i < ROWS; ++i) {
            const uint32_t lead = step[i] * 0x00800080u + 0x03800380u, minus = step[i] * 0x00800080u + 0x80008000u;
            st_shared16(st + ((i & 1) ? off1 : off0) + 1024u * (i >> 1), codes_bf16(code[i].x, lead, minus),
                        codes_bf16(code[i].x >> 8, lead, minus), codes_bf16(code[i].y, lead, minus),
                        codes_bf16(code[i].y >> 8, lead, minus));
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(full_b(slot));
      }
      g += m.iters;
    }
  } else if (warp < WG_TMA) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(S::REGS_OUT));
    ok = wg_write<S>(a, &out_map, base + WG_RING, acc_full(0), acc_empty(0), tmem);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::REGS_REST));
    if (warp == WG_TMA) {
    // ------------------------------------------------ dy tiles by TMA
    if (TMA && lane == 0) {
      for (int i = blockIdx.x; ok && i < a.items; i += gridDim.x) {
        const WgItem m = item_at(i);
        for (int it = 0; it < m.iters; ++it, ++g) {
          const int s = g % STAGES;
          if (!(ok = mbar_wait(empty(s), ((g / STAGES) & 1) ^ 1))) break;
          mbar_expect(full_a(s), PARTS * A_BYTES);
          const uint32_t st = base + (uint32_t)s * S::STAGE;
          const int y = (int)(m.t0 + (int64_t)it * KT);
#pragma unroll
          for (int p = 0; p < PARTS; ++p)
#pragma unroll
            for (int b = 0; b < S::M / 64; ++b)
              tma_load_3d(st + p * A_BYTES + b * BLOCK, &dy_map, (int)m.n0 + 64 * b, y, p, full_a(s));
        }
      }
      // its copies in flight write this CTA's memory: see them land
      if (!ok)
        for (int j = max(0, g - STAGES); j < g; ++j) mbar_wait(full_a(j % STAGES), (j / STAGES) & 1);
    }
    } else if (warp == WG_MMA) {
    // ------------------------------------------------ MMA
    if (lane == 0) {
      uint32_t used0 = 0u, used1 = 0u;  // chains so far of each accumulator
      for (int i = blockIdx.x; ok && i < a.items; i += gridDim.x) {
        const WgItem m = item_at(i);
        const uint32_t nd = (uint32_t)((min((int64_t)WG_N, a.k - m.k0) + 15) / 16 * 16);
        // fp32 accumulator, bf16 operands, both MN-major, N, M = 128
        const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 15) | (1u << 16) | ((nd >> 3) << 17) | (8u << 24);
        auto arrived = [&](int q) {
          const int s = q % STAGES;
          const uint32_t ph = (q / STAGES) & 1;
          const bool in = (!TMA || mbar_wait(full_a(s), ph)) && mbar_wait(full_b(s), ph);
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          return in;
        };
        // a chain begins where the one before has been read out
        auto vacant = [&](int h) {
          const bool in = mbar_wait(acc_empty(h), ((h ? used1++ : used0++) & 1) ^ 1);
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          return in;
        };
        auto multiply = [&](int q, int h, bool first) {
          const uint32_t st = base + (uint32_t)(q % STAGES) * S::STAGE;
#pragma unroll
          for (int j = 0; j < KT / 16; ++j) {
            const uint64_t db = mn_desc(st + PARTS * A_BYTES + j * 2048, BLOCK);
            if (PARTS == 1) {
              mma_f16(tmem + 256u * h, mn_desc(st + h * 2 * BLOCK + j * 2048, BLOCK), db, idesc, !first || j > 0);
            } else {
#pragma unroll
              for (int p = 0; p < PARTS; ++p)
                mma_f16(tmem + (p ? 256u : 0u), mn_desc(st + p * A_BYTES + j * 2048, BLOCK), db, idesc, !first || j > 0 || p > 1);
            }
          }
        };
        int end0 = wg_chain_end<S>(m.iters, 0, 0), end1 = m.halves == 2 ? wg_chain_end<S>(m.iters, 1, 0) : m.iters + 1;
        bool new0 = true, new1 = m.halves == 2;
        for (int pos = 0; ok && pos < m.iters;) {
          const int stop = min(end0, end1);
          if (new0 || new1) {
            // the other accumulator goes on with the stages at hand while
            // the one whose chain begins is still read out, which catches up
            const int lead = min(stop - pos, STAGES), h = new0 && !new1 && m.halves == 2 ? 1 : 0;
            ok = !(h ? new1 : new0) || vacant(h);
            for (int q = 0; ok && q < lead; ++q) {
              if (!(ok = arrived(g + pos + q))) break;
              multiply(g + pos + q, h, (h ? new1 : new0) && q == 0);
              if (m.halves == 1) mma_commit(empty((g + pos + q) % STAGES));
            }
            if (m.halves == 2) {
              ok = ok && vacant(1 - h);
              for (int q = 0; ok && q < lead; ++q) {
                multiply(g + pos + q, 1 - h, q == 0);
                mma_commit(empty((g + pos + q) % STAGES));
              }
            }
            pos += lead;
          }
          for (; ok && pos < stop; ++pos) {
            if (!(ok = arrived(g + pos))) break;
            multiply(g + pos, 0, false);
            if (m.halves == 2) multiply(g + pos, 1, false);
            mma_commit(empty((g + pos) % STAGES));
          }
          new0 = end0 == stop, new1 = end1 == stop;
          if (new0) mma_commit(acc_full(0)), end0 = wg_chain_end<S>(m.iters, 0, pos);
          if (new1) mma_commit(acc_full(1)), end1 = wg_chain_end<S>(m.iters, 1, pos);
        }
        g += m.iters;
      }
      if (!ok) {
        // MMAs in flight read this CTA's memory: see them end (by a barrier of
        // their own: either accumulator's chain may be done while the other's runs)
        mma_commit(drained);
        mbar_wait(drained, 0);
      }
    }
    }
  }
  if (!ok) atomicOr(a.diag + DIAG_ERR, GC_DIAG_TIMEOUT);
  __syncwarp();
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (warp == WG_MMA)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

// dw = (dw +) cscale * the splits' sums in their order, four columns per
// thread and eight sums' loads at a time.  vec: rows of dw on 16-byte
// boundaries.  Bound by L2 and latency: four sums of 1024 x 1024 take 6 us.
__global__ void __launch_bounds__(256) k_weight_grad_join(const float4* part, int splits, int64_t n, int64_t k, int64_t fours,
                                                          const void* cscale, int ctype, float* dw, int64_t lddw,
                                                          int accumulate, bool vec) {
  chain_wait();
  const int64_t total = n * fours;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t r = total < (int64_t(1) << 32) ? (int64_t)((uint32_t)i / (uint32_t)fours) : i / fours;
    const int64_t c = (i - r * fours) * 4;
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int p = 0; p < splits; p += 8) {
      float4 v[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] = p + q < splits ? __ldg(part + (p + q) * total + i) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        s[0] = __fadd_rn(s[0], v[q].x), s[1] = __fadd_rn(s[1], v[q].y);
        s[2] = __fadd_rn(s[2], v[q].z), s[3] = __fadd_rn(s[3], v[q].w);
      }
    }
    float* o = dw + r * lddw + c;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (c + e >= k) break;
      if (cscale) s[e] = __fmul_rn(s[e], load_as_f32(cscale, ctype, c + e));
      if (accumulate) s[e] = __fadd_rn(o[e], s[e]);
    }
    if (vec && c + 4 <= k) {
      *reinterpret_cast<float4*>(o) = make_float4(s[0], s[1], s[2], s[3]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (c + e < k) o[e] = s[e];
    }
  }
}

// The bf16 terms of dy, one [rows, ldt] after another: the upper halves of
// what is left, by truncation, so that nothing overflows and the rest is exact.
// Bound by memory: 8192 x 1024 in fp16 takes 8 us.
template <typename T, int PARTS, bool SPAN>
__global__ void __launch_bounds__(256, 4) k_split(const T* dy, int64_t ld, Tiling t, __nv_bfloat16* terms, int64_t ldt) {
  constexpr int AHEAD = 8 / (int)(sizeof(T) / 2);
  __shared__ float4 shared[Rows<T, SPAN>::bytes(AHEAD, 256) / 16];
  chain_wait();
  const Place p = place(t);
  Rows<T, SPAN> in(shared, 256, dy + p.r * ld, p.step * ld, p.c8, p.n, t.cols);
  __nv_bfloat16* to = terms + p.r * ldt + (int64_t)p.c8 * CHUNK;
  int64_t r = p.r, next = p.r;
  auto copy = [&](int slot) {
    in.copy(slot, next < p.end);
    copy_group();
    next += p.step;
  };
#pragma unroll
  for (int i = 0; i < AHEAD - 1; ++i) copy(i);
  int slot = 0;
  for (int64_t lead = (int64_t)blockIdx.y * t.slab; lead < p.end; lead += p.step, r += p.step, to += p.step * ldt) {
    float v[CHUNK];
    wait_groups<AHEAD - 2>();
    in.landed();
    in.take(slot, r < p.end ? p.n : 0, v);
    in.done();
    copy((slot + AHEAD - 1) % AHEAD);
    slot = (slot + 1) % AHEAD;
    const bool put = r < p.end && (int64_t)p.c8 * CHUNK < ldt;
#pragma unroll
    for (int q = 0; q < PARTS; ++q) {
      uint32_t x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = __byte_perm(__float_as_uint(v[2 * j]), __float_as_uint(v[2 * j + 1]), 0x7632);
      if (q + 1 < PARTS) {
#pragma unroll
        for (int e = 0; e < CHUNK; ++e) {
          const float top = __uint_as_float(__float_as_uint(v[e]) & 0xFFFF0000u);
          v[e] = isinf(v[e]) ? 0.0f : __fsub_rn(v[e], top);
        }
      }
      if (put) *reinterpret_cast<uint4*>(to + q * t.rows * ldt) = make_uint4(x[0], x[1], x[2], x[3]);
    }
  }
}

constexpr int WG_SMS = 152;  // of a GB300

static int64_t wg_span(int64_t rows, int64_t splits) { return ((rows + splits - 1) / splits + 63) / 64 * 64; }
static int64_t wg_tiles_m(int64_t n, int32_t dtype) {
  const int m = dtype == GC_BF16 ? WgShape<1, true>::M : WgShape<2, false>::M;
  return (n + m - 1) / m;
}
// Splits of the rows where there are fewer tiles than SMs.  In us: 64 rows take
// STAGE, a split's sums take 8 bytes an element at 7 TB/s and 0.1 to write and
// to join, the join's launch 2; with s splits STAGE * stages / s + each * s, least
// for their root.  (500 x 4096 x 1024 in bf16 takes 13.6 us whole and 19.8 in
// two; 1000 x 333 x 1001 in fp32 15.0 in six, 15.6 in four, 23.9 whole.)
struct WgSplit {
  int64_t stages;
  double stage, each;
};
static WgSplit wg_split(int64_t rows, int64_t n, int64_t k, int32_t dtype) {
  return {(rows + 63) / 64, dtype == GC_F32 ? 1.0 : 0.67, (double)n * (double)k * 8.0 / 7e6 + 0.1};
}
// The most that so many rows, or fewer, are split into: it never falls as rows
// grow, where the splits themselves do, by how the rows divide into stages.
static int wg_most_splits(int64_t rows, int64_t n, int64_t k, int32_t dtype) {
  const WgSplit w = wg_split(rows, n, k, dtype);
  const int64_t most = WG_SMS / (wg_tiles_m(n, dtype) * ((k + WG_N - 1) / WG_N));
  const int64_t s = (int64_t)(std::sqrt((double)w.stages * w.stage / w.each) + 0.5);
  return (int)(s < most ? s : most);
}
static int wg_splits(int64_t rows, int64_t n, int64_t k, int32_t dtype) {
  const WgSplit w = wg_split(rows, n, k, dtype);
  int64_t s = wg_most_splits(rows, n, k, dtype);
  if (s < 2) return 1;
  const int64_t span = wg_span(rows, s);
  s = (rows + span - 1) / span;
  return (double)(span / 64) * w.stage + (double)s * w.each + 2.0 < (double)w.stages * w.stage ? (int)s : 1;
}
static int64_t wg_ldp(int64_t k) { return (k + 3) / 4 * 4; }  // row stride of the splits' sums

// The terms of dy as a 3-D tensor (n, rows, term) of 64 x 64 boxes under the
// 128-byte swizzle.
static bool make_dy_map(CUtensorMap* m, const WgArgs& a, int parts) {
  const TensorMapEncode encode = tensor_map_encode();
  const cuuint64_t dims[3] = {(cuuint64_t)a.n, (cuuint64_t)a.rows, (cuuint64_t)parts};
  const cuuint64_t strides[2] = {(cuuint64_t)a.lddy * 2, (cuuint64_t)a.lddy * 2 * (cuuint64_t)a.rows};
  const cuuint32_t box[3] = {64, 64, 1}, step[3] = {1, 1, 1};
  return encode && encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<__nv_bfloat16*>(a.dy), dims, strides, box, step,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// The result as a 3-D tensor (k, n, split) of 32 x 32 boxes.
static bool make_out_map(CUtensorMap* m, const WgArgs& a) {
  const TensorMapEncode encode = tensor_map_encode();
  const cuuint64_t dims[3] = {(cuuint64_t)a.k, (cuuint64_t)a.n, (cuuint64_t)a.splits};
  const cuuint64_t strides[2] = {(cuuint64_t)a.ldo * 4, (cuuint64_t)a.ldo * 4 * (cuuint64_t)a.n};
  const cuuint32_t box[3] = {32, 32, 1}, step[3] = {1, 1, 1};
  return encode && encode(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, a.out, dims, strides, box, step,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int PARTS, bool TMA>
static bool launch_wg(const WgArgs& a, cudaStream_t s) {
  auto kern = k_weight_grad<PARTS, TMA>;
  // the registers that the groups share out are those of the launch: with
  // fewer the kernel would wait for more, so it is not launched (a compiler
  // that gives it other than 96 asks for other shares above)
  static PerDevice ready;
  const auto prepare = [=] {
    cudaFuncAttributes at;
    if (cudaFuncGetAttributes(&at, kern) != cudaSuccess) return (void)cudaGetLastError(), 0;
    return at.numRegs == WG_REGS && grant_shared(kern, WG_SMEM) ? 1 : 0;
  };
  CUtensorMap dy_map = {}, out_map = {};
  if (!ready.get(current_device(), prepare) || (TMA && !make_dy_map(&dy_map, a, PARTS)) || (a.bulk && !make_out_map(&out_map, a))) return false;
  launch_chained(kern, (unsigned)(a.items < WG_SMS ? a.items : WG_SMS), WG_THREADS, WG_SMEM, s, dy_map, out_map, a);
  return true;
}

template <typename T, int PARTS>
static void launch_split(const void* dy, int64_t lddy, int64_t rows, int64_t n, __nv_bfloat16* terms, int64_t ldt,
                         cudaStream_t s) {
  const bool span = sizeof(T) == 4 || !aligned16(dy) || lddy % 8 != 0;
  // a bf16 dy comes here only as spans, fp32 always does
  constexpr auto ALIGNED = &k_split<T, PARTS, PARTS != 2>, ANY = &k_split<T, PARTS, true>;
  dim3 grid;
  const Tiling t = make_tiling(rows, n, span, span ? resident<ANY>() : resident<ALIGNED>(), &grid);
  launch_chained(span ? ANY : ALIGNED, grid, 256, 0, s, static_cast<const T*>(dy), lddy, t, terms, ldt);
}

// Workspace: the diagnostic words, dy's terms (none for a bf16 dy whose n
// elements per row can lie on 16-byte boundaries), room for the sums of the most
// splits, so that what holds many rows holds fewer (at most 40 MB: there are
// splits only where all their tiles fit the SMs).
struct WgSpace {
  int parts, splits;
  int64_t ldt;  // row stride of the terms
  size_t terms, sums, bytes;
};
static WgSpace wg_space(int64_t rows, int64_t n, int64_t k, int32_t dtype) {
  WgSpace w;
  w.parts = dtype == GC_BF16 ? 1 : dtype == GC_F16 ? 2 : 3;
  w.splits = wg_splits(rows, n, k, dtype);
  w.ldt = (n + 7) / 8 * 8;
  w.terms = DIAG_BYTES;
  w.sums = w.terms + (dtype == GC_BF16 && n % 8 == 0 ? 0 : align_up((size_t)w.parts * rows * w.ldt * 2, 256));
  const int most = wg_most_splits(rows, n, k, dtype);
  w.bytes = w.sums + (most > 1 ? (size_t)most * n * wg_ldp(k) * sizeof(float) : 0);
  return w;
}

}  // namespace gc

using namespace gc;

extern "C" gc_status gc_act_weight_grad_workspace_size(int64_t rows, int64_t n, int64_t k, int32_t dtype,
                                                       size_t* bytes) {
  gc_status st = validate_matrix(rows, n, dtype);
  if (st == GC_OK) st = validate_matrix(rows, k, dtype);
  if (st != GC_OK) return st;
  if (!bytes) return GC_ERR_INVALID_ARG;
  *bytes = wg_space(rows, n, k, dtype).bytes;
  return GC_OK;
}

extern "C" gc_status gc_act_weight_grad(const void* dy, int64_t lddy, int32_t dtype, int64_t rows, int64_t n,
                                        const int8_t* codes, const uint8_t* steps, int64_t k, const void* col_scale,
                                        int32_t col_scale_dtype, float* dw, int64_t lddw, uint32_t flags,
                                        void* workspace, size_t ws_bytes, void* stream) {
  NvtxRange nvtx_range("gc_act_weight_grad");
  size_t need = 0;
  gc_status st = gc_act_weight_grad_workspace_size(rows, n, k, dtype, &need);
  if (st != GC_OK) return st;
  if ((col_scale && !valid_dtype(col_scale_dtype)) || (flags & ~GC_ACCUMULATE)) return GC_ERR_INVALID_ARG;
  if ((st = check_workspace(workspace, ws_bytes, need)) != GC_OK || (st = check_matrix(dw, lddw, k, GC_F32)) != GC_OK ||
      (st = check_vector(col_scale, col_scale_dtype)) != GC_OK)
    return st;
  if (rows > 0 && ((st = check_matrix(dy, lddy, n, dtype)) != GC_OK || (st = check_codes(codes, steps)) != GC_OK))
    return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const WgSpace w = wg_space(rows, n, k, dtype);
  const int splits = w.splits, acc = (flags & GC_ACCUMULATE) ? 1 : 0;
  const int64_t tiles_n = (k + WG_N - 1) / WG_N, items = wg_tiles_m(n, dtype) * tiles_n * splits;
  if (items > INT64_C(1073741823)) return GC_ERR_LAYOUT;
  unsigned char* const ws = static_cast<unsigned char*>(workspace);
  float* part = reinterpret_cast<float*>(ws + w.sums);
  if (rows > 0) {
    WgArgs a;
    a.dy = static_cast<const __nv_bfloat16*>(dy), a.lddy = lddy, a.rows = rows, a.n = n, a.k = k, a.ldc = act_ldc(k);
    a.codes = codes, a.steps = steps;
    a.cscale = splits > 1 ? nullptr : col_scale, a.ctype = col_scale_dtype;
    a.accumulate = splits > 1 ? 0 : acc;
    a.out = splits > 1 ? part : dw, a.ldo = splits > 1 ? wg_ldp(k) : lddw;
    a.bulk = !(aligned16(a.out) && a.ldo % 4 == 0) ? WG_NONE : splits > 1 || k % 4 == 0 ? WG_ALL : WG_WHOLE;
    a.splits = splits, a.tiles_n = (int)tiles_n, a.items = (int)items;
    a.span = wg_span(rows, splits);
    a.diag = reinterpret_cast<uint32_t*>(ws);
    const bool bulk = dtype == GC_BF16 && aligned16(dy) && lddy % 8 == 0;  // dy as it is
    if (!bulk && w.sums > w.terms) {
      __nv_bfloat16* terms = reinterpret_cast<__nv_bfloat16*>(ws + w.terms);
      if (dtype == GC_BF16)
        launch_split<__nv_bfloat16, 1>(dy, lddy, rows, n, terms, w.ldt, s);
      else if (dtype == GC_F16)
        launch_split<__half, 2>(dy, lddy, rows, n, terms, w.ldt, s);
      else
        launch_split<float, 3>(dy, lddy, rows, n, terms, w.ldt, s);
      a.dy = terms, a.lddy = w.ldt;
    }
    const bool ok = w.parts == 2   ? launch_wg<2, true>(a, s)
                    : w.parts == 3 ? launch_wg<3, true>(a, s)
                    : bulk || w.sums > w.terms ? launch_wg<1, true>(a, s) : launch_wg<1, false>(a, s);
    if (!ok) return GC_ERR_CUDA;
  } else if (!zero_chained(ws, DIAG_BYTES, s)) {
    return GC_ERR_CUDA;
  }
  if (splits > 1 || rows == 0) {
    const int64_t fours = wg_ldp(k) / 4, blocks = (n * fours + 255) / 256;
    launch_chained(k_weight_grad_join, (unsigned)(blocks < 152 * 16 ? blocks : 152 * 16), 256, 0, s,
                   reinterpret_cast<const float4*>(part), rows == 0 ? 0 : splits, n, k, fours, col_scale,
                   (int)col_scale_dtype, dw, lddw, acc, aligned16(dw) && lddw % 4 == 0);
  }
  return cudaGetLastError() == cudaSuccess ? GC_OK : GC_ERR_CUDA;
}
