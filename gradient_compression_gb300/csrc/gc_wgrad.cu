// Weight gradient from an activation checkpoint on the fifth-generation
// tensor cores: dw[n, k] = sum_t dy[t, n] * q[t, k], q = code * step.
#include <cuda.h>

#include <type_traits>

#include "gc_act.cuh"
#include "gc_host.h"

namespace gc {

// Mathematics and precision.  q's code has 7 bits and its step is a power of
// two, so q is exact in bf16; a bf16 dy is too, an fp16 dy is the exact sum
// of two bf16 terms (11 bits = 8 + 3) and an fp32 dy of three (24 = 8 + 8 +
// 8).  Every product is therefore exact and only the fp32 sums round.
//
// Tile.  A CTA computes 256 (n) x 256 (k) of dw: two accumulators of 128 x
// 256 fp32, all 512 columns of the SM's tensor memory.  q has to be unpacked
// from codes by ordinary instructions, and the unpacked tile serves both
// accumulators: 16 codes per clock at the tensor cores' full rate, about 45%
// of the SM's issue slots at 2.5 instructions each.  A 128 x 256 tile would
// need 32 codes per clock.
//
// Both operands have the summed index t as their slow dimension in memory,
// so both are staged "MN-major": 128-byte rows of 64 consecutive n (or k) of
// one t, 16-byte chunk c of row t at chunk c ^ (t & 7) (the 128-byte
// swizzle), 64-wide column blocks one after another.
constexpr int WG_M = 256, WG_N = 256;      // n and k of a CTA's tile
// The unpacking warps work in teams, each on every WG_TEAMS-th stage: a team
// has as many stages' time for its own, so the latency of its loads of codes
// is hidden without keeping several stages' codes in registers.
constexpr int WG_TEAMS = 3, WG_TEAM = 4;   // teams, warps of a team
constexpr int WG_CONV = WG_TEAMS * WG_TEAM;     // warps that unpack codes, then write the result
constexpr int WG_THREADS = (WG_CONV + 2) * 32;  // + one warp issuing TMA loads, one issuing MMAs
constexpr int WG_SMEM = 192 * 1024;

struct WgArgs {
  const void* dy;
  int64_t lddy, rows, n, k, ldc;
  const int8_t* codes;
  const uint8_t* steps;
  const void* cscale;
  int ctype, accumulate;
  float* dw;       // or the partial sums, one [n, k] after another
  int64_t lddw;
  int splits, tiles_n;          // tiles along k
  int64_t span;                 // rows of a split, a multiple of 64
  uint32_t* diag;
};

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
// Waits for the phase of the given parity to complete, a bounded number of
// polls (each suspended by the hardware for at most about a microsecond).
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity) {
  for (int i = 0; i < (1 << 22); ++i) {
    uint32_t done;
    asm volatile(
        "{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 1000;\nselp.b32 %0, 1, 0, p;\n}\n"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    if (done) return true;
  }
  return false;
}
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(map), "r"(bar), "r"(x), "r"(y)
      : "memory");
}

__device__ __forceinline__ void st_shared16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// Shared-memory operand descriptor of an MN-major tile under the 128-byte
// swizzle: 64-wide blocks `block` bytes apart, groups of 8 t 1024 bytes apart.
__device__ __forceinline__ uint64_t mn_desc(uint32_t addr, uint32_t block) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)(block >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         (uint64_t(1) << 46) | (uint64_t(2) << 61);
}
// D[128 x N] (+)= A^T B over 16 t: bf16 operands, fp32 accumulator in tensor memory.
__device__ __forceinline__ void mma_bf16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\ntcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tmem_load32(float (&v)[32], uint32_t addr) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
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
// The bytes of a word come out in the order 0, 2, 1, 3: column 4 q + p of the
// tile holds column 4 q + (0, 2, 1, 3)[p] of q, which the result undoes.
__device__ __forceinline__ int wg_column(int c) { return (c & ~3) | ((c & 1) << 1) | ((c >> 1) & 1); }

// 8 elements of dy from column c on, as fp32; 0 outside [0, n).
template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T* row, int64_t c, int64_t n, float (&v)[8]) {
  if (VEC && c + 8 <= n) {
    if constexpr (sizeof(T) == 4) {
      const float4 a = *reinterpret_cast<const float4*>(row + c), b = *reinterpret_cast<const float4*>(row + c + 4);
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
      const uint4 a = *reinterpret_cast<const uint4*>(row + c);
      const T* e = reinterpret_cast<const T*>(&a);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = to_f32(e[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c + i < n ? to_f32(row[c + i]) : 0.0f;
  }
}

// TMA: dy is bf16 and its rows start on 16-byte boundaries, so that its
// tiles come by bulk tensor copies; else the unpacking warps load it too,
// split into PARTS bf16 terms.
// WIDE: the rows of q in a stage may span 2^32 bytes.
template <typename T, int PARTS, bool TMA, bool VEC, bool WIDE>
__global__ void __launch_bounds__(WG_THREADS, 1) k_weight_grad(const __grid_constant__ CUtensorMap map, const WgArgs a) {
  constexpr int KT = TMA ? 64 : 32;                     // t of a stage
  constexpr int BLOCK = KT * 128;                       // bytes of a 64-wide column block
  constexpr int A_BYTES = 4 * BLOCK, B_BYTES = 4 * BLOCK, STAGE = PARTS * A_BYTES + B_BYTES;
  constexpr int STAGES = WG_SMEM / STAGE;
  constexpr int ROWS = KT / WG_TEAM;                    // t per unpacking warp and stage
  extern __shared__ __align__(1024) unsigned char smem[];
  __shared__ __align__(8) uint64_t bars[3 * 8 + 1];
  __shared__ uint32_t tmem_base;
  __shared__ volatile int failed;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t base = smem_u32(smem), bar0 = smem_u32(bars);
  auto full_a = [&](int s) { return bar0 + 8u * s; };
  auto full_b = [&](int s) { return bar0 + 64u + 8u * s; };
  auto empty = [&](int s) { return bar0 + 128u + 8u * s; };
  const uint32_t done = bar0 + 192u;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) mbar_init(full_a(s), 1), mbar_init(full_b(s), WG_TEAM), mbar_init(empty(s), 1);
    mbar_init(done, 1);
    failed = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == WG_CONV + 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&tmem_base)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = tmem_base;
  chain_wait();
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.diag = 0u;

  const int split = blockIdx.x % a.splits;
  const int tile = blockIdx.x / a.splits;
  const int64_t n0 = (int64_t)(tile / a.tiles_n) * WG_M, k0 = (int64_t)(tile % a.tiles_n) * WG_N;
  const int64_t t0 = split * a.span, t1 = min(t0 + a.span, a.rows);
  const int iters = t1 > t0 ? (int)((t1 - t0 + KT - 1) / KT) : 0;
  const int halves = n0 + 128 < a.n ? 2 : 1;
  auto fail = [&]() {
    failed = 1;
    atomicOr(a.diag, GC_DIAG_TIMEOUT);
  };

  if (warp < WG_CONV) {
    // ------------------------------------------------ unpack q (and split dy)
    // Lanes past q's last column read the last columns again: what they put
    // into the tile reaches only columns of the accumulators that are not
    // written out.
    using Off = typename std::conditional<WIDE, int64_t, uint32_t>::type;
    const int team = warp / WG_TEAM, w = warp % WG_TEAM;  // rows w, w + 4, ...
    const int64_t kc = min(k0 + 8 * lane, a.ldc - 8), groups = a.ldc >> 5;
    const int8_t* cp = a.codes + (t0 + (int64_t)team * KT) * a.ldc;
    const uint8_t* sp = a.steps + (t0 + (int64_t)team * KT) * groups;
    const Off co = (Off)(w * a.ldc + kc), so = (Off)(w * groups + (kc >> 5));
    const uint32_t off0 = (uint32_t)(lane >> 3) * BLOCK + (uint32_t)w * 128u + (uint32_t)(((lane & 7) ^ w) << 4);
    const uint32_t off1 = (uint32_t)(lane >> 3) * BLOCK + (uint32_t)w * 128u + 512u + (uint32_t)(((lane & 7) ^ (w + 4)) << 4);
    bool ok = true;
    for (int it = team; it < iters; it += WG_TEAMS) {
      uint2 code[ROWS];
      uint32_t step[ROWS];
      if ((int64_t)(it + 1) * KT <= t1 - t0) {
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
          code[i] = __ldg(reinterpret_cast<const uint2*>(cp + (co + (Off)(WG_TEAM * i) * (Off)a.ldc)));
          step[i] = __ldg(sp + (so + (Off)(WG_TEAM * i) * (Off)groups));
        }
      } else {
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {  // rows past the split's end: zeros
          const bool in = (int64_t)it * KT + WG_TEAM * i + w < t1 - t0;
          code[i] = in ? __ldg(reinterpret_cast<const uint2*>(cp + (co + (Off)(WG_TEAM * i) * (Off)a.ldc))) : make_uint2(0u, 0u);
          step[i] = in ? __ldg(sp + (so + (Off)(WG_TEAM * i) * (Off)groups)) : 1u;
        }
      }
      cp += WG_TEAMS * KT * a.ldc;
      sp += WG_TEAMS * KT * groups;
      const int slot = it % STAGES;
      if (!(ok = mbar_wait(empty(slot), ((it / STAGES) & 1) ^ 1))) break;
      const uint32_t st = base + (uint32_t)slot * STAGE;
      if constexpr (!TMA) {
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
          const int64_t t = t0 + (int64_t)it * KT + WG_TEAM * i + w;
          float v[8];
          if (t < t1) {
            load8<T, VEC>(static_cast<const T*>(a.dy) + t * a.lddy, n0 + 8 * lane, a.n, v);
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = 0.0f;
          }
#pragma unroll
          for (int p = 0; p < PARTS; ++p) {
            uint32_t x[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              // the upper halves: truncation to bf16, so that nothing overflows
              x[j] = __byte_perm(__float_as_uint(v[2 * j]), __float_as_uint(v[2 * j + 1]), 0x7632);
              if (p + 1 < PARTS) {
#pragma unroll
                for (int e = 2 * j; e < 2 * j + 2; ++e) {
                  const float h = __uint_as_float(__float_as_uint(v[e]) & 0xFFFF0000u);
                  v[e] = isinf(v[e]) ? 0.0f : __fsub_rn(v[e], h);
                }
              }
            }
            st_shared16(st + p * A_BYTES + ((i & 1) ? off1 : off0) + 1024u * (i >> 1), x[0], x[1], x[2], x[3]);
          }
        }
      }
      uint32_t odd = 0u;
#pragma unroll
      for (int i = 0; i < ROWS; ++i) odd = max(odd, step[i] - 1u);
      if (__any_sync(FULL, odd >= 247u)) {
#pragma unroll
        for (int i = 0; i < ROWS; ++i)
          st_shared16(st + PARTS * A_BYTES + ((i & 1) ? off1 : off0) + 1024u * (i >> 1), codes_bf16_any(code[i].x, step[i]),
                      codes_bf16_any(code[i].x >> 8, step[i]), codes_bf16_any(code[i].y, step[i]),
                      codes_bf16_any(code[i].y >> 8, step[i]));
      } else {
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
          const uint32_t lead = step[i] * 0x00800080u + 0x03800380u, minus = step[i] * 0x00800080u + 0x80008000u;
          st_shared16(st + PARTS * A_BYTES + ((i & 1) ? off1 : off0) + 1024u * (i >> 1), codes_bf16(code[i].x, lead, minus),
                      codes_bf16(code[i].x >> 8, lead, minus), codes_bf16(code[i].y, lead, minus),
                      codes_bf16(code[i].y >> 8, lead, minus));
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(full_b(slot));
    }
    if (!ok) fail();
  } else if (warp == WG_CONV) {
    // ------------------------------------------------ dy tiles by TMA
    if (TMA && lane == 0) {
      bool ok = true;
      int it = 0;
      for (; it < iters; ++it) {
        const int s = it % STAGES;
        if (!(ok = mbar_wait(empty(s), ((it / STAGES) & 1) ^ 1))) break;
        mbar_expect(full_a(s), A_BYTES);
        const uint32_t st = base + (uint32_t)s * STAGE;
        const int y = (int)(t0 + (int64_t)it * KT);
        for (int b = 0; b < 4; ++b) tma_load_2d(st + b * BLOCK, &map, (int)n0 + 64 * b, y, full_a(s));
      }
      if (!ok) {
        fail();
        for (int j = max(0, it - STAGES); j < it; ++j) mbar_wait(full_a(j % STAGES), (j / STAGES) & 1);
      }
    }
    __syncwarp();
  } else if (lane == 0) {
    // ------------------------------------------------ MMA
    const int kw = (int)min((int64_t)WG_N, a.k - k0);
    const uint32_t nd = (uint32_t)((kw + 15) / 16 * 16);
    // fp32 accumulator, bf16 operands, both MN-major, N, M = 128
    const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 15) | (1u << 16) | ((nd >> 3) << 17) | (8u << 24);
    bool ok = true;
    for (int it = 0; it < iters; ++it) {
      const int s = it % STAGES;
      const uint32_t ph = (it / STAGES) & 1;
      if (!(ok = (!TMA || mbar_wait(full_a(s), ph)) && mbar_wait(full_b(s), ph))) break;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const uint32_t st = base + (uint32_t)s * STAGE;
#pragma unroll
      for (int j = 0; j < KT / 16; ++j) {
        const uint64_t db = mn_desc(st + PARTS * A_BYTES + j * 2048, BLOCK);
#pragma unroll
        for (int p = 0; p < PARTS; ++p)
          for (int h = 0; h < halves; ++h)
            mma_bf16(tmem + 256u * h, mn_desc(st + p * A_BYTES + h * 2 * BLOCK + j * 2048, BLOCK), db, idesc,
                     it > 0 || j > 0 || p > 0);
      }
      mma_commit(empty(s));
    }
    mma_commit(done);
    if (!ok) {
      fail();
      mbar_wait(done, 0);
    }
  }
  __syncwarp();

  if (warp < WG_CONV && !failed) {
    // -------------------------------------------------- the result, row by row
    const bool finished = mbar_wait(done, 0);
    __syncwarp();
    if (__all_sync(FULL, finished)) {
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      float* buf = reinterpret_cast<float*>(smem) + warp * 32 * 33;
      float* out = a.dw + (a.splits > 1 ? (int64_t)split * a.n * a.lddw : 0);
      for (int item = warp / 4; item < 2 * (WG_N / 32); item += WG_TEAMS) {  // 32 columns of an accumulator
        const int h = item / (WG_N / 32), c0 = item % (WG_N / 32) * 32;
        const int64_t r0 = n0 + 128 * h + 32 * (warp & 3);
        if (k0 + c0 >= a.k || r0 >= a.n) continue;
        float v[32];
        if (iters > 0) {
          tmem_load32(v, tmem + ((uint32_t)(32 * (warp & 3)) << 16) + 256u * h + c0);
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = 0.0f;
        }
#pragma unroll
        for (int j = 0; j < 32; ++j) buf[lane * 33 + j] = v[j];
        __syncwarp();
        const int64_t c = k0 + c0 + lane;
        if (c < a.k) {
          const float cs = a.splits == 1 && a.cscale ? load_as_f32(a.cscale, a.ctype, c) : 1.0f;
          const int rows = (int)min((int64_t)32, a.n - r0);
          for (int r = 0; r < rows; ++r) {
            float* o = out + (r0 + r) * a.lddw + c;
            const float x = __fmul_rn(buf[r * 33 + wg_column(lane)], cs);
            *o = a.splits == 1 && a.accumulate ? __fadd_rn(*o, x) : x;
          }
        }
        __syncwarp();
      }
    } else {
      fail();
    }
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (warp == WG_CONV + 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

// dw = (dw +) cscale * the splits' sums in their order.
__global__ void __launch_bounds__(256) k_weight_grad_join(const float* part, int splits, int64_t n, int64_t k,
                                                          const void* cscale, int ctype, float* dw, int64_t lddw,
                                                          int accumulate) {
  chain_wait();
  const int64_t total = n * k;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    float s = part[i];
    for (int p = 1; p < splits; ++p) s = __fadd_rn(s, part[p * total + i]);
    const int64_t r = i / k, c = i - r * k;
    if (cscale) s = __fmul_rn(s, load_as_f32(cscale, ctype, c));
    float* o = dw + r * lddw + c;
    *o = accumulate ? __fadd_rn(*o, s) : s;
  }
}

constexpr int WG_SMS = 152;  // of a GB300

// Splits of the rows: as many as keep every SM busy when there are few
// tiles, each of at least 256 rows.
static int wg_splits(int64_t rows, int64_t n, int64_t k) {
  const int64_t tiles = ((n + WG_M - 1) / WG_M) * ((k + WG_N - 1) / WG_N);
  int64_t s = WG_SMS / tiles;
  if (s > rows / 256) s = rows / 256;
  return (int)(s < 1 ? 1 : s);
}

// dy as a 2-D tensor of 64 x 64 boxes under the 128-byte swizzle.
static bool make_dy_map(CUtensorMap* m, const void* dy, int64_t lddy, int64_t rows, int64_t n) {
  using Encode = decltype(&cuTensorMapEncodeTiled);
  static const Encode encode = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<Encode>(f);
  }();
  if (!encode) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)n, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)lddy * 2};
  const cuuint32_t box[2] = {64, 64}, step[2] = {1, 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(dy), dims, strides, box, step,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int PARTS, bool TMA, bool VEC, bool WIDE = false>
static bool launch_wg(const CUtensorMap& map, const WgArgs& a, unsigned grid, cudaStream_t s) {
  auto kern = k_weight_grad<T, PARTS, TMA, VEC, WIDE>;
  static const bool ready = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, WG_SMEM) == cudaSuccess;
  if (!ready) return false;
  launch_chained(kern, grid, WG_THREADS, WG_SMEM, s, map, a);
  return true;
}

}  // namespace gc

using namespace gc;

extern "C" gc_status gc_act_weight_grad_workspace_size(int64_t rows, int64_t n, int64_t k, int32_t dtype,
                                                       size_t* bytes) {
  gc_status st = validate_matrix(rows, n, dtype);
  if (st == GC_OK) st = validate_matrix(rows, k, dtype);
  if (st != GC_OK) return st;
  if (!bytes) return GC_ERR_INVALID_ARG;
  const int splits = wg_splits(rows, n, k);
  *bytes = DIAG_BYTES + (splits > 1 ? (size_t)splits * (size_t)n * (size_t)k * sizeof(float) : 0);
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
  if ((st = check_workspace(workspace, ws_bytes, need)) != GC_OK || (st = check_matrix(dw, lddw, k, GC_F32)) != GC_OK)
    return st;
  if (rows > 0 && ((st = check_matrix(dy, lddy, n, dtype)) != GC_OK || (st = check_codes(codes, steps)) != GC_OK))
    return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int splits = wg_splits(rows, n, k);
  const int64_t tiles_n = (k + WG_N - 1) / WG_N, tiles = (n + WG_M - 1) / WG_M * tiles_n;
  if (tiles * splits > INT64_C(2147483647)) return GC_ERR_LAYOUT;
  WgArgs a;
  a.dy = dy, a.lddy = lddy, a.rows = rows, a.n = n, a.k = k, a.ldc = act_ldc(k);
  a.codes = codes, a.steps = steps, a.cscale = col_scale, a.ctype = col_scale_dtype;
  a.accumulate = (flags & GC_ACCUMULATE) ? 1 : 0;
  float* part = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + DIAG_BYTES);
  a.dw = splits > 1 ? part : dw;
  a.lddw = splits > 1 ? k : lddw;
  a.splits = splits, a.tiles_n = (int)tiles_n;
  a.span = ((rows + splits - 1) / splits + 63) / 64 * 64;
  a.diag = static_cast<uint32_t*>(workspace);
  const unsigned grid = (unsigned)(tiles * splits);
  const bool vec = aligned16(dy) && lddy % 8 == 0;
  CUtensorMap map = {};
  bool ok;
  if (a.ldc >= (int64_t(1) << 25)) {  // 64 rows of q span 2^31 bytes
    ok = dtype == GC_BF16  ? launch_wg<__nv_bfloat16, 1, false, false, true>(map, a, grid, s)
         : dtype == GC_F16 ? launch_wg<__half, 2, false, false, true>(map, a, grid, s)
                           : launch_wg<float, 3, false, false, true>(map, a, grid, s);
  } else if (dtype == GC_BF16 && vec && rows > 0) {
    ok = make_dy_map(&map, dy, lddy, rows, n) && launch_wg<__nv_bfloat16, 1, true, true>(map, a, grid, s);
  } else if (dtype == GC_BF16) {
    ok = launch_wg<__nv_bfloat16, 1, false, false>(map, a, grid, s);
  } else if (dtype == GC_F16) {
    ok = vec ? launch_wg<__half, 2, false, true>(map, a, grid, s) : launch_wg<__half, 2, false, false>(map, a, grid, s);
  } else {
    ok = vec ? launch_wg<float, 3, false, true>(map, a, grid, s) : launch_wg<float, 3, false, false>(map, a, grid, s);
  }
  if (!ok) return GC_ERR_CUDA;
  if (splits > 1) {
    const int64_t blocks = (n * k + 255) / 256;
    launch_chained(k_weight_grad_join, (unsigned)(blocks < 152 * 16 ? blocks : 152 * 16), 256, 0, s, (const float*)part,
                   splits, n, k, col_scale, (int)col_scale_dtype, dw, lddw, a.accumulate);
  }
  return cudaGetLastError() == cudaSuccess ? GC_OK : GC_ERR_CUDA;
}
