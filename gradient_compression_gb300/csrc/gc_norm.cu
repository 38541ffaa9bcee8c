// RMS norm with the residual's addition, its checkpoint and its gradient.
#include "gc_act.cuh"
#include "gc_host.h"

namespace gc {

// A row is held in registers by W warps, N chunks of 8 columns per lane (chunk
// (j W + w) 32 + lane), so that it is read once; a CTA of up to 8 warps (W, if
// that is more) works on 8 / W rows at a time and walks over the rows.  Rows
// wider than 16384 are read twice (the _wide kernels).
constexpr int NTHREADS = 256;
constexpr int64_t NORM_WIDEST = 16384;
constexpr int THREADS_80 = 768, THREADS_128 = 512;  // of an SM, 80 or 128 registers each

struct RowShape {
  int warps;    // W
  int threads;  // of a CTA
};

// The sum over a row's warps of each thread's V values, the same bits in all of
// its threads.  `red` holds 2 x 32 floats and is used alternately: one barrier.
// With V = 2 a warp stands for two, w and w + W, of the order with V = 1: a row
// gives the same bits on twice the warps.
template <int V>
__device__ __forceinline__ float row_sum(float (&v)[V], int W, int w, float (&red)[2][32], int& turn) {
#pragma unroll
  for (int o = 16; o; o >>= 1)
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = __fadd_rn(v[i], __shfl_xor_sync(FULL, v[i], o));
  if (W == 1) return V == 1 ? v[0] : __fadd_rn(v[0], v[V - 1]);
  float* const of = &red[turn][((int)(threadIdx.x >> 5) - w) * V];  // w: this warp of the row's W
  if ((threadIdx.x & 31) == 0) {
#pragma unroll
    for (int i = 0; i < V; ++i) of[i * W + w] = v[i];
  }
  __syncthreads();
  float s = __fadd_rn(of[0], of[1]);
  for (int i = 2; i + 1 < V * W; i += 2) s = __fadd_rn(s, __fadd_rn(of[i], of[i + 1]));
  if (V == 1 && (W & 1)) s = __fadd_rn(s, of[W - 1]);
  turn ^= 1;
  return s;
}

// share = 1 / cols
__device__ __forceinline__ float rms_inverse(float ss, float share, float eps) {
  return __frsqrt_rn(__fadd_rn(__fmul_rn(ss, share), eps));
}

// The weights as fp32 in shared memory, once per CTA: the first and the last
// four of every chunk apart, so that a warp's 16-byte loads meet no bank
// twice.  Ones without weights, zeros past the row's end.  Read 16 bytes a lane:
// element by element this took every CTA's start 2.3 us longer.
__device__ __forceinline__ void stage_weights(float4* ws, const void* weight, int wtype, int64_t cols, int chunks) {
  const bool lanes = ((uintptr_t)weight & 15u) == 0;
#pragma unroll 2
  for (int c = threadIdx.x; c < chunks; c += blockDim.x) {
    const int n = (int)min(cols - (int64_t)c * CHUNK, (int64_t)CHUNK);
    float w[CHUNK];
    if (weight && lanes && n == CHUNK) {
      if (wtype == GC_F32) {
        const float4* from = static_cast<const float4*>(weight) + 2 * c;
        const float4 a = __ldg(from), b = __ldg(from + 1);
        w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
      } else {
        const uint4 a = __ldg(static_cast<const uint4*>(weight) + c);
        if (wtype == GC_BF16)
          unpack(*reinterpret_cast<const Raw8<__nv_bfloat16>*>(&a), w);
        else
          unpack(*reinterpret_cast<const Raw8<__half>*>(&a), w);
      }
    } else {
#pragma unroll
      for (int e = 0; e < CHUNK; ++e) w[e] = e < n ? (weight ? load_as_f32(weight, wtype, (int64_t)c * CHUNK + e) : 1.0f) : 0.0f;
    }
    ws[c] = make_float4(w[0], w[1], w[2], w[3]), ws[chunks + c] = make_float4(w[4], w[5], w[6], w[7]);
  }
  __syncthreads();
}

__device__ __forceinline__ void load_weights(const float4* ws, int chunks, int c8, float (&w)[CHUNK]) {
  const int c = min(c8, chunks - 1);  // a lane past the row's end weighs nothing
  const float4 a = ws[c], b = ws[chunks + c];
  w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
}

// How a row lies on its warps.
constexpr int ROW_SPAN = 0;    // any rows: a warp's 32 chunks as a span
constexpr int ROW_CHUNKS = 1;  // 16-bit rows on 16-byte boundaries: each lane its own
constexpr int ROW_FULL = 2;    // and every lane has N whole chunks: no bounds inside a row

// A thread's N chunks of a row: the first, and the others 32 W chunks apart.
template <int N, int MODE>
struct RowChunks {
  int first, apart;  // chunks
  int len[N];        // elements of each inside the row
  int chunks;        // of a row, pad included
  int sub, per;      // this warp's row of those that the CTA takes at a time
  int W;             // warps per row
  __device__ __forceinline__ RowChunks(int warps, int64_t cols, int64_t groups) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    W = warps, per = (int)(blockDim.x >> 5) / warps, sub = warp / warps;
    first = warp % warps * 32 + lane, apart = warps * 32, chunks = 4 * (int)groups;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int left = (int)cols - c8(j) * CHUNK;  // cols <= NORM_WIDEST
      len[j] = left < 0 ? 0 : (left < CHUNK ? left : CHUNK);
    }
  }
  __device__ __forceinline__ int c8(int j) const { return first + j * apart; }
  __device__ __forceinline__ int n(int j) const { return MODE == ROW_FULL ? CHUNK : len[j]; }
  __device__ __forceinline__ bool held(int j) const { return MODE == ROW_FULL || c8(j) < chunks; }  // in the checkpoint
};

// Rows ahead come through rings in shared memory: one row is in flight while
// one is worked on (none for the widest rows that are spans or fp32, whose
// second slot does not fit).  Registers for the rows ahead cost the warps that
// hide the latency: 0.5 of a copy's rate; three or four slots measured no faster.
template <typename T, int N, int MODE>
struct RowShared {
  static constexpr bool SPAN = MODE == ROW_SPAN;
  static constexpr int SLOTS = N * sizeof(T) <= 8 && !(SPAN && N == 4) ? 2 : 1;
  static constexpr size_t rows(int threads) { return N * Rows<T, SPAN>::bytes(SLOTS, threads); }  // of one matrix
  static constexpr size_t stage(int threads) { return SPAN ? (size_t)(threads / 32) * RowsOut<T, SPAN>::STAGE * 16 : 0; }
  static constexpr size_t forward(int threads) { return 2 * rows(threads) + stage(threads); }
  static constexpr size_t backward(int threads) {
    return 2 * rows(threads) + stage(threads) + CodeRing::bytes(N * SLOTS, threads);
  }
};

// The N chunks of a matrix's rows.
template <typename T, int N, int MODE>
struct RowIn {
  static constexpr bool SPAN = MODE == ROW_SPAN;
  Rows<T, SPAN> in;
  int64_t jump;  // elements from chunk to chunk
  int len[N];    // of each chunk, or of each span
  __device__ __forceinline__ RowIn(char* shared, const T* row, int64_t stride, const RowChunks<N, MODE>& at, int cols)
      : in(shared, (int)blockDim.x, row, stride, at.first, at.n(0), cols), jump((int64_t)at.apart * CHUNK) {
#pragma unroll
    for (int j = 0; j < N; ++j)
      len[j] = SPAN ? min(max(cols - (at.c8(j) - (int)(threadIdx.x & 31)) * CHUNK, 0), 32 * CHUNK) : at.n(j);
  }
  __device__ __forceinline__ void copy(int slot, bool there) {
    const T* row = in.next;
    if (there) {
#pragma unroll
      for (int j = 0; j < N; ++j) {
        in.next = row + j * jump, in.len = len[j];
        if (MODE == ROW_FULL)
          in.copy_whole(slot * N + j);
        else
          in.copy(slot * N + j, true);
      }
    }
    in.next = row + in.step;
  }
  // a span's columns are whole lines apart: all N share the row's misalignment
  __device__ __forceinline__ void take(int slot, int j, int n, float (&v)[CHUNK]) const { in.take(slot * N + j, n, v); }
};
template <typename T, int N, int MODE>
struct RowTo {
  static constexpr bool SPAN = MODE == ROW_SPAN;
  RowsOut<T, SPAN> to;
  int64_t jump;
  int len[N];
  __device__ __forceinline__ RowTo(T* row, int64_t stride, const RowChunks<N, MODE>& at, int cols)
      : to(row, stride, at.first, cols), jump((int64_t)at.apart * CHUNK) {
#pragma unroll
    for (int j = 0; j < N; ++j) len[j] = SPAN ? min(max(cols - (at.c8(j) - (int)(threadIdx.x & 31)) * CHUNK, 0), 32 * CHUNK) : 0;
  }
  // chunk j of the current row
  __device__ __forceinline__ void put(int j, const float (&v)[CHUNK], int n, bool there, float4* stage) {
    T* row = to.next;
    to.next = row + j * jump, to.len = len[j];
    to.put(v, n, there, stage);
    to.next = row;
  }
  __device__ __forceinline__ void done() { to.next += to.step; }
};

// One pass, bound by memory and by what a row's warps wait for each other:
// 16384 x 4096 in bf16 with residual, h, rstd and checkpoint takes 94 us (0.97
// of a copy's rate), 5120 columns 118 us (0.97), 8192 202 us (0.90), fp32 195 us (0.88), rows of
// 4095 150 us (0.60: spans, bound by instructions); one row 2.7 us.  The bounds stand
// for registers: 80 a thread, three CTAs of 256 per SM (four of 64: 104 us, two
// 99), or 128 and two for spans (12 and 25 us more, rows of 4095 and fp32, with
// three).
template <typename T, int N, int MODE>
__global__ void __launch_bounds__(N == 2 && MODE != ROW_SPAN ? THREADS_80 : THREADS_128, 1)
    k_rmsnorm(const T* x, int64_t ldx, const T* res, int64_t ldr, const void* weight, int wtype, float eps, int64_t rows,
              int64_t cols, int64_t groups, int warps, T* y, int64_t ldy, T* h, int64_t ldh, float* rstd, int8_t* codes,
              uint8_t* steps) {
  using S = RowShared<T, N, MODE>;
  constexpr int SLOTS = S::SLOTS;
  __shared__ float red[2][32];
  extern __shared__ float4 shared[];  // the weights, then the rings and the warps' staging
  chain_wait();
  const RowChunks<N, MODE> at(warps, cols, groups);
  char* const rings = reinterpret_cast<char*>(shared + 2 * at.chunks);
  const size_t one = S::rows((int)blockDim.x);
  float4* const own = reinterpret_cast<float4*>(rings + 2 * one) + (threadIdx.x >> 5) * RowsOut<T, S::SPAN>::STAGE;
  const int64_t stride = (int64_t)gridDim.x * at.per, start = at.first * CHUNK;
  int64_t r = (int64_t)blockIdx.x * at.per + at.sub, next = r;
  RowIn<T, N, MODE> xin(rings, x + r * ldx, stride * ldx, at, (int)cols);
  RowIn<T, N, MODE> rin(rings + one, res + r * ldr, stride * ldr, at, (int)cols);
  RowTo<T, N, MODE> hto(h + r * ldh, stride * ldh, at, (int)cols), yto(y + r * ldy, stride * ldy, at, (int)cols);
  auto copy = [&](int slot) {
    xin.copy(slot, next < rows);
    if (res) rin.copy(slot, next < rows);
    copy_group();
    next += stride;
  };
  if (SLOTS == 2) copy(0);
  if (y) stage_weights(shared, weight, wtype, cols, at.chunks);
  const float share = __fdiv_rn(1.0f, (float)cols);
  int8_t* pc = codes + r * groups * ACT_GROUP + start;
  uint8_t* ps = steps + r * groups + (at.first >> 2);
  int turn = 0, slot = 0;
  for (int64_t lead = (int64_t)blockIdx.x * at.per; lead < rows; lead += stride, r += stride) {
    const bool in = r < rows;
    float v[N][CHUNK], ss[2] = {0.0f, 0.0f};
    if (SLOTS == 1) copy(0);
    wait_groups<0>();
    xin.in.landed();
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int n = in ? at.n(j) : 0;
      xin.take(slot, j, n, v[j]);
      if (res) {
        float t[CHUNK];
        rin.take(slot, j, n, t);
#pragma unroll
        for (int e = 0; e < CHUNK; e += 2) put2(v[j] + e, add2(get2(v[j] + e), get2(t + e)));
      }
#pragma unroll
      for (int e = 0; e < CHUNK; e += 2) put2(ss, fma2(get2(v[j] + e), get2(v[j] + e), get2(ss)));
    }
    xin.in.done();
    if (res) rin.in.done();
    if (SLOTS == 2) {
      copy(slot ^ 1);
      slot ^= 1;
    }
    if (h) {
#pragma unroll
      for (int j = 0; j < N; ++j) hto.put(j, v[j], at.n(j), in, own);
      hto.done();
    }
    float sum[1] = {__fadd_rn(ss[0], ss[1])};
    const float rs = rms_inverse(row_sum(sum, at.W, at.first >> 5, red, turn), share, eps);
    if (rstd && in && threadIdx.x % (32 * at.W) == 0) rstd[r] = rs;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int n = in ? at.n(j) : 0;
#pragma unroll
      for (int e = 0; e < CHUNK; e += 2) put2(v[j] + e, mul2(get2(v[j] + e), f2(rs)));
      if (codes) {
        // past the row's end the values are 0 * rstd, which a rstd that is
        // not finite would turn into NaN
        if (MODE != ROW_FULL && n < CHUNK) {
#pragma unroll
          for (int e = 0; e < CHUNK; ++e)
            if (e >= n) v[j][e] = 0.0f;
        }
        const uint32_t b = chunk_step(v[j]);
        const uint2 q = chunk_codes(v[j], b);
        if (in && at.held(j)) {
          *reinterpret_cast<uint2*>(pc + j * at.apart * CHUNK) = q;
          if ((at.first & 3) == 0) ps[j * (at.apart >> 2)] = (uint8_t)b;
        }
      }
      if (y) {
        float t[CHUNK];
        load_weights(shared, at.chunks, at.c8(j), t);
#pragma unroll
        for (int e = 0; e < CHUNK; e += 2) put2(t + e, mul2(get2(v[j] + e), get2(t + e)));
        yto.put(j, t, at.n(j), in, own);
      }
    }
    yto.done();
    pc += stride * groups * ACT_GROUP, ps += stride * groups;
  }
}

// Gradient: gw = dy * weight, dx = rstd (gw - q mean(gw q)) + dh, and each
// thread's share of dw = sum dy q of its columns over the rows that its CTA
// walks over, one partial sum per CTA.
// Bound by memory and by the waits within a row, as above.  With four chunks
// per lane (rows on 16-byte boundaries) fewer warps wait for a row; gw and q do
// not fit into registers next to dw across that wait and are worked out AGAIN
// from the rings (88 us with two chunks where four took 81, and four without
// AGAIN 130).  16384 x 4096 in bf16 with dh and dw: 76 us (0.93 of a copy's rate),
// 8192 columns 148 us (0.96), 16384 columns 281 us (1.0).  Spans and fp32, bound by
// instructions, keep two chunks: rows of 4095 126 us (0.56), fp32 161 us (0.81);
// with four 30 and 60 us more.
template <typename T, int N, int MODE>
__global__ void __launch_bounds__(THREADS_128, 1)
    k_rmsnorm_backward(const T* dy, int64_t lddy, const T* dh, int64_t lddh, const int8_t* codes, const uint8_t* steps,
                       const float* rstd, const void* weight, int wtype, int64_t rows, int64_t cols, int64_t groups,
                       int warps, T* dx, int64_t lddx, float* part) {
  using S = RowShared<T, N, MODE>;
  constexpr int SLOTS = S::SLOTS;
  constexpr bool AGAIN = N == 4;
  constexpr int V = N / 2;
  __shared__ float red[2][32];
  extern __shared__ float4 shared[];
  chain_wait();
  const RowChunks<N, MODE> at(warps, cols, groups);
  char* const rings = reinterpret_cast<char*>(shared + 2 * at.chunks);
  const size_t one = S::rows((int)blockDim.x);
  float4* const own = reinterpret_cast<float4*>(rings + 2 * one) + (threadIdx.x >> 5) * RowsOut<T, S::SPAN>::STAGE;
  const CodeRing code(rings + 2 * one + S::stage((int)blockDim.x), (int)blockDim.x);
  const int64_t stride = (int64_t)gridDim.x * at.per, ldc = groups * ACT_GROUP, start = at.first * CHUNK;
  int64_t r = (int64_t)blockIdx.x * at.per + at.sub, next = r;
  RowIn<T, N, MODE> din(rings, dy + r * lddy, stride * lddy, at, (int)cols);
  RowIn<T, N, MODE> hin(rings + one, dh + r * lddh, stride * lddh, at, (int)cols);
  RowTo<T, N, MODE> to(dx + r * lddx, stride * lddx, at, (int)cols);
  const int8_t* pc = codes + r * ldc + start;
  const uint8_t* ps = steps + r * groups + (at.first >> 2);
  auto copy = [&](int slot) {
    din.copy(slot, next < rows);
    if (dh) hin.copy(slot, next < rows);
    if (next < rows) {
#pragma unroll
      for (int j = 0; j < N; ++j)
        if (at.held(j)) code.copy(slot * N + j, pc + j * at.apart * CHUNK);
    }
    copy_group();
    next += stride, pc += stride * ldc;
  };
  // step bytes and rstd, a row ahead
  uint32_t b[N];
  float rs;
  auto fetch = [&](int64_t row) {
    const bool in = row < rows;
#pragma unroll
    for (int j = 0; j < N; ++j) b[j] = in && at.held(j) ? __ldg(ps + j * (at.apart >> 2)) : 1u;
    rs = in ? __ldg(rstd + row) : 0.0f;
    ps += stride * groups;
  };
  if (SLOTS == 2) copy(0);
  fetch(r);
  stage_weights(shared, weight, wtype, cols, at.chunks);
  const float share = __fdiv_rn(1.0f, (float)cols);
  int turn = 0, slot = 0;
  float dw[N][CHUNK];
#pragma unroll
  for (int j = 0; j < N; ++j)
#pragma unroll
    for (int e = 0; e < CHUNK; ++e) dw[j][e] = 0.0f;
  for (int64_t lead = (int64_t)blockIdx.x * at.per; lead < rows; lead += stride, r += stride) {
    const bool in = r < rows;
    uint32_t step[N];
#pragma unroll
    for (int j = 0; j < N; ++j) step[j] = b[j];
    const float inverse = rs;
    if (SLOTS == 1) copy(0);
    wait_groups<0>();
    din.in.landed();
    if (SLOTS == 2) copy(slot ^ 1);
    if (lead + stride < rows) fetch(r + stride);
    float gw[N][CHUNK], q[N][CHUNK], s[V][2] = {};
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int n = in ? at.n(j) : 0;
      float w[CHUNK];
      din.take(slot, j, n, gw[j]);
      chunk_values(code.take(slot * N + j), step[j], q[j]);
      load_weights(shared, at.chunks, at.c8(j), w);
      // past the row's end q is nothing (what was not copied, or a NaN's step)
      if (n < CHUNK) {
#pragma unroll
        for (int e = 0; e < CHUNK; ++e)
          if (MODE == ROW_FULL || e >= n) q[j][e] = 0.0f;
      }
#pragma unroll
      for (int e = 0; e < CHUNK; e += 2) {
        const F2 g = get2(gw[j] + e), qe = get2(q[j] + e), ge = mul2(g, get2(w + e));
        put2(dw[j] + e, fma2(g, qe, get2(dw[j] + e)));
        put2(gw[j] + e, ge);
        put2(s[j % V], fma2(ge, qe, get2(s[j % V])));
      }
    }
    float sum[V];
#pragma unroll
    for (int i = 0; i < V; ++i) sum[i] = __fadd_rn(s[i][0], s[i][1]);
    const float minus_mean = __fmul_rn(row_sum(sum, at.W, at.first >> 5, red, turn), -share);
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int n = in ? at.n(j) : 0;
      float t[CHUNK];
      if (dh) hin.take(slot, j, n, t);
      if (AGAIN) {
        float w[CHUNK];
        din.take(slot, j, n, gw[j]);
        load_weights(shared, at.chunks, at.c8(j), w);
#pragma unroll
        for (int e = 0; e < CHUNK; e += 2) put2(gw[j] + e, mul2(get2(gw[j] + e), get2(w + e)));
      }
      if (AGAIN || sizeof(T) == 4) chunk_values(code.take(slot * N + j), step[j], q[j]);
#pragma unroll
      for (int e = 0; e < CHUNK; e += 2) {
        const F2 v = fma2(get2(q[j] + e), f2(minus_mean), get2(gw[j] + e));
        put2(gw[j] + e, dh ? fma2(f2(inverse), v, get2(t + e)) : mul2(f2(inverse), v));
      }
      to.put(j, gw[j], at.n(j), in, own);
    }
    to.done();
    din.in.done();
    if (dh) hin.in.done();
    if (SLOTS == 2) slot ^= 1;
  }
  if (!part) return;
  part += (int64_t)blockIdx.x * ldc;
  if (at.per == 1) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      float4* o = reinterpret_cast<float4*>(part + start + j * at.apart * CHUNK);
      if (at.held(j)) {
        o[0] = make_float4(dw[j][0], dw[j][1], dw[j][2], dw[j][3]);
        o[1] = make_float4(dw[j][4], dw[j][5], dw[j][6], dw[j][7]);
      }
    }
    return;
  }
  // the rows at a time of narrow matrices, added up in their order by way of
  // the rings' memory
  static_assert((N > 2 && MODE == ROW_SPAN) || 2 * N * sizeof(float4) <= 2 * N * sizeof(T) * CHUNK * SLOTS, "room for the sums");
  float4* const sums = reinterpret_cast<float4*>(rings);
  __syncthreads();
#pragma unroll
  for (int j = 0; j < N; ++j) {
    sums[(2 * j) * blockDim.x + threadIdx.x] = make_float4(dw[j][0], dw[j][1], dw[j][2], dw[j][3]);
    sums[(2 * j + 1) * blockDim.x + threadIdx.x] = make_float4(dw[j][4], dw[j][5], dw[j][6], dw[j][7]);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * N * at.apart; i += blockDim.x) {
    const int half = i / at.apart, lane = i - half * at.apart, c8 = lane + (half >> 1) * at.apart;
    float4 t = sums[half * blockDim.x + lane];
    for (int p = 1; p < at.per; ++p) {
      const float4 v = sums[half * blockDim.x + p * at.apart + lane];
      t.x = __fadd_rn(t.x, v.x), t.y = __fadd_rn(t.y, v.y), t.z = __fadd_rn(t.z, v.z), t.w = __fadd_rn(t.w, v.w);
    }
    if (c8 < at.chunks) reinterpret_cast<float4*>(part)[2 * c8 + (half & 1)] = t;
  }
}

// dw[c] = (dw[c] +) the partial sums in a fixed order: 32 columns per CTA, 32
// warps each over every 32nd sum, its loads issued eight at a time: bound by
// their latency.  1031 x 1001 in fp32 takes 7.1 us with its backward pass.
__global__ void __launch_bounds__(1024) k_rmsnorm_dw_join(const float* part, int parts, int64_t cols, int64_t ldp, float* dw,
                                                          int accumulate) {
  __shared__ float sum[32][33];
  chain_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;  // ldp columns exist
  float s = 0.0f;
  for (int p = warp; p < parts; p += 256) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = p + 32 * i < parts ? __ldg(part + (int64_t)(p + 32 * i) * ldp + c) : 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s = __fadd_rn(s, v[i]);
  }
  sum[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < cols) {
    float t = sum[0][lane];
#pragma unroll
    for (int i = 1; i < 32; ++i) t = __fadd_rn(t, sum[i][lane]);
    dw[c] = accumulate ? __fadd_rn(dw[c], t) : t;
  }
}

// ---------------------------------------------------------------- wide rows
// The plain way for rows that no CTA's registers hold: read twice, the second
// time mostly from L2, and dw by a pass of its own.
// The sum over the CTA, the same bits in every thread.
__device__ __forceinline__ float cta_sum(float v, float* red) {
  for (int o = 16; o; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(FULL, v, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = red[0];
  for (int w = 1; w < NTHREADS / 32; ++w) s = __fadd_rn(s, red[w]);
  return s;
}

// One CTA per row: the sum of squares, then the outputs, a warp per group.
template <typename T>
__global__ void __launch_bounds__(NTHREADS)
    k_rmsnorm_wide(const T* x, int64_t ldx, const T* res, int64_t ldr, const void* weight, int wtype, float eps,
                   int64_t rows, int64_t cols, int64_t groups, T* y, int64_t ldy, T* h, int64_t ldh, float* rstd,
                   int8_t* codes, uint8_t* steps) {
  __shared__ float red[NTHREADS / 32];
  chain_wait();
  const int lane = threadIdx.x & 31;
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    auto sum_at = [&](int64_t c) {
      const float v = to_f32(x[r * ldx + c]);
      return res ? __fadd_rn(v, to_f32(res[r * ldr + c])) : v;
    };
    float ss = 0.0f;
    for (int64_t c = threadIdx.x; c < cols; c += NTHREADS) {
      const float v = sum_at(c);
      ss = __fmaf_rn(v, v, ss);
    }
    const float rs = rms_inverse(cta_sum(ss, red), __fdiv_rn(1.0f, (float)cols), eps);
    if (rstd && threadIdx.x == 0) rstd[r] = rs;
    for (int64_t g = threadIdx.x >> 5; g < groups; g += NTHREADS / 32) {
      const int64_t c = g * 32 + lane;
      const float v = c < cols ? sum_at(c) : 0.0f;
      const float q = c < cols ? __fmul_rn(v, rs) : 0.0f;
      if (c < cols) {
        if (h) h[r * ldh + c] = from_f32<T>(v);
        if (y) y[r * ldy + c] = from_f32<T>(weight ? __fmul_rn(q, load_as_f32(weight, wtype, c)) : q);
      }
      if (codes) {
        const uint32_t b = act_step(__reduce_max_sync(FULL, __float_as_uint(fabsf(q))));
        codes[(r * groups + g) * 32 + lane] = (int8_t)act_code(q, act_inverse(b));
        if (lane == 0) steps[r * groups + g] = (uint8_t)b;
      }
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(NTHREADS)
    k_rmsnorm_backward_wide(const T* dy, int64_t lddy, const T* dh, int64_t lddh, const int8_t* codes,
                            const uint8_t* steps, const float* rstd, const void* weight, int wtype, int64_t rows,
                            int64_t cols, int64_t groups, T* dx, int64_t lddx) {
  __shared__ float red[NTHREADS / 32];
  chain_wait();
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    auto terms = [&](int64_t c, float* q) {
      *q = __fmul_rn((float)codes[r * groups * 32 + c], act_scale(steps[r * groups + c / 32]));
      const float d = to_f32(dy[r * lddy + c]);
      return weight ? __fmul_rn(d, load_as_f32(weight, wtype, c)) : d;
    };
    float s = 0.0f;
    for (int64_t c = threadIdx.x; c < cols; c += NTHREADS) {
      float q;
      const float gw = terms(c, &q);
      s = __fmaf_rn(gw, q, s);
    }
    s = __fdiv_rn(cta_sum(s, red), (float)cols);
    const float rs = rstd[r];
    for (int64_t c = threadIdx.x; c < cols; c += NTHREADS) {
      float q;
      const float gw = terms(c, &q);
      float v = __fmul_rn(rs, __fmaf_rn(-q, s, gw));
      if (dh) v = __fadd_rn(v, to_f32(dh[r * lddh + c]));
      dx[r * lddx + c] = from_f32<T>(v);
    }
  }
}

// dw[c] over rows [p * span, (p + 1) * span) of part p: a thread per column.
template <typename T>
__global__ void __launch_bounds__(NTHREADS)
    k_rmsnorm_dw_wide(const T* dy, int64_t lddy, const int8_t* codes, const uint8_t* steps, int64_t rows, int64_t cols,
                      int64_t groups, int64_t span, float* part) {
  chain_wait();
  const int64_t c = (int64_t)blockIdx.x * NTHREADS + threadIdx.x;
  if (c >= cols) return;
  const int64_t r0 = blockIdx.y * span, r1 = min(r0 + span, rows);
  float s = 0.0f;
  for (int64_t r = r0; r < r1; ++r)
    s = __fmaf_rn(to_f32(dy[r * lddy + c]),
                  __fmul_rn((float)codes[r * groups * 32 + c], act_scale(steps[r * groups + c / 32])), s);
  part[blockIdx.y * groups * 32 + c] = s;
}

// ---------------------------------------------------------------- shapes
constexpr int NORM_SMS = 152;  // of a GB300

// Chunks per lane: two up to 8192 columns, four beyond; but four in the
// backward pass of 16-bit rows on 16-byte boundaries (up to 512 columns have
// one warp either way).
static int norm_chunks(int64_t cols, bool four) { return cols <= (four ? 512 : 8192) ? 2 : 4; }
// Warps: an even number with two chunks, half of it with four, so that both add
// up a row in the same order; as many as 1024 columns each take (5120 columns
// on 16 warps of two chunks took 202 us for 16384 rows, on ten 118).
static RowShape norm_shape(int64_t cols, int chunks) {
  RowShape s;
  s.warps = cols <= 512 ? 1 : (int)((cols + 1023) / 1024) * (chunks == 2 ? 2 : 1);
  s.threads = s.warps * (s.warps < 8 ? 8 / s.warps : 1) * 32;
  return s;
}
// CTAs: one per set of rows, at most `waves` times as many as the SMs hold,
// each SM `threads` threads.
static int norm_grid(int64_t rows, const RowShape& s, int threads, int waves) {
  const int per = s.threads / 32 / s.warps;
  const int64_t ctas = (rows + per - 1) / per, most = (int64_t)NORM_SMS * (threads / s.threads) * waves;
  return (int)(ctas < most ? ctas : most);
}
// Shared memory for the widest rows, asked for once per kernel and GPU.
template <auto KERN>
static bool allow_shared() {
  static PerDevice granted;
  return granted.get(current_device(), [] { return grant_shared(KERN, 232192) ? 1 : 0; }) != 0;
}
static int row_mode(int64_t cols, const RowShape& s, int chunks, bool vec) {
  if (!vec) return ROW_SPAN;
  return cols == (int64_t)s.warps * chunks * 256 ? ROW_FULL : ROW_CHUNKS;
}
template <int N>
struct Chunks {
  static constexpr int value = N;
};
// What the SMs hold by the kernels' registers: two waves forward (94 us for 16384 x 4096 in bf16; one wave 101, four 94), one
// backward, whose sums of dw grow with the CTAs.
static int forward_grid(int64_t rows, const RowShape& s, int chunks, int mode) {
  return norm_grid(rows, s, chunks == 2 && mode != ROW_SPAN ? THREADS_80 : THREADS_128, 2);
}
static int backward_grid(int64_t rows, const RowShape& s) { return norm_grid(rows, s, THREADS_128, 1); }
static int dw_parts(int64_t rows, int64_t cols) {
  if (rows < 1) return 1;
  if (cols > NORM_WIDEST) return (int)(rows < 64 ? rows : 64);
  const int two = backward_grid(rows, norm_shape(cols, norm_chunks(cols, false)));
  const int four = backward_grid(rows, norm_shape(cols, norm_chunks(cols, true)));
  return two > four ? two : four;
}

}  // namespace gc

using namespace gc;

extern "C" gc_status gc_rmsnorm(const void* x, int64_t ldx, const void* residual, int64_t ldr, int32_t dtype,
                                const void* weight, int32_t weight_dtype, float eps, int64_t rows, int64_t cols,
                                void* y, int64_t ldy, void* h, int64_t ldh, float* rstd, int8_t* codes,
                                uint8_t* steps, void* stream) {
  NvtxRange nvtx_range("gc_rmsnorm");
  gc_status st = validate_matrix(rows, cols, dtype);
  if (st != GC_OK) return st;
  if (!(eps >= 0.0f) || (weight && !valid_dtype(weight_dtype))) return GC_ERR_INVALID_ARG;
  if (rows == 0) return GC_OK;
  if ((st = check_matrix(x, ldx, cols, dtype)) != GC_OK ||
      (residual && (st = check_matrix(residual, ldr, cols, dtype)) != GC_OK) ||
      (y && (st = check_matrix(y, ldy, cols, dtype)) != GC_OK) ||
      (h && (st = check_matrix(h, ldh, cols, dtype)) != GC_OK) ||
      ((codes || steps) && (st = check_codes(codes, steps)) != GC_OK) ||
      (st = check_vector(weight, weight_dtype)) != GC_OK || (st = check_vector(rstd, GC_F32)) != GC_OK)
    return st;
  const int64_t groups = act_ldc(cols) / 32;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cols > NORM_WIDEST) {
    const unsigned grid = (unsigned)(rows < 152 * 64 ? rows : 152 * 64);
    GC_BY_DTYPE(dtype, T, launch_chained(k_rmsnorm_wide<T>, grid, NTHREADS, 0, s, static_cast<const T*>(x), ldx,
                                         static_cast<const T*>(residual), ldr, weight, weight_dtype, eps, rows, cols,
                                         groups, static_cast<T*>(y), ldy, static_cast<T*>(h), ldh, rstd, codes, steps));
    return cudaGetLastError() == cudaSuccess ? GC_OK : GC_ERR_CUDA;
  }
  const int chunks = norm_chunks(cols, false);
  const RowShape shape = norm_shape(cols, chunks);
  const bool vec = chunk_aligned(x, ldx, dtype) && (!residual || chunk_aligned(residual, ldr, dtype)) &&
                   (!y || chunk_aligned(y, ldy, dtype)) && (!h || chunk_aligned(h, ldh, dtype));
  const int mode = row_mode(cols, shape, chunks, vec);
  GC_BY_DTYPE(dtype, T, {
    auto go = [&](auto per_lane) -> bool {
      constexpr int N = decltype(per_lane)::value;
      constexpr bool ANY = sizeof(T) == 4;  // fp32 rows are spans always
      auto run = [&](auto kern, size_t ring) -> bool {
        launch_chained(kern, (unsigned)forward_grid(rows, shape, chunks, mode), shape.threads,
                       (size_t)groups * ACT_GROUP * sizeof(float) + ring, s, static_cast<const T*>(x), ldx,
                       static_cast<const T*>(residual), ldr, weight, weight_dtype, eps, rows, cols, groups, shape.warps,
                       static_cast<T*>(y), ldy, static_cast<T*>(h), ldh, rstd, codes, steps);
        return true;
      };
      constexpr int FULL = ANY ? ROW_SPAN : ROW_FULL, LANES = ANY ? ROW_SPAN : ROW_CHUNKS;
      if (mode == ROW_FULL) return allow_shared<k_rmsnorm<T, N, FULL>>() && run(k_rmsnorm<T, N, FULL>, RowShared<T, N, FULL>::forward(shape.threads));
      if (mode == ROW_CHUNKS) return allow_shared<k_rmsnorm<T, N, LANES>>() && run(k_rmsnorm<T, N, LANES>, RowShared<T, N, LANES>::forward(shape.threads));
      return allow_shared<k_rmsnorm<T, N, ROW_SPAN>>() && run(k_rmsnorm<T, N, ROW_SPAN>, RowShared<T, N, ROW_SPAN>::forward(shape.threads));
    };
    if (!(chunks == 2 ? go(Chunks<2>()) : go(Chunks<4>()))) return GC_ERR_CUDA;
  });
  return cudaGetLastError() == cudaSuccess ? GC_OK : GC_ERR_CUDA;
}

extern "C" gc_status gc_rmsnorm_backward_workspace_size(int64_t rows, int64_t cols, size_t* bytes) {
  const gc_status st = validate_matrix(rows, cols, GC_F32);
  if (st != GC_OK) return st;
  if (!bytes) return GC_ERR_INVALID_ARG;
  *bytes = (size_t)dw_parts(rows, cols) * (size_t)act_ldc(cols) * sizeof(float);
  return GC_OK;
}

extern "C" gc_status gc_rmsnorm_backward(const void* dy, int64_t lddy, const void* dh, int64_t lddh, int32_t dtype,
                                         const int8_t* codes, const uint8_t* steps, const float* rstd,
                                         const void* weight, int32_t weight_dtype, int64_t rows, int64_t cols,
                                         void* dx, int64_t lddx, float* dw, uint32_t flags, void* workspace,
                                         size_t ws_bytes, void* stream) {
  NvtxRange nvtx_range("gc_rmsnorm_backward");
  gc_status st = validate_matrix(rows, cols, dtype);
  if (st != GC_OK) return st;
  if ((weight && !valid_dtype(weight_dtype)) || (flags & ~GC_ACCUMULATE)) return GC_ERR_INVALID_ARG;
  if (dw) {
    size_t need = 0;
    gc_rmsnorm_backward_workspace_size(rows, cols, &need);
    if ((st = check_workspace(workspace, ws_bytes, need)) != GC_OK) return st;
    if ((st = check_vector(dw, GC_F32)) != GC_OK) return st;
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t groups = act_ldc(cols) / 32;
  const int acc = (flags & GC_ACCUMULATE) ? 1 : 0;
  float* part = dw ? static_cast<float*>(workspace) : nullptr;
  auto join = [&](int parts) {
    launch_chained(k_rmsnorm_dw_join, (unsigned)groups, 1024, 0, s, (const float*)part, parts, cols, groups * 32, dw, acc);
  };
  if (rows == 0) {
    if (dw && !acc) join(0);
    return cudaGetLastError() == cudaSuccess ? GC_OK : GC_ERR_CUDA;
  }
  if ((st = check_matrix(dy, lddy, cols, dtype)) != GC_OK || (dh && (st = check_matrix(dh, lddh, cols, dtype)) != GC_OK) ||
      (st = check_matrix(dx, lddx, cols, dtype)) != GC_OK || (st = check_codes(codes, steps)) != GC_OK ||
      (st = check_vector(weight, weight_dtype)) != GC_OK || (st = check_vector(rstd, GC_F32)) != GC_OK)
    return st;
  if (!rstd) return GC_ERR_INVALID_ARG;
  const int parts = dw_parts(rows, cols);
  if (cols > NORM_WIDEST) {
    const unsigned grid = (unsigned)(rows < 152 * 64 ? rows : 152 * 64);
    GC_BY_DTYPE(dtype, T, {
      if (dw) {  // before dx, which may overwrite dy
        launch_chained(k_rmsnorm_dw_wide<T>, dim3((unsigned)((cols + NTHREADS - 1) / NTHREADS), parts), NTHREADS, 0, s,
                       static_cast<const T*>(dy), lddy, codes, steps, rows, cols, groups, (rows + parts - 1) / parts, part);
        join(parts);
      }
      launch_chained(k_rmsnorm_backward_wide<T>, grid, NTHREADS, 0, s, static_cast<const T*>(dy), lddy,
                     static_cast<const T*>(dh), lddh, codes, steps, rstd, weight, weight_dtype, rows, cols, groups,
                     static_cast<T*>(dx), lddx);
    });
    return cudaGetLastError() == cudaSuccess ? GC_OK : GC_ERR_CUDA;
  }
  const bool vec = chunk_aligned(dy, lddy, dtype) && (!dh || chunk_aligned(dh, lddh, dtype)) && chunk_aligned(dx, lddx, dtype);
  const int chunks = norm_chunks(cols, vec);
  const RowShape shape = norm_shape(cols, chunks);
  const int grid = backward_grid(rows, shape);
  const int mode = row_mode(cols, shape, chunks, vec);
  GC_BY_DTYPE(dtype, T, {
    auto go = [&](auto per_lane) -> bool {
      constexpr int N = decltype(per_lane)::value;
      constexpr bool ANY = sizeof(T) == 4;  // fp32 rows are spans always
      auto run = [&](auto kern, size_t ring) -> bool {
        launch_chained(kern, (unsigned)grid, shape.threads,
                       (size_t)groups * ACT_GROUP * sizeof(float) + ring, s, static_cast<const T*>(dy), lddy,
                       static_cast<const T*>(dh), lddh, codes, steps, rstd, weight, weight_dtype, rows, cols, groups,
                       shape.warps, static_cast<T*>(dx), lddx, part);
        return true;
      };
      constexpr int FULL = ANY ? ROW_SPAN : ROW_FULL, LANES = ANY ? ROW_SPAN : ROW_CHUNKS;
      if (mode == ROW_FULL) return allow_shared<k_rmsnorm_backward<T, N, FULL>>() && run(k_rmsnorm_backward<T, N, FULL>, RowShared<T, N, FULL>::backward(shape.threads));
      if (mode == ROW_CHUNKS) return allow_shared<k_rmsnorm_backward<T, N, LANES>>() && run(k_rmsnorm_backward<T, N, LANES>, RowShared<T, N, LANES>::backward(shape.threads));
      return allow_shared<k_rmsnorm_backward<T, N, ROW_SPAN>>() && run(k_rmsnorm_backward<T, N, ROW_SPAN>, RowShared<T, N, ROW_SPAN>::backward(shape.threads));
    };
    if (!(chunks == 2 ? go(Chunks<2>()) : go(Chunks<4>()))) return GC_ERR_CUDA;
  });
  if (dw) join(grid);
  return cudaGetLastError() == cudaSuccess ? GC_OK : GC_ERR_CUDA;
}
