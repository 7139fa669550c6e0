// Normalisations around the layer, fused with the block's gate, residual scale
// and residual sum (sm_100a).
//
// For every row (token) of width D, with the residual stream r and a block's
// output o:
//   n  = o / sqrt(mean(o^2) + eps)                 (w_post given; else n = o)
//   r' = r + c * sg(a) * (n * w_post)              (c: scale, a: gate logits)
//   h  = r' / sqrt(mean(r'^2) + eps) * w_next      (the next block's input)
// and, given dr' and dh, the chain rule (mean over the row's D channels):
//   x  = r' rstd_next,  e = dh w_next,  G = dr' + rstd_next (e - x mean(e x))
//   dr = G,  A = sum over rows of G sg(a) n,  dscale = w_post A,
//   dw_post = c A,  dw_next = sum over rows of dh x,
//   da = G c n w_post sg(a)(1 - sg(a)),
//   f  = G c sg(a) w_post,  do = rstd_post (f - n mean(f n)).
// Both parameter gradients of the block need one sum A only: w_post and c do
// not depend on the row.
//
// Bound by memory: each stream is read once and each result written once, so
// a row stays in registers between its two reductions.  One CTA takes a row at a
// time, 16 bytes per thread and stream (4 bytes, or single elements, where D
// makes the rows unaligned), and walks over the rows with its columns' weights in
// registers.  Its next rows are on their way meanwhile: every thread copies its
// own pieces to shared memory asynchronously (so no barrier goes with them) and
// reads them back when their turn comes.  All statistics and sums in fp32, by the
// packed operations on two neighbouring channels (backward, 16384 x 4096: 209 us,
// 234 with single ones, whose instructions filled 60% of the cycles).
//
// Measured (device time, bf16, every part): forward 65536 x 4096 450 us, 6.0 TB/s;
// backward 16384 x 4096 205 us, 5.2 TB/s, 8192 x 768 28 us, 3.7 TB/s; one token 3.3
// us; fp32, 16384 x 4096: 241 and 430 us.  What keeps the backward below the copy rate: its sums and weights take the
// registers of all but 16 warps per SM, which two reductions a row stop in turn.
#include "common.cuh"
#include "f32x2.cuh"
#include "kernels.h"
#include "pdl.cuh"

namespace infini {

namespace {

constexpr int kSMs = 148;
constexpr int kMaxThreads = 512;
constexpr int kFwdThreads = 1024;  // threads per SM that the registers allow
constexpr int kBwdThreads = 512;   // (8192 x 768: 28 us; with 640, by fewer registers, 31)

template <int BYTES> struct RawVec;
template <> struct RawVec<2> { using type = unsigned short; };
template <> struct RawVec<4> { using type = unsigned int; };
template <> struct RawVec<16> { using type = uint4; };

// V consecutive elements of T, as loaded.
template <typename T, int V>
struct Pack {
  static constexpr int kBytes = V * (int)sizeof(T);
  typename RawVec<kBytes>::type raw;
  __device__ __forceinline__ void clear() { raw = {}; }
  static constexpr int kLanes = V > 1 ? V / 2 : 1;
  using L = typename LaneOf<V>::type;
  __device__ __forceinline__ L get(int i) const {
    if constexpr (V == 1) {
      return to_f32<T>(*reinterpret_cast<const T*>(&raw));
    } else if constexpr (sizeof(T) == 4) {
      return reinterpret_cast<const float2*>(&raw)[i];
    } else {
      const uint32_t w = reinterpret_cast<const uint32_t*>(&raw)[i];
      return {__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)};
    }
  }
  __device__ __forceinline__ void set(int i, L x) {
    if constexpr (V == 1) {
      *reinterpret_cast<T*>(&raw) = from_f32<T>(x);
    } else if constexpr (sizeof(T) == 4) {
      reinterpret_cast<float2*>(&raw)[i] = x;
    } else {
      const __nv_bfloat162 v = __floats2bfloat162_rn(x.x, x.y);
      reinterpret_cast<uint32_t*>(&raw)[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
  }
  __device__ __forceinline__ void store(void* base, size_t at) const {
    *reinterpret_cast<decltype(raw)*>(static_cast<T*>(base) + at) = raw;
  }
};

// A thread's pieces of a row's streams: N vectors of each of ARRAYS streams, with
// STAGES - 1 rows on their way (STAGES = 1: loaded when they are needed, which
// 2-byte pieces have to be).
template <typename T, int V, int N, int ARRAYS, int STAGES>
struct Streams {
  using P = Pack<T, V>;
  uint8_t* smem;                   // this thread's first piece
  const uint8_t* next[ARRAYS];     // its place in the row that is started next (null: not there, reads as zero)
  long long row;                   // that row
  int nvec;
  __device__ __forceinline__ Streams(uint8_t* ring, const void* const (&base)[ARRAYS], int width) {
    smem = ring + threadIdx.x * P::kBytes;
    nvec = width / V;
    row = blockIdx.x;
    const size_t off = ((size_t)row * width + (size_t)threadIdx.x * V) * sizeof(T);
#pragma unroll
    for (int a = 0; a < ARRAYS; ++a) next[a] = base[a] ? static_cast<const uint8_t*>(base[a]) + off : nullptr;
  }
  __device__ __forceinline__ uint8_t* at(int stage, int a, int i) const {
    return smem + (size_t)((stage * ARRAYS + a) * N + i) * blockDim.x * P::kBytes;
  }
  __device__ __forceinline__ void advance(size_t row_step) {
#pragma unroll
    for (int a = 0; a < ARRAYS; ++a)
      if (next[a]) next[a] += row_step;
    row += gridDim.x;
  }
  // Starts the next row's copies (row_step: bytes to the row after it).
  __device__ __forceinline__ void start(int stage, long long rows, size_t row_step) {
    if constexpr (STAGES > 1) {
      if (row < rows) {
#pragma unroll
        for (int a = 0; a < ARRAYS; ++a)
          if (next[a]) {
#pragma unroll
            for (int i = 0; i < N; ++i)
              if (threadIdx.x + i * blockDim.x < nvec) {
                const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(at(stage, a, i)));
                const uint8_t* from = next[a] + (size_t)i * blockDim.x * P::kBytes;
                if constexpr (P::kBytes == 16)
                  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
                else
                  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(from) : "memory");
              }
          }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
      advance(row_step);
    }
  }
  __device__ __forceinline__ static void wait() {
    if constexpr (STAGES > 1) asm volatile("cp.async.wait_group %0;" ::"n"(STAGES > 1 ? STAGES - 2 : 0) : "memory");
  }
  __device__ __forceinline__ void read(int stage, P (&x)[ARRAYS][N], size_t row_step) {
#pragma unroll
    for (int a = 0; a < ARRAYS; ++a)
#pragma unroll
      for (int i = 0; i < N; ++i) {
        x[a][i].clear();
        if (next[a] && threadIdx.x + i * blockDim.x < nvec) {
          const uint8_t* from = STAGES > 1 ? at(stage, a, i) : next[a] + (size_t)i * blockDim.x * P::kBytes;
          x[a][i].raw = *reinterpret_cast<const decltype(x[a][i].raw)*>(from);
        }
      }
    if constexpr (STAGES == 1) advance(row_step);
  }
};

// V consecutive fp32 weights; 1 where the vector is absent or `in` is false.
template <int V>
__device__ __forceinline__ void load_weights(const float* w, int at, bool in, float (&x)[V]) {
  if (w == nullptr || !in) {
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = 1.f;
  } else if constexpr (V % 4 == 0) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const float4 t = __ldg(reinterpret_cast<const float4*>(w + at + i));
      x[i] = t.x; x[i + 1] = t.y; x[i + 2] = t.z; x[i + 3] = t.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = __ldg(w + at + i);
  }
}

// A thread's columns of a weight vector: in registers for the kernel's whole life
// where MOST of them fit, read for every row otherwise.
template <int V, int N, int MOST>
struct Weights {
  static constexpr bool kKept = N * V <= MOST;
  const float *w, *times;  // times: a second vector, multiplied in
  float kept[kKept ? N : 1][V];
  __device__ __forceinline__ void read(int v, bool in, float (&x)[V]) const {
    load_weights<V>(w, v * V, in, x);
    if (times) {
      float y[V];
      load_weights<V>(times, v * V, in, y);
#pragma unroll
      for (int e = 0; e < V; ++e) x[e] *= y[e];
    }
  }
  __device__ __forceinline__ void load(const float* w_, int nvec, const float* times_ = nullptr) {
    w = w_;
    times = times_;
    if constexpr (kKept) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        read(v, v < nvec, kept[i]);
      }
    }
  }
  using L = typename LaneOf<V>::type;
  static constexpr int kLanes = V > 1 ? V / 2 : 1;
  __device__ __forceinline__ void get(int i, L (&x)[kLanes]) const {
    const auto lanes = [&](const float(&from)[V]) {
#pragma unroll
      for (int e = 0; e < kLanes; ++e) {
        if constexpr (V == 1) x[e] = from[0];
        else x[e] = {from[2 * e], from[2 * e + 1]};
      }
    };
    if constexpr (kKept) {
      lanes(kept[i]);
    } else {
      float now[V];
      read(threadIdx.x + i * blockDim.x, true, now);
      lanes(now);
    }
  }
};

__device__ __forceinline__ float ex2(float x) {
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(x));
  return x;
}
__device__ __forceinline__ float rcp(float x) {
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(x));
  return x;
}
__device__ __forceinline__ float ex2_lanes(float x) { return ex2(x); }
__device__ __forceinline__ float2 ex2_lanes(float2 x) { return {ex2(x.x), ex2(x.y)}; }
__device__ __forceinline__ float rcp_lanes(float x) { return rcp(x); }
__device__ __forceinline__ float2 rcp_lanes(float2 x) { return {rcp(x.x), rcp(x.y)}; }
__device__ __forceinline__ float most(float x, float y) { return fmaxf(x, y); }
__device__ __forceinline__ float2 most(float2 x, float y) { return {fmaxf(x.x, y), fmaxf(x.y, y)}; }
__device__ __forceinline__ float least(float x, float y) { return fminf(x, y); }
__device__ __forceinline__ float2 least(float2 x, float y) { return {fminf(x.x, y), fminf(x.y, y)}; }

// Logistic of a gate logit, u, and 1 - u (as e^-a u, which keeps its digits
// where u rounds to 1), by the hardware's approximations of 2^x (2^-22) and 1 / x (2^-23).
// 0 and 1 in the limits, NaN for NaN.  u is 0 from e^-a = 2^126 on, where 1 / x would be
// subnormal, and 1 - u is then wanted times u only; the bound keeps infinity times 0 out of it.
// The product a log2(e) is rounded to fp32, which e^-a feels |a| 2^-24 of: within 2^-17.5
// up to |a| = 88, little beside bf16's 2^-8.  EXACT (fp32 rows) puts its remainder back
// and keeps u to 2^-20.8 and 1 - u to 2^-20.
template <bool EXACT, typename L>
__device__ __forceinline__ L sigmoid(L a, L& rest) {
  const L y = mul(a, both<L>(-1.4426950408889634f));
  L t = ex2_lanes(y);
  if constexpr (EXACT) {
    // What the rounding of y and of log2(e) left, times ln 2.  (NaN or infinite where a or y
    // is infinite: some factor then that leaves 0 and infinity what they are.)
    const L left = fma(a, both<L>(-1.4426950408889634f), mul(y, both<L>(-1.f)));
    const L e = mul(fma(a, both<L>(-1.9259629911266175e-8f), left), both<L>(0.6931471805599453f));
    t = mul(t, add(least(most(e, -0.5f), 0.5f), both<L>(1.f)));
  }
  const L u = rcp_lanes(add(t, both<L>(1.f)));
  rest = mul(least(t, 0x1p126f), u);
  return u;
}

// Sum over the CTA, the same value in every thread.  `turn` alternates
// between two slots, so one barrier per sum is enough.
__device__ __forceinline__ float block_sum(float x, float (*slots)[32], int& turn) {
  x = warp_sum(x);
  const int nw = blockDim.x >> 5;
  if (nw == 1) return x;
  const int lane = threadIdx.x & 31;
  if (lane == 0) slots[turn][threadIdx.x >> 5] = x;
  __syncthreads();
  x = warp_sum(lane < nw ? slots[turn][lane] : 0.f);
  turn ^= 1;
  return x;
}

// Rows in flight: by a thread's bytes of one row, so that the rings of an SM's
// CTAs fit into its shared memory (512 threads of 96 bytes take 4 x 48 KB).
constexpr int stages_of(int bytes, bool copies) { return !copies ? 1 : bytes <= 96 ? 4 : bytes <= 192 ? 2 : 1; }

// (512 threads that hold one vector each: two CTAs an SM; the registers of wider
// rows leave room for one.)
template <typename T, int V, int N>
__global__ void __launch_bounds__(kMaxThreads, N == 1 ? 2 : 1)
block_norm_fwd_kernel(BlockNormProblem p) {
  constexpr int STAGES = stages_of(3 * N * V * (int)sizeof(T), V * sizeof(T) >= 4);
  __shared__ float slots[2][32];
  extern __shared__ __align__(16) uint8_t ring[];
  int turn = 0;
  const int D = p.width, nvec = D / V;
  const float inv_d = 1.f / (float)D;
  using S = Streams<T, V, N, 3, STAGES>;
  using L = typename S::P::L;
  constexpr int W = S::P::kLanes;
  const void* const from[3] = {p.r, p.o, p.gate};
  S in(ring, from, D);
  Weights<V, N, 16> wb, wn;  // wb: scale w_post
  wb.load(p.w_post, nvec, p.scale);
  wn.load(p.w_next, nvec);
  const size_t row_step = (size_t)gridDim.x * D * sizeof(T);
#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s) in.start(s, p.rows, row_step);
  int stage = 0;
  // This thread's first element of the row, from the start of an array.
  size_t here = (size_t)blockIdx.x * D + (size_t)threadIdx.x * V;
  for (long long row = blockIdx.x; row < p.rows; row += gridDim.x, here += (size_t)gridDim.x * D) {
    typename S::P raw[3][N];  // r, o, gate
    S::wait();
    in.read(stage, raw, row_step);
    in.start(stage > 0 ? stage - 1 : STAGES - 1, p.rows, row_step);
    stage = stage + 1 < STAGES ? stage + 1 : 0;
    L x[N][W];
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int e = 0; e < W; ++e) x[i][e] = raw[0][i].get(e);
    if (p.o) {
      float rp = 1.f;
      if (p.w_post) {
        L ss = both<L>(0.f);
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
          for (int e = 0; e < W; ++e) ss = fma(raw[1][i].get(e), raw[1][i].get(e), ss);
        rp = rsqrtf(block_sum(sum(ss), slots, turn) * inv_d + p.eps);
        if (p.rstd_post && threadIdx.x == 0) p.rstd_post[row] = rp;
      }
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        if (v < nvec) {
          L c[W];  // scale w_post
          wb.get(i, c);
          typename S::P out;
#pragma unroll
          for (int e = 0; e < W; ++e) {
            L rest;
            const L n = mul(raw[1][i].get(e), both<L>(rp));
            x[i][e] = fma(n, p.gate ? mul(sigmoid<sizeof(T) == 4>(raw[2][i].get(e), rest), c[e]) : c[e], x[i][e]);
            out.set(e, x[i][e]);
          }
          out.store(p.r_out, here + (size_t)i * blockDim.x * V);
        }
      }
    }
    if (p.w_next) {
      // The norm of the sum before its rounding to T: h is as near the
      // formula as its own type allows.
      L ss = both<L>(0.f);
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int e = 0; e < W; ++e) ss = fma(x[i][e], x[i][e], ss);
      const float rn = rsqrtf(block_sum(sum(ss), slots, turn) * inv_d + p.eps);
      if (p.rstd_next && threadIdx.x == 0) p.rstd_next[row] = rn;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        if (v < nvec) {
          L next[W];
          wn.get(i, next);
          typename S::P out;
#pragma unroll
          for (int e = 0; e < W; ++e) out.set(e, mul(mul(x[i][e], both<L>(rn)), next[e]));
          out.store(p.h, here + (size_t)i * blockDim.x * V);
        }
      }
    }
  }
}

template <typename T, int V, int N>
__global__ void __launch_bounds__(kMaxThreads, 1)
block_norm_bwd_kernel(BlockNormProblem p) {
  constexpr int STAGES = stages_of(5 * N * V * (int)sizeof(T), V * sizeof(T) >= 4);
  __shared__ float slots[2][32];
  extern __shared__ __align__(16) uint8_t ring[];
  int turn = 0;
  const int D = p.width, nvec = D / V;
  const float inv_d = 1.f / (float)D;
  const bool want_a = p.scale || p.w_post;
  using S = Streams<T, V, N, 5, STAGES>;
  using L = typename S::P::L;
  constexpr int W = S::P::kLanes;
  const void* const from[5] = {p.dr_out, p.dh, p.w_next ? p.r : nullptr, p.o, p.gate};
  S in(ring, from, D);
  Weights<V, N, 8> wb, wn;  // (the sums take as many registers); wb: scale w_post
  wb.load(p.w_post, nvec, p.scale);
  wn.load(p.w_next, nvec);
  L acc_n[N][W], acc_a[N][W];  // this CTA's rows' shares of dw_next and A
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int e = 0; e < W; ++e) acc_n[i][e] = acc_a[i][e] = both<L>(0.f);
  const size_t row_step = (size_t)gridDim.x * D * sizeof(T);
#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s) in.start(s, p.rows, row_step);
  int stage = 0;
  float rn_next = p.w_next ? p.rstd_next[blockIdx.x] : 0.f, rp_next = p.w_post ? p.rstd_post[blockIdx.x] : 1.f;
  // This thread's first element of the row, from the start of an array.
  size_t here = (size_t)blockIdx.x * D + (size_t)threadIdx.x * V;
  for (long long row = blockIdx.x; row < p.rows; row += gridDim.x, here += (size_t)gridDim.x * D) {
    typename S::P raw[5][N];  // dr_out, dh, r_out, o, gate
    const float rn = rn_next, rp = rp_next;
    if (row + gridDim.x < p.rows) {
      if (p.w_next) rn_next = p.rstd_next[row + gridDim.x];
      if (p.w_post) rp_next = p.rstd_post[row + gridDim.x];
    }
    S::wait();
    in.read(stage, raw, row_step);
    in.start(stage > 0 ? stage - 1 : STAGES - 1, p.rows, row_step);
    stage = stage + 1 < STAGES ? stage + 1 : 0;
    L G[N][W];
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int e = 0; e < W; ++e) G[i][e] = raw[0][i].get(e);
    if (p.w_next) {
      L dot = both<L>(0.f);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (threadIdx.x + i * blockDim.x < nvec) {
          L next[W];
          wn.get(i, next);
#pragma unroll
          for (int e = 0; e < W; ++e) {
            const L n = mul(raw[2][i].get(e), both<L>(rn)), dh = raw[1][i].get(e);
            acc_n[i][e] = fma(dh, n, acc_n[i][e]);
            dot = fma(mul(dh, next[e]), n, dot);
          }
        }
      }
      const float m = block_sum(sum(dot), slots, turn) * inv_d;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        if (v < nvec) {
          L next[W];
          wn.get(i, next);
          typename S::P out;
#pragma unroll
          for (int e = 0; e < W; ++e) {
            const L n = mul(raw[2][i].get(e), both<L>(rn));
            G[i][e] = fma(both<L>(rn), fma(n, both<L>(-m), mul(raw[1][i].get(e), next[e])), G[i][e]);
            out.set(e, G[i][e]);
          }
          out.store(p.dr, here + (size_t)i * blockDim.x * V);
        }
      }
    }
    if (p.o) {
      L f[N][W], dot = both<L>(0.f);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        if (v < nvec) {
          L c[W];  // scale w_post
          wb.get(i, c);
          typename S::P da;
#pragma unroll
          for (int e = 0; e < W; ++e) {
            L rest = both<L>(0.f), gu = G[i][e];
            if (p.gate) gu = mul(gu, sigmoid<sizeof(T) == 4>(raw[4][i].get(e), rest));
            const L n = mul(raw[3][i].get(e), both<L>(rp));
            acc_a[i][e] = fma(gu, n, acc_a[i][e]);
            f[i][e] = mul(gu, c[e]);
            const L fn = mul(f[i][e], n);
            dot = add(dot, fn);
            if (p.gate) da.set(e, mul(fn, rest));
          }
          if (p.gate) da.store(p.dgate, here + (size_t)i * blockDim.x * V);
        } else {
#pragma unroll
          for (int e = 0; e < W; ++e) f[i][e] = both<L>(0.f);
        }
      }
      if (p.w_post) {
        const float m = block_sum(sum(dot), slots, turn) * inv_d;
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
          for (int e = 0; e < W; ++e)
            f[i][e] = mul(both<L>(rp), fma(mul(raw[3][i].get(e), both<L>(rp)), both<L>(-m), f[i][e]));
      }
      // (Without the norm do does not depend on o: f, and not f - o 0, NaN for an infinite o.)
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        if (v < nvec) {
          typename S::P out;
#pragma unroll
          for (int e = 0; e < W; ++e) out.set(e, f[i][e]);
          out.store(p.d_o, here + (size_t)i * blockDim.x * V);
        }
      }
    }
  }
  // Partials [CTA][2][D]; the second kernel adds them in CTA order.
  float* part = p.part + (size_t)blockIdx.x * 2 * D;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    if (v < nvec) {
#pragma unroll
      for (int e = 0; e < W; ++e) {
        if (p.w_next) put(part + v * V, e, acc_n[i][e]);
        if (want_a) put(part + D + v * V, e, acc_a[i][e]);
      }
    }
  }
  pdl_trigger();
}

// Column sums of the partials, in a fixed order: thread (x, y) adds every
// kSumRows-th CTA's share of its column, then a warp adds a column's kSumRows sums.
// 8 columns a CTA (a 32-byte sector of each partial), so that narrow rows still
// spread over the GPU and no thread adds more than 37 values.
constexpr int kSumCols = 8, kSumRows = 64;

__global__ void __launch_bounds__(kSumCols * kSumRows)
block_norm_reduce_kernel(BlockNormProblem p, int n_part) {
  __shared__ float sums[kSumRows][kSumCols + 1];
  pdl_wait();
  const int D = p.width;
  const int col = blockIdx.x * kSumCols + threadIdx.x;
  const bool second = blockIdx.y == 1;  // 0: dw_next, 1: A
  float s = 0.f;
  if (col < D && (second ? (p.scale || p.w_post) : p.w_next != nullptr)) {
    const float* part = p.part + (second ? D : 0) + col;
    constexpr int kU = 12;  // in flight together
    for (int c0 = threadIdx.y; c0 < n_part; c0 += kU * kSumRows) {
      float v[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int c = c0 + u * kSumRows;
        v[u] = c < n_part ? __ldcg(part + (size_t)c * 2 * D) : 0.f;
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) s += v[u];
    }
  }
  sums[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  const int t = threadIdx.y * kSumCols + threadIdx.x, lane = t & 31, warp = t >> 5;
  if (warp >= kSumCols) return;
  const float total = warp_sum(sums[lane][warp] + sums[lane + 32][warp]);
  const int out = blockIdx.x * kSumCols + warp;
  if (lane != 0 || out >= D) return;
  if (!second) {
    if (p.dw_next) p.dw_next[out] = total;
  } else {
    if (p.dscale) p.dscale[out] = p.w_post ? total * p.w_post[out] : total;
    if (p.dw_post) p.dw_post[out] = p.scale ? total * p.scale[out] : total;
  }
}

struct Shape {
  int vec, n, threads, per_sm;
  size_t smem;
};

// The widest pieces that the rows' alignment allows; as few of them per thread as
// kMaxThreads threads need (a power of two); as many CTAs per SM as `sm_threads`
// threads are (registers), at most 16.  One piece a thread up to 512 threads, not
// two from 256 threads on: 65536 x 4096 bf16 forward 462 us against 486, 16384 x
// 4096 backward 209 against 249.
Shape row_shape(int width, int elem, int arrays, int sm_threads) {
  Shape s;
  const int bytes = (width * elem) % 16 == 0 ? 16 : (width * elem) % 4 == 0 ? 4 : 2;
  s.vec = bytes / elem;
  const int nvec = width / s.vec;
  s.n = 1;
  while (s.n * kMaxThreads < nvec) s.n *= 2;
  s.threads = ((nvec + s.n - 1) / s.n + 31) / 32 * 32;
  s.per_sm = sm_threads / (s.n > 1 && sm_threads > kMaxThreads ? 2 : 1) / s.threads;
  s.per_sm = s.per_sm < 1 ? 1 : s.per_sm > 16 ? 16 : s.per_sm;
  const int piece = arrays * s.n * bytes, stages = stages_of(piece, bytes >= 4);
  s.smem = stages > 1 ? (size_t)piece * s.threads * stages : 0;
  return s;
}

int row_grid(long long rows, const Shape& s) {
  const long long most = (long long)kSMs * s.per_sm;
  return (int)(rows < most ? rows : most);
}

// The limit of a kernel's shared memory belongs to the kernel, not to the call: it is set
// to the most that any width asks of this instance (PIECE: a thread's bytes of a row), the
// same value by every host thread.
template <int PIECE, bool COPIES, typename K>
cudaError_t run(K kernel, const BlockNormProblem& p, const Shape& s, cudaStream_t st) {
  constexpr int stages = stages_of(PIECE, COPIES), most = stages > 1 ? PIECE * kMaxThreads * stages : 0;
  if (most + 1024 > 48 * 1024) {  // (some of the default is the sums')
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e != cudaSuccess) return e;
  }
  kernel<<<row_grid(p.rows, s), s.threads, s.smem, st>>>(p);
  return cudaGetLastError();
}

template <bool BWD, typename T, int V, int N>
cudaError_t launch_n(const BlockNormProblem& p, const Shape& s, cudaStream_t st) {
  constexpr int bytes = V * (int)sizeof(T);
  if constexpr (BWD) return run<5 * N * bytes, bytes >= 4>(block_norm_bwd_kernel<T, V, N>, p, s, st);
  else return run<3 * N * bytes, bytes >= 4>(block_norm_fwd_kernel<T, V, N>, p, s, st);
}

template <bool BWD, typename T, int V>
cudaError_t launch_v(const BlockNormProblem& p, const Shape& s, cudaStream_t st) {
  constexpr int kMost = kBlockNormMaxWidth / V / kMaxThreads;  // vectors per thread
  switch (s.n) {
    case 1: return launch_n<BWD, T, V, 1>(p, s, st);
    case 2: return launch_n<BWD, T, V, 2>(p, s, st);
    case 4: return launch_n<BWD, T, V, 4>(p, s, st);
    case 8: if constexpr (kMost >= 8) return launch_n<BWD, T, V, 8>(p, s, st); else break;
    case 16: if constexpr (kMost >= 16) return launch_n<BWD, T, V, 16>(p, s, st); else break;
    case 32: if constexpr (kMost >= 32) return launch_n<BWD, T, V, 32>(p, s, st); else break;
  }
  return cudaErrorInvalidValue;
}

template <bool BWD>
cudaError_t launch_any(const BlockNormProblem& p, const Shape& s, cudaStream_t st) {
  if (p.bf16) {
    if (s.vec == 8) return launch_v<BWD, __nv_bfloat16, 8>(p, s, st);
    if (s.vec == 2) return launch_v<BWD, __nv_bfloat16, 2>(p, s, st);
    return launch_v<BWD, __nv_bfloat16, 1>(p, s, st);
  }
  return s.vec == 4 ? launch_v<BWD, float, 4>(p, s, st) : launch_v<BWD, float, 1>(p, s, st);
}

Shape fwd_shape(int width, int elem) { return row_shape(width, elem, 3, kFwdThreads); }
Shape bwd_shape(int width, int elem) { return row_shape(width, elem, 5, kBwdThreads); }

}  // namespace

bool block_norm_supported(int width) { return width >= 1 && width <= kBlockNormMaxWidth; }

int block_norm_partials(long long rows, int width) {
  // The most that either element type needs.
  const int a = row_grid(rows, bwd_shape(width, 2)), b = row_grid(rows, bwd_shape(width, 4));
  return a > b ? a : b;
}

cudaError_t launch_block_norm_forward(const BlockNormProblem& p, cudaStream_t st) {
  return launch_any<false>(p, fwd_shape(p.width, p.bf16 ? 2 : 4), st);
}

cudaError_t launch_block_norm_backward(const BlockNormProblem& p, cudaStream_t st) {
  const Shape s = bwd_shape(p.width, p.bf16 ? 2 : 4);
  const cudaError_t e = launch_any<true>(p, s, st);
  if (e != cudaSuccess || !(p.w_next || p.scale || p.w_post)) return e;
  return launch_pdl(true, block_norm_reduce_kernel, dim3((p.width + kSumCols - 1) / kSumCols, 2),
                    dim3(kSumCols, kSumRows), 0, st, p,
                    row_grid(p.rows, s));
}

}  // namespace infini
