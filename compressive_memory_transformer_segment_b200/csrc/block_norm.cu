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
// a row stays in registers between its two reductions.  One CTA per row at a
// time, 16 bytes per thread and stream (element by element where D makes the
// rows unaligned); every statistic and sum in fp32.
#include "common.cuh"
#include "kernels.h"
#include "pdl.cuh"

namespace infini {

namespace {

constexpr int kSMs = 148;
constexpr int kMaxThreads = 512;
constexpr int kRegThreads = 512;  // threads per SM at the backward's register count

template <int BYTES> struct RawVec;
template <> struct RawVec<2> { using type = unsigned short; };
template <> struct RawVec<4> { using type = unsigned int; };
template <> struct RawVec<16> { using type = uint4; };

// Streams pass through once: they stay out of L1, which keeps the weights.
__device__ __forceinline__ void ld_stream(const void* p, uint4& r) {
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
}
__device__ __forceinline__ void ld_stream(const void* p, unsigned int& r) {
  asm volatile("ld.global.L1::no_allocate.u32 %0, [%1];" : "=r"(r) : "l"(p));
}
__device__ __forceinline__ void ld_stream(const void* p, unsigned short& r) {
  asm volatile("ld.global.L1::no_allocate.u16 %0, [%1];" : "=h"(r) : "l"(p));
}

// V consecutive elements of T, as loaded.
template <typename T, int V>
struct Pack {
  typename RawVec<V * (int)sizeof(T)>::type raw;
  __device__ __forceinline__ void load(const void* base, size_t at) {
    ld_stream(static_cast<const T*>(base) + at, raw);
  }
  __device__ __forceinline__ void clear() { raw = {}; }
  __device__ __forceinline__ float get(int i) const {
    return to_f32<T>(reinterpret_cast<const T*>(&raw)[i]);
  }
  __device__ __forceinline__ void set(int i, float x) { reinterpret_cast<T*>(&raw)[i] = from_f32<T>(x); }
  __device__ __forceinline__ void store(void* base, size_t at) const {
    *reinterpret_cast<decltype(raw)*>(static_cast<T*>(base) + at) = raw;
  }
};

// V consecutive fp32 weights; 1 where the vector is absent.
template <int V>
__device__ __forceinline__ void load_weights(const float* w, int at, float (&x)[V]) {
  if (w == nullptr) {
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

// Logistic of a gate logit, u, and 1 - u (as e^-a u, which keeps its digits
// where u rounds to 1).  0 and 1 in the limits, NaN for NaN; the bound only
// keeps infinity times 0 out of 1 - u, where u is 0 and wanted as such.
__device__ __forceinline__ float sigmoid(float a, float& rest) {
  const float t = __expf(-a);
  const float u = __fdividef(1.f, 1.f + t);
  rest = fminf(t, 1e30f) * u;
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

template <typename T, int V, int N>
__global__ void __launch_bounds__(kMaxThreads)
block_norm_fwd_kernel(BlockNormProblem p) {
  __shared__ float slots[2][32];
  int turn = 0;
  const int D = p.width, nvec = D / V;
  const float inv_d = 1.f / (float)D;
  for (long long row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const size_t base = (size_t)row * D;
    Pack<T, V> r[N], o[N], a[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      r[i].clear(); o[i].clear(); a[i].clear();
      if (v < nvec) {
        r[i].load(p.r, base + (size_t)v * V);
        if (p.o) o[i].load(p.o, base + (size_t)v * V);
        if (p.gate) a[i].load(p.gate, base + (size_t)v * V);
      }
    }
    float x[N][V];
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int e = 0; e < V; ++e) x[i][e] = r[i].get(e);
    if (p.o) {
      float rp = 1.f;
      if (p.w_post) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
          for (int e = 0; e < V; ++e) ss = fmaf(o[i].get(e), o[i].get(e), ss);
        rp = rsqrtf(block_sum(ss, slots, turn) * inv_d + p.eps);
        if (p.rstd_post && threadIdx.x == 0) p.rstd_post[row] = rp;
      }
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        if (v < nvec) {
          float wp[V], c[V];
          load_weights<V>(p.w_post, v * V, wp);
          load_weights<V>(p.scale, v * V, c);
          Pack<T, V> out;
#pragma unroll
          for (int e = 0; e < V; ++e) {
            float rest;
            const float u = p.gate ? sigmoid(a[i].get(e), rest) : 1.f;
            x[i][e] = fmaf(o[i].get(e) * rp * wp[e], u * c[e], x[i][e]);
            out.set(e, x[i][e]);
          }
          out.store(p.r_out, base + (size_t)v * V);
        }
      }
    }
    if (p.w_next) {
      // The norm of the sum before its rounding to T: h is as near the
      // formula as its own type allows.
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e) ss = fmaf(x[i][e], x[i][e], ss);
      const float rn = rsqrtf(block_sum(ss, slots, turn) * inv_d + p.eps);
      if (p.rstd_next && threadIdx.x == 0) p.rstd_next[row] = rn;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        if (v < nvec) {
          float wn[V];
          load_weights<V>(p.w_next, v * V, wn);
          Pack<T, V> out;
#pragma unroll
          for (int e = 0; e < V; ++e) out.set(e, x[i][e] * rn * wn[e]);
          out.store(p.h, base + (size_t)v * V);
        }
      }
    }
  }
}

// One row's streams of the backward.
template <typename T, int V, int N>
struct BwdRow {
  Pack<T, V> dr[N], dh[N], x[N], o[N], a[N];
  __device__ __forceinline__ void load(const BlockNormProblem& p, long long row, int nvec) {
    const size_t base = (size_t)row * p.width;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      dr[i].clear(); dh[i].clear(); x[i].clear(); o[i].clear(); a[i].clear();
      if (v < nvec) {
        const size_t at = base + (size_t)v * V;
        if (p.dr_out) dr[i].load(p.dr_out, at);
        if (p.w_next) {
          dh[i].load(p.dh, at);
          x[i].load(p.r, at);
        }
        if (p.o) o[i].load(p.o, at);
        if (p.gate) a[i].load(p.gate, at);
      }
    }
  }
};

template <typename T, int V, int N>
__global__ void __launch_bounds__(kMaxThreads, 1)
block_norm_bwd_kernel(BlockNormProblem p) {
  __shared__ float slots[2][32];
  int turn = 0;
  const int D = p.width, nvec = D / V;
  const float inv_d = 1.f / (float)D;
  const bool want_a = p.scale || p.w_post;
  float acc_n[N][V], acc_a[N][V];  // this CTA's rows' shares of dw_next and A
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int e = 0; e < V; ++e) acc_n[i][e] = acc_a[i][e] = 0.f;

  BwdRow<T, V, N> cur;
  if (blockIdx.x < p.rows) cur.load(p, blockIdx.x, nvec);
  for (long long row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const size_t base = (size_t)row * D;
    float G[N][V];
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int e = 0; e < V; ++e) G[i][e] = cur.dr[i].get(e);
    if (p.w_next) {
      const float rn = p.rstd_next[row];
      float dot = 0.f;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        if (v < nvec) {
          float wn[V];
          load_weights<V>(p.w_next, v * V, wn);
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const float n = cur.x[i].get(e) * rn, dh = cur.dh[i].get(e);
            acc_n[i][e] = fmaf(dh, n, acc_n[i][e]);
            dot = fmaf(dh * wn[e], n, dot);
          }
        }
      }
      const float m = block_sum(dot, slots, turn) * inv_d;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        if (v < nvec) {
          float wn[V];
          load_weights<V>(p.w_next, v * V, wn);
          Pack<T, V> out;
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const float n = cur.x[i].get(e) * rn;
            G[i][e] = fmaf(rn, fmaf(-n, m, cur.dh[i].get(e) * wn[e]), G[i][e]);
            out.set(e, G[i][e]);
          }
          out.store(p.dr, base + (size_t)v * V);
        }
      }
    }
    if (p.o) {
      const float rp = p.w_post ? p.rstd_post[row] : 1.f;
      float f[N][V], dot = 0.f;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        if (v < nvec) {
          float wp[V], c[V];
          load_weights<V>(p.w_post, v * V, wp);
          load_weights<V>(p.scale, v * V, c);
          Pack<T, V> da;
#pragma unroll
          for (int e = 0; e < V; ++e) {
            float rest = 0.f;
            const float u = p.gate ? sigmoid(cur.a[i].get(e), rest) : 1.f;
            const float n = cur.o[i].get(e) * rp;
            const float gu = G[i][e] * u;
            acc_a[i][e] = fmaf(gu, n, acc_a[i][e]);
            f[i][e] = gu * c[e] * wp[e];
            dot = fmaf(f[i][e], n, dot);
            da.set(e, f[i][e] * n * rest);
          }
          if (p.gate) da.store(p.dgate, base + (size_t)v * V);
        } else {
#pragma unroll
          for (int e = 0; e < V; ++e) f[i][e] = 0.f;
        }
      }
      float m = 0.f;
      if (p.w_post) m = block_sum(dot, slots, turn) * inv_d;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        if (v < nvec) {
          Pack<T, V> out;
#pragma unroll
          for (int e = 0; e < V; ++e)
            out.set(e, rp * fmaf(-(cur.o[i].get(e) * rp), m, f[i][e]));
          out.store(p.d_o, base + (size_t)v * V);
        }
      }
    }
    if (row + gridDim.x < p.rows) cur.load(p, row + gridDim.x, nvec);
  }
  // Partials [CTA][2][D]; the second kernel adds them in CTA order.
  float* part = p.part + (size_t)blockIdx.x * 2 * D;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    if (v < nvec) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        if (p.w_next) part[v * V + e] = acc_n[i][e];
        if (want_a) part[D + v * V + e] = acc_a[i][e];
      }
    }
  }
  pdl_trigger();
}

// Column sums of the partials, in a fixed order: thread (x, y) adds every
// 32nd CTA's share of its column, then the 32 sums are added in turn.
__global__ void __launch_bounds__(1024)
block_norm_reduce_kernel(BlockNormProblem p, int n_part) {
  __shared__ float sums[32][33];
  pdl_wait();
  const int D = p.width;
  const int col = blockIdx.x * 32 + threadIdx.x;
  const bool second = blockIdx.y == 1;  // 0: dw_next, 1: A
  float s = 0.f;
  if (col < D && (second ? (p.scale || p.w_post) : p.w_next != nullptr)) {
    const float* part = p.part + (second ? D : 0) + col;
#pragma unroll 8
    for (int c = threadIdx.y; c < n_part; c += 32) s += __ldcg(part + (size_t)c * 2 * D);
  }
  sums[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  // One warp per column: rows of `sums` transposed, so a warp adds 32 values.
  const float total = warp_sum(sums[threadIdx.x][threadIdx.y]);
  const int out = blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x != 0 || out >= D) return;
  if (!second) {
    if (p.dw_next) p.dw_next[out] = total;
  } else {
    if (p.dscale) p.dscale[out] = p.w_post ? total * p.w_post[out] : total;
    if (p.dw_post) p.dw_post[out] = p.scale ? total * p.scale[out] : total;
  }
}

// Threads of a CTA for rows of nvec vectors, N vectors per thread.
int row_threads(int nvec, int n) {
  const int t = ((nvec + n - 1) / n + 31) / 32 * 32;
  return t < kMaxThreads ? t : kMaxThreads;
}

struct Shape {
  int vec, n, threads;
};

// 16-byte vectors where the rows are 16-byte aligned, single elements
// otherwise; as few vectors per thread as kMaxThreads threads need.
Shape row_shape(int width, int elem) {
  Shape s;
  s.vec = (width * elem) % 16 == 0 ? 16 / elem : 1;
  const int nvec = width / s.vec;
  s.n = 1;
  while (s.n * kMaxThreads < nvec) s.n *= 2;
  s.threads = row_threads(nvec, s.n);
  return s;
}

template <typename T, int V>
cudaError_t launch_fwd(const BlockNormProblem& p, const Shape& s, cudaStream_t st) {
  const unsigned grid = (unsigned)(p.rows < 0x7fffffffLL ? p.rows : 0x7fffffffLL);
  switch (s.n) {
    case 1: block_norm_fwd_kernel<T, V, 1><<<grid, s.threads, 0, st>>>(p); break;
    case 2: block_norm_fwd_kernel<T, V, 2><<<grid, s.threads, 0, st>>>(p); break;
    case 4: block_norm_fwd_kernel<T, V, 4><<<grid, s.threads, 0, st>>>(p); break;
    default:
      if constexpr (V <= 4) {
        if (s.n == 8) { block_norm_fwd_kernel<T, V, 8><<<grid, s.threads, 0, st>>>(p); break; }
      }
      if constexpr (V == 1) {
        if (s.n == 16) { block_norm_fwd_kernel<T, V, 16><<<grid, s.threads, 0, st>>>(p); break; }
        if (s.n == 32) { block_norm_fwd_kernel<T, V, 32><<<grid, s.threads, 0, st>>>(p); break; }
      }
      return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

template <typename T, int V>
cudaError_t launch_bwd(const BlockNormProblem& p, const Shape& s, int grid, cudaStream_t st) {
  switch (s.n) {
    case 1: block_norm_bwd_kernel<T, V, 1><<<grid, s.threads, 0, st>>>(p); break;
    case 2: block_norm_bwd_kernel<T, V, 2><<<grid, s.threads, 0, st>>>(p); break;
    case 4: block_norm_bwd_kernel<T, V, 4><<<grid, s.threads, 0, st>>>(p); break;
    default:
      if constexpr (V <= 4) {
        if (s.n == 8) { block_norm_bwd_kernel<T, V, 8><<<grid, s.threads, 0, st>>>(p); break; }
      }
      if constexpr (V == 1) {
        if (s.n == 16) { block_norm_bwd_kernel<T, V, 16><<<grid, s.threads, 0, st>>>(p); break; }
        if (s.n == 32) { block_norm_bwd_kernel<T, V, 32><<<grid, s.threads, 0, st>>>(p); break; }
      }
      return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

int bwd_grid(long long rows, int threads) {
  const int per_sm = kRegThreads / threads;
  const long long most = (long long)kSMs * (per_sm < 1 ? 1 : per_sm);
  return (int)(rows < most ? rows : most);
}

}  // namespace

bool block_norm_supported(int width) { return width >= 1 && width <= kBlockNormMaxWidth; }

int block_norm_partials(long long rows, int width) {
  // The most that any element type and alignment of this width needs.
  int most = 0;
  for (int elem = 2; elem <= 4; elem += 2) {
    const int g = bwd_grid(rows, row_shape(width, elem).threads);
    most = g > most ? g : most;
  }
  return most;
}

cudaError_t launch_block_norm_forward(const BlockNormProblem& p, cudaStream_t st) {
  const Shape s = row_shape(p.width, p.bf16 ? 2 : 4);
  if (p.bf16)
    return s.vec > 1 ? launch_fwd<__nv_bfloat16, 8>(p, s, st) : launch_fwd<__nv_bfloat16, 1>(p, s, st);
  return s.vec > 1 ? launch_fwd<float, 4>(p, s, st) : launch_fwd<float, 1>(p, s, st);
}

cudaError_t launch_block_norm_backward(const BlockNormProblem& p, cudaStream_t st) {
  const Shape s = row_shape(p.width, p.bf16 ? 2 : 4);
  const int grid = bwd_grid(p.rows, s.threads);
  cudaError_t e;
  if (p.bf16)
    e = s.vec > 1 ? launch_bwd<__nv_bfloat16, 8>(p, s, grid, st) : launch_bwd<__nv_bfloat16, 1>(p, s, grid, st);
  else
    e = s.vec > 1 ? launch_bwd<float, 4>(p, s, grid, st) : launch_bwd<float, 1>(p, s, grid, st);
  if (e != cudaSuccess || !(p.w_next || p.scale || p.w_post)) return e;
  return launch_pdl(true, block_norm_reduce_kernel, dim3((p.width + 31) / 32, 2), dim3(32, 32), 0, st, p,
                    grid);
}

}  // namespace infini
