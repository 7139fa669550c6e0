// Decode step over a segment buffer held in 4 bits (sm_100a).
//
// The streaming decode step of decode.cu with the current segment's keys and
// values as 4-bit codes: in groups of 32 channels, value = s q + m with q in
// 0..15 and bf16 s (scale) and m (minimum).  For the query heads h of one KV
// head (groups j of channels):
//   score_r = sum_j s_rj (sum over j of q_r x) + m_rj (sum over j of x),
//   a_dot   = sum_r p_r v_r / sum_r p_r,
//   sum_r p_r v_r[e] = sum_r (p_r s_rj) q_r[e] + sum_r p_r m_rj   (e in group j)
// so both products run over the codes themselves (integers, exact in bf16) on
// the tensor cores, with the scales on the outside of the first and folded
// into the probabilities of the second.  Probabilities times scale are
// rounded to bf16 for bf16 heads (2^-8 of each term, as in the bf16 forward);
// fp32 heads carry queries and probabilities as three bf16 parts each.
//
// Bound by the buffer's bytes (5 bits per value): with 4 query heads per KV
// head a CUDA-core version would need 8 multiply-adds per value besides the
// conversions, about 1.5 times what the memory allows; as matrix products
// (16 rows x 8 heads, mma.sync) the arithmetic is left to the conversions.
// One warp takes 16 rows at a time:
//   S^T = K Q^T   rows of codes are the A operand (lane 4 i + c: rows i, i + 8),
//   O^T = V^T P^T V's codes are the A operand with the rows along k, P^T the
//                 B operand: the scores' fragments, transposed in registers.
// The buffer's layout is such that a lane's fragments are one contiguous load
// per row (see the header), so rows go from global memory to the tensor cores
// without shared memory; the next 16 rows are loaded while these are used.
//
// Grid: CTA 0 of a (batch row, KV head, chunk of 8 query heads) reads the
// memory (sigma(q) M, sigma(q) z), the others up to `chunk` rows each; the
// last one of them to finish (a ticket) merges and writes the output.  The
// number of rows is read from device memory, so one captured launch serves
// every position.
#include "common.cuh"
#include "kernels.h"
#include "q4_common.cuh"

namespace infini {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kHeads = 8;               // query heads of a CTA (columns of a product)
constexpr int kUnit = kWarps * 16;      // rows a CTA takes at a time
constexpr int kSMs = 148;

template <int BYTES> struct RawBytes;
template <> struct RawBytes<2> { using type = unsigned short; };
template <> struct RawBytes<4> { using type = uint32_t; };
template <> struct RawBytes<8> { using type = uint2; };
template <> struct RawBytes<16> { using type = uint4; };

__device__ __forceinline__ void ld_once(const void* p, uint4& r) { r = ld_once_16(p); }
__device__ __forceinline__ void ld_once(const void* p, uint2& r) {
  asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "l"(p));
}
__device__ __forceinline__ void ld_once(const void* p, uint32_t& r) {
  asm volatile("ld.global.L1::no_allocate.u32 %0, [%1];" : "=r"(r) : "l"(p));
}
__device__ __forceinline__ void ld_once(const void* p, unsigned short& r) {
  asm volatile("ld.global.L1::no_allocate.u16 %0, [%1];" : "=h"(r) : "l"(p));
}

template <int BYTES>
struct Raw {
  typename RawBytes<BYTES>::type v;
  __device__ __forceinline__ void load(const void* p, bool in) {
    v = {};
    if (in) ld_once(p, v);
  }
  __device__ __forceinline__ uint32_t word(int j) const { return reinterpret_cast<const uint32_t*>(&v)[j]; }
  __device__ __forceinline__ uint32_t half(int j) const {
    return reinterpret_cast<const unsigned short*>(&v)[j];
  }
  // Scale and minimum of group j (a bf16 pair).
  __device__ __forceinline__ float scale(int j) const { return __uint_as_float(word(j) << 16); }
  __device__ __forceinline__ float minimum(int j) const { return __uint_as_float(word(j) & 0xffff0000u); }
};

// Transposes an 8 x 8 matrix of 16-bit elements held across the warp (lane
// 4 i + c: row i, columns 2c, 2c + 1).
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

// Sum (maximum) over the lanes that hold the same columns (lane 4 i + c: all i).
__device__ __forceinline__ float column_sum(float x) {
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
__device__ __forceinline__ float column_max(float x) {
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}

// One row x[0..D-1] into the buffer, by one warp: lane l holds channel l of
// each group.  fp32 arithmetic with one rounding per operation; a group with
// a NaN becomes NaN.
template <typename T, int D, bool KEY>
__device__ __forceinline__ void store_row(const T* x, uint8_t* codes, __nv_bfloat16* sm, int lane) {
  constexpr int NJ = D / 32;
  float v[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) v[j] = to_f32<T>(x[32 * j + lane]);
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const float lo = -warp_max(-v[j]), hi = warp_max(v[j]);
    __nv_bfloat162 par;
    par.y = __float2bfloat16_rn(lo);
    const float m = __bfloat162float(par.y);
    par.x = __float2bfloat16_rn(__fmul_rn(fmaxf(__fsub_rn(hi, m), 0.f), 1.f / 15.f));
    const float s = __bfloat162float(par.x);
    if (__any_sync(0xffffffffu, v[j] != v[j])) par = __floats2bfloat162_rn(NAN, NAN);
    const float t = s > 0.f ? rintf(__fdiv_rn(__fsub_rn(v[j], m), s)) : 0.f;
    const uint32_t q = (uint32_t)fminf(fmaxf(t, 0.f), 15.f);
    if constexpr (KEY) {
      const int o = lane & 7, c = lane >> 3;
      uint32_t w = q << ((o & 1) ? 2 * o + 14 : 2 * o);
      w |= __shfl_xor_sync(0xffffffffu, w, 1);
      w |= __shfl_xor_sync(0xffffffffu, w, 2);
      w |= __shfl_xor_sync(0xffffffffu, w, 4);
      if (o == 0) reinterpret_cast<uint32_t*>(codes)[c * NJ + j] = w;
    } else {
      const int t4 = lane & 3, i = lane >> 2;
      uint32_t w = q << (4 * t4);
      w |= __shfl_xor_sync(0xffffffffu, w, 1);
      w |= __shfl_xor_sync(0xffffffffu, w, 2);
      if (t4 == 0) reinterpret_cast<unsigned short*>(codes)[i * NJ + j] = (unsigned short)w;
    }
    if (lane == 0) reinterpret_cast<__nv_bfloat162*>(sm)[j] = par;
  }
}

// The queries of head i at 8 channels as B fragments of `parts` bf16 parts.
template <typename T> struct Parts;
template <> struct Parts<__nv_bfloat16> { static constexpr int n = 1; };
template <> struct Parts<float> { static constexpr int n = 3; };

// One warp's 16 rows as loaded: keys of rows i, i + 8 (chunk c), values of
// rows 2c, 2c + 1, 2c + 8, 2c + 9 (chunk i), and the parameters of rows i,
// i + 8.  Rows from r1 on read as zero, whatever the buffer holds there.
template <int D>
struct Tile {
  Raw<D / 8> k[2];
  Raw<D / 8> kp[2], vp[2];
  Raw<D / 16> v[4];
  __device__ __forceinline__ void load(const Q4Problem& p, size_t bh, int r, int r1, int i, int c) {
    const size_t row0 = bh * p.S;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int row = r + i + 8 * e;
      const bool in = row < r1;
      k[e].load(p.k_codes + (row0 + row) * (D / 2) + c * (D / 8), in);
      kp[e].load(p.k_scale + (row0 + row) * (D / 16), in);
      vp[e].load(p.v_scale + (row0 + row) * (D / 16), in);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int row = r + 2 * c + (e & 1) + 8 * (e >> 1);
      v[e].load(p.v_codes + (row0 + row) * (D / 2) + i * (D / 16), row < r1);
    }
  }
};

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, Parts<T>::n == 1 ? 2 : 1)
q4_decode_kernel(Q4Problem p) {
  constexpr int NJ = D / 32;           // groups
  constexpr int E = D / 32;            // channels per lane in the merges
  constexpr int NP = Parts<T>::n;
  __shared__ float red[kWarps][kHeads][D + 2];
  __shared__ int last;

  const int bh = blockIdx.y;
  const int b = bh / p.H_kv, hk = bh - b * p.H_kv;
  const int pos = p.pos[b];
  if (pos < 0 || pos >= p.S) {  // an idle stream; nothing of it is touched
    if (pos != -1 && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(p.status, kStatusRange);
    return;
  }
  const int nch = pos / p.chunk + 1;
  if ((int)blockIdx.x > nch) return;
  const int g = p.H_q / p.H_kv;
  const int hq0 = hk * g + blockIdx.z * kHeads;
  const int ng = min(kHeads, g - (int)blockIdx.z * kHeads);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const size_t head0 = (size_t)b * p.H_q + hq0;
  const T* q_t = static_cast<const T*>(p.q_t) + head0 * D;

  if (blockIdx.x > 0) {
    // ------------------------------------------------ attention partial
    const int r0 = (blockIdx.x - 1) * p.chunk, r1 = min(r0 + p.chunk, pos + 1);
    const int i = lane >> 2, c = lane & 3;
    if (r1 == pos + 1) {
      // This CTA's rows include the token's own: it is stored first (by every
      // head chunk, the same bytes) and then read like any other.
      const size_t row = (size_t)bh * p.S + pos;
      if (warp == 0)
        store_row<T, D, true>(static_cast<const T*>(p.k_t) + (size_t)bh * D, p.k_codes + row * (D / 2),
                              p.k_scale + row * (D / 16), lane);
      else if (warp == 1)
        store_row<T, D, false>(static_cast<const T*>(p.v_t) + (size_t)bh * D, p.v_codes + row * (D / 2),
                               p.v_scale + row * (D / 16), lane);
      __syncthreads();
    }
    int r = r0 + warp * 16;
    Tile<D> next;
    if (r < r1) next.load(p, bh, r, r1, i, c);

    // Queries of head i as B fragments, and every head's sum over each group.
    uint32_t qf[NJ][NP][4];
    float qsum[NJ][2];
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = 0.f;
      if (i < ng) {
        const T* src = q_t + (size_t)i * D + 32 * j + 8 * c;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = to_f32<T>(src[e]);
      }
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) s += x[e];
      s += __shfl_xor_sync(0xffffffffu, s, 1);
      s += __shfl_xor_sync(0xffffffffu, s, 2);
      qsum[j][0] = __shfl_sync(0xffffffffu, s, 8 * c);
      qsum[j][1] = __shfl_sync(0xffffffffu, s, 8 * c + 4);
#pragma unroll
      for (int part = 0; part < NP; ++part)
#pragma unroll
        for (int t = 0; t < 4; ++t) qf[j][part][t] = split_bf16(x[2 * t], x[2 * t + 1]);
    }
    const float sl2 = rsqrtf((float)D) * 1.4426950408889634f;

    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};  // heads 2c, 2c + 1; l over rows i, i + 8
    float o[2 * NJ][4], omin[NJ][2];
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      omin[j][0] = omin[j][1] = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) o[2 * j][e] = o[2 * j + 1][e] = 0.f;
    }
    for (; r < r1; r += kUnit) {
      const Tile<D> cur = next;
      if (r + kUnit < r1) next.load(p, bh, r + kUnit, r1, i, c);
      // Scores of rows i (s[0], s[1]) and i + 8 (s[2], s[3]).
      float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        uint32_t fa[4], fb[4];
        unpack_codes(cur.k[0].word(j), kCodeBias2, fa);
        unpack_codes(cur.k[1].word(j), kCodeBias2, fb);
        float t[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int part = 0; part < NP; ++part) {
          mma_bf16(t, fa[0], fb[0], fa[1], fb[1], qf[j][part][0], qf[j][part][1]);
          mma_bf16(t, fa[2], fb[2], fa[3], fb[3], qf[j][part][2], qf[j][part][3]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
          s[e] = fmaf(cur.kp[e >> 1].scale(j), t[e], fmaf(cur.kp[e >> 1].minimum(j), qsum[j][e & 1], s[e]));
      }
      const bool in0 = r + i < r1, in1 = r + i + 8 < r1;
      float pr[4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float s0 = in0 ? s[h] * sl2 : -INFINITY, s1 = in1 ? s[2 + h] * sl2 : -INFINITY;
        const float mn = fmaxf(m[h], column_max(fmaxf(s0, s1)));
        const float corr = exp2f(m[h] - mn);  // 0 for the first rows
        m[h] = mn;
        pr[h] = exp2f(s0 - mn);
        pr[2 + h] = exp2f(s1 - mn);
        l[h] = fmaf(l[h], corr, pr[h] + pr[2 + h]);
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          omin[j][h] = fmaf(pr[h], cur.vp[0].minimum(j), fmaf(pr[2 + h], cur.vp[1].minimum(j), omin[j][h] * corr));
          o[2 * j][h] *= corr; o[2 * j][2 + h] *= corr;
          o[2 * j + 1][h] *= corr; o[2 * j + 1][2 + h] *= corr;
        }
      }
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        // Codes of group j: element t of a lane's four is channel
        // 32 j + 4 i + t, rows 2c, 2c + 1 (lo) and 2c + 8, 2c + 9 (hi).
        uint32_t lo[4], hi[4];
        unpack_codes(cur.v[0].half(j) | (cur.v[1].half(j) << 16), kCodeBias2, lo);
        unpack_codes(cur.v[2].half(j) | (cur.v[3].half(j) << 16), kCodeBias2, hi);
        float w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = pr[e] * cur.vp[e >> 1].scale(j);
#pragma unroll
        for (int part = 0; part < NP; ++part) {
          const uint32_t b0 = transpose8(split_bf16(w[0], w[1])), b1 = transpose8(split_bf16(w[2], w[3]));
          mma_bf16(o[2 * j], lo[0], lo[1], hi[0], hi[1], b0, b1);
          mma_bf16(o[2 * j + 1], lo[2], lo[3], hi[2], hi[3], b0, b1);
        }
      }
    }
    // This warp's (max, sum, acc) of heads 2c, 2c + 1.
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] = column_sum(l[h]);
      if (i == 0) {
        red[warp][2 * c + h][D] = m[h];
        red[warp][2 * c + h][D + 1] = l[h];
      }
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const float add = column_sum(omin[j][h]);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          red[warp][2 * c + h][32 * j + 4 * i + 2 * u] = o[2 * j + u][h] + add;
          red[warp][2 * c + h][32 * j + 4 * i + 2 * u + 1] = o[2 * j + u][2 + h] + add;
        }
      }
    }
    __syncthreads();
    for (int at = threadIdx.x; at < ng * D; at += kThreads) {
      const int hh = at / D, e = at - hh * D;
      float mx = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, red[w][hh][D]);
      float ls = 0.f, as = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        // A warp without rows has m = -inf, l = acc = 0.
        const float f = red[w][hh][D] == -INFINITY ? 0.f : exp2f(red[w][hh][D] - mx);
        ls = fmaf(red[w][hh][D + 1], f, ls);
        as = fmaf(red[w][hh][e], f, as);
      }
      float* part = p.part + ((head0 + hh) * p.nsplit + blockIdx.x - 1) * (D + 2);
      part[2 + e] = as;
      if (e == 0) {
        part[0] = mx;
        part[1] = ls;
      }
    }
  } else {
    // ------------------------------------------------ retrieval
    // Warp w sums M's rows [w D/8, (w+1) D/8), lane l columns l + 32 k.
    float(*sq)[D] = reinterpret_cast<float(*)[D]>(&red[0][0][0]);  // [kHeads][D], before the sums
    for (int at = threadIdx.x; at < kHeads * D; at += kThreads) {
      const int hh = at / D, e = at - hh * D;
      sq[hh][e] = hh < ng ? elu1(to_f32<T>(q_t[(size_t)hh * D + e])) : 0.f;
    }
    __syncthreads();
    const float* zv = p.z + (size_t)bh * D;
    const float* Mh = p.M + (size_t)bh * D * D;
    float* ret = p.ret + head0 * (D + 1);
    if (warp < ng) {
      float dp = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) dp = fmaf(sq[warp][lane + 32 * e], zv[lane + 32 * e], dp);
      dp = warp_sum(dp);
      if (lane == 0) ret[(size_t)warp * (D + 1) + D] = dp;
    }
    float acc[kHeads][E];
#pragma unroll
    for (int hh = 0; hh < kHeads; ++hh)
#pragma unroll
      for (int e = 0; e < E; ++e) acc[hh][e] = 0.f;
    constexpr int kRowsPerWarp = D / kWarps;
#pragma unroll 8
    for (int k = 0; k < kRowsPerWarp; ++k) {
      const int row = warp * kRowsPerWarp + k;
      float mrow[E];
#pragma unroll
      for (int e = 0; e < E; ++e) mrow[e] = Mh[(size_t)row * D + lane + 32 * e];
#pragma unroll
      for (int hh = 0; hh < kHeads; ++hh) {
        const float w = sq[hh][row];
#pragma unroll
        for (int e = 0; e < E; ++e) acc[hh][e] = fmaf(w, mrow[e], acc[hh][e]);
      }
    }
    __syncthreads();  // sq has been read
#pragma unroll
    for (int hh = 0; hh < kHeads; ++hh)
#pragma unroll
      for (int e = 0; e < E; ++e) red[warp][hh][lane + 32 * e] = acc[hh][e];
    __syncthreads();
    for (int at = threadIdx.x; at < ng * D; at += kThreads) {
      const int hh = at / D, e = at - hh * D;
      float num = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) num += red[w][hh][e];
      ret[(size_t)hh * (D + 1) + e] = num;
    }
  }

  // ------------------------------------------------ the last CTA finishes
  __threadfence();  // this thread's workspace writes, before the ticket
  __syncthreads();
  unsigned int* ctr = p.ctr + (size_t)bh * gridDim.z + blockIdx.z;
  if (threadIdx.x == 0) last = atomicAdd(ctr, 1u) == (unsigned int)nch;
  __syncthreads();
  if (!last) return;
  __threadfence();  // every other CTA's writes of this group are visible
  if (warp < ng) {
    // Warp w merges head w's partials, in chunk order; lane l columns l + 32 e.
    const float* part = p.part + (head0 + warp) * p.nsplit * (D + 2);
    const float* ret = p.ret + (head0 + warp) * (D + 1);
    float num[E];
#pragma unroll
    for (int e = 0; e < E; ++e) num[e] = __ldcg(ret + lane + 32 * e);
    const float den = __ldcg(ret + D);
    const float gm = gate_sigmoid(p.beta[hq0 + warp]);
    float mx = -INFINITY, ls = 0.f, as[E];
#pragma unroll
    for (int e = 0; e < E; ++e) as[e] = 0.f;
    constexpr int kU = 8;  // partials in flight
    for (int c0 = 0; c0 < nch; c0 += kU) {
      float mc[kU], lc[kU], ac[kU][E];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const bool in = c0 + u < nch;
        const float* pc = part + (size_t)(c0 + u) * (D + 2);
        mc[u] = in ? __ldcg(pc) : -INFINITY;
        lc[u] = in ? __ldcg(pc + 1) : 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) ac[u][e] = in ? __ldcg(pc + 2 + lane + 32 * e) : 0.f;
      }
      float nm = mx;
#pragma unroll
      for (int u = 0; u < kU; ++u) nm = fmaxf(nm, mc[u]);
      const float corr = exp2f(mx - nm);  // 0 for the first partials
      ls *= corr;
#pragma unroll
      for (int e = 0; e < E; ++e) as[e] *= corr;
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const float f = exp2f(mc[u] - nm);  // 0 past the last partial
        ls = fmaf(lc[u], f, ls);
#pragma unroll
        for (int e = 0; e < E; ++e) as[e] = fmaf(ac[u][e], f, as[e]);
      }
      mx = nm;
    }
    T* out = static_cast<T*>(p.out_t) + (head0 + warp) * D;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float a_mem = den != 0.f ? num[e] / den : 0.f;
      out[lane + 32 * e] = from_f32<T>(gm * a_mem + (1.f - gm) * (as[e] / ls));
    }
  }
  if (threadIdx.x == 0) *ctr = 0u;  // ready for the next step
}

// Rows of k and v [B, H_kv, n, D] into the buffers from row pos[b] on: one
// warp per row and buffer.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) q4_append_kernel(Q4Problem p, int n) {
  const long long unit = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const long long total = (long long)p.B * p.H_kv * n;
  if (unit >= total) return;
  const long long bh = unit / n;
  const int t = (int)(unit - bh * n);
  const int pos = p.pos[bh / p.H_kv];
  if (pos < 0 || pos > p.S - n) {
    if (pos != -1 && lane == 0) atomicOr(p.status, kStatusRange);
    return;
  }
  const size_t row = (size_t)bh * p.S + pos + t;
  if (blockIdx.y == 0)
    store_row<T, D, true>(static_cast<const T*>(p.k_t) + unit * D, p.k_codes + row * (D / 2),
                          p.k_scale + row * (D / 16), lane);
  else
    store_row<T, D, false>(static_cast<const T*>(p.v_t) + unit * D, p.v_codes + row * (D / 2),
                           p.v_scale + row * (D / 16), lane);
}

// The values of rows 0..n-1 as k and v [B, H_kv, n, D]: a thread takes 8
// channels (a key word) or 4 (a value halfword) of a row.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) q4_read_kernel(Q4Problem p, int n, T* k, T* v) {
  constexpr int NJ = D / 32;
  const bool key = blockIdx.y == 0;
  const int per_row = key ? D / 8 : D / 4;
  const long long total = (long long)p.B * p.H_kv * n * per_row;
  for (long long at = (long long)blockIdx.x * kThreads + threadIdx.x; at < total;
       at += (long long)gridDim.x * kThreads) {
    const long long unit = at / per_row;
    const int w = (int)(at - unit * per_row);  // word of the row: channels 8w.. or 4w..
    const long long bh = unit / n;
    const size_t row = (size_t)bh * p.S + (unit - bh * n);
    const int j = key ? w / 4 : w / 8;
    const __nv_bfloat162 par =
        reinterpret_cast<const __nv_bfloat162*>((key ? p.k_scale : p.v_scale) + row * (D / 16))[j];
    const float s = __low2float(par), m = __high2float(par);
    T* dst = (key ? k : v) + unit * D + (key ? 8 : 4) * w;
    if (key) {
      const uint32_t word = reinterpret_cast<const uint32_t*>(p.k_codes + row * (D / 2))[(w & 3) * NJ + j];
#pragma unroll
      for (int o = 0; o < 8; ++o)
        dst[o] = from_f32<T>(fmaf(s, (float)((word >> ((o & 1) ? 2 * o + 14 : 2 * o)) & 15u), m));
    } else {
      const uint32_t half =
          reinterpret_cast<const unsigned short*>(p.v_codes + row * (D / 2))[(w & 7) * NJ + j];
#pragma unroll
      for (int t = 0; t < 4; ++t) dst[t] = from_f32<T>(fmaf(s, (float)((half >> (4 * t)) & 15u), m));
    }
  }
}

template <typename T, int D>
cudaError_t launch(const Q4Problem& p, Q4What what, int n, void* k, void* v, cudaStream_t st) {
  const long long rows = (long long)p.B * p.H_kv * n;
  switch (what) {
    case Q4What::kStep: {
      const int g = p.H_q / p.H_kv;
      q4_decode_kernel<T, D><<<dim3(p.nsplit + 1, p.B * p.H_kv, (g + kHeads - 1) / kHeads), kThreads, 0, st>>>(p);
      break;
    }
    case Q4What::kAppend:
      q4_append_kernel<T, D><<<dim3((unsigned)((rows + kWarps - 1) / kWarps), 2), kThreads, 0, st>>>(p, n);
      break;
    case Q4What::kRead: {
      const long long blocks = (rows * (D / 8) + kThreads - 1) / kThreads;
      const unsigned grid = (unsigned)(blocks < kSMs * 32 ? blocks : kSMs * 32);
      q4_read_kernel<T, D><<<dim3(grid, 2), kThreads, 0, st>>>(p, n, static_cast<T*>(k), static_cast<T*>(v));
      break;
    }
  }
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_type(const Q4Problem& p, Q4What what, int n, void* k, void* v, cudaStream_t st) {
  switch (p.d) {
    case 32: return launch<T, 32>(p, what, n, k, v, st);
    case 64: return launch<T, 64>(p, what, n, k, v, st);
    case 128: return launch<T, 128>(p, what, n, k, v, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

int q4_head_chunks(int g) { return (g + kHeads - 1) / kHeads; }

// Rows per CTA: one unit of 128 while that fills the GPU, then as many as
// leave about four waves of resident CTAs (two per SM), at most 16 units.
int q4_chunk_rows(long long groups, int S) {
  const long long units = groups * ((S + kUnit - 1) / kUnit);
  long long n = units / (kSMs * 2 * 4);
  n = n < 1 ? 1 : n > 16 ? 16 : n;
  return (int)n * kUnit;
}

cudaError_t launch_q4(const Q4Problem& p, Q4What what, int n, void* k, void* v, cudaStream_t st) {
  return p.bf16 ? launch_type<__nv_bfloat16>(p, what, n, k, v, st) : launch_type<float>(p, what, n, k, v, st);
}

}  // namespace infini
