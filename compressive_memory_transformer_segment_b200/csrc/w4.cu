// Projections of a few tokens with 4-bit weights (sm_100a).
//
//   y[t][n] = sum over k of x[t][k] w[n][k] (+ bias[n]),
//   w[n][k] = scales[n][k / G] (q[n][k] - zeros[n][k / G])
// with 4-bit codes q, and for the query/key/value projection the head split
// and rotary embedding of infini_attn_qkv_project in the epilogue.
//
// Bound by the weights' bytes: each is read once for all tokens of a pass and
// used for 2 operations per token.  Multiplying them on the CUDA cores would
// cost a conversion and a multiply-add per weight and token; instead a warp
// turns 8 codes into 4 bf16 pairs (q - zero, exact) and multiplies 16 rows by
// 8 tokens at a time on the tensor cores (mma.sync: the 128-row tiles of
// tcgen05 would carry at most a few tokens).  The sums over a group are taken
// over the integers, and the group's scale multiplies the fp32 sum: no
// rounding of the weights anywhere.  fp32 tokens go in as three bf16 parts,
// which hold all their bits.
//
// Layout (see the header): a row's 128-channel blocks are stored so that the
// 16 bytes lane 4 i + c loads hold exactly the codes that lane's fragments
// need (chunk c of the block: word j = channels 32 j + 8 c .. + 7), and the
// same 8 channels of a token are 16 contiguous bytes.  So both operands go
// from global memory to the tensor cores without shared memory or shuffles.
//
// A CTA takes 16 rows; its 8 warps share out the row's blocks, and their sums
// are added in warp order through shared memory.
#include "common.cuh"
#include "kernels.h"
#include "q4_common.cuh"

namespace infini {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kBlock = 128;  // channels of a packed block
constexpr int kTile = 16;    // rows of a CTA

// Scale (fp32) and bias pair (bf16x2 of 128 + zero) of a row's groups in one
// block; NG groups of 128 / NG channels.
template <int NG>
struct GroupParams {
  __nv_bfloat16 s[NG];
  uint8_t z[NG];
  // Groups from `groups` on hold no channel below K; their scale is taken as
  // 0, whatever the array holds there.
  __device__ __forceinline__ void load(const __nv_bfloat16* scales, const uint8_t* zeros, size_t row,
                                       int per_row, int blk, int groups) {
#pragma unroll
    for (int i = 0; i < NG; ++i) {
      const int at = blk * NG + i;
      const bool in = at < groups;
      s[i] = in ? scales[row * per_row + at] : __float2bfloat16_rn(0.f);
      z[i] = in && zeros ? zeros[row * per_row + at] : (uint8_t)8;
    }
  }
  __device__ __forceinline__ float scale(int i) const { return __bfloat162float(s[i]); }
  __device__ __forceinline__ uint32_t bias(int i) const { return kCodeBias2 + z[i] * 0x00010001u; }
};

// 8 channels of a token as B fragments: parts of 4 bf16 pairs.
template <typename T> struct TokenFrag;
template <> struct TokenFrag<__nv_bfloat16> {
  static constexpr int kParts = 1;
  uint32_t b[1][4];
  __device__ __forceinline__ void load(const __nv_bfloat16* x, bool in) {
    const uint4 v = in ? __ldg(reinterpret_cast<const uint4*>(x)) : uint4{0, 0, 0, 0};
    b[0][0] = v.x; b[0][1] = v.y; b[0][2] = v.z; b[0][3] = v.w;
  }
};
template <> struct TokenFrag<float> {
  static constexpr int kParts = 3;
  uint32_t b[3][4];
  __device__ __forceinline__ void load(const float* x, bool in) {
    float4 v[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
    if (in) {
      v[0] = __ldg(reinterpret_cast<const float4*>(x));
      v[1] = __ldg(reinterpret_cast<const float4*>(x) + 1);
    }
#pragma unroll
    for (int part = 0; part < 3; ++part) {
      b[part][0] = split_bf16(v[0].x, v[0].y);
      b[part][1] = split_bf16(v[0].z, v[0].w);
      b[part][2] = split_bf16(v[1].x, v[1].y);
      b[part][3] = split_bf16(v[1].z, v[1].w);
    }
  }
};

// Row of the weight matrix that row m of tile `tile` is.  A plain layer takes
// 16 consecutive rows; a projection into heads takes rows i0 .. i0 + 7 of one
// head and their partners i + d/2, so that one lane holds both halves of a
// rotation.
template <bool QKV>
__device__ __forceinline__ int tile_row(const W4Problem& p, int tile, int m) {
  if constexpr (!QKV) return tile * kTile + m;
  const int per_head = p.d / kTile;
  const int head = tile / per_head, i0 = (tile - head * per_head) * 8;
  return head * p.d + i0 + (m < 8 ? m : m - 8 + p.d / 2);
}

template <typename T, int NT, int NG, bool QKV>
__global__ void __launch_bounds__(kThreads)
w4_kernel(W4Problem p) {
  constexpr int kTok = NT * 8;
  constexpr int kParts = TokenFrag<T>::kParts;
  __shared__ float red[kWarps][kTile][kTok + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int i = lane >> 2, c = lane & 3;
  const int t0 = blockIdx.y * kTok;
  const int nt = min(kTok, p.M - t0);
  const int nblk = (p.K + kBlock - 1) / kBlock;
  const int groups = (p.K + kBlock / NG - 1) / (kBlock / NG);
  // Rows past the last are read as the last one and never stored.
  const size_t row_a = min(tile_row<QKV>(p, blockIdx.x, i), p.N - 1);
  const size_t row_b = min(tile_row<QKV>(p, blockIdx.x, i + 8), p.N - 1);
  const uint8_t* wa_p = p.packed + row_a * nblk * (kBlock / 2) + c * 16;
  const uint8_t* wb_p = p.packed + row_b * nblk * (kBlock / 2) + c * 16;
  const T* x = static_cast<const T*>(p.x);

  float acc[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[n][e] = 0.f;

  uint4 na = {0, 0, 0, 0}, nb = {0, 0, 0, 0};
  GroupParams<NG> pa, pb;
  if (warp < nblk) {
    na = ld_once_16(wa_p + (size_t)warp * (kBlock / 2));
    nb = ld_once_16(wb_p + (size_t)warp * (kBlock / 2));
    pa.load(p.scales, p.zeros, row_a, nblk * NG, warp, groups);
    pb.load(p.scales, p.zeros, row_b, nblk * NG, warp, groups);
  }
  for (int blk = warp; blk < nblk; blk += kWarps) {
    const uint32_t wa[4] = {na.x, na.y, na.z, na.w}, wb[4] = {nb.x, nb.y, nb.z, nb.w};
    const GroupParams<NG> ga = pa, gb = pb;
    const int next = blk + kWarps;
    if (next < nblk) {
      na = ld_once_16(wa_p + (size_t)next * (kBlock / 2));
      nb = ld_once_16(wb_p + (size_t)next * (kBlock / 2));
      pa.load(p.scales, p.zeros, row_a, nblk * NG, next, groups);
      pb.load(p.scales, p.zeros, row_b, nblk * NG, next, groups);
    }
    float sum[NT][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int g = j * NG / 4;
      uint32_t fa[4], fb[4];
      unpack_codes(wa[j], ga.bias(g), fa);
      unpack_codes(wb[j], gb.bias(g), fb);
      const bool first = j % (4 / NG) == 0, last = (j + 1) % (4 / NG) == 0;
      const int k0 = blk * kBlock + 32 * j + 8 * c;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if (first) sum[n][0] = sum[n][1] = sum[n][2] = sum[n][3] = 0.f;
        const int t = n * 8 + i;
        TokenFrag<T> f;
        f.load(x + (size_t)(t0 + t) * p.K + k0, t < nt && k0 < p.K);
#pragma unroll
        for (int part = 0; part < kParts; ++part) {
          mma_bf16(sum[n], fa[0], fb[0], fa[1], fb[1], f.b[part][0], f.b[part][1]);
          mma_bf16(sum[n], fa[2], fb[2], fa[3], fb[3], f.b[part][2], f.b[part][3]);
        }
        if (last) {
          acc[n][0] = fmaf(ga.scale(g), sum[n][0], acc[n][0]);
          acc[n][1] = fmaf(ga.scale(g), sum[n][1], acc[n][1]);
          acc[n][2] = fmaf(gb.scale(g), sum[n][2], acc[n][2]);
          acc[n][3] = fmaf(gb.scale(g), sum[n][3], acc[n][3]);
        }
      }
    }
  }
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    red[warp][i][n * 8 + 2 * c] = acc[n][0];
    red[warp][i][n * 8 + 2 * c + 1] = acc[n][1];
    red[warp][i + 8][n * 8 + 2 * c] = acc[n][2];
    red[warp][i + 8][n * 8 + 2 * c + 1] = acc[n][3];
  }
  __syncthreads();
  auto total = [&](int m, int t) {
    float s = red[0][m][t];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) s += red[w][m][t];
    return s;
  };
  if constexpr (!QKV) {
    for (int at = threadIdx.x; at < kTile * nt; at += kThreads) {
      const int t = at / kTile, m = at % kTile;
      const int row = blockIdx.x * kTile + m;
      if (row < p.N) {
        float y = total(m, t);
        if (p.bias) y += p.bias[row];
        static_cast<T*>(p.y)[(size_t)(t0 + t) * p.N + row] = from_f32<T>(y);
      }
    }
  } else {
    const int half = p.d / 2;
    for (int at = threadIdx.x; at < 8 * nt; at += kThreads) {
      const int t = at / 8, m = at % 8;
      const int row = tile_row<true>(p, blockIdx.x, m);
      const int head = row / p.d, e = row - head * p.d;
      float y0 = total(m, t), y1 = total(m + 8, t);
      if (p.bias) {
        y0 += p.bias[row];
        y1 += p.bias[row + half];
      }
      const int tok = t0 + t, b = tok / p.L, l = tok - b * p.L;
      if (p.rope_cos && head < p.H_q + p.H_kv) {
        const int pos = p.positions ? p.positions[tok] : l;
        if (pos >= 0 && pos < p.n_pos) {
          const float cs = p.rope_cos[(size_t)pos * half + e], sn = p.rope_sin[(size_t)pos * half + e];
          const float r0 = y0 * cs - y1 * sn;
          y1 = y1 * cs + y0 * sn;
          y0 = r0;
        } else {
          atomicOr(p.status, kStatusRange);
        }
      }
      T* out;
      int heads, h = head;
      if (h < p.H_q) {
        out = static_cast<T*>(p.q); heads = p.H_q;
      } else if (h < p.H_q + p.H_kv) {
        out = static_cast<T*>(p.k); heads = p.H_kv; h -= p.H_q;
      } else {
        out = static_cast<T*>(p.v); heads = p.H_kv; h -= p.H_q + p.H_kv;
      }
      out += ((size_t)(b * heads + h) * p.L + l) * p.d + e;
      out[0] = from_f32<T>(y0);
      out[half] = from_f32<T>(y1);
    }
  }
}

template <typename T, int NG, bool QKV>
cudaError_t launch_tokens(const W4Problem& p, cudaStream_t st) {
  const unsigned tiles = (p.N + kTile - 1) / kTile;
  // 8, 16, 32 or 64 tokens a pass: the least that holds them all.
  if (p.M <= 8)
    w4_kernel<T, 1, NG, QKV><<<dim3(tiles, 1), kThreads, 0, st>>>(p);
  else if (p.M <= 16)
    w4_kernel<T, 2, NG, QKV><<<dim3(tiles, 1), kThreads, 0, st>>>(p);
  else if (p.M <= 32)
    w4_kernel<T, 4, NG, QKV><<<dim3(tiles, 1), kThreads, 0, st>>>(p);
  else
    w4_kernel<T, 8, NG, QKV><<<dim3(tiles, (p.M + 63) / 64), kThreads, 0, st>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_type(const W4Problem& p, cudaStream_t st) {
  const bool qkv = p.q != nullptr;
  switch (p.group) {
    case 32: return qkv ? launch_tokens<T, 4, true>(p, st) : launch_tokens<T, 4, false>(p, st);
    case 64: return qkv ? launch_tokens<T, 2, true>(p, st) : launch_tokens<T, 2, false>(p, st);
    case 128: return qkv ? launch_tokens<T, 1, true>(p, st) : launch_tokens<T, 1, false>(p, st);
    default: return cudaErrorInvalidValue;
  }
}

// ---------------------------------------------------------------- layout
// Bit of channel ch (0..127) in its block: word j of chunk c holds channels
// 32 j + 8 c + o, o even in bits 2 o .. 2 o + 3, o odd 16 bits further up.
__device__ __forceinline__ int code_bit(int ch) {
  const int j = ch >> 5, c = (ch >> 3) & 3, o = ch & 7;
  return 32 * (4 * c + j) + 4 * (o >> 1) + 16 * (o & 1);
}

// One warp per row and block of 128 channels; lane l holds channels l, l + 32,
// l + 64, l + 96.  Codes go to shared memory and leave as 16 words.
__device__ __forceinline__ void store_block(const int (&q)[4], uint32_t (*words)[16], int w, int lane,
                                            uint32_t* dst) {
  if (lane < 16) words[w][lane] = 0u;
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int bit = code_bit(32 * j + lane);
    atomicOr(&words[w][bit >> 5], (uint32_t)q[j] << (bit & 31));
  }
  __syncwarp();
  if (lane < 16) dst[lane] = words[w][lane];
}

template <typename T>
__global__ void __launch_bounds__(kThreads) w4_quantize_kernel(W4PackProblem p) {
  __shared__ uint32_t words[kWarps][16];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nblk = (p.K + kBlock - 1) / kBlock, ng = kBlock / p.group;
  const long long unit = (long long)blockIdx.x * kWarps + warp;
  if (unit >= (long long)p.N * nblk) return;
  const int row = (int)(unit / nblk), blk = (int)(unit - (long long)row * nblk);
  const T* w = static_cast<const T*>(p.w) + (size_t)row * p.K;
  float v[4], lo[4], hi[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int k = blk * kBlock + 32 * j + lane;
    v[j] = k < p.K ? to_f32<T>(w[k]) : 0.f;
    lo[j] = -warp_max(-v[j]);
    hi[j] = warp_max(v[j]);
  }
  int q[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    // Range of the channel's group, 0 included (a code for 0 always exists).
    const int per = 4 / ng, g = j / per;
    float a = 0.f, b = 0.f;
#pragma unroll
    for (int t = 0; t < 4; ++t)
      if (t / per == g) {
        a = fminf(a, lo[t]);
        b = fmaxf(b, hi[t]);
      }
    float s, z = 8.f;
    if (p.zeros) {
      s = __bfloat162float(__float2bfloat16_rn((b - a) * (1.f / 15.f)));
      z = s > 0.f ? fminf(fmaxf(rintf(__fdiv_rn(-a, s)), 0.f), 15.f) : 8.f;
    } else {
      s = __bfloat162float(__float2bfloat16_rn(fmaxf(-a, b) * (1.f / 7.f)));
    }
    const float t = s > 0.f ? rintf(__fdiv_rn(v[j], s)) + z : z;
    q[j] = (int)fminf(fmaxf(t, 0.f), 15.f);
    if (lane == 0 && j % per == 0) {
      const size_t at = ((size_t)row * nblk + blk) * ng + g;
      const bool in = blk * kBlock + g * p.group < p.K;
      p.scales[at] = __float2bfloat16_rn(in ? s : 0.f);
      if (p.zeros) p.zeros[at] = (uint8_t)z;
    }
  }
  store_block(q, words, warp, lane, reinterpret_cast<uint32_t*>(p.packed) + unit * 16);
}

__global__ void __launch_bounds__(kThreads) w4_pack_kernel(W4PackProblem p) {
  __shared__ uint32_t words[kWarps][16];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nblk = (p.K + kBlock - 1) / kBlock;
  const long long unit = (long long)blockIdx.x * kWarps + warp;
  if (unit >= (long long)p.N * nblk) return;
  const int row = (int)(unit / nblk), blk = (int)(unit - (long long)row * nblk);
  const uint8_t* codes = static_cast<const uint8_t*>(p.w) + (size_t)row * p.K;
  int q[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int k = blk * kBlock + 32 * j + lane;
    q[j] = k < p.K ? codes[k] & 15 : 0;
  }
  store_block(q, words, warp, lane, reinterpret_cast<uint32_t*>(p.packed) + unit * 16);
}

template <typename T>
__global__ void __launch_bounds__(kThreads) w4_dequantize_kernel(W4PackProblem p) {
  const int nblk = (p.K + kBlock - 1) / kBlock, ng = kBlock / p.group;
  const long long total = (long long)p.N * p.K;
  for (long long at = (long long)blockIdx.x * kThreads + threadIdx.x; at < total;
       at += (long long)gridDim.x * kThreads) {
    const long long row = at / p.K;
    const int k = (int)(at - row * p.K), blk = k / kBlock, ch = k % kBlock;
    const int bit = code_bit(ch);
    const uint32_t w = reinterpret_cast<const uint32_t*>(p.packed)[(row * nblk + blk) * 16 + (bit >> 5)];
    const size_t g = (size_t)(row * nblk + blk) * ng + ch / p.group;
    const int zero = p.zeros ? p.zeros[g] : 8;
    static_cast<T*>(const_cast<void*>(p.w))[at] =
        from_f32<T>(__bfloat162float(p.scales[g]) * (float)((int)((w >> (bit & 31)) & 15u) - zero));
  }
}

}  // namespace

cudaError_t launch_w4(const W4Problem& p, cudaStream_t st) {
  return p.bf16 ? launch_type<__nv_bfloat16>(p, st) : launch_type<float>(p, st);
}

cudaError_t launch_w4_layout(const W4PackProblem& p, W4Layout what, cudaStream_t st) {
  const long long units = (long long)p.N * ((p.K + kBlock - 1) / kBlock);
  const unsigned grid = (unsigned)((units + kWarps - 1) / kWarps);
  switch (what) {
    case W4Layout::kQuantize:
      if (p.bf16) w4_quantize_kernel<__nv_bfloat16><<<grid, kThreads, 0, st>>>(p);
      else w4_quantize_kernel<float><<<grid, kThreads, 0, st>>>(p);
      break;
    case W4Layout::kPack: w4_pack_kernel<<<grid, kThreads, 0, st>>>(p); break;
    case W4Layout::kDequantize: {
      const unsigned g = grid < 148u * 16u ? grid : 148u * 16u;
      if (p.bf16) w4_dequantize_kernel<__nv_bfloat16><<<g, kThreads, 0, st>>>(p);
      else w4_dequantize_kernel<float><<<g, kThreads, 0, st>>>(p);
      break;
    }
  }
  return cudaGetLastError();
}

}  // namespace infini
