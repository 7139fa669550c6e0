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
// same 8 channels of a token are 16 contiguous bytes.  So no operand is shuffled
// between lanes; shared memory only holds codes on their way (split) or the tokens
// that four warps share (rows).
//
// A CTA takes 16 rows, whose blocks its 8 warps share out (their sums are added
// in warp order through shared memory), or, for 9 tokens and more and where that
// still fills the GPU, 64 rows, whose 4 warps take a tile each and share the
// tokens' channels.
//
// Measured (device time): one token through 4096 -> 6144 (13 MB) 6.8 us, 1.9
// TB/s, of which about 3 us are the launch and the last wave's drain; 16 tokens,
// 4096 -> 16384 (36 MB) 21 us, 1.8 TB/s.  The second is bound by the warps' own
// instructions: 290 of them per 16 rows x 128 channels (88 to make operands of the
// codes, 16 products, the rest loads, scales and addresses), issued in 43% of the
// cycles with 7 warps per SM; the order of the products and twice the warps
// changed it by 3% or less.  One token through 4096 -> 131072 (272 MB) takes 84 us,
// 3.3 TB/s, for the same reason.
#include "common.cuh"
#include "kernels.h"
#include "q4_common.cuh"

namespace infini {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kBlock = 128;  // channels of a packed block
constexpr int kTile = 16;    // rows of a tile
constexpr int kSMs = 148;

// Scales and zeros of a row's NG groups (of 128 / NG channels) in one block, as
// they lie in memory.
template <int NG>
struct GroupParams {
  uint32_t s[NG == 4 ? 2 : 1];  // bf16
  uint32_t z;                   // bytes
  __device__ __forceinline__ void load(const __nv_bfloat16* scales, const uint8_t* zeros) {
    z = 0x08080808u;
    if constexpr (NG == 4) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(scales));
      s[0] = v.x; s[1] = v.y;
      if (zeros) z = __ldg(reinterpret_cast<const uint32_t*>(zeros));
    } else if constexpr (NG == 2) {
      s[0] = __ldg(reinterpret_cast<const uint32_t*>(scales));
      if (zeros) z = __ldg(reinterpret_cast<const unsigned short*>(zeros));
    } else {
      s[0] = __ldg(reinterpret_cast<const unsigned short*>(scales));
      if (zeros) z = __ldg(zeros);
    }
  }
  // The scales of groups without a channel below K count as 0, whatever the
  // array holds there: only `groups` (at least one) of the block's do.
  __device__ __forceinline__ void cut(int groups) {
#pragma unroll
    for (int g = 1; g < NG; ++g)
      if (g >= groups) s[g >> 1] &= g & 1 ? 0x0000ffffu : 0xffff0000u;
  }
  __device__ __forceinline__ float scale(int g) const {
    return __uint_as_float(g & 1 ? s[g >> 1] & 0xffff0000u : s[g >> 1] << 16);
  }
  // bf16x2 of 128 + zero.
  __device__ __forceinline__ uint32_t bias(int g) const {
    return kCodeBias2 + __byte_perm(z, 0, 0x4040 + g * 0x0101);
  }
};

// 8 channels of a token as B fragments: parts of 4 bf16 pairs.
template <typename T> struct TokenFrag;
template <> struct TokenFrag<__nv_bfloat16> {
  static constexpr int kParts = 1;
  uint32_t b[1][4];
  __device__ __forceinline__ void load(const __nv_bfloat16* x, bool in) {
    const uint4 v = in ? *reinterpret_cast<const uint4*>(x) : uint4{0, 0, 0, 0};
    b[0][0] = v.x; b[0][1] = v.y; b[0][2] = v.z; b[0][3] = v.w;
  }
};
template <> struct TokenFrag<float> {
  static constexpr int kParts = 3;
  uint32_t b[3][4];
  __device__ __forceinline__ void load(const float* x, bool in) {
    float4 v[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
    if (in) {
      v[0] = *reinterpret_cast<const float4*>(x);
      v[1] = reinterpret_cast<const float4*>(x)[1];
    }
    set(v);
  }
  __device__ __forceinline__ void set(float4 (&v)[2]) {
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
__device__ __forceinline__ int tile_row(const W4Problem& p, int tile, int m) {
  if (p.q == nullptr) return tile * kTile + m;
  const int per_head = p.d / kTile;
  const int head = tile / per_head, i0 = (tile - head * per_head) * 8;
  return head * p.d + i0 + (m < 8 ? m : m - 8 + p.d / 2);
}

// A row tile's codes of a block (rows a and b of this lane) times NT token tiles,
// into acc; piece(j, f): the tokens' fragments of channels 32 j ...  The second and
// third parts of fp32 tokens have a sum of their own, added to the first's once a group:
// the tensor cores truncate every sum, the small ones then at 2^-8 of the large (128
// channels: error 2.4e-7 with one sum, 4e-8 with two; 64 tokens, 4096 -> 16384: 157 and 134
// us, the two being chains that do not wait for each other).
template <typename T, int NT, int NG, typename F>
__device__ __forceinline__ void multiply(const uint4& a, const uint4& b, const GroupParams<NG>& pa,
                                         const GroupParams<NG>& pb, F&& piece, float (&acc)[NT][4]) {
  const uint32_t wa[4] = {a.x, a.y, a.z, a.w}, wb[4] = {b.x, b.y, b.z, b.w};
  constexpr bool kParts = TokenFrag<T>::kParts > 1;
  float s[NT][4], small[kParts ? NT : 1][4];
  uint32_t ba = 0, bb = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int g = j * NG / 4;
    const bool first = j % (4 / NG) == 0, last = (j + 1) % (4 / NG) == 0;
    if (first) {
      ba = pa.bias(g);
      bb = pb.bias(g);
    }
    uint32_t fa[4], fb[4];
    unpack_codes(wa[j], ba, fa);
    unpack_codes(wb[j], bb, fb);
    TokenFrag<T> f[NT];
    piece(j, f);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if (first)
        mma_bf16_first(s[n], fa[0], fb[0], fa[1], fb[1], f[n].b[0][0], f[n].b[0][1]);
      else
        mma_bf16(s[n], fa[0], fb[0], fa[1], fb[1], f[n].b[0][0], f[n].b[0][1]);
      mma_bf16(s[n], fa[2], fb[2], fa[3], fb[3], f[n].b[0][2], f[n].b[0][3]);
#pragma unroll
      for (int part = 1; part < TokenFrag<T>::kParts; ++part) {
        if (first && part == 1)
          mma_bf16_first(small[n], fa[0], fb[0], fa[1], fb[1], f[n].b[part][0], f[n].b[part][1]);
        else
          mma_bf16(small[n], fa[0], fb[0], fa[1], fb[1], f[n].b[part][0], f[n].b[part][1]);
        mma_bf16(small[n], fa[2], fb[2], fa[3], fb[3], f[n].b[part][2], f[n].b[part][3]);
      }
      if constexpr (kParts) {
        if (last) {
#pragma unroll
          for (int e = 0; e < 4; ++e) s[n][e] += small[n][e];
        }
      }
      if (last) {
        const float sa = pa.scale(g), sb = pb.scale(g);
        acc[n][0] = fmaf(sa, s[n][0], acc[n][0]);
        acc[n][1] = fmaf(sa, s[n][1], acc[n][1]);
        acc[n][2] = fmaf(sb, s[n][2], acc[n][2]);
        acc[n][3] = fmaf(sb, s[n][3], acc[n][3]);
      }
    }
  }
}

// Where a lane's row of the weights lies.
template <int NG>
struct Row {
  const uint8_t* codes;  // its 16 bytes of the first block
  const __nv_bfloat16* scales;
  const uint8_t* zeros;  // or null
  __device__ __forceinline__ Row(const W4Problem& p, int tile, int m, int nblk, int c) {
    // Rows past the last are read as the last one and never stored.
    const size_t row = min(tile_row(p, tile, m), p.N - 1);
    codes = p.packed + row * nblk * (kBlock / 2) + c * 16;
    scales = p.scales + row * nblk * NG;
    zeros = p.zeros ? p.zeros + row * nblk * NG : nullptr;
  }
  __device__ __forceinline__ const uint8_t* block(int blk) const { return codes + (uint32_t)blk * (kBlock / 2); }
  __device__ __forceinline__ void load(GroupParams<NG>& to, int blk) const {
    to.load(scales + blk * NG, zeros ? zeros + blk * NG : nullptr);
  }
};

// A finished tile to the outputs: value(m, t) is row m's sum for token t of this
// pass; `threads` threads, this one `thread`.
template <typename T, typename F>
__device__ __forceinline__ void write_tile(const W4Problem& p, int tile, int t0, int nt, int thread, int threads,
                                           F&& value) {
  if (p.q == nullptr) {
    for (int at = thread; at < kTile * nt; at += threads) {
      const int t = at / kTile, m = at % kTile, n = tile * kTile + m;
      if (n < p.N) {
        float y = value(m, t);
        if (p.bias) y += p.bias[n];
        static_cast<T*>(p.y)[(size_t)(t0 + t) * p.N + n] = from_f32<T>(y);
      }
    }
    return;
  }
  const int half = p.d / 2, first = tile_row(p, tile, 0);
  for (int at = thread; first < p.N && at < 8 * nt; at += threads) {
    const int t = at / 8, m = at % 8, n = first + m;
    const int head = n / p.d, e = n - head * p.d;
    float y0 = value(m, t), y1 = value(m + 8, t);
    if (p.bias) {
      y0 += p.bias[n];
      y1 += p.bias[n + half];
    }
    const int tok = t0 + t, b = tok / p.L, l = tok - b * p.L;
    if (p.rope_cos && head < p.H_q + p.H_kv) {
      const int pos = p.positions ? p.positions[tok] : l;
      if (pos >= 0 && pos < p.n_pos) {
        const float cs = p.rope_cos[(size_t)pos * half + e], sn = p.rope_sin[(size_t)pos * half + e];
        const float r0 = y0 * cs - y1 * sn;
        y1 = y1 * cs + y0 * sn;
        y0 = r0;
      } else if (pos != -1) {
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

// A CTA per tile of 16 rows, whose 8 warps share out the blocks: the most
// parallelism for few tokens or few rows.  A warp has the codes of its next four
// blocks on their way (all of its blocks, up to 4096 channels), copied to shared
// memory by the lanes that will read them, so that they take no registers and
// need no barrier.  (CTAs that stay and go on to further tiles with the ring
// running on were slower: their addresses and bounds are more instructions than a new
// CTA's; one token, 4096 -> 131072, 100 us against 84.)  8 warps and three CTAs an SM:
// one token, 4096 -> 16384, 13.2 us; 4 warps 14.2, two CTAs 15.3, four 14.3 (spills).
// NT: tiles of 8 tokens.
template <typename T, int NT, int NG>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 3 : NT == 2 ? 2 : 1)
w4_split_kernel(W4Problem p) {
  constexpr int kTok = NT * 8, kAhead = 4;
  __shared__ float red[kWarps][kTile][kTok + 1];
  extern __shared__ __align__(16) uint8_t smem[];  // [kWarps][kAhead][2][32] pieces of 16 bytes
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int i = lane >> 2, c = lane & 3;
  const int t0 = blockIdx.y * kTok;
  const int nt = min(kTok, p.M - t0);
  const int nblk = (p.K + kBlock - 1) / kBlock;
  const Row<NG> ra(p, blockIdx.x, i, nblk, c), rb(p, blockIdx.x, i + 8, nblk, c);
  const T* x = static_cast<const T*>(p.x) + (size_t)(t0 + i) * p.K + 8 * c;  // this lane's first token
  uint4* mine = reinterpret_cast<uint4*>(smem) + warp * kAhead * 64 + lane;
  GroupParams<NG> par[kAhead][2];
  auto start = [&](int u, int blk) {
    if (blk < nblk) {
      const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(mine + u * 64));
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(ra.block(blk)) : "memory");
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + 512), "l"(rb.block(blk)) : "memory");
      ra.load(par[u][0], blk);
      rb.load(par[u][1], blk);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int u = 0; u < kAhead; ++u) start(u, warp + u * kWarps);
  float acc[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[n][e] = 0.f;
  // bf16 tokens of a block are loaded together, fp32 ones (twice the registers,
  // and three parts) piece by piece.
  constexpr bool kTogether = TokenFrag<T>::kParts == 1 && NT <= 2;
#pragma unroll 1
  for (int b0 = warp; b0 < nblk; b0 += kWarps * kAhead) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int blk = b0 + u * kWarps;
      if (blk < nblk) {
        const T* xb = x + (uint32_t)blk * kBlock;
        const int left = p.K - blk * kBlock - 8 * c;  // channels from this lane's on
        auto tokens = [&](int j, TokenFrag<T>(&to)[NT]) {
#pragma unroll
          for (int n = 0; n < NT; ++n) to[n].load(xb + (size_t)(n * 8) * p.K + 32 * j, n * 8 + i < nt && 32 * j < left);
        };
        TokenFrag<T> f[kTogether ? 4 : 1][NT];
        if constexpr (kTogether) {
#pragma unroll
          for (int j = 0; j < 4; ++j) tokens(j, f[j]);
        }
        asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
        const uint4 ca = mine[u * 64], cb = mine[u * 64 + 32];
        if (NG > 1 && blk == nblk - 1) {
          const int groups = (p.K - blk * kBlock + kBlock / NG - 1) / (kBlock / NG);
          par[u][0].cut(groups);
          par[u][1].cut(groups);
        }
        multiply<T, NT, NG>(ca, cb, par[u][0], par[u][1], [&](int j, TokenFrag<T>(&to)[NT]) {
          if constexpr (kTogether) {
#pragma unroll
            for (int n = 0; n < NT; ++n) to[n] = f[j][n];
          } else {
            tokens(j, to);
          }
        }, acc);
        start(u, blk + kWarps * kAhead);
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
  write_tile<T>(p, blockIdx.x, t0, nt, threadIdx.x, kThreads, [&](int m, int t) {
    float s = red[0][m][t];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) s += red[w][m][t];
    return s;
  });
}

// A CTA per 64 rows, one tile a warp, all blocks in turn: the tokens' channels of
// a block are copied to shared memory once for the four tiles, two blocks ahead
// (one ahead for 64 fp32 tokens, whose blocks are 32 KB: with three slots two CTAs
// fit an SM, with four one, and 4096 -> 16384 takes 134 us, 162 against 311 when that was measured), and a
// warp's codes are loaded three blocks ahead into registers.
constexpr int kRowWarps = 4;
template <typename T, int NT>
constexpr int kRowStages = NT * 8 * kBlock * sizeof(T) >= 32768 ? 3 : 4;

template <typename T, int NT, int NG>
__global__ void __launch_bounds__(kRowWarps * 32, NT <= 2 ? 4 : NT == 4 ? 3 : 2)
w4_rows_kernel(W4Problem p) {
  constexpr int kTok = NT * 8, kStages = kRowStages<T, NT>;
  constexpr int kRowBytes = kBlock * (int)sizeof(T), kPieces = kRowBytes / 16;  // of a token and block
  extern __shared__ __align__(16) uint8_t smem[];                               // [kStages][kTok][kRowBytes]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int i = lane >> 2, c = lane & 3;
  const int t0 = blockIdx.y * kTok;
  const int nt = min(kTok, p.M - t0);
  const int nblk = (p.K + kBlock - 1) / kBlock;
  const int tile = blockIdx.x * kRowWarps + warp;
  const Row<NG> ra(p, tile, i, nblk, c), rb(p, tile, i + 8, nblk, c);
  const uint8_t* x = reinterpret_cast<const uint8_t*>(static_cast<const T*>(p.x) + (size_t)t0 * p.K);
  // Piece q of token t lies at q ^ swizzle(t): the 8 lanes that read together
  // (two tokens, 4 or 8 pieces apart) then reach different banks.
  auto swizzle = [](int t) { return sizeof(T) == 2 ? (t & 1) * 4 : 0; };
  auto copy = [&](int blk) {
    if (blk < nblk) {
      uint8_t* stage = smem + (blk % kStages) * (kTok * kRowBytes);
      const int left = (p.K - blk * kBlock) * (int)sizeof(T);  // bytes of a row from here
#pragma unroll
      for (int e = threadIdx.x; e < kTok * kPieces; e += kRowWarps * 32) {
        const int t = e / kPieces, q = e % kPieces;
        uint8_t* dst = stage + t * kRowBytes + (q ^ swizzle(t)) * 16;
        if (t < nt && q * 16 < left) {
          const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to),
                       "l"(x + ((size_t)t * p.K + blk * kBlock) * sizeof(T) + q * 16) : "memory");
        } else {
          *reinterpret_cast<uint4*>(dst) = uint4{0, 0, 0, 0};
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  float acc[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[n][e] = 0.f;
  struct Block {
    uint4 a, b;
    GroupParams<NG> pa, pb;
  } w[3];
  auto load = [&](Block& to, int blk) {
    if (blk < nblk) {
      to.a = ld_once_16(ra.block(blk));
      to.b = ld_once_16(rb.block(blk));
      ra.load(to.pa, blk);
      rb.load(to.pb, blk);
    }
  };
#pragma unroll
  for (int e = 0; e < 3; ++e) load(w[e], e);
#pragma unroll
  for (int e = 0; e < kStages - 2; ++e) copy(e);
  auto use = [&](Block& r, int blk) {
    copy(blk + kStages - 2);  // (its slot was last read two blocks ago, before the last barrier)
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
    __syncthreads();
    const uint8_t* stage = smem + (blk % kStages) * (kTok * kRowBytes);
    if (NG > 1 && blk == nblk - 1) {
      const int groups = (p.K - blk * kBlock + kBlock / NG - 1) / (kBlock / NG);
      r.pa.cut(groups);
      r.pb.cut(groups);
    }
    multiply<T, NT, NG>(r.a, r.b, r.pa, r.pb, [&](int j, TokenFrag<T>(&to)[NT]) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int t = n * 8 + i;
        const int q = (sizeof(T) == 2 ? 4 * j + c : 8 * j + 2 * c) ^ swizzle(t);
        to[n].load(reinterpret_cast<const T*>(stage + t * kRowBytes + q * 16), true);
      }
    }, acc);
    load(r, blk + 3);
  };
#pragma unroll 1
  for (int blk = 0; blk < nblk; blk += 3) {
    use(w[0], blk);
    if (blk + 1 < nblk) use(w[1], blk + 1);
    if (blk + 2 < nblk) use(w[2], blk + 2);
  }
  // Each warp's sums to its own part of shared memory, in order of rows.
  __syncthreads();
  float(*mine)[kTok + 1] = reinterpret_cast<float(*)[kTok + 1]>(smem) + warp * kTile;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    mine[i][n * 8 + 2 * c] = acc[n][0];
    mine[i][n * 8 + 2 * c + 1] = acc[n][1];
    mine[i + 8][n * 8 + 2 * c] = acc[n][2];
    mine[i + 8][n * 8 + 2 * c + 1] = acc[n][3];
  }
  __syncwarp();
  write_tile<T>(p, tile, t0, nt, lane, 32, [&](int m, int t) { return mine[m][t]; });
}

template <typename T, int NT, int NG>
cudaError_t launch_tokens(const W4Problem& p, cudaStream_t st) {
  const unsigned tiles = (p.N + kTile - 1) / kTile, passes = (p.M + NT * 8 - 1) / (NT * 8);
  // 64 rows a CTA where that gives every SM one.  bf16 tokens, 4096 channels, us with 64
  // rows a CTA / with the blocks shared out:
  //   tokens         16            17            32            64
  //   4096 rows   15.0 /  6.3   19.1 /  9.5   19.3 / 11.4   30.1 / 23.1
  //   6144 rows   16.5 / 10.5   20.4 / 13.2   20.7 / 16.2   31.1 / 33.5
  //   16384 rows  20.8 / 21.8   26.6 / 32.9   27.2 / 38.6   42.0 / 79.1
  // and fp32 tokens:
  //   6144 rows   32.3 / 17.0   64.5 / 29.8   66.1 / 30.9  116.5 / 87.5
  //   16384 rows  43.5 / 38.2   72.3 / 72.8   73.9 / 75.6  134.1 / 216.1
  // With 8 tokens or fewer there is little to share, and the split is as fast or faster.
  if constexpr (NT > 1) {
    if (tiles >= (unsigned)(kRowWarps * kSMs)) {
      constexpr int copies = kRowStages<T, NT> * NT * 8 * kBlock * (int)sizeof(T), sums = kRowWarps * kTile * (NT * 8 + 1) * 4;
      constexpr int bytes = copies > sums ? copies : sums;
      if (bytes > 48 * 1024) {
        cudaError_t e =
            cudaFuncSetAttribute(w4_rows_kernel<T, NT, NG>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
      }
      w4_rows_kernel<T, NT, NG><<<dim3((tiles + kRowWarps - 1) / kRowWarps, passes), kRowWarps * 32, bytes, st>>>(p);
      return cudaGetLastError();
    }
  }
  constexpr int ring = kWarps * 4 * 64 * 16, fixed = kWarps * kTile * (NT * 8 + 1) * 4;
  if (ring + fixed > 48 * 1024) {
    cudaError_t e = cudaFuncSetAttribute(w4_split_kernel<T, NT, NG>, cudaFuncAttributeMaxDynamicSharedMemorySize, ring);
    if (e != cudaSuccess) return e;
  }
  w4_split_kernel<T, NT, NG><<<dim3(tiles, passes), kThreads, ring, st>>>(p);
  return cudaGetLastError();
}

// 8, 16, 32 or 64 tokens a pass: the least that holds them all.
template <typename T, int NG>
cudaError_t launch_group(const W4Problem& p, cudaStream_t st) {
  if (p.M <= 8) return launch_tokens<T, 1, NG>(p, st);
  if (p.M <= 16) return launch_tokens<T, 2, NG>(p, st);
  if (p.M <= 32) return launch_tokens<T, 4, NG>(p, st);
  return launch_tokens<T, 8, NG>(p, st);
}

template <typename T>
cudaError_t launch_type(const W4Problem& p, cudaStream_t st) {
  switch (p.group) {
    case 32: return launch_group<T, 4>(p, st);
    case 64: return launch_group<T, 2>(p, st);
    case 128: return launch_group<T, 1>(p, st);
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
      const unsigned g = grid < kSMs * 16u ? grid : kSMs * 16u;
      if (p.bf16) w4_dequantize_kernel<__nv_bfloat16><<<g, kThreads, 0, st>>>(p);
      else w4_dequantize_kernel<float><<<g, kThreads, 0, st>>>(p);
      break;
    }
  }
  return cudaGetLastError();
}

}  // namespace infini
