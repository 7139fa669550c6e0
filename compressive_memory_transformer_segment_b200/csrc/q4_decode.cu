// Decode step over a segment buffer held in 4 bits (sm_100a).
//
// The streaming decode step of decode.cu with the current segment's keys and
// values as 4-bit codes: in groups of 32 channels, value = s q + m with q in
// 0..15 and bf16 s (scale) and m (minimum).  For the query heads h of one KV
// head (groups j of channels):
//   score_r = sum_j s_rj (sum over j of q_r x) + m_rj (sum over j of x),
//   a_dot   = sum_r p_r v_r / sum_r p_r,
//   sum_r p_r v_r[e] = sum_r (p_r s_rj) q_r[e] + sum_r p_r m_rj   (e in group j)
// so both products run over the codes themselves on the tensor cores, with the
// scales on the outside of the first and folded into the probabilities of the
// second.  Queries and probabilities times scale meet the codes as fp16, in its
// range by powers of two (see Attention).
//
// The floor is the buffer's bytes (5 bits per value), but what bounds it at 64
// streams is the instructions around them: with 4 query heads per KV head half of
// each product's 8 columns are empty, and making operands of the codes, the
// scales and the probabilities take more cycles than the bytes.  A CUDA-core
// version would need 8 multiply-adds per value besides the conversions.
// One warp takes 16 rows at a time (mma.sync: 16 rows x 8 heads):
//   S^T = K Q^T   rows of codes are the A operand (lane 4 i + c: rows i, i + 8),
//   O^T = V^T P^T V's codes are the A operand with the rows along k, P^T the
//                 B operand: the scores' fragments, transposed in registers.
// The layout (see the header) is such that a lane's fragments are contiguous.
// Rows come by asynchronous copies through a ring in shared memory, a warp's own
// (no barrier), three tiles ahead.
//
// Measured (device time): 2 streams at the end of 2048-row segments, 32/8 heads of
// 128, 14 us (6 MB: latency alone); 64 streams at ragged positions below 8192 112
// us for 370 MB, 3.3 TB/s, 0.50 of the copy rate; 8 x 8 x 1500 rows appended and read
// back 34 us for 137 MB, 4.0 TB/s (bound by the instructions that choose the codes).
//
// Grid: the rows of all (stream, KV head, chunk of 8 query heads) are shared out
// in equal parts over as many CTAs as the GPU holds, whatever the streams'
// lengths (read from device memory: one captured launch serves every
// position), and the rows of the memory for sigma(q) M, sigma(q) z with them.
// The last of a head chunk's CTAs to finish (a ticket) merges their partials in
// order and writes the output.  No CTA waits for another.
#include <cuda_fp16.h>

#include "common.cuh"
#include "f32x2.cuh"
#include "kernels.h"
#include "q4_common.cuh"

namespace infini {

namespace {

constexpr int kThreads = 128;       // of a CTA that attends
constexpr int kMoveThreads = 256;   // of one that appends or reads rows
constexpr int kWarps = kThreads / 32;
constexpr int kHeads = 8;               // query heads of a CTA (columns of a product)
constexpr int kUnit = kWarps * 32;      // rows of the smallest share of the work
constexpr int kSMs = 148;
// What a segment costs besides its rows, in units of 128 rows (the latencies of
// its first loads, the memory's rows and its partial's way to the workspace), for every
// shape: 64 streams at ragged positions below 8192, us with 2 / 4 / 8 / 12 / 20:
//   4 heads per KV head, d = 128   148 / 123 / 113 / 119 / 122
//   d = 64                         103 /  78 /  69 /  73 /  77
//   d = 32                          69 /  59 /  50 /  52 /  58
//   1 head per KV head             139 / 116 / 111 / 117 / 120
//   8 heads per KV head            179 / 145 / 128 / 135 / 139
//   fp32 heads, d = 128            200 / 196 / 197 / 201 / 207
//   fp32 heads, d = 64             144 / 128 / 125 / 128 / 131
// and 256 streams below 1024, d = 128: 153 / 132 / 123 / 124 / 130.
constexpr int kLeadUnits = 8;
constexpr int kResident = 3;  // CTAs per SM (bf16 heads; two for fp32 ones)

template <int BYTES> struct RawBytes;
template <> struct RawBytes<2> { using type = unsigned short; };
template <> struct RawBytes<4> { using type = uint32_t; };
template <> struct RawBytes<8> { using type = uint2; };
template <> struct RawBytes<16> { using type = uint4; };

template <int BYTES>
struct Raw {
  typename RawBytes<BYTES>::type v;
  __device__ __forceinline__ void load(const uint8_t* p) { v = *reinterpret_cast<const decltype(v)*>(p); }
  __device__ __forceinline__ uint32_t word(int j) const {
    if constexpr (BYTES == 2) return v;
    else return reinterpret_cast<const uint32_t*>(&v)[j];
  }
  // Halfword j of this and of `other`, in the low and the high half.
  __device__ __forceinline__ uint32_t half_pair(const Raw& other, int j) const {
    return __byte_perm(word(j / 2), other.word(j / 2), j % 2 == 0 ? 0x5410 : 0x7632);
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

__device__ __forceinline__ float max_or_nan(float a, float b) {
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(a) : "f"(b));
  return a;
}

// 8 channels 8 w .. 8 w + 7 of a row, held by one lane, into the buffer; the 4
// lanes of a 32-channel group are neighbours and call together.  fp32
// arithmetic with one rounding per operation; a group with a NaN becomes NaN.
template <int D>
__device__ __forceinline__ void store_group(const float (&x)[8], int w, bool key, uint8_t* codes,
                                            __nv_bfloat16* sm, bool active) {
  constexpr int NJ = D / 32;
  const int j = w >> 2, c = w & 3;
  float lo = x[0], hi = x[0];  // hi is NaN once a value is
#pragma unroll
  for (int e = 1; e < 8; ++e) {
    lo = fminf(lo, x[e]);
    hi = max_or_nan(hi, x[e]);
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = max_or_nan(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  __nv_bfloat162 par;
  par.y = __float2bfloat16_rn(lo);
  const float m = __bfloat162float(par.y);
  const float range = __fsub_rn(hi, m);
  par.x = __float2bfloat16_rn(__fmul_rn(fmaxf(range, 0.f), 1.f / 15.f));
  const float s = __bfloat162float(par.x);
  if (range != range) par = __floats2bfloat162_rn(NAN, NAN);
  // Codes: the quotient (x - m) / s rounded to the nearest integer, ties to even,
  // in 0..15.  An approximate quotient finds the half h = k + 1/2 nearest to it; the
  // sign of x - m - h s, which one fused operation gives exactly (h s fits 13 bits),
  // then says on which side of h the quotient lies.  Rounding the quotient to fp32
  // first changes nothing: where x - m is not h s it differs by 2^-24 of it or
  // more, and half a step at h is less.  Ties are not rare (bf16 values and a bf16
  // scale: about one group in eight has one), so no branch looks for them.
  float2 d[4];
  float s1 = s;
#pragma unroll
  for (int e = 0; e < 4; ++e) d[e] = add({x[2 * e], x[2 * e + 1]}, {-m, -m});
  if (!(s >= 0x1p-100f && s < INFINITY)) {  // all codes 0, or a scale whose reciprocal overflows
    const bool none = !(s > 0.f && s < INFINITY);
    s1 = none ? 1.f : s * 0x1p100f;
#pragma unroll
    for (int e = 0; e < 4; ++e) d[e] = none ? float2{0.f, 0.f} : mul(d[e], {0x1p100f, 0x1p100f});
  }
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s1));
  inv *= 1.f / 14.f;
  constexpr float kRound = 12582912.f;  // 1.5 2^23: a sum with it has an integer in its low bits
  uint32_t q[8];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 part = {__saturatef(fmaf(d[e].x, inv, -0.5f / 14.f)), __saturatef(fmaf(d[e].y, inv, -0.5f / 14.f))};
    const float2 u = fma(part, {14.f, 14.f}, {kRound, kRound});
    // (k - 2^23 3 / 2 and the half in two steps: the constant of one is no fp32.)
    const float2 r = fma(add(add(u, {-kRound, -kRound}), {0.5f, 0.5f}), {-s1, -s1}, d[e]);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t k = __float_as_uint(h ? u.y : u.x) & 15u;
      q[2 * e + h] = k + (__float_as_int(h ? r.y : r.x) + (int)(k & 1u) > 0);  // r > 0, or 0 and k odd
    }
  }
  if (!active) return;
  uint32_t word = 0;
  if (key) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      word += q[e] << ((e & 1) ? 2 * e + 14 : 2 * e);
    reinterpret_cast<uint32_t*>(codes)[c * NJ + j] = word;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) word += q[e] << 4 * e;
    unsigned short* halves = reinterpret_cast<unsigned short*>(codes);
    halves[2 * c * NJ + j] = (unsigned short)word;
    halves[(2 * c + 1) * NJ + j] = (unsigned short)(word >> 16);
  }
  if (c == 0) reinterpret_cast<__nv_bfloat162*>(sm)[j] = par;
}

// 8 consecutive elements as floats (16- or 32-byte aligned).
__device__ __forceinline__ void load8(const __nv_bfloat16* x, float (&v)[8]) {
  const uint4 r = *reinterpret_cast<const uint4*>(x);
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[2 * e] = __uint_as_float(w[e] << 16);
    v[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load8(const float* x, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(x)[0], b = reinterpret_cast<const float4*>(x)[1];
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void store8(__nv_bfloat16* x, const float (&v)[8]) {
  uint4 r;
  uint32_t* w = reinterpret_cast<uint32_t*>(&r);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const __nv_bfloat162 t = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
    w[e] = *reinterpret_cast<const uint32_t*>(&t);
  }
  *reinterpret_cast<uint4*>(x) = r;
}
__device__ __forceinline__ void store8(float* x, const float (&v)[8]) {
  reinterpret_cast<float4*>(x)[0] = {v[0], v[1], v[2], v[3]};
  reinterpret_cast<float4*>(x)[1] = {v[4], v[5], v[6], v[7]};
}

// The token's key and value into row `row` of the buffer, by one warp: half of
// it for each.
template <typename T, int D>
__device__ __forceinline__ void store_token(const Q4Problem& p, size_t bh, size_t row, int lane) {
  const bool key = lane < 16, active = (lane & 15) < D / 8;
  const int w = lane & 15 & (D / 8 - 1);
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (active) load8(static_cast<const T*>(key ? p.k_t : p.v_t) + bh * D + 8 * w, v);
  store_group<D>(v, w, key, (key ? p.k_codes : p.v_codes) + row * (D / 2),
                 (key ? p.k_scale : p.v_scale) + row * (D / 16), active);
}

// fp16 parts that hold a query of this type.
template <typename T> struct Parts;
template <> struct Parts<__nv_bfloat16> { static constexpr int n = 1; };
template <> struct Parts<float> { static constexpr int n = 2; };

// The index of a product along 16 rows (i and i + 8, or 2c, 2c + 1, 2c + 8, 2c +
// 9) stands for row k_row(index) of its eight: an order in which the key loads
// from shared memory have no bank conflict and the value loads two-way ones.
__device__ __forceinline__ int k_row(int i) { return (i & 1) ? 4 + ((i >> 1) ^ 1) : i >> 1; }

// 16 rows as a lane needs them.  Keys: chunk c of rows k_row(i), + 8, their
// parameters, and their minima (scales) in two groups as A fragments: groups
// 2 (c & 1) and the next for d = 128, 0 and 1 for 64, 0 and 0 for 32.
template <int D>
struct KeyTile {
  Raw<D / 8> k[2], kp[2];
  uint32_t kmin[2], kcen[2];
};
// Values: chunk i of rows k_row(2c), k_row(2c + 1), + 8, + 8; parameters of rows
// k_row(i), + 8.
template <int D>
struct ValueTile {
  Raw<D / 8> vp[2];
  Raw<D / 16> v[4];
};

// A warp's ring in shared memory, filled by asynchronous copies of 16 rows at a
// time: the next slots' loads are in flight while two are used (one's keys, the
// one before's values), without registers to hold them.
template <int D>
struct Ring {
  static constexpr int kRows = 16;
  static constexpr int kCodes = kRows * (D / 2), kParams = kRows * (D / 8);  // bytes of a slot's rows
  static constexpr int kSlot = 2 * kCodes + 2 * kParams;
  static constexpr int kStages = 4;
  // The ring first carries the warp's rows of the memory M, kMem at a time.
  static constexpr int kMem = kSlot / (D * 4);
  static_assert(kMem * D * 4 == kSlot, "whole rows");
  uint8_t* smem;
  const uint8_t *k, *v, *kp, *vp;  // the first row
  const float* mem;                // the warp's first row of M
  int n, lane;                     // rows
  int mem_rows, mem_items;
  int first;                       // the warp's first row behind them

  __device__ __forceinline__ void set(const Q4Problem& p, uint8_t* ring, size_t row0, int rows, int lane_) {
    smem = ring; n = rows; lane = lane_;
    k = p.k_codes + row0 * (D / 2);
    v = p.v_codes + row0 * (D / 2);
    kp = reinterpret_cast<const uint8_t*>(p.k_scale) + row0 * (D / 8);
    vp = reinterpret_cast<const uint8_t*>(p.v_scale) + row0 * (D / 8);
  }
  template <int BYTES>
  __device__ __forceinline__ static void copy(uint32_t to, const uint8_t* src) {
    if constexpr (BYTES == 16)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(src) : "memory");
    else
      asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(src), "n"(BYTES) : "memory");
  }
  // BYTES zeros instead of a copy.
  template <int BYTES>
  __device__ __forceinline__ static void zero(uint32_t to) {
#pragma unroll
    for (int e = 0; e < BYTES; e += 4) asm volatile("st.shared.u32 [%0], %1;" ::"r"(to + e), "r"(0) : "memory");
  }
  // Two arrays a and b of kRows rows of ROW bytes each, in pieces of BYTES, to
  // `to` and behind one another; lanes take neighbouring pieces.
  template <int ROW, int BYTES, bool FULL>
  __device__ __forceinline__ void rows(uint32_t to, const uint8_t* a, const uint8_t* b, int left) const {
    constexpr int kPieces = kRows * ROW / BYTES;  // of one array
    static_assert(2 * kPieces % 32 == 0 && (kPieces % 32 == 0 || kPieces == 16), "whole turns of the warp");
#pragma unroll
    for (int e = 0; e < 2 * kPieces / 32; ++e) {
      int piece = lane + 32 * (kPieces >= 32 ? e % (kPieces >= 32 ? kPieces / 32 : 1) : 0);
      const uint8_t* src = kPieces >= 32 ? (e < kPieces / 32 ? a : b) : (lane < 16 ? a : b);
      if (kPieces < 32) piece &= 15;
      const uint32_t dst = to + (lane + 32 * e) * BYTES;
      if (FULL || piece * BYTES / ROW < left) copy<BYTES>(dst, src + piece * BYTES);
      else zero<BYTES>(dst);
    }
  }
  template <bool FULL>
  __device__ __forceinline__ void fill_rows(int slot, int r) const {
    const uint32_t s = static_cast<uint32_t>(__cvta_generic_to_shared(smem)) + slot * kSlot;
    const size_t code = (size_t)r * (D / 2), par = (size_t)r * (D / 8);
    rows<D / 2, 16, FULL>(s, k + code, v + code, n - r);
    rows<D / 8, D / 8, FULL>(s + 2 * kCodes, kp + par, vp + par, n - r);
  }
  // Starts the copy of rows r .. r + kRows - 1; rows from n on become zeros,
  // whatever the buffer holds there.
  __device__ __forceinline__ void fill(int slot, int r) const {
    if (__builtin_expect(r + kRows <= n, 1)) fill_rows<true>(slot, r);
    else fill_rows<false>(slot, r);
  }
  // Starts the copy of the warp's item x: kMem rows of M, or 16 rows.
  __device__ __forceinline__ void next(int slot, int x) const {
    if (x >= mem_items) {
      const int r = first + (x - mem_items) * kWarps * kRows;
      if (r < n) fill(slot, r);
    } else {
      const uint32_t s = static_cast<uint32_t>(__cvta_generic_to_shared(smem)) + slot * kSlot;
      const uint8_t* src = reinterpret_cast<const uint8_t*>(mem + (size_t)x * kMem * D);
      const int bytes = min(kMem, mem_rows - x * kMem) * D * 4;
#pragma unroll
      for (int e = 0; e < kSlot; e += 512)
        if (e + lane * 16 < bytes) copy<16>(s + e + lane * 16, src + e + lane * 16);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  // Waits until at most LEFT groups of this lane are in flight.
  template <int LEFT>
  __device__ __forceinline__ static void wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
    __syncwarp();
  }
  __device__ __forceinline__ void read(KeyTile<D>& t, int slot) const {
    const int i = lane >> 2, c = lane & 3, kr = k_row(i);
    const uint8_t* s = smem + slot * kSlot;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint8_t* par = s + 2 * kCodes + (kr + 8 * e) * (D / 8);
      t.k[e].load(s + (kr + 8 * e) * (D / 2) + c * (D / 8));
      t.kp[e].load(par);
      uint32_t a = t.kp[e].word(0), b = t.kp[e].word(D / 32 > 1 ? 1 : 0);
      if constexpr (D == 128) {
        const uint2 w = *reinterpret_cast<const uint2*>(par + (c & 1) * 8);
        a = w.x; b = w.y;
      }
      t.kmin[e] = __byte_perm(a, b, 0x7632);
      t.kcen[e] = __byte_perm(a, b, 0x5410);
    }
  }
  __device__ __forceinline__ void read(ValueTile<D>& t, int slot) const {
    const int i = lane >> 2, c = lane & 3, kr = k_row(i);
    const uint8_t* s = smem + slot * kSlot;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = 8 * e;
      t.vp[e].load(s + 2 * kCodes + kParams + (kr + 8 * e) * (D / 8));
      t.v[2 * e].load(s + kCodes + (c + r) * (D / 2) + i * (D / 16));
      t.v[2 * e + 1].load(s + kCodes + (4 + (c ^ 1) + r) * (D / 2) + i * (D / 16));
    }
  }
};

// 4-bit codes as fp16 operands without arithmetic: the fp16 with the bits of a
// small integer n is n 2^-24 (subnormals, and the first exponent, are linear
// up to 2^11 2^-24), so masking is all the conversion there is.  Of the four
// codes of a 16-bit half the first and third (after one shift by 8) come out as
// q, the second and fourth, masked where they stand, as 16 q; whoever uses
// them has 1/16 in the other operand or in the result.
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t (&out)[4]) {
  out[0] = w & 0x000f000fu;
  out[1] = w & 0x00f000f0u;
  out[2] = (w >> 8) & 0x000f000fu;
  out[3] = (w >> 8) & 0x00f000f0u;
}
// The tensor cores align such products by their operands' exponents, zeros in
// front included, which drops what lies 2^-13 of a code below the largest product:
// at most 2^-13 of the span of a sum's codes, and about 2^-16 of a sum of 16 terms
// of a size.  That is right for bf16 heads, not for fp32 ones.  Those take q - 8 as a
// normal number: 1024 + q by insertion, minus 1032; 1024 + 16 q, over 16 and minus
// 72 (both exact).  (For bf16 heads the codes three bits further up, by one shift
// more in two: 114.6 us against 111.3 for 64 streams.)
template <bool EXACT>
__device__ __forceinline__ void code_pairs(uint32_t w, uint32_t (&out)[4]) {
  codes_f16(w, out);
  if constexpr (EXACT) {
    const __half2 one = __floats2half2_rn(-1032.f, -1032.f), sixteenth = __floats2half2_rn(0.0625f, 0.0625f),
                  shift = __floats2half2_rn(-72.f, -72.f);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t bits = out[e] | 0x64006400u;
      const __half2 n = *reinterpret_cast<const __half2*>(&bits);
      const __half2 v = e % 2 == 0 ? __hadd2(n, one) : __hfma2(n, sixteenth, shift);
      out[e] = *reinterpret_cast<const uint32_t*>(&v);
    }
  }
}

// f16x2 of (lo, hi), and what it leaves of them.
__device__ __forceinline__ uint32_t split_f16(float& lo, float& hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  lo -= __low2float(v);
  hi -= __high2float(v);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// 2^e, -126 <= e <= 127.
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }

// Running attention of one warp over its rows, for 8 heads: fragments of
// heads 2c, 2c + 1.  The operands that meet the codes are fp16.
// Queries are kept in its range by a power of two per head, set by the largest
// element: bf16 heads in one part (exact down to 2^-27 of that), fp32 heads in two
// (2^-22 of an element, and 2^-39 of the largest).
// The weights, probabilities times scale, go in as two parts (2^-22 of a weight, for
// bf16 heads 2^-21): one part, 2^-11 at most, would be the sum's largest error, since it
// counts by the codes, which all lie on one side of zero (bf16 heads, 2048 rows: 4e-4 of
// the output against 2e-5).  With at most 4 query heads per KV head and one part per
// query (kPaired) the second parts take the columns of heads 4 .. 7, whose lanes hold the
// same four heads again: 64 streams of 4 heads 112 us, against 107 with one part and 125 with
// two products.  (8 heads: 124 us by two products, 110 with one part.)
// fp32 heads add a tile's products, and the second parts' of a score, to their sums by
// fp32 additions: the tensor cores truncate the sums they go on with (2048 rows: error 5.1e-7
// against 2.5e-7; 64 streams 197 against 202 us).
// The weights' range is a power of two for each head and group (`unit`): their largest
// so far lies at 2^8 .. 2^15 (lower() and rebase() see to it), so that what fp16
// drops, 2^-24, is 2^-32 of it or less, whatever the scales of other groups, of rows of
// little probability, and of what other heads attend to.
template <int D, int NP, bool WIDE>
struct Attention {
  static constexpr int NJ = D / 32;
  static constexpr bool kExact = NP > 1;
  static constexpr float kUnit1 = kExact ? 1.f : 0x1p24f;        // of a product with q, or with q - 8
  static constexpr float kOdd = kExact ? 1.f : 0.0625f;          // second and fourth codes
  static constexpr float kCenter = kExact ? 8.f : 0.f;
  static constexpr float kLead = 7.f;
  static constexpr bool kPaired = NP == 1 && !WIDE;
  static constexpr int VP = kPaired ? 1 : 2;                     // parts of a weight in a lane
  static constexpr float kMostUnit = 0x1p120f;
  uint32_t qf[NJ][NP][4];  // queries of head i as B fragments, times 2^e (pairs 1, 3: kOdd of that)
  // Sums of head i's scaled query over each group, in units of a code, as a B
  // operand of bf16 parts: index 4 part + group (d = 128), 2 part + group (64),
  // 2 part (32) along the minima.
  uint32_t qs[2], qc[2];   // (qc: times kCenter)
  float f1, f2[2];         // log2(e) / sqrt(d) kUnit1, 2^-e: scores to powers of two
  float m[2], l[2];        // reference of the powers; their sum over this lane's rows
  float o[2 * NJ][4];      // O^T without the minima, times unit / kUnit1 (rows i + 8: over kOdd too)
  float omin[NJ][2];       // sum of p (minimum + kCenter scale) over this lane's rows
  float unit[NJ][2];       // powers of two: p scale unit is what group j's products get
  float minus;             // kPaired: 0 in the lanes of the first parts, -1 of the second

  // q_t: this KV head's first query; ng: heads of it that exist.
  template <typename T>
  __device__ __forceinline__ void init(const T* q_t, int ng, int lane) {
    const int i = lane >> 2, c = lane & 3, head = kPaired ? i & 3 : i;
    minus = c < 2 ? 0.f : -1.f;
    float x[NJ][8], top = 0.f;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[j][e] = 0.f;
      if (head < ng) load8(q_t + (size_t)head * D + 32 * j + 8 * c, x[j]);
#pragma unroll
      for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(x[j][e]));
    }
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    // The largest element goes to 2^14 .. 2^15.
    const int e = min(14 + 127 - (__float_as_int(top) >> 23), 100);
    const float up = pow2(e);
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      float s = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        x[j][k] *= up;
        s += x[j][k];
      }
      s += __shfl_xor_sync(0xffffffffu, s, 1);
      s += __shfl_xor_sync(0xffffffffu, s, 2);
      sum[j] = s * (1.f / kUnit1);
#pragma unroll
      for (int k = 2; k < 8; k += 4) {
        x[j][k] *= kOdd;
        x[j][k + 1] *= kOdd;
      }
#pragma unroll
      for (int part = 0; part < NP; ++part)
#pragma unroll
        for (int k = 0; k < 4; ++k) qf[j][part][k] = split_f16(x[j][2 * k], x[j][2 * k + 1]);
    }
    // This lane's indexes along the minima: 2c, 2c + 1 (b0), 2c + 8, 2c + 9 (b1).
    {
      const bool upper = NJ == 4 && (c & 1);
      float lo = upper ? sum[2] : sum[0], hi = upper ? sum[3] : sum[1];
      uint32_t part[3];
#pragma unroll
      for (int k = 0; k < 3; ++k) part[k] = split_bf16(lo, hi);
      if constexpr (NJ == 4) {
        qs[0] = c < 2 ? part[0] : part[1];
        qs[1] = c < 2 ? part[2] : 0u;
      } else {
        qs[0] = c == 0 ? part[0] : c == 1 ? part[1] : c == 2 ? part[2] : 0u;
        qs[1] = 0u;
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const __nv_bfloat162 v = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&qs[k]),
                                         __floats2bfloat162_rn(kCenter, kCenter));  // a power of two
        qc[k] = *reinterpret_cast<const uint32_t*>(&v);
      }
    }
    f1 = rsqrtf((float)D) * 1.4426950408889634f * kUnit1;
    f2[0] = pow2(-__shfl_sync(0xffffffffu, e, 8 * c));
    f2[1] = pow2(-__shfl_sync(0xffffffffu, e, 8 * c + 4));
    clear();
  }

  // Before the first row.
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      omin[j][0] = omin[j][1] = 0.f;
      unit[j][0] = unit[j][1] = kMostUnit;
#pragma unroll
      for (int k = 0; k < 4; ++k) o[2 * j][k] = o[2 * j + 1][k] = 0.f;
    }
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;
  }

  // 1 / x of a power of two, 2^-126 <= x <= 2^126.
  __device__ __forceinline__ static float inverse(float x) { return __int_as_float((254 << 23) - __float_as_int(x)); }
  // O^T of group j and head h, times x.
  __device__ __forceinline__ void scale_o(int j, int h, float x) {
    o[2 * j][h] *= x; o[2 * j][2 + h] *= x;
    o[2 * j + 1][h] *= x; o[2 * j + 1][2 + h] *= x;
  }

  // The reference becomes the maximum so far.  The weights that were the largest
  // are now smaller by the factor corr: the units grow by the power of two below 1 / corr.
  __device__ __forceinline__ void rebase(float top0, float top1) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float mn = fmaxf(m[h], column_max(h ? top1 : top0));
      const float corr = exp2_approx(m[h] - mn);  // 0 for the first rows
      const float grow = pow2((int)fminf(mn - m[h], 126.f));
      m[h] = mn;
      l[h] *= corr;
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const float to = fminf(unit[j][h] * grow, kMostUnit);
        omin[j][h] *= corr;
        scale_o(j, h, corr * (to * inverse(unit[j][h])));
        unit[j][h] = to;
      }
    }
  }

  // A weight of this tile reached 2^15 (the first rows' do, but for scales next to 0):
  // the unit of its head and group moves so that the largest lies at 2^8 .. 2^9.
  __device__ __forceinline__ void lower(const ValueTile<D>& t, const float (&pr)[4]) {
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float top = 0.f;  // the largest over 2^8: no product of finite values is infinite
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float w = (pr[2 * e + h] * 0x1p-8f) * t.vp[e].scale(j);
          top = fmaxf(top, w < INFINITY ? w : 0.f);  // (a lost group or score has no say)
        }
        top = column_max(top);
        if (top * 0x1p-7f * unit[j][h] >= 1.f) {
          const float to = pow2(127 - (__float_as_int(top) >> 23));
          scale_o(j, h, to * inverse(unit[j][h]));
          unit[j][h] = to;
        }
      }
  }

  // Scores (as powers of two) of rows k_row(i) (x[0], x[1]) and + 8 (x[2],
  // x[3]) of a tile; minus infinity for rows from `left` on.
  __device__ __forceinline__ void scores(const KeyTile<D>& t, int left, int kr, float (&x)[4]) const {
    // The minima's share first: (minima of a row) times (sums of the queries).
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    mma_bf16(s, t.kmin[0], t.kmin[1], t.kmin[0], t.kmin[1], qs[0], qs[1]);
    if constexpr (kExact) mma_bf16(s, t.kcen[0], t.kcen[1], t.kcen[0], t.kcen[1], qc[0], qc[1]);
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      uint32_t fa[4], fb[4];
      code_pairs<kExact>(t.k[0].word(j), fa);
      code_pairs<kExact>(t.k[1].word(j), fb);
      float d[4];
      mma_f16_first(d, fa[0], fb[0], fa[1], fb[1], qf[j][0][0], qf[j][0][1]);
      mma_f16(d, fa[2], fb[2], fa[3], fb[3], qf[j][0][2], qf[j][0][3]);
#pragma unroll
      for (int part = 1; part < NP; ++part) {
        float small[4];
        mma_f16_first(small, fa[0], fb[0], fa[1], fb[1], qf[j][part][0], qf[j][part][1]);
        mma_f16(small, fa[2], fb[2], fa[3], fb[3], qf[j][part][2], qf[j][part][3]);
#pragma unroll
        for (int e = 0; e < 4; ++e) d[e] += small[e];
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float sc = t.kp[e].scale(j);
#pragma unroll
        for (int h = 0; h < 2; ++h) s[2 * e + h] = fmaf(sc, d[2 * e + h], s[2 * e + h]);
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = kr + 8 * (e >> 1) < left ? s[e] * f1 * f2[e & 1] : -INFINITY;
  }

  // A tile's weights p scale unit as fp16 parts: [group][rows k_row(i), + 8][part].
  __device__ __forceinline__ void weigh(const ValueTile<D>& t, const float (&pr)[4], uint32_t (&w)[NJ][2][VP]) const {
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float sc = t.vp[e].scale(j);
        float x[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) x[h] = pr[2 * e + h] * unit[j][h] * sc;
        if constexpr (kPaired) {
          // The leading 11 bits (which is what truncating to fp16 leaves), or the rest.
          const float2 lead = {__uint_as_float(__float_as_uint(x[0]) & 0xffffe000u),
                               __uint_as_float(__float_as_uint(x[1]) & 0xffffe000u)};
          const float2 part = fma(lead, {minus, minus}, {x[0], x[1]});
          asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(w[j][e][0]) : "f"(part.y), "f"(part.x));
        } else {
#pragma unroll
          for (int part = 0; part < VP; ++part) w[j][e][part] = split_f16(x[0], x[1]);
        }
      }
  }

  // O^T += V^T P^T of a tile with probabilities pr.
  __device__ __forceinline__ void values(const ValueTile<D>& t, const float (&pr)[4]) {
    uint32_t w[NJ][2][VP];
    weigh(t, pr, w);
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < NJ; ++j) top = __vmaxu2(top, __vmaxu2(w[j][0][0], w[j][1][0]));
    if (__builtin_expect(__any_sync(0xffffffffu, max(top & 0xffffu, top >> 16) >= 0x7800u), 0)) {
      lower(t, pr);
      weigh(t, pr, w);
    }
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      // Codes of group j: element t of a lane's four is channel 32 j + 4 i + t,
      // indexes 2c, 2c + 1 (lo) and 2c + 8, 2c + 9 (hi) along the rows.
      uint32_t lo[4], hi[4];
      code_pairs<kExact>(t.v[0].half_pair(t.v[1], j), lo);
      code_pairs<kExact>(t.v[2].half_pair(t.v[3], j), hi);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float sc = t.vp[e].scale(j);
        const float mn = kExact ? fmaf(kCenter, sc, t.vp[e].minimum(j)) : t.vp[e].minimum(j);
#pragma unroll
        for (int h = 0; h < 2; ++h) omin[j][h] = fmaf(pr[2 * e + h], mn, omin[j][h]);
      }
#pragma unroll
      for (int part = 0; part < VP; ++part) {
        const uint32_t b0 = transpose8(w[j][0][part]), b1 = transpose8(w[j][1][part]);
        if constexpr (kExact) {
          float t[2][4];
          mma_f16_first(t[0], lo[0], lo[1], hi[0], hi[1], b0, b1);
          mma_f16_first(t[1], lo[2], lo[3], hi[2], hi[3], b0, b1);
#pragma unroll
          for (int e = 0; e < 8; ++e) o[2 * j + e / 4][e % 4] += t[e / 4][e % 4];
        } else {
          mma_f16(o[2 * j], lo[0], lo[1], hi[0], hi[1], b0, b1);
          mma_f16(o[2 * j + 1], lo[2], lo[3], hi[2], hi[3], b0, b1);
        }
      }
    }
  }

  // Probabilities (powers of two relative to a reference m, at most 2^kLead) of
  // a tile from its scores x.  A maximum is taken over the warp only when a score
  // leaves that room (and by the first rows), not for every tile.
  __device__ __forceinline__ void probabilities(const float (&x)[4], float (&pr)[4]) {
    const float top0 = fmaxf(x[0], x[2]), top1 = fmaxf(x[1], x[3]);
    if (__builtin_expect(__any_sync(0xffffffffu, fmaxf(top0 - m[0], top1 - m[1]) > kLead), 0)) rebase(top0, top1);
#pragma unroll
    for (int e = 0; e < 4; ++e) pr[e] = exp2_approx(x[e] - m[e & 1]);
    l[0] += pr[0] + pr[2];
    l[1] += pr[1] + pr[3];
  }

  // All of a ring's rows of this warp (every kWarps-th 16), from item mem_items
  // on, which lies in `slot`.  A turn computes one tile's scores and the tile
  // before's products with the values: two chains that do not wait for each
  // other, in the code of one tile.
  __device__ __forceinline__ void run(const Ring<D>& ring, int slot) {
    using R = Ring<D>;
    const int kr = k_row(ring.lane >> 2);
    float pr[4] = {0.f, 0.f, 0.f, 0.f};
    int before = slot > 0 ? slot - 1 : R::kStages - 1, x = ring.mem_items;
#pragma unroll 1
    for (int r = ring.first; r < ring.n; r += kWarps * R::kRows, ++x) {
      // Of the kStages - 1 groups before this turn's the first is needed; the
      // slot of the tile before is read below and filled again.
      R::template wait<R::kStages - 2>();
      KeyTile<D> keys;
      ring.read(keys, slot);
      float s[4];
      scores(keys, ring.n - r, kr, s);
      ValueTile<D> val;
      if (r > ring.first) {
        ring.read(val, before);
        values(val, pr);
        __syncwarp();  // every lane has read the slot
      }
      ring.next(before, x + R::kStages - 1);
      probabilities(s, pr);
      before = slot;
      slot = slot + 1 < R::kStages ? slot + 1 : 0;
    }
    if (ring.first < ring.n) {
      ValueTile<D> val;
      ring.read(val, before);
      values(val, pr);
    }
    __syncwarp();
  }
};

// Units of a segment of stream b (0: idle): p.lead for what a segment costs
// whatever its length, then one for each p.unit rows.
__device__ __forceinline__ uint32_t stream_units(const Q4Problem& p, int b) {
  const int pos = p.pos[b];
  return pos >= 0 && pos < p.S ? p.lead + pos / p.unit + 1 : 0;
}

// How the units of all segments are shared out.  A segment is what one (stream,
// KV head, chunk of 8 query heads) attends to; segments lie one after another
// (stream by stream, segs of equal length each), and CTA k of `ctas` takes
// units [k U / ctas, (k + 1) U / ctas) of the U in all: equal work whatever
// the streams' lengths are.  (A launch whose units are no more than its CTAs has
// one unit per CTA: none then has two segments.)
struct Share {
  uint32_t units, ctas, per, rest;  // units = ctas per + rest
  __device__ __forceinline__ void set(uint32_t total, uint32_t most) {
    units = total;
    ctas = min(most, total);
    per = ctas ? total / ctas : 0;
    rest = total - per * ctas;
  }
  // (rest is 0 or ctas at most a few hundred: the product fits.)
  __device__ __forceinline__ uint32_t first(uint32_t k) const { return k * per + k * rest / ctas; }
  __device__ __forceinline__ uint32_t owner(uint32_t u) const {
    // Near enough that a turn or two set it right.
    uint32_t k = min((uint32_t)((float)u * ((float)ctas / (float)units)), ctas - 1);
    while (first(k) > u) --k;
    while (k + 1 < ctas && first(k + 1) <= u) ++k;
    return k;
  }
};

// Adds up the streams' units, shares them out, and finds the stream that this
// CTA's first unit lies in, and the stream's first unit.  Every warp does it for
// itself, 32 streams at a time: no barrier.
__device__ __forceinline__ void locate(const Q4Problem& p, uint32_t segs, Share& share, uint32_t& stream,
                                       uint32_t& start) {
  const int lane = threadIdx.x & 31;
  uint32_t total = 0, mine = 0;
#pragma unroll 1
  for (int b = lane; b < p.B; b += 32) total += mine = stream_units(p, b) * segs;
  share.set(__reduce_add_sync(0xffffffffu, total), p.ctas);
  if (blockIdx.x >= share.ctas) return;
  const uint32_t want = share.first(blockIdx.x);
  start = 0;
#pragma unroll 1
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    if (p.B > 32) mine = b0 + lane < p.B ? stream_units(p, b0 + lane) * segs : 0;
    uint32_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    const uint32_t behind = __ballot_sync(0xffffffffu, want < start + incl);
    if (behind) {  // the first such lane's stream (`want` lies below the total)
      stream = b0 + __ffs(behind) - 1;
      start += __shfl_sync(0xffffffffu, incl - mine, __ffs(behind) - 1);
      return;
    }
    start += __shfl_sync(0xffffffffu, incl, 31);
  }
  share.ctas = 0;  // (only if the positions changed meanwhile)
}

// A run of units of one segment, and the segment's place.
struct Run {
  uint32_t b, off, seg;  // stream, its first unit, segment of the stream
  uint32_t s0, s1;       // the segment's units of rows
  uint32_t u, end;       // the run's
  int pos, hk, hq0, ng;  // token's row; KV head; query heads hq0 .. hq0 + ng - 1
  __device__ __forceinline__ size_t bh(const Q4Problem& p) const { return (size_t)b * p.H_kv + hk; }
  __device__ __forceinline__ size_t head0(const Q4Problem& p) const { return (size_t)b * p.H_q + hq0; }
  __device__ __forceinline__ bool whole() const { return u == s0 && end == s1; }
};

// What a CTA leaves of a run, per head: the attention over its rows (max
// reference m, sum l, acc[D]) and its share of the retrieval, sigma(q) M and
// sigma(q) z.
template <int D>
struct Partial {
  float acc[D];
  float num[D];
  float m, l, den, unused;  // 16 bytes, read as one
};

// E neighbouring floats that another CTA wrote.
template <int E>
__device__ __forceinline__ void load_columns(const float* p, float (&x)[E]) {
  if constexpr (E == 4) {
    const float4 v = __ldcg(reinterpret_cast<const float4*>(p));
    x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
  } else if constexpr (E == 2) {
    const float2 v = __ldcg(reinterpret_cast<const float2*>(p));
    x[0] = v.x; x[1] = v.y;
  } else {
    x[0] = __ldcg(p);
  }
}

// The ticket of a segment, taken once a CTA's share of it is in the workspace;
// the last CTA merges the partials in CTA order, with the gate.  The whole CTA
// calls it; no CTA waits for another.
template <typename T, int D>
__device__ __forceinline__ void finish(const Q4Problem& p, const Share& share, const Run& r, uint32_t segs) {
  constexpr int E = D / 32, kU = 8;  // channels per lane; partials in flight
  __shared__ int last;       // partials to merge, 0 if this CTA is not the last
  __shared__ uint32_t first_cta;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  unsigned int* ctr = p.ctr + (size_t)r.b * segs + r.seg;
  Partial<D>* part = reinterpret_cast<Partial<D>*>(p.part);
  __syncthreads();  // every thread's share is written
  if (threadIdx.x == 0) {
    const uint32_t k0 = r.whole() ? blockIdx.x : share.owner(r.s0);
    const uint32_t n = r.whole() ? 1 : share.owner(r.s1 - 1) - k0 + 1;
    __threadfence();  // (cumulative: the barrier put the CTA's writes before it)
    last = n == 1 || atomicAdd(ctr, 1u) == n - 1 ? (int)n : 0;
    first_cta = k0;
    __threadfence();  // every other CTA's writes are visible
  }
  __syncthreads();
  const int np = last;
  if (np == 0) return;
  const size_t head0 = r.head0(p);
  // Partial x of head hh: a CTA that has the segment whole leaves it at the
  // heads' own place; of several the first may have had another before this one.
  const bool later = np > 1 && share.first(first_cta) < r.s0 - p.lead;
  const Partial<D>* mine = part + (np == 1 ? head0 : (size_t)p.B * p.H_q + (size_t)first_cta * 2 * kHeads);
  for (int hh = warp; hh < r.ng; hh += kWarps) {
    auto at = [&](int x) { return mine + (size_t)x * 2 * kHeads + (x == 0 && later ? kHeads : 0) + hh; };
    // 32 partials a turn: (m, l, den) one per lane, and 8 at a time every lane's
    // E columns (E l .. E l + E - 1), the first 8 before the weights are needed.
    float mx = -INFINITY, ls = 0.f, den = 0.f, w = 0.f, as[E], num[E];
#pragma unroll
    for (int e = 0; e < E; ++e) as[e] = num[e] = 0.f;
#pragma unroll 1
    for (int k0 = 0; k0 < np; k0 += kU) {
      const bool turn = k0 % 32 == 0;
      float4 t = {-INFINITY, 0.f, 0.f, 0.f};
      if (turn && k0 + lane < np) t = __ldcg(reinterpret_cast<const float4*>(&at(k0 + lane)->m));
      float av[kU][E], nv[kU][E];
#pragma unroll
      for (int k = 0; k < kU; ++k) {
        const Partial<D>* q = at(min(k0 + k, np - 1));
        load_columns<E>(q->acc + E * lane, av[k]);
        load_columns<E>(q->num + E * lane, nv[k]);
      }
      if (turn) {
        const float nm = fmaxf(mx, warp_max(t.x)), corr = exp2_approx(mx - nm);  // 0 for the first
        w = exp2_approx(t.x - nm);  // 0 past the last
        mx = nm;
        ls = fmaf(ls, corr, warp_sum(t.y * w));
        den += warp_sum(t.z);
#pragma unroll
        for (int e = 0; e < E; ++e) as[e] *= corr;
      }
#pragma unroll
      for (int k = 0; k < kU; ++k) {
        const float wk = __shfl_sync(0xffffffffu, w, (k0 + k) & 31);
        if (k0 + k < np) {
#pragma unroll
          for (int e = 0; e < E; ++e) {
            as[e] = fmaf(av[k][e], wk, as[e]);
            num[e] += nv[k][e];
          }
        }
      }
    }
    const float gm = gate_sigmoid(p.beta[r.hq0 + hh]);
    T* out = static_cast<T*>(p.out_t) + (head0 + hh) * D;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float a_mem = den != 0.f ? num[e] / den : 0.f;
      out[E * lane + e] = from_f32<T>(gm * a_mem + (1.f - gm) * (as[e] / ls));
    }
  }
  if (threadIdx.x == 0) *ctr = 0u;  // ready for the next step
}

// A warp's share of the retrieval: its rows of M, which come through the ring
// before the segment's, times sigma(q) (sq: of the warp's first row on), to
// num[kHeads][D].  Returns the slot behind them.
template <int D>
__device__ __forceinline__ int retrieve(const Ring<D>& ring, const float (*sq)[kHeads], float (*num)[D]) {
  using R = Ring<D>;
  constexpr int E = D / 32;  // columns E l .. E l + E - 1 of lane l
  float acc[kHeads][E];
#pragma unroll
  for (int hh = 0; hh < kHeads; ++hh)
#pragma unroll
    for (int e = 0; e < E; ++e) acc[hh][e] = 0.f;
  int slot = 0, before = R::kStages - 1;
#pragma unroll 1
  for (int x = 0; x < ring.mem_items; ++x) {
    R::template wait<R::kStages - 2>();
    ring.next(before, x + R::kStages - 1);  // (read in the turn before)
    const float* rows = reinterpret_cast<const float*>(ring.smem + slot * R::kSlot) + E * ring.lane;
    const int n = min(R::kMem, ring.mem_rows - x * R::kMem);
#pragma unroll 1
    for (int k = 0; k < n; ++k) {
      float mv[E];
      if constexpr (E == 4) {
        const float4 v = *reinterpret_cast<const float4*>(rows + k * D);
        mv[0] = v.x; mv[1] = v.y; mv[2] = v.z; mv[3] = v.w;
      } else if constexpr (E == 2) {
        const float2 v = *reinterpret_cast<const float2*>(rows + k * D);
        mv[0] = v.x; mv[1] = v.y;
      } else {
        mv[0] = rows[k * D];
      }
      const float4 lo = *reinterpret_cast<const float4*>(sq[x * R::kMem + k]);
      const float4 hi = *reinterpret_cast<const float4*>(sq[x * R::kMem + k] + 4);
      const float w[kHeads] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
      for (int hh = 0; hh < kHeads; ++hh)
#pragma unroll
        for (int e = 0; e < E; ++e) acc[hh][e] = fmaf(w[hh], mv[e], acc[hh][e]);
    }
    __syncwarp();  // every lane has read the slot
    before = slot;
    slot = slot + 1 < R::kStages ? slot + 1 : 0;
  }
#pragma unroll
  for (int hh = 0; hh < kHeads; ++hh)
#pragma unroll
    for (int e = 0; e < E; ++e) num[hh][E * ring.lane + e] = acc[hh][e];
  return slot;
}

template <int D> constexpr int kRingBytes = kWarps * Ring<D>::kStages * Ring<D>::kSlot;
template <int D> constexpr int kSumBytes = kWarps * kHeads * (D + 2) * 4;
template <int D> constexpr int kNumBytes = kWarps * kHeads * D * 4;
template <int D> constexpr int kSmemBytes = kRingBytes<D> + kSumBytes<D> + kNumBytes<D>;

template <typename T, int D, bool WIDE>
__global__ void __launch_bounds__(kThreads, Parts<T>::n == 1 ? kResident : 2)
q4_decode_kernel(Q4Problem p) {
  static_assert(kThreads == 16 * kHeads, "16 threads a head");
  constexpr int NP = Parts<T>::n;
  using R = Ring<D>;
  constexpr int kTurn = kWarps * R::kRows;  // rows the CTA's warps take at a time
  extern __shared__ __align__(16) uint8_t smem[];
  float(*red)[kHeads][D + 2] = reinterpret_cast<float(*)[kHeads][D + 2]>(smem + kRingBytes<D>);  // [kWarps]
  float(*sq)[kHeads] = reinterpret_cast<float(*)[kHeads]>(smem + kRingBytes<D>);  // [D], before the sums
  float(*num)[kHeads][D] = reinterpret_cast<float(*)[kHeads][D]>(smem + kRingBytes<D> + kSumBytes<D>);  // [kWarps]

  const int g = p.H_q / p.H_kv, zc = (g + kHeads - 1) / kHeads;
  const uint32_t segs = (uint32_t)(p.H_kv * zc);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int i = lane >> 2, c = lane & 3;
  if (blockIdx.x == 0) {
    // A position that is neither a row nor -1: reported, the stream left alone.
#pragma unroll 1
    for (int b = threadIdx.x; b < p.B; b += kThreads)
      if (p.pos[b] < -1 || p.pos[b] >= p.S) atomicOr(p.status, kStatusRange);
  }
  Share share;
  Run run;
  locate(p, segs, share, run.b, run.off);
  if (blockIdx.x >= share.ctas) return;
  const uint32_t u_end = share.first(blockIdx.x + 1);
  run.end = share.first(blockIdx.x);
  R ring;
  Attention<D, NP, WIDE> at;
  float den = 0.f;  // sigma(q) z over the run's rows of M, of head threadIdx.x / 16
  at.clear();
#pragma unroll 1
  for (int turn = 0;; ++turn) {
    // The next run: from run.end, to its segment's end or this CTA's.  Its rows
    // are on their way before the last one is put away.
    const Run done = run;
    run.u = run.end;
    bool more = run.end < u_end;
    int k0 = 0, k1 = 0;
    if (more) {
      uint32_t n = stream_units(p, run.b);
      while (run.u >= run.off + segs * n && (int)run.b + 1 < p.B) {
        run.off += segs * n;
        n = stream_units(p, ++run.b);
      }
      run.pos = p.pos[run.b];
      // Positions that change while the step runs give no result worth having, but
      // must not lead out of the buffer either.
      if (run.pos < 0 || run.pos >= p.S || n <= (uint32_t)p.lead || run.u >= run.off + segs * n) return;
      run.seg = (run.u - run.off) / n;
      n -= p.lead;
      run.s0 = run.off + run.seg * (n + p.lead) + p.lead;
      run.s1 = run.s0 + n;
      run.end = min(u_end, run.s1);
      run.u = max(run.u, run.s0);
      more = run.u < run.end;  // (else only of a segment's lead: its rows are the next CTA's)
      if (more) {
        run.hk = zc == 1 ? run.seg : run.seg / zc;
        run.hq0 = run.hk * g + (run.seg - run.hk * zc) * kHeads;
        run.ng = min(kHeads, (run.hk + 1) * g - run.hq0);
        const int r0 = (run.u - run.s0) * p.unit;
        const int r1 = (int)min((long long)(run.end - run.s0) * p.unit, (long long)run.pos + 1);
        if (r1 == run.pos + 1 && (run.pos - r0) / R::kRows % kWarps == warp) {
          // The warp that will read the token's own row stores it first (with
          // several head chunks each does, the same bytes).
          store_token<T, D>(p, run.bh(p), run.bh(p) * p.S + run.pos, lane);
          __syncwarp();
        }
        // M's rows k0 .. k1 - 1 go with the run's units, a quarter to each warp.
        k0 = (run.u - run.s0) * D / n;  // (at most 2^30 / 128 units)
        k1 = (run.end - run.s0) * D / n;
        const int w0 = (k1 - k0) * warp / kWarps, w1 = (k1 - k0) * (warp + 1) / kWarps;
        ring.set(p, smem + warp * R::kStages * R::kSlot, run.bh(p) * p.S + r0, r1 - r0, lane);
        ring.mem = p.M + (run.bh(p) * D + k0 + w0) * D;
        ring.mem_rows = w1 - w0;
        ring.mem_items = (w1 - w0 + R::kMem - 1) / R::kMem;
        ring.first = warp * R::kRows;
#pragma unroll 1
        for (int e = 0; e < R::kStages - 1; ++e) ring.next(e, e);
      }
    }

    if (turn > 0) {
      // The last run's partial: of a CTA that has the segment whole, at the
      // heads' own place; of others, at the CTA's (its first run, or its last).
      Partial<D>* part = reinterpret_cast<Partial<D>*>(p.part) +
                         (done.whole() ? done.head0(p)
                                       : (size_t)p.B * p.H_q + ((size_t)blockIdx.x * 2 + (turn > 1)) * kHeads);
      if (threadIdx.x % 16 == 0 && (int)threadIdx.x / 16 < done.ng) part[threadIdx.x / 16].den = den;
      __syncthreads();  // sigma(q) has been read
      // This warp's (max, sum, acc) of heads 2c, 2c + 1.
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        at.l[h] = column_sum(at.l[h]);
        if (i == 0) {
          red[warp][2 * c + h][D] = at.m[h];
          red[warp][2 * c + h][D + 1] = at.l[h];
        }
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
          const float add = column_sum(at.omin[j][h]), unit = at.inverse(at.unit[j][h]);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float* to = &red[warp][2 * c + h][32 * j + 4 * i + 2 * k];
            if constexpr (Attention<D, NP, WIDE>::kPaired) {
              at.o[2 * j + k][h] += __shfl_xor_sync(0xffffffffu, at.o[2 * j + k][h], 2);
              at.o[2 * j + k][2 + h] += __shfl_xor_sync(0xffffffffu, at.o[2 * j + k][2 + h], 2);
            }
            to[0] = at.o[2 * j + k][h] * at.kUnit1 * unit + add;
            to[1] = at.o[2 * j + k][2 + h] * (at.kUnit1 * at.kOdd) * unit + add;
          }
        }
      }
      __syncthreads();
#pragma unroll 1
      for (int x = threadIdx.x; x < done.ng * D; x += kThreads) {
        const int hh = x / D, e = x - hh * D;
        float mx = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, red[w][hh][D]);
        float ls = 0.f, as = 0.f, ns = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          // A warp without rows has m = -inf, l = acc = 0.
          const float f = red[w][hh][D] == -INFINITY ? 0.f : exp2_approx(red[w][hh][D] - mx);
          ls = fmaf(red[w][hh][D + 1], f, ls);
          as = fmaf(red[w][hh][e], f, as);
          ns += num[w][hh][e];
        }
        part[hh].acc[e] = as;
        part[hh].num[e] = ns;
        if (e == 0) {
          part[hh].m = mx;
          part[hh].l = ls;
        }
      }
      finish<T, D>(p, share, done, segs);  // (its barriers also free the sums)
    }
    if (!more) return;

    // sigma(q) and its product with z: 16 threads a head, all loads first.
    {
      const int hh = threadIdx.x / 16, t = threadIdx.x % 16;
      const T* q = static_cast<const T*>(p.q_t) + (run.head0(p) + (hh < run.ng ? hh : 0)) * D + k0;
      const float* z = p.z + run.bh(p) * D + k0;
      float qv[D / 16], zv[D / 16];
#pragma unroll
      for (int e = 0; e < D / 16; ++e) {
        const bool in = t + 16 * e < k1 - k0;
        qv[e] = in ? to_f32<T>(q[t + 16 * e]) : 0.f;
        zv[e] = in ? z[t + 16 * e] : 0.f;
      }
      at.init(static_cast<const T*>(p.q_t) + run.head0(p) * D, run.ng, lane);
      den = 0.f;
#pragma unroll
      for (int e = 0; e < D / 16; ++e) {
        const float s = elu1(qv[e]);
        if (t + 16 * e < k1 - k0) sq[t + 16 * e][hh] = s;
        den = fmaf(s, zv[e], den);
      }
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
    }
    __syncthreads();
    const int slot = retrieve<D>(ring, sq + (k1 - k0) * warp / kWarps, num[warp]);
    at.run(ring, slot);
  }
}

// Rows of k and v [B, H_kv, n, D] into the buffers from row pos[b] on.  A
// thread takes 8 channels (16 bytes of bf16) of kPerThread rows: 4 neighbours hold
// a group and agree on its range by two exchanges, and each has whole words of
// the layout.
constexpr int kPerThread = 4;

template <typename T, int D>
__global__ void __launch_bounds__(kMoveThreads) q4_append_kernel(Q4Problem p, int n) {
  const bool key = blockIdx.z == 0;
  constexpr int PR = D / 8, kStep = kMoveThreads / PR;  // threads per row, rows at a time
  const int bh = blockIdx.y;
  const int pos = p.pos[bh / p.H_kv];
  if (pos < 0 || pos > p.S - n) {
    if (pos != -1 && threadIdx.x == 0) atomicOr(p.status, kStatusRange);
    return;
  }
  const int t0 = blockIdx.x * (kStep * kPerThread) + threadIdx.x / PR, w = threadIdx.x % PR;
  const T* src = static_cast<const T*>(key ? p.k_t : p.v_t) + ((size_t)bh * n + t0) * D + 8 * w;
  const size_t row = (size_t)bh * p.S + pos + t0;
  uint8_t* codes = (key ? p.k_codes : p.v_codes) + row * (D / 2);
  __nv_bfloat16* sm = (key ? p.k_scale : p.v_scale) + row * (D / 16);
  float v[kPerThread][8];
#pragma unroll
  for (int e = 0; e < kPerThread; ++e) {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[e][k] = 0.f;
    if (t0 + e * kStep < n) load8(src + e * (kStep * D), v[e]);
  }
#pragma unroll
  for (int e = 0; e < kPerThread; ++e)
    store_group<D>(v[e], w, key, codes + e * (kStep * D / 2), sm + e * (kStep * D / 16),
                   t0 + e * kStep < n);
}

// The values of rows 0..n-1 as k and v [B, H_kv, n, D]: a thread writes 8
// channels (one key word, two value halfwords) of kPerThread rows.
template <typename T, int D, bool KEY>
__device__ __forceinline__ void read_rows(const uint8_t* codes, const __nv_bfloat16* sm, int w,
                                          int left, T* to) {
  constexpr int NJ = D / 32, kStep = kMoveThreads / (D / 8);
  const int j = w >> 2, c = w & 3;
  uint32_t word[kPerThread], par[kPerThread];
#pragma unroll
  for (int e = 0; e < kPerThread; ++e) {
    word[e] = par[e] = 0;
    if (e * kStep < left) {
      par[e] = reinterpret_cast<const uint32_t*>(sm + e * (kStep * D / 16))[j];
      if (KEY) {
        word[e] = reinterpret_cast<const uint32_t*>(codes + e * (kStep * D / 2))[c * NJ + j];
      } else {
        const unsigned short* halves =
            reinterpret_cast<const unsigned short*>(codes + e * (kStep * D / 2)) + 2 * c * NJ + j;
        word[e] = halves[0] | (uint32_t)halves[NJ] << 16;
      }
    }
  }
#pragma unroll
  for (int e = 0; e < kPerThread; ++e) {
    const float s = __uint_as_float(par[e] << 16), m = __uint_as_float(par[e] & 0xffff0000u);
    float out[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // codes i and i + 4 from the lowest bits on: 2^23 + 16^i code, less 2^23
      constexpr float kBase = 8388608.f;
      const float at = 1.f / (1 << 4 * i);
      const uint32_t mask = 15u << 4 * i;
      const float2 n = {__uint_as_float((word[e] & mask) | 0x4b000000u),
                        __uint_as_float((word[e] >> 16 & mask) | 0x4b000000u)};
      const float2 y = fma({s, s}, fma(n, {at, at}, {-kBase * at, -kBase * at}), {m, m});
      out[KEY ? 2 * i : i] = y.x;
      out[KEY ? 2 * i + 1 : i + 4] = y.y;
    }
    if (e * kStep < left) store8(to + e * (kStep * D), out);
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kMoveThreads) q4_read_kernel(Q4Problem p, int n, T* k, T* v) {
  constexpr int PR = D / 8, kStep = kMoveThreads / PR;
  const int bh = blockIdx.y;
  const int t0 = blockIdx.x * (kStep * kPerThread) + threadIdx.x / PR, w = threadIdx.x % PR;
  const size_t row = (size_t)bh * p.S + t0, at = ((size_t)bh * n + t0) * D + 8 * w;
  if (blockIdx.z == 0)
    read_rows<T, D, true>(p.k_codes + row * (D / 2), p.k_scale + row * (D / 16), w, n - t0, k + at);
  else
    read_rows<T, D, false>(p.v_codes + row * (D / 2), p.v_scale + row * (D / 16), w, n - t0, v + at);
}

int chunks_of(int g) { return (g + kHeads - 1) / kHeads; }

// Rows of a unit, and CTAs that attend.  A buffer whose full segments have at
// most 2 units of 128 rows for each CTA that the GPU holds is cut into longer
// units, one per CTA, none across a segment's end; with more work the units are
// 128 rows and every CTA takes an equal run of them.
struct Q4Plan {
  int unit, lead;
  long long ctas;
};
Q4Plan q4_plan(int B, int H_q, int H_kv, int S) {
  const long long segments = (long long)B * H_kv * chunks_of(H_q / H_kv), most = kSMs * kResident;
  const long long units = segments * ((S + kUnit - 1) / kUnit);
  if (units > 2 * most) return {kUnit, kLeadUnits, most};
  const int per = (int)((units + most - 1) / most);
  return {per * kUnit, 0, segments * ((S + per * kUnit - 1) / (per * kUnit))};
}

template <typename T, int D>
cudaError_t launch(const Q4Problem& p, Q4What what, int n, void* k, void* v, cudaStream_t st) {
  constexpr int kRowsPerCta = kMoveThreads / (D / 8) * kPerThread;
  const dim3 rows((unsigned)(((long long)n + kRowsPerCta - 1) / kRowsPerCta), p.B * p.H_kv, 2);
  switch (what) {
    case Q4What::kStep: {
      constexpr int bytes = kSmemBytes<D>;
      // WIDE: the second parts of the weights find no free columns (fp32 heads always take
      // products of their own, next to those of the queries' two parts).
      constexpr bool kAlways = Parts<T>::n > 1;
      auto* kernel = kAlways || p.H_q / p.H_kv > kHeads / 2 ? q4_decode_kernel<T, D, true>
                                                            : q4_decode_kernel<T, D, kAlways>;
      if (bytes > 48 * 1024) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
      }
      const Q4Plan plan = q4_plan(p.B, p.H_q, p.H_kv, p.S);
      Q4Problem q = p;
      q.ctas = (int)plan.ctas;
      q.unit = plan.unit;
      q.lead = plan.lead;
      kernel<<<(unsigned)plan.ctas, kThreads, bytes, st>>>(q);
      break;
    }
    case Q4What::kAppend: q4_append_kernel<T, D><<<rows, kMoveThreads, 0, st>>>(p, n); break;
    case Q4What::kRead:
      q4_read_kernel<T, D><<<rows, kMoveThreads, 0, st>>>(p, n, static_cast<T*>(k), static_cast<T*>(v));
      break;
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

int q4_head_chunks(int g) { return chunks_of(g); }

bool q4_units_ok(int B, int H_q, int H_kv, int S) {
  return (long long)B * H_kv * chunks_of(H_q / H_kv) * (kLeadUnits + S / kUnit + 1) <= 0x7fffffffLL;
}

// Bytes of the partials: one per query head, and two sets of kHeads per CTA.
size_t q4_partial_bytes(int B, int H_q, int H_kv, int S, int d) {
  return ((size_t)B * H_q + (size_t)q4_plan(B, H_q, H_kv, S).ctas * 2 * kHeads) * (2 * d + 4) * 4;
}

cudaError_t launch_q4(const Q4Problem& p, Q4What what, int n, void* k, void* v, cudaStream_t st) {
  return p.bf16 ? launch_type<__nv_bfloat16>(p, what, n, k, v, st) : launch_type<float>(p, what, n, k, v, st);
}

}  // namespace infini
