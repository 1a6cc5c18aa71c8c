// checkpoint.hpp -- writing an activation's 8-bit checkpoint, a tile at a time:
// for its own kernel (checkpoint.hip) and for work-groups of other kernels that
// have the input at hand.
//
// 127 x has at most 15 significant bits and the quotient 127 x / a is correctly
// rounded, so a tie of the exact quotient is a tie here: codes do not depend on
// the order of anything.  A quotient that is no tie lies at least 2^-16 of itself
// from one, the quotient's rounding moves it by 2^-24.
#pragma once

#include "common.hpp"
#include "launch.hpp"

namespace qlora {

constexpr int kCkThreads = 256;
constexpr int kCkCols = 512;                // columns of a work-group: 32 lanes of 16
constexpr int kCkTokens = kCkThreads / 32;  // its tokens
constexpr uint32_t kNoScale = 0x7FC0u;  // NaN
// below 2^-100 and from 2^100 on a block is scaled first: 127 / a or 127 x
// would leave fp32's range
constexpr uint32_t kTiny = 0x0D80u, kHuge = 0x7180u;

typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t,
                            __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
}

// Largest of the lane's quad.
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true));  // lanes 1, 0, 3, 2
  return max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true));  // lanes 2, 3, 0, 1
}

// 16 bf16 of a block whose constant (bf16 bits, sign cleared) is a -> 16 codes.
// q = 127 x / a: the product with r = fl(1 / a), then its residual (exact in
// one fused step) taken back, which rounds the quotient correctly.  Adding
// 1.5 2^23 rounds to a whole number, ties to even, and leaves it in the low
// byte.
__device__ __forceinline__ u32x4 encode16(const u32x4& lo, const u32x4& hi, uint32_t a) {
  if (a == 0u || a == kNoScale) return u32x4{0u, 0u, 0u, 0u};
  const float up = a < kTiny ? 0x1p64f : (a >= kHuge ? 0x1p-64f : 1.0f);
  const float af = __uint_as_float(a << 16) * up, f127 = 127.0f * up;
  const float r = 1.0f / af;
  auto code = [&](float x) {
    const float n = x * f127, q = n * r;
    return __float_as_uint(fmaf(fmaf(-q, af, n), r, q) + 12582912.0f);
  };
  u32x4 out;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w0 = i < 2 ? lo[2 * i] : hi[2 * i - 4], w1 = i < 2 ? lo[2 * i + 1] : hi[2 * i - 3];
    const uint32_t p = perm(code(bf16_hi(w0)), code(bf16_lo(w0)), 0x0C0C0400u);
    const uint32_t s = perm(code(bf16_hi(w1)), code(bf16_lo(w1)), 0x0C0C0400u);
    out[i] = p | (s << 16);
  }
  return out;
}

// Tile number `tile` of a checkpoint, eight tokens of 512 columns, by 256 threads:
// four lanes share a block, each with 16 of its columns in two loads.  `as` holds
// the tile's constants.
typedef uint16_t CkConstants[kCkCols / kBlock][kCkTokens];
__device__ __forceinline__ void ck_save_tile(const CkJob& job, int tile, CkConstants& as) {
  const int M = job.M, k = job.k;
  const int nct = ((k - 1) / kCkCols + 1), ct = tile % nct;
  const int col = ct * kCkCols + ((int)threadIdx.x & 31) * 16, row = (int)threadIdx.x >> 5;
  const int m0 = tile / nct * kCkTokens, m = m0 + row;
  u32x4 lo = {0u, 0u, 0u, 0u}, hi = lo;
  if (m < M && col < k) {
    const uint16_t* x = job.X + (size_t)m * k + col;
    lo = *reinterpret_cast<const u32x4*>(x);
    hi = *reinterpret_cast<const u32x4*>(x + 8);
  }
  uint32_t v = 0u;
#pragma unroll
  for (int q = 0; q < 4; ++q) v = max_u16x2(v, max_u16x2(lo[q] & 0x7FFF7FFFu, hi[q] & 0x7FFF7FFFu));
  uint32_t a = quad_max(max(v & 0xFFFFu, v >> 16));
  if (a >= 0x7F80u) a = kNoScale;
  if ((threadIdx.x & 3) == 0) as[(threadIdx.x & 31) >> 2][row] = (uint16_t)a;
  const u32x4 c = encode16(lo, hi, a);
  if (m < M && col < k) *reinterpret_cast<u32x4*>(job.codes + (size_t)m * k + col) = c;
  __syncthreads();
  // a row of constants has room for whole groups of tokens
  const int b = (int)threadIdx.x, kb = ct * (kCkCols / kBlock) + b;
  if (b < kCkCols / kBlock && kb < k / kBlock)
    *reinterpret_cast<u32x4*>(job.absmax + (size_t)kb * job.ldm + m0) = *reinterpret_cast<const u32x4*>(&as[b][0]);
}

inline int ck_tiles(int M, int k) { return ((k - 1) / kCkCols + 1) * ((M + kCkTokens - 1) / kCkTokens); }

}  // namespace qlora
