// checkpoint.hip -- activations kept at 8 bits between a forward and its
// backward.
//
// A block is 64 consecutive columns of one token (so it lies inside a row, as
// the weight's blocks do).  With a = max |x| over the block, kept in bf16 and
// so exactly,
//
//   c = rint(127 x / a)  (ties to even, int8),   x^ = bf16(fl32(c fl32(a fl32(1/127)))).
//
// c = 127 gives a back exactly.  A block with an infinity or a NaN has no scale:
// its a is NaN and so is all that it stands for.
//
// Codes are M x k as the activations are.  The constants are kept by column
// block, tokens contiguous (k/64 rows of roundup(M, 64)): the backward's
// reduction over tokens takes 32 tokens of one column block at a time, whose
// constants are then 64 bytes in a row.
#include "checkpoint.hpp"

namespace qlora {

// (Four times the tokens a work-group, all in flight together: 1001 x 4160 save 5.9
// us, load 5.3, against 4.3 and 4.1; 4096 x 4096 10.8 and 11.3 against 9.9 and 11.3;
// 4096 x 22016 50.4 and 53.6 against 49.6 and 47.3, 5.5 and 5.8 TB/s.)  Bound by
// memory.
__global__ __launch_bounds__(kCkThreads) void k_ck_save(CkJob job) {
  __shared__ __attribute__((aligned(16))) CkConstants as;
  ck_save_tile(job, (int)blockIdx.x, as);
}

__global__ __launch_bounds__(kCkThreads) void k_ck_load(const uint8_t* __restrict__ codes,
                                                        const uint16_t* __restrict__ absmax, int M, int k, int ldm,
                                                        uint16_t* __restrict__ X) {
  const int nct = ((k - 1) / kCkCols + 1);
  const int col = (int)blockIdx.x % nct * kCkCols + ((int)threadIdx.x & 31) * 16;
  const int m = (int)blockIdx.x / nct * kCkTokens + ((int)threadIdx.x >> 5);
  if (m >= M || col >= k) return;
  const u32x4 c = *reinterpret_cast<const u32x4*>(codes + (size_t)m * k + col);
  const float a = ck_scale(absmax[(size_t)(col / kBlock) * ldm + m]);
  uint16_t* x = X + (size_t)m * k + col;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    u32x4 o;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t w = c[2 * h + (q >> 1)] >> (16 * (q & 1));
      o[q] = pack_bf16x2(ck_value(w, a), ck_value(w >> 8, a));
    }
    *reinterpret_cast<u32x4*>(x + 8 * h) = o;
  }
}

hipError_t launch_ck_save(const CkJob& job, hipStream_t st) {
  QLORA_LAUNCH("ck_save", st, k_ck_save, dim3((unsigned)ck_tiles(job.M, job.k)), dim3(kCkThreads), 0, st, job);
  return hipGetLastError();
}

hipError_t launch_ck_load(const uint8_t* codes, const uint16_t* absmax, int M, int k, uint16_t* X, hipStream_t st) {
  QLORA_LAUNCH("ck_load", st, k_ck_load, dim3((unsigned)ck_tiles(M, k)), dim3(kCkThreads), 0, st, codes, absmax, M, k, tsave_ld(M), X);
  return hipGetLastError();
}

}  // namespace qlora
