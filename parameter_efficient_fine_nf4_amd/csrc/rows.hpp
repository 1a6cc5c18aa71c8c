// rows.hpp -- device helpers of the kernels that read rows of a head's logits
// (loss.hip, scores.hip): a row's pieces, its exponentials and their sums.
#pragma once

#include <algorithm>
#include <cmath>
#include <cstring>
#include <limits>

#include "common.hpp"

namespace qlora {

constexpr double kLog2e = 1.4426950408889634074;
constexpr double kLn2 = 0.69314718055994530942;
constexpr float kNegInf = -__builtin_inff();

template <typename E>
struct Elem;
template <>
struct Elem<uint16_t> {
  static constexpr int kPer16 = 8;
  static constexpr uint32_t kFill = 0xFF80FF80u;  // -inf, -inf
  static __device__ __forceinline__ float get(const uint16_t* p) { return bf16_to_f32(*p); }
  static __device__ __forceinline__ void put(uint16_t* p, float v) { *p = (uint16_t)pack_bf16x2(v, 0.0f); }
  static __device__ __forceinline__ void unpack(const u32x4& w, float (&f)[8]) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      f[2 * q] = bf16_lo(w[q]);
      f[2 * q + 1] = bf16_hi(w[q]);
    }
  }
  static __device__ __forceinline__ u32x4 pack(const float (&f)[8]) {
    return u32x4{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7])};
  }
};
template <>
struct Elem<float> {
  static constexpr int kPer16 = 4;
  static constexpr uint32_t kFill = 0xFF800000u;  // -inf
  static __device__ __forceinline__ float get(const float* p) { return *p; }
  static __device__ __forceinline__ void put(float* p, float v) { *p = v; }
  static __device__ __forceinline__ void unpack(const u32x4& w, float (&f)[4]) {
#pragma unroll
    for (int q = 0; q < 4; ++q) f[q] = __uint_as_float(w[q]);
  }
  static __device__ __forceinline__ u32x4 pack(const float (&f)[4]) {
    return u32x4{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])};
  }
};

// A 16-byte piece of a gradient.  `stream`: the gradient as a whole is larger
// than half the last-level cache and would only push the logits out of it
// (T = 4096, V = 32000, bf16, 40 % masked: the next call's log-probabilities
// take 31 us after such stores and 47 us after ordinary ones, whose lines it
// has to write back first; the gradient itself 68 and 74 us).  A template
// argument: of a branch between the two the compiler makes one ordinary store.
template <bool STREAM>
__device__ __forceinline__ void put16(void* out, const u32x4& v) {
  if constexpr (STREAM)
    __builtin_nontemporal_store(v, reinterpret_cast<u32x4_any*>(out));
  else
    *reinterpret_cast<u32x4_any*>(out) = v;
}

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// Maximum and sum over the work-group of T threads; every thread gets the
// result.  `red` holds one float per wave.
template <int T>
__device__ __forceinline__ float block_max(float v, float* red) {
  v = wave_max(v);
  if (T == 64) return v;
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  float r = red[0];
#pragma unroll
  for (int i = 1; i < T / 64; ++i) r = fmaxf(r, red[i]);
  return r;
}

template <int T>
__device__ __forceinline__ float block_sum(float v, float* red) {
  v = wave_sum(v);
  if (T == 64) return v;
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  float r = red[0];
#pragma unroll
  for (int i = 1; i < T / 64; ++i) r += red[i];
  return r;
}

// c = tau log2 e = hi + lo, lo > 0: a masked word's -inf stays -inf in either.
struct Scale {
  double c;
  float one, hi, lo;  // one: fl(c)
  __device__ __forceinline__ float times(float d) const { return fmaf(d, hi, d * lo); }
};

// How a row's exponentials are formed from its maximum m.
struct RowExp {
  Scale c;
  float k, m;
  bool far;
  __device__ __forceinline__ RowExp(float m_, const Scale& c_)
      : c(c_), k((float)((double)m_ * c_.c)), m(m_), far(!(fabsf(k) < 512.0f)) {}
  __device__ __forceinline__ float near_e(float z) const { return exp2_hw(fmaf(z, c.lo, fmaf(z, c.hi, -k))); }
  __device__ __forceinline__ float far_e(float z) const { return exp2_hw(c.times(z - m)); }
  // for a gradient of type E
  template <typename E>
  __device__ __forceinline__ float near_g(float z) const {
    return sizeof(E) == 2 ? exp2_hw(fmaf(z, c.one, -k)) : near_e(z);
  }
  __device__ __forceinline__ float e(float z) const { return far ? far_e(z) : near_e(z); }
  // factor of near_e over far_e: what k's rounding is
  __device__ __forceinline__ float shift() const {
    return far ? 1.0f : exp2_hw((float)((double)m * c.c - (double)k));
  }
  // ln of the sum of exp(tau (z - m)), from the sum s of e()
  __device__ __forceinline__ double ln_sum(float s) const {
    return log((double)s) + (far ? 0.0 : kLn2 * ((double)k - (double)m * c.c));
  }
};

// The same piece, as far as the compiler knows another one: each pass over a
// row in registers unpacks its pieces one at a time.  Otherwise the values of
// one pass, or those that two branches share, are all kept at once (twice the
// registers of the row, for bf16).
template <int PASS>
__device__ __forceinline__ u32x4 anew(u32x4 w) {
  if (PASS == 0) asm volatile("; maximum" : "+v"(w));
  if (PASS == 1) asm volatile("; near" : "+v"(w));
  if (PASS == 2) asm volatile("; far" : "+v"(w));
  if (PASS == 3) asm volatile("; near, streamed" : "+v"(w));
  if (PASS == 4) asm volatile("; far, streamed" : "+v"(w));
  return w;
}

// A row as 16-byte pieces: nv of them from the first 16-byte boundary on
// (element `head`), and fewer than 16 single elements before and after, one a
// thread.  Rows of an odd stride start anywhere; read or written at their own
// boundaries they take no longer than aligned ones (V = ld = 131071, bf16,
// policy loss and gradient: 549 us at the rows' starts).
struct RowSpan {
  int head, nv, rest;  // rest: this thread's single element, or one past the row
  template <typename E>
  __device__ __forceinline__ RowSpan(const E* z, int V) {
    constexpr int kPer = Elem<E>::kPer16;
    const int h = (int)((16u - ((uint32_t)(uintptr_t)z & 15u)) & 15u) / (int)sizeof(E);
    head = h < V ? h : V;
    nv = (V - head) / kPer;
    rest = (int)threadIdx.x < head ? (int)threadIdx.x : (int)threadIdx.x + nv * kPer;
    if (threadIdx.x >= 16 || rest > V) rest = V;
  }
};
// A row of V elements in the registers of T threads: N pieces each and a
// single element.  What is past the end holds -inf.
template <typename E, int T, int N>
struct RowRegs {
  static constexpr int kPer = Elem<E>::kPer16;
  u32x4 w[N];
  float last;

  __device__ __forceinline__ void load(const E* z, int V, const RowSpan& at) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int i = j * T + threadIdx.x;
      w[j] = u32x4{Elem<E>::kFill, Elem<E>::kFill, Elem<E>::kFill, Elem<E>::kFill};
      if (i < at.nv) w[j] = *reinterpret_cast<const u32x4*>(z + at.head + (size_t)i * kPer);
    }
    last = kNegInf;
    if (at.rest < V) last = Elem<E>::get(z + at.rest);
  }
  __device__ __forceinline__ float max() const {
    float m = last;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      float f[kPer];
      Elem<E>::unpack(anew<0>(w[j]), f);
#pragma unroll
      for (int q = 0; q < kPer; ++q) m = fmaxf(m, f[q]);
    }
    return m;
  }
  template <bool FAR>
  __device__ __forceinline__ float sum_of(const RowExp& x) const {
    float s[2] = {FAR ? x.far_e(last) : x.near_e(last), 0.0f};
#pragma unroll
    for (int j = 0; j < N; ++j) {
      float f[kPer];
      Elem<E>::unpack(anew<1 + FAR>(w[j]), f);
#pragma unroll
      for (int q = 0; q < kPer; ++q) s[q & 1] += FAR ? x.far_e(f[q]) : x.near_e(f[q]);
    }
    return s[0] + s[1];
  }
  __device__ __forceinline__ float sum(const RowExp& x) const { return x.far ? sum_of<true>(x) : sum_of<false>(x); }
};

// Running maximum and sum of exp2((z - m) c), for rows read in pieces.  A
// maximum of -inf (nothing but masked values so far) is read as 0 in the
// exponents: -inf - (-inf) would make a NaN of it.
struct Online {
  float m = kNegInf, s = 0.0f;
  template <typename E, int N>
  __device__ __forceinline__ void add(const u32x4 (&w)[N], const Scale& c) {
    constexpr int kPer = Elem<E>::kPer16;
    float f[kPer], mx = m;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      Elem<E>::unpack(anew<0>(w[j]), f);
#pragma unroll
      for (int q = 0; q < kPer; ++q) mx = fmaxf(mx, f[q]);
    }
    const float ref = mx == kNegInf ? 0.0f : mx;
    float sum = s * exp2_hw(c.times(m - ref));
#pragma unroll
    for (int j = 0; j < N; ++j) {
      Elem<E>::unpack(anew<2>(w[j]), f);
#pragma unroll
      for (int q = 0; q < kPer; ++q) sum += exp2_hw(c.times(f[q] - ref));
    }
    m = mx;
    s = sum;
  }
  __device__ __forceinline__ void add_one(float f, const Scale& c) {
    const float mx = fmaxf(m, f), ref = mx == kNegInf ? 0.0f : mx;
    s = s * exp2_hw(c.times(m - ref)) + exp2_hw(c.times(f - ref));
    m = mx;
  }
};

// Maximum and sum of a row of any length, in pieces.
template <typename E, int T, int N>
__device__ __forceinline__ Online row_pieces(const E* z, int V, const RowSpan& at, const Scale& c) {
  constexpr int kPer = Elem<E>::kPer16;
  Online o;
  for (int i0 = threadIdx.x; i0 < at.nv; i0 += N * T) {
    u32x4 w[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
      w[j] = u32x4{Elem<E>::kFill, Elem<E>::kFill, Elem<E>::kFill, Elem<E>::kFill};
      if (i0 + j * T < at.nv) w[j] = *reinterpret_cast<const u32x4*>(z + at.head + (size_t)(i0 + j * T) * kPer);
    }
    o.template add<E, N>(w, c);
  }
  if (at.rest < V) o.add_one(Elem<E>::get(z + at.rest), c);
  return o;
}

template <typename E, int T, bool STREAM>
__device__ __forceinline__ void row_zero_of(E* out, const RowSpan& at) {
  for (int i = threadIdx.x; i < at.nv; i += T)
    put16<STREAM>(out + at.head + (size_t)i * Elem<E>::kPer16, u32x4{0u, 0u, 0u, 0u});
}
template <typename E, int T>
__device__ __forceinline__ void row_zero(E* out, int cols, bool stream) {
  const RowSpan at(out, cols);
  if (stream)
    row_zero_of<E, T, true>(out, at);
  else
    row_zero_of<E, T, false>(out, at);
  if (at.rest < cols) Elem<E>::put(out + at.rest, 0.0f);
}

__device__ __forceinline__ bool is_counted(int label, int V) { return (uint32_t)label < (uint32_t)V; }

// ------------------------------------------------------------- host -----

// The row kernels' work-groups have a row each (in a loop over rows the fp64
// logarithm's constants would stay in registers through the whole of it, 20 of
// a thread's); a launch has up to 2^20 of them, below 2^32 threads.
constexpr int64_t kRowsALaunch = (int64_t)1 << 20;

// Half of the 256 MB last-level cache.
inline bool past_cache(int64_t T, int64_t ldd, int f32) { return T * ldd * (f32 ? 4 : 2) > ((int64_t)128 << 20); }

// Finite for every finite tau (the row's maximum has 0 times it), and lo above 0
// where c has no bits left for it.
inline Scale exp2_scale(float tau) {
  const double c = std::min((double)tau * kLog2e, (double)std::numeric_limits<float>::max());
  float hi = (float)c;
  if ((double)hi > c) hi = std::nextafter(hi, 0.0f);
  uint32_t bits;
  std::memcpy(&bits, &hi, 4);
  if (std::isnormal(hi)) bits &= 0xFFFFFF00u;
  std::memcpy(&hi, &bits, 4);
  const float lo = std::max((float)(c - (double)hi), std::numeric_limits<float>::denorm_min());
  return Scale{(double)hi + (double)lo, (float)((double)hi + (double)lo), hi, lo};
}

}  // namespace qlora
