// muon.hip -- optimiser step that orthogonalises an adapter factor's update.
//
// Per matrix of R x C parameters (a LoRA factor: A is r x k, B is d x r), with
// gradient g, momentum buffer m and master weights w:
//
//   m <- mu m + g;    u = g + mu m (nesterov) or m
//   X = u / (|u|_F + eps);   steps times  X <- (a I + b G + c G^2) X,  G = X X^T
//   w <- (1 - lr wd) w - lr scale X;    p = bf16(w)
//
// (for R > C with X^T X on the other side).  The shorter side S of a factor
// is its rank, at most 64, so the iteration is not run on the R x C matrix:
// every iterate is a polynomial in the S x S matrix G_0 = u u^T / |u|^2 times
// u.  With P_i = a I + b G_i + c G_i^2,
//
//   G_{i+1} = P_i G_i P_i,   Q = P_{n-1} ... P_0,   X_n = Q u / (|u| + eps),
//
// all of it commuting, and |u|^2 is the trace of u u^T.  Two passes over the
// parameters remain (the Gram product; the update), 20 bytes a parameter
// that no form can avoid plus 6 of m and g read again.
//
// G_0 and the iteration are held in fp64: a small singular value s of X enters
// G as s^2, which fp32 loses below 3e-4 of the largest, while the iteration
// amplifies it by a^n (485 for the usual five steps).
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "common.hpp"
#include "launch.hpp"

namespace qlora {

constexpr int kMuThreads = 256;
// Elements of a matrix with S <= 16 up to which one work-group takes it whole
// (8 x 256: 8.4 us a call against 12.1 in two launches; 8 x 1024: 12.2 against
// 11.8, as one CU's loads no longer keep up with many).
constexpr int64_t kMuWhole = 4096;

struct MuShape {
  int64_t nmat, rows, cols;
  int S, L, tall;  // short and long side; rows > cols
};

static MuShape mu_shape(int64_t nmat, int64_t rows, int64_t cols) {
  MuShape s{nmat, rows, cols, 0, 0, rows > cols};
  s.S = (int)(s.tall ? cols : rows);
  s.L = (int)(s.tall ? rows : cols);
  return s;
}

__device__ __forceinline__ float mu_momentum(float m, float g, float mu) { return __fadd_rn(__fmul_rn(mu, m), g); }
__device__ __forceinline__ float mu_update(float m, float g, float mu, int nesterov) {
  return nesterov ? __fadd_rn(g, __fmul_rn(mu, m)) : m;
}

typedef __attribute__((ext_vector_type(4))) double f64x4;

__device__ __forceinline__ f64x4 mfma_f64(double a, double b, f64x4 c) {
  return __builtin_amdgcn_mfma_f64_16x16x4f64(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma_f32(float a, float b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

// N consecutive values at element alignment (rows of odd lengths start
// anywhere).  VEC: one vector access; otherwise one by one, where only the
// first n exist (a load repeats the last of them, so that no load depends on a
// branch; n >= 1 at an address the caller has clamped into the matrix).
template <int N>
struct Vec {
  typedef float __attribute__((ext_vector_type(N), aligned(4))) F;
  typedef uint16_t __attribute__((ext_vector_type(N), aligned(2))) H;
};
template <>
struct Vec<1> {
  typedef float F;
  typedef uint16_t H;
};
// N bf16 values, two to a register.
template <int N>
struct Halves {
  uint32_t w[(N + 1) / 2];
  __device__ __forceinline__ float f32(int i) const { return i % 2 ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]); }
};
__device__ __forceinline__ int clamp_at(int i, int n) { return i < n ? i : (n > 1 ? n - 1 : 0); }

// An access is a wave-uniform base (scalar registers) plus a lane's 32-bit
// offset in elements: row and step go into the base, so that the many rows of
// a step in flight take no vector registers for addresses.  A matrix has
// fewer than 2^29 elements.  Vectors are accessed by casts of the pointer to
// their types in place: a type's alignment is lost where the type is a
// template argument.
template <typename E>
__device__ __forceinline__ E* lane_at(E* base, uint32_t at) {
  typedef typename std::conditional<std::is_const<E>::value, const char, char>::type B;
  return reinterpret_cast<E*>(reinterpret_cast<B*>(base) + at * (uint32_t)sizeof(E));
}

// STREAM (with VEC): past the caches.
template <bool VEC, bool STREAM, int N>
__device__ __forceinline__ void load_f(const float* p, uint32_t at, int n, float (&v)[N]) {
  if constexpr (VEC) {
    typename Vec<N>::F x;
    if constexpr (STREAM)
      x = __builtin_nontemporal_load(reinterpret_cast<const typename Vec<N>::F*>(lane_at(p, at)));
    else
      x = *reinterpret_cast<const typename Vec<N>::F*>(lane_at(p, at));
    __builtin_memcpy(v, &x, N * 4);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = *lane_at(p, at + clamp_at(i, n));
  }
}
template <bool VEC, int N>
__device__ __forceinline__ void load_h(const uint16_t* p, uint32_t at, int n, Halves<N>& v) {
  if constexpr (VEC && N == 3) {
    // 4 and 2 bytes: the compiler reads a vector of three as four, which past a
    // matrix's last three is past the end of G; and a copy of 6 bytes into two
    // registers goes through scratch memory
    const typename Vec<2>::H x = *reinterpret_cast<const typename Vec<2>::H*>(lane_at(p, at));
    __builtin_memcpy(v.w, &x, 4);
    v.w[1] = *lane_at(p, at + 2);
  } else if constexpr (VEC) {
    const typename Vec<N>::H x = *reinterpret_cast<const typename Vec<N>::H*>(lane_at(p, at));
    v.w[(N - 1) / 2] = 0;
    __builtin_memcpy(v.w, &x, N * 2);
  } else {
#pragma unroll
    for (int i = 0; i < (N + 1) / 2; ++i)
      v.w[i] = (uint32_t)*lane_at(p, at + clamp_at(2 * i, n)) |
               (uint32_t)*lane_at(p, at + clamp_at(2 * i + 1, n)) << 16;
  }
}
template <bool VEC, bool STREAM, int N>
__device__ __forceinline__ void store_f(float* p, uint32_t at, int n, const float (&v)[N]) {
  if constexpr (VEC) {
    if (n > 0) {
      typename Vec<N>::F x;
      __builtin_memcpy(&x, v, N * 4);
      if constexpr (STREAM)
        __builtin_nontemporal_store(x, reinterpret_cast<typename Vec<N>::F*>(lane_at(p, at)));
      else
        *reinterpret_cast<typename Vec<N>::F*>(lane_at(p, at)) = x;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < n) *lane_at(p, at + i) = v[i];
  }
}
template <bool VEC, bool STREAM, int N>
__device__ __forceinline__ void store_bf16(uint16_t* p, uint32_t at, int n, const float (&v)[N]) {
  uint32_t h[(N + 1) / 2];
#pragma unroll
  for (int i = 0; i < N; i += 2) h[i / 2] = pack_bf16x2(v[i], i + 1 < N ? v[i + 1 < N ? i + 1 : i] : 0.0f);
  if constexpr (VEC) {
    if (n > 0) {
      typename Vec<N>::H x;
      __builtin_memcpy(&x, h, N * 2);
      if constexpr (STREAM)
        __builtin_nontemporal_store(x, reinterpret_cast<typename Vec<N>::H*>(lane_at(p, at)));
      else
        *reinterpret_cast<typename Vec<N>::H*>(lane_at(p, at)) = x;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < n) *lane_at(p, at + i) = (uint16_t)(h[i / 2] >> (16 * (i % 2)));
  }
}
__device__ __forceinline__ int room(int end, int at) { return at < end ? end - at : 0; }

// The Gram matrix and everything made of it are symmetric: of the NT x NT
// tiles of 16 x 16 only those (t, t2) with t <= t2 are formed, numbered u.
constexpr int mu_tiles(int nt) { return nt * (nt + 1) / 2; }

// The whole steps of one wave over a matrix's long axis: the waves of all its
// work-groups take neighbouring steps in turn.  Each matrix starts at its own
// place (and goes round): rows of a power of two of bytes would otherwise put
// every work-group of a stack on the same memory channels at the same time.
// What is left of the axis (all of it where no step is whole) comes after, in
// steps from `rest` on.
struct Steps {
  int i, n, first, rest, stride, step;
  __device__ __forceinline__ Steps(const MuShape& s, int64_t mat, int wave, int waves, int step_)
      : i(wave), n(s.L / step_), stride(waves), step(step_) {
    first = (int)(mat * n / s.nmat);
    // (past the axis for every wave but the one whose turn it is; L + step
    // fits an int as a matrix has fewer than 2^29 elements)
    rest = n * step < s.L ? (int)min((int64_t)s.L, ((int64_t)n + (i + stride - n % stride) % stride) * step) : s.L;
  }
  __device__ __forceinline__ bool valid() const { return i < n; }
  __device__ __forceinline__ int j0(int at) const { return (first + at < n ? first + at : first + at - n) * step; }
};

// A work-group's matrix and split.  Work-groups go to the 8 dies in turn; each
// die takes neighbouring ones of the stack, so that a line of memory that two
// of them share is read once and written whole by one L2 (27 x 64 x 10704,
// pass 1: 50 us in plain order, 46 so).  last_first: a die's from the last to
// the first.
struct MuPlace {
  int64_t mat;
  int split, group;
  __device__ __forceinline__ MuPlace(const MuShape& s, int splits, bool last_first) {
    const int all = (int)s.nmat * splits, die = blockIdx.x % 8, i = blockIdx.x / 8;
    const int each = all / 8, more = all % 8, n = each + (die < more);
    group = die * each + min(die, more) + (last_first ? n - 1 - i : i);
    mat = group / splits;
    split = group % splits;
  }
};

// -------------------------------------------------------------- pass 1 ----
//
// m <- mu m + g, and one fp64 partial of u u^T per (matrix, split), as the
// tiles' MFMA accumulators (16 x 16 x 4: operand lane l holds index l % 16 of
// position l / 16; the same registers are both operands).  A wave takes 32
// long positions at a time, 8 per lane; the order of the positions inside an
// MFMA does not matter to the sum, so each lane loads consecutive values:
//
//   not tall: 8 positions of row 16 t + l % 16 (a row's 32 are a 128-byte
//             line of m), tile index i of t is row 16 t + i;
//   tall:     NT consecutive short indexes of 8 long positions 4 apart, tile
//             index i of t is NT i + t, or, in the last vector of a row, S -
//             NT + t (k_muon_poly undoes the order).
template <int NT, bool TALL>
struct GramLoad {
  static constexpr int A = TALL ? 8 : NT, B = TALL ? NT : 8;  // A vectors of B consecutive values
  float m[A][B];
  Halves<B> g[A];

  // Vector a of a lane starts at base(a) + lane_part(a) (clamped into the
  // matrix) and has count(a) values.  VEC: all positions of the step exist.
  // Tall, with S not a multiple of NT, the last vector of a row starts NT
  // before the row's end: its first values (`again` of them) are the vector
  // before's too, count for nothing in the sums and are stored twice alike.
  template <bool VEC>
  static __device__ __forceinline__ int base(const MuShape& s, int j0, int a) {
    if (TALL) return VEC ? (j0 + 4 * a) * s.S : 0;
    return VEC ? 16 * a * s.L + j0 : 0;
  }
  template <bool VEC>
  static __device__ __forceinline__ uint32_t lane_part(const MuShape& s, int j0, int lane, int a) {
    if (TALL) {
      const int i = NT * (lane & 15), last = s.S - NT, j = j0 + 4 * a + lane / 16;
      return (VEC ? lane / 16 : (j < s.L ? j : s.L - 1)) * s.S + (i < last ? i : last);
    }
    const int i = 16 * a + (lane & 15), j = j0 + 8 * (lane / 16);
    if (VEC) return ((a < NT - 1 || i < s.S ? i : s.S - 1) - 16 * a) * s.L + 8 * (lane / 16);
    return (i < s.S ? i : s.S - 1) * s.L + (j < s.L ? j : s.L - 1);
  }
  template <bool VEC>
  static __device__ __forceinline__ int count(const MuShape& s, int j0, int lane, int a) {
    if (TALL) return NT * (lane & 15) < s.S && (VEC || j0 + lane / 16 + 4 * a < s.L) ? NT : 0;
    if (16 * a + (lane & 15) >= s.S) return 0;
    return VEC ? 8 : room(s.L, j0 + 8 * (lane / 16));
  }
  static __device__ __forceinline__ int again(const MuShape& s, int lane) {
    const int i = NT * (lane & 15);
    return TALL && i < s.S && i + NT > s.S ? i + NT - s.S : 0;
  }
  template <bool VEC>
  __device__ __forceinline__ void load(const uint16_t* G, const float* M, const MuShape& s, int j0, int lane) {
#pragma unroll
    for (int a = 0; a < A; ++a) {
      const int n = count<VEC>(s, j0, lane, a), first = base<VEC>(s, j0, a);
      load_f<VEC, false, B>(M + first, lane_part<VEC>(s, j0, lane, a), n, m[a]);
      load_h<VEC, B>(G + first, lane_part<VEC>(s, j0, lane, a), n, g[a]);
    }
  }
  // m <- mu m + g; the tiles' sums take u.
  template <bool VEC>
  __device__ __forceinline__ void use(float* M, const MuShape& s, int j0, int lane, float mu, int nesterov,
                                      f64x4 (&acc)[mu_tiles(NT)]) {
    float v[A][B];
    const int dup = again(s, lane);
#pragma unroll
    for (int a = 0; a < A; ++a) {
      const int n = count<VEC>(s, j0, lane, a);
#pragma unroll
      for (int b = 0; b < B; ++b) {
        m[a][b] = mu_momentum(m[a][b], g[a].f32(b), mu);
        v[a][b] = (b < n && b >= dup) ? mu_update(m[a][b], g[a].f32(b), mu, nesterov) : 0.0f;
      }
      store_f<VEC, false, B>(M + base<VEC>(s, j0, a), lane_part<VEC>(s, j0, lane, a), n, m[a]);
    }
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      double d[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) d[t] = (double)(TALL ? v[TALL ? c : 0][TALL ? t : 0] : v[TALL ? 0 : t][TALL ? 0 : c]);
#pragma unroll
      for (int t2 = 0; t2 < NT; ++t2)
#pragma unroll
        for (int t = 0; t <= t2; ++t) acc[mu_tiles(t2) + t] = mfma_f64(d[t], d[t2], acc[mu_tiles(t2) + t]);
    }
  }
};

// The sums of one wave (`wave` of `waves`) over a matrix.
template <int NT, bool TALL>
__device__ __forceinline__ void gram_sums(const uint16_t* G, float* M, const MuShape& s, int64_t mat, int wave, int waves,
                                          int lane, float mu, int nesterov, f64x4 (&acc)[mu_tiles(NT)]) {
#pragma unroll
  for (int u = 0; u < mu_tiles(NT); ++u) acc[u] = f64x4{0.0, 0.0, 0.0, 0.0};
  Steps at(s, mat, wave, waves, 32);
  GramLoad<NT, TALL> x;
#pragma unroll 1
  for (; at.valid(); at.i += at.stride) {
    x.template load<true>(G, M, s, at.j0(at.i), lane);
    x.template use<true>(M, s, at.j0(at.i), lane, mu, nesterov, acc);
  }
#pragma unroll 1
  for (int64_t j0 = at.rest; j0 < s.L; j0 += (int64_t)at.stride * 32) {
    x.template load<false>(G, M, s, (int)j0, lane);
    x.template use<false>(M, s, (int)j0, lane, mu, nesterov, acc);
  }
}

// The W waves' sums to wave 0, halving: the upper half of the waves left hand
// theirs to the lower half.  red: W / 2 x U x 256 doubles.
template <int NT, int W>
__device__ __forceinline__ void gram_reduce(f64x4 (&acc)[mu_tiles(NT)], double* red, int wave, int lane) {
  constexpr int U = mu_tiles(NT);
#pragma unroll
  for (int half = W / 2; half >= 1; half /= 2) {
    if (wave >= half && wave < 2 * half) {
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int q = 0; q < 4; ++q) red[((wave - half) * U + u) * 256 + q * 64 + lane] = acc[u][q];
    }
    __syncthreads();
    if (wave < half) {
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[u][q] += red[(wave * U + u) * 256 + q * 64 + lane];
    }
    __syncthreads();
  }
}

// Bound by memory, 10 bytes a parameter, where S is large (80 x 64 x 8192: 90
// us, 420 MB at 4.7 TB/s; the fp64 MFMAs of a triangle of tiles take 51 us of
// the matrix units beside it), by the latency of its few steps where it is
// not (32 x 11008 x 16: 11 us, 56 MB).  Three waves a SIMD: at two the loads of
// one step do not cover the sums (368 us for the whole call, 336 with three).
template <int NT, bool TALL>
__global__ __launch_bounds__(kMuThreads, 3) void k_muon_gram(const uint16_t* __restrict__ G, float* __restrict__ M,
                                                             MuShape s, float mu, int nesterov, int splits,
                                                             double* __restrict__ part) {
  constexpr int U = mu_tiles(NT);
  __shared__ double red[2 * U * 256];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const MuPlace at(s, splits, false);
  const int64_t base = at.mat * s.rows * s.cols;
  f64x4 acc[U];
  gram_sums<NT, TALL>(G + base, M + base, s, at.mat, at.split * 4 + wave, splits * 4, lane, mu, nesterov,
                      acc);
  gram_reduce<NT, 4>(acc, red, wave, lane);
  if (wave == 0) {
    double* out = part + (size_t)at.group * U * 256;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int q = 0; q < 4; ++q) out[u * 256 + q * 64 + lane] = acc[u][q];
  }
}

// ---------------------------------------------------- S x S iteration ----
//
// One matrix per work-group, on fp64 MFMA tiles with the four matrices G, P,
// Q, R in LDS, padded with zeros to N = 16 NT.  All of them are polynomials in
// G_0, so they are symmetric and commute: an operand's fragment (lane l: index
// l % 16, k = l / 16) is read as row k, sixteen consecutive doubles, for
// either side, and a tile is written both as it is and transposed.  Element
// (k, i) lies at column i ^ (k % 16), and for even NT in the other 16-column
// half for odd k (N = 16 and 48 put odd rows into the other half of the LDS
// banks by themselves): then the two rows that a half-wave reads or writes,
// and the two columns it writes transposed, meet no bank twice.
//
// D of the instruction: lane l, register q holds row l / 16 + 4 q, column
// l % 16.
//
// Per step: P from G G; then P Q and P G, which read the same matrices, in one
// phase; then (P G) P.  The last step needs no G.
template <int NT>
struct PolyLds {
  static constexpr int N = 16 * NT;
  static __device__ __forceinline__ int at(int k, int i) {
    return k * N + (i ^ (NT % 2 == 0 ? (k & 15) | ((k & 1) << 4) : k & 15));
  }
};

// Four waves per SIMD (one would leave the matrix unit idle over its own LDS
// traffic; S = 64: two 36.7 us, four 34.5) share the tiles in turn; the second
// of two products that run in one phase starts with the wave at which the
// first one's tiles ended.
//
// 17 products in five steps at S = 64 are 2720 MFMAs of 64 cycles, 18 us of
// the four matrix units of the one CU that a matrix has; the rest are 15 LDS
// phases and the sum of the partials (S = 48: 24 us, S = 32: 14).
constexpr int kPolyWaves = 16;
template <int NT>
constexpr int kPolyTiles = (mu_tiles(NT) + kPolyWaves - 1) / kPolyWaves;

// Tile e of this wave of the first (turn 0) or second product of a phase.
struct PolyTile {
  int u, t, t2;
};
template <int NT>
__device__ __forceinline__ PolyTile poly_tile(int turn, int e) {
  constexpr int W = kPolyWaves, U = mu_tiles(NT);
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int u = (wave + (turn ? W - U % W : 0)) % W + W * e;
  const int t2 = (u >= 1) + (u >= 3) + (u >= 6);
  return PolyTile{u, u - t2 * (t2 + 1) / 2, t2};
}

// The wave's tiles of x y, handed element by element to f(q, i, k, value,
// add(i, k)); add is called before the products, so that the LDS reads in it
// do not wait for f's writes one by one (S = 32: 18.1 us, 16.9 so).
template <int NT, typename A, typename F>
__device__ __forceinline__ void poly_mul(int turn, const double* x, const double* y, A add, F f) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int e = 0; e < kPolyTiles<NT>; ++e) {
    const PolyTile p = poly_tile<NT>(turn, e);
    if (p.u >= mu_tiles(NT)) break;
    // row lane / 16; row + 4 k differs in bits 2 and 3 of the column
    const int xo = PolyLds<NT>::at(lane / 16, 16 * p.t + (lane & 15));
    const int yo = PolyLds<NT>::at(lane / 16, 16 * p.t2 + (lane & 15));
    double more[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) more[q] = add(16 * p.t + lane / 16 + 4 * q, 16 * p.t2 + (lane & 15));
    f64x4 acc = {0.0, 0.0, 0.0, 0.0};
#pragma unroll
    for (int k = 0; k < 4 * NT; ++k)
      acc = mfma_f64(x[(xo ^ (4 * (k & 3))) + k * 64 * NT], y[(yo ^ (4 * (k & 3))) + k * 64 * NT], acc);
#pragma unroll
    for (int q = 0; q < 4; ++q) f(4 * e + q, 16 * p.t + lane / 16 + 4 * q, 16 * p.t2 + (lane & 15), acc[q], more[q]);
  }
}

template <int NT>
__device__ __forceinline__ void poly_put(double* m, int i, int k, double v) {
  m[PolyLds<NT>::at(i, k)] = v;
  if ((i ^ k) >> 4) m[PolyLds<NT>::at(k, i)] = v;
}

// Short index -> the index 16 t + i that the Gram matrix's tiles give it.
template <int NT, bool TALL>
__device__ __forceinline__ int poly_index(int e, int S) {
  if (!TALL) return e;
  return e < S / NT * NT ? e % NT * 16 + e / NT : (e - (S - NT)) * 16 + S / NT;
}

// G (in LDS) -> Q / (|u| + eps), rounded to fp32: N x N, zeros past S, and
// zeros for u = 0 (whose X is 0 also where a^n / eps is past fp32).
template <int NT, bool TALL>
__device__ __forceinline__ void poly_run(double* G, double* P, double* Q, double* R, const MuonCoef& co, float eps,
                                         float* out, int S) {
  using At = PolyLds<NT>;
  constexpr int N = At::N, U = mu_tiles(NT), kThreads = 64 * kPolyWaves;
  const auto none = [](int, int) { return 0.0; };
  const int lane = threadIdx.x & 63;
  double trace = lane < N ? G[At::at(lane, lane)] : 0.0;
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) trace += __shfl_xor(trace, o, 64);
  const double inv = 1.0 / (sqrt(trace) + (double)eps);
  __syncthreads();
  for (int e = threadIdx.x; e < N * N; e += kThreads) G[e] *= inv * inv;
  __syncthreads();
#pragma unroll 1
  for (int n = 0; n < co.n; ++n) {
    const double ca = co.c[n][0], cb = co.c[n][1], cc = co.c[n][2];
    const bool last = n + 1 == co.n;
    poly_mul<NT>(
        0, G, G, [&](int i, int k) { return fma(cb, G[At::at(i, k)], i == k ? ca : 0.0); },
        [&](int, int i, int k, double v, double add) {
          const double p = fma(cc, v, add);
          poly_put<NT>(P, i, k, p);
          if (n == 0) poly_put<NT>(Q, i, k, p);
        });
    __syncthreads();
    double hold[4 * kPolyTiles<NT>];  // P Q, until every wave has read Q
    if (n > 0) poly_mul<NT>(0, P, Q, none, [&](int e, int, int, double v, double) { hold[e] = v; });
    if (!last) poly_mul<NT>(1, P, G, none, [&](int, int i, int k, double v, double) { poly_put<NT>(R, i, k, v); });
    __syncthreads();
    if (n > 0) {
#pragma unroll
      for (int e = 0; e < kPolyTiles<NT>; ++e) {
        const PolyTile p = poly_tile<NT>(0, e);
        if (p.u >= U) break;
#pragma unroll
        for (int q = 0; q < 4; ++q)
          poly_put<NT>(Q, 16 * p.t + lane / 16 + 4 * q, 16 * p.t2 + (lane & 15), hold[4 * e + q]);
      }
    }
    if (!last) poly_mul<NT>(0, R, P, none, [&](int, int i, int k, double v, double) { poly_put<NT>(G, i, k, v); });
    __syncthreads();
  }
  for (int e = threadIdx.x; e < N * N; e += kThreads) {
    const int i = e / N, k = e % N;
    out[e] = i < S && k < S && trace != 0.0
                 ? (float)(Q[At::at(poly_index<NT, TALL>(i, S), poly_index<NT, TALL>(k, S))] * inv)
                 : 0.0f;
  }
}

// S <= 16: one tile, one wave, no LDS.  The accumulator's register q holds row
// l / 16 + 4 q of column l % 16, which is just what operand step k = q of the
// next product takes: every product feeds the next one in place.
__device__ __forceinline__ f64x4 poly_mul16(const f64x4& x, const f64x4& y) {
  f64x4 acc = {0.0, 0.0, 0.0, 0.0};
#pragma unroll
  for (int k = 0; k < 4; ++k) acc = mfma_f64(x[k], y[k], acc);
  return acc;
}

__device__ __forceinline__ void poly_run16(f64x4 G, const MuonCoef& co, float eps, float* out, int S, int lane) {
  f64x4 one;
  double trace = 0.0;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    one[q] = lane / 16 + 4 * q == (lane & 15) ? 1.0 : 0.0;
    trace += one[q] != 0.0 ? G[q] : 0.0;
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) trace += __shfl_xor(trace, o, 64);
  const double inv = 1.0 / (sqrt(trace) + (double)eps);
  G *= inv * inv;
  f64x4 Q = one;
#pragma unroll 1
  for (int n = 0; n < co.n; ++n) {
    const f64x4 sq = poly_mul16(G, G);
    f64x4 P;
#pragma unroll
    for (int q = 0; q < 4; ++q) P[q] = fma(co.c[n][2], sq[q], fma(co.c[n][1], G[q], co.c[n][0] * one[q]));
    Q = n > 0 ? poly_mul16(P, Q) : P;
    if (n + 1 < co.n) G = poly_mul16(poly_mul16(P, G), P);
  }
#pragma unroll
  for (int q = 0; q < 4; ++q)
    out[64 * q + lane] = lane / 16 + 4 * q < S && (lane & 15) < S && trace != 0.0 ? (float)(Q[q] * inv) : 0.0f;
}

// A wave's share of the sum of the splits' partials.
__device__ __forceinline__ f64x4 poly_sum16(const double* __restrict__ src, int wave, int splits, int lane) {
  f64x4 sum = {0.0, 0.0, 0.0, 0.0}, v[8];  // at most 32 partials: all of them in flight
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    v[j] = f64x4{0.0, 0.0, 0.0, 0.0};
    if (wave + 4 * j < splits)
#pragma unroll
      for (int q = 0; q < 4; ++q) v[j][q] = src[(size_t)(wave + 4 * j) * 256 + q * 64 + lane];
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) sum += v[j];
  return sum;
}

// The sum of many partials (a quarter of a tile of a matrix a work-group), so
// that the one work-group of the iteration need not read them all.
constexpr int kSumWaves = 16;
__global__ __launch_bounds__(64 * kSumWaves) void k_muon_sum(const double* __restrict__ part, int splits, int quarters,
                                                             double* __restrict__ sums) {
  __shared__ double red[kSumWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x / 64;
  const double* src = part + ((int64_t)(blockIdx.x / quarters) * splits * quarters + blockIdx.x % quarters) * 64 + lane;
  double sum = 0.0;
#pragma unroll 1
  for (int k = wave; k < splits; k += 8 * kSumWaves) {
    double v[8];  // in flight
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int at = k + j * kSumWaves;
      v[j] = at < splits ? src[(int64_t)at * quarters * 64] : 0.0;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) sum += v[j];
  }
  red[wave][lane] = sum;
  __syncthreads();
  if (wave == 0) {
#pragma unroll
    for (int j = 1; j < kSumWaves; ++j) sum += red[j][lane];
    sums[(int64_t)blockIdx.x * 64 + lane] = sum;
  }
}

// part -> Q / (|u| + eps): N x N, zeros past S.
template <int NT, bool TALL>
__global__ __launch_bounds__(64 * kPolyWaves) void k_muon_poly(const double* __restrict__ part, int splits, int S,
                                                               MuonCoef co, float eps, float* __restrict__ Qout) {
  constexpr int N = 16 * NT, U = mu_tiles(NT);
  __shared__ double m[4][N * N];
  // the partials' sum, in order, several partials' loads in flight for every
  // element of a thread
  constexpr int kThreads = 64 * kPolyWaves, E = (U * 256 + kThreads - 1) / kThreads;
  constexpr int J = NT == 4 ? 8 : 16;
  const double* src = part + (size_t)blockIdx.x * splits * U * 256;
  double sum[E] = {};
#pragma unroll 1
  for (int k = 0; k < splits; k += J) {
    double v[J][E];
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int at = e * kThreads + threadIdx.x;
        v[j][e] = 0.0;
        if (k + j < splits && at < U * 256) v[j][e] = src[(size_t)(k + j) * U * 256 + at];
      }
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int e = 0; e < E; ++e) sum[e] += v[j][e];
  }
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int at = e * kThreads + threadIdx.x;
    const int u = at / 256, q = at / 64 % 4, lane = at % 64, t2 = (u >= 1) + (u >= 3) + (u >= 6);
    if (u < U) poly_put<NT>(m[0], 16 * (u - t2 * (t2 + 1) / 2) + lane / 16 + 4 * q, 16 * t2 + (lane & 15), sum[e]);
  }
  __syncthreads();
  poly_run<NT, TALL>(m[0], m[1], m[2], m[3], co, eps, Qout + (size_t)blockIdx.x * N * N, S);
}

// -------------------------------------------------------------- pass 2 ----
//
// X = Q u on fp32 MFMA tiles (16 x 16 x 4: A[i][k] lane l: i = l % 16, k = l /
// 16; D lane l, register q: row 4 (l / 16) + q, column l % 16), the weights
// and their bf16 copy.  Q is the A operand; rows of D are short indexes,
// columns long positions.  As in pass 1 lanes load consecutive values and the
// order inside an MFMA follows:
//
//   not tall: lane l has C positions C (l % 16) + c of row k = 4 s + l / 16,
//             and D gives it the same C positions of rows 16 t + 4 (l / 16) + q;
//   tall:     a step's positions are one run of memory, which the lanes load
//             and store in consecutive fours whatever S is; u and X change
//             between that order and the operands' (k of MFMA (s, c) is 16 s +
//             4 (l / 16) + c of position l % 16; D: short indexes 16 t + 4 (l /
//             16) + q of that position) in LDS of the wave's own.  Loaded in
//             the operands' order, rows of 64 took 222 us where this takes
//             108 (80 x 8192 x 64).
//
// Q is in LDS (64 x 64 of it would take the registers of the loads in flight),
// in rows of a stride that puts an operand's four rows, next to each other or
// four apart, into four sets of banks.
template <int NT, bool TALL>
struct ApplyShape {
  // positions per lane (not tall) or 16-position groups per step (tall): as
  // much in flight as two waves' share of the registers holds
  static constexpr int C = NT >= 3 ? 2 : 4;
  static constexpr int kStep = 16 * C;
  static constexpr int kQRow = 16 * NT + (TALL ? 4 : NT % 2 == 0 ? 16 : 0);
  static constexpr int kScratch = TALL ? kStep * (16 * NT + 4) : 0;  // floats of a wave
};

// Q (N x N) into an operand's place.
template <int NT, bool TALL>
__device__ __forceinline__ void put_q(const float* Q, float* qs, int threads) {
  constexpr int N = 16 * NT;
  for (int e = threadIdx.x; e < N * N; e += threads) qs[e / N * ApplyShape<NT, TALL>::kQRow + e % N] = Q[e];
}

struct ApplyArgs {
  const uint16_t* G;
  float* M;
  float* W;
  uint16_t* P;
  float mu, decay, step;
  int nesterov;
};

__device__ __forceinline__ float mu_weight(const ApplyArgs& a, float w, float x) {
  return __fsub_rn(__fmul_rn(w, a.decay), __fmul_rn(a.step, x));
}

// The LDS of a wave in the tall form: a row of S + pad floats a position.  Pad
// makes the stride an odd number of 16-byte slots where S is a multiple of 4
// (a quarter wave then reads its 16 positions' slots without a conflict);
// other strides are read and written by single values.
template <int NT>
struct TallLds {
  static constexpr int E = ApplyShape<NT, true>::C * NT;  // fours a lane
  float* lds;
  int S, row, fours;
  bool quads;
  int off[E];  // of the lane's fours in LDS

  __device__ __forceinline__ TallLds(float* lds_, int S_, int lane)
      : lds(lds_), S(S_), row(S_ + (S_ % 8 == 0 ? 4 : 0)), fours(ApplyShape<NT, true>::kStep / 4 * S_),
        quads(S_ % 4 == 0) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int at = 4 * four(e, lane);
      off[e] = row == S ? at : at + 4 * (at / S);
    }
  }
  __device__ __forceinline__ int four(int e, int lane) const {
    const int f = lane + 64 * e;
    return f < fours ? f : fours - 1;
  }
  __device__ __forceinline__ void get4(int e, float (&v)[4]) const {
    const f32x4 x = *reinterpret_cast<const f32x4*>(lds + off[e]);
#pragma unroll
    for (int c = 0; c < 4; ++c) v[c] = x[c];
  }
  __device__ __forceinline__ void put4(int e, const float (&v)[4]) const {
    *reinterpret_cast<f32x4*>(lds + off[e]) = f32x4{v[0], v[1], v[2], v[3]};
  }
  // four of a position from short index i on; past S any finite ones (they
  // meet zeros of Q)
  __device__ __forceinline__ f32x4 get(int pos, int i) const {
    const float* p = lds + pos * row;
    if (quads) return *reinterpret_cast<const f32x4*>(p + (i < S ? i : S - 4));
    f32x4 v;
#pragma unroll
    for (int c = 0; c < 4; ++c) v[c] = p[i + c < S ? i + c : S - 1];
    return v;
  }
  __device__ __forceinline__ void put(int pos, int i, const f32x4& v) const {
    float* p = lds + pos * row;
    if (quads) {
      if (i < S) *reinterpret_cast<f32x4*>(p + i) = v;
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (i + c < S) p[i + c] = v[c];
    }
  }
};

// The wave's own LDS accesses take effect in order; this keeps the compiler to
// it across lanes.
__device__ __forceinline__ void wave_lds_order() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_wave_barrier();
}

// VEC: all positions of the step exist.
template <int NT, bool VEC, bool STREAM>
__device__ __forceinline__ void apply_tall(const ApplyArgs& p, const MuShape& s, int j0, int lane, const float* qs,
                                           const TallLds<NT>& x) {
  constexpr int K = ApplyShape<NT, true>::C, E = TallLds<NT>::E;
  const int first = j0 * s.S, there = (s.L - j0) * s.S;  // elements from the step's first on
  float m[E][4], w[E][4];
  Halves<4> g[E];
  auto at = [&](int e) { return (uint32_t)(VEC ? 4 * x.four(e, lane) : min(4 * x.four(e, lane), there - 1)); };
  auto count = [&](int e) { return VEC ? 4 : room(there, 4 * x.four(e, lane)); };
#pragma unroll
  for (int e = 0; e < E; ++e) {
    load_f<VEC, false, 4>(p.M + first, at(e), count(e), m[e]);
    load_h<VEC, 4>(p.G + first, at(e), count(e), g[e]);
    load_f<VEC, STREAM, 4>(p.W + first, at(e), count(e), w[e]);
  }
  if constexpr (VEC) __builtin_amdgcn_sched_barrier(0);  // all of the step's loads go out first
#pragma unroll
  for (int e = 0; e < E; ++e) {
    float u[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) u[c] = mu_update(m[e][c], g[e].f32(c), p.mu, p.nesterov);
    x.put4(e, u);
  }
  wave_lds_order();
  f32x4 acc[K][NT];
#pragma unroll
  for (int a = 0; a < K; ++a)
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[a][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int k4 = 0; k4 < NT; ++k4) {
    f32x4 u[K];
#pragma unroll
    for (int a = 0; a < K; ++a) u[a] = x.get(16 * a + (lane & 15), 16 * k4 + 4 * (lane / 16));
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      float q[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t)
        q[t] = qs[(16 * k4 + 4 * (lane / 16) + c) * ApplyShape<NT, true>::kQRow + 16 * t + (lane & 15)];
#pragma unroll
      for (int a = 0; a < K; ++a)
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[a][t] = mfma_f32(q[t], u[a][c], acc[a][t]);
    }
  }
  wave_lds_order();
#pragma unroll
  for (int a = 0; a < K; ++a)
#pragma unroll
    for (int t = 0; t < NT; ++t) x.put(16 * a + (lane & 15), 16 * t + 4 * (lane / 16), acc[a][t]);
  wave_lds_order();
#pragma unroll
  for (int e = 0; e < E; ++e) {
    float o[4];
    x.get4(e, o);
#pragma unroll
    for (int c = 0; c < 4; ++c) w[e][c] = mu_weight(p, w[e][c], o[c]);
    store_f<VEC, STREAM, 4>(p.W + first, at(e), count(e), w[e]);
    store_bf16<VEC, STREAM, 4>(p.P + first, at(e), count(e), w[e]);
  }
  wave_lds_order();
}

template <int NT, bool VEC, bool STREAM>
__device__ __forceinline__ void apply_wide(const ApplyArgs& p, const MuShape& s, int j0, int lane, const float* qs) {
  constexpr int C = ApplyShape<NT, false>::C;
  const int j = j0 + C * (lane & 15);
  const int nj = VEC ? C : room(s.L, j), col = VEC ? C * (lane & 15) : (j < s.L ? j : s.L - 1);
  float m[4 * NT][C], w[NT][4][C];
  Halves<C> g[4 * NT];
  // row first + of_lane: only the last tile of 16 can go past S, in its first
  // row too (the base's row is clamped on its own, so that a lane's offset
  // from it is never negative)
  auto row0 = [&](int first) { return first < 16 * (NT - 1) || first < s.S ? first : s.S - 1; };
  auto base = [&](int first) { return VEC ? row0(first) * s.L + j0 : 0; };
  auto at = [&](int first, int of_lane) -> uint32_t {
    if (VEC && first < 16 * (NT - 1)) return of_lane * s.L + col;
    const int i = first + of_lane < s.S ? first + of_lane : s.S - 1;
    return (VEC ? i - row0(first) : i) * s.L + col;
  };
#pragma unroll
  for (int k = 0; k < 4 * NT; ++k) {
    load_f<VEC, false, C>(p.M + base(4 * k), at(4 * k, lane / 16), nj, m[k]);
    load_h<VEC, C>(p.G + base(4 * k), at(4 * k, lane / 16), nj, g[k]);
  }
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int q = 0; q < 4; ++q)
      load_f<VEC, STREAM, C>(p.W + base(16 * t + q), at(16 * t + q, 4 * (lane / 16)), nj, w[t][q]);
  // all of the step's loads go out first, and Q stays in LDS from step to step
  if constexpr (VEC) __builtin_amdgcn_sched_barrier(0);
  asm volatile("" ::: "memory");
  f32x4 acc[NT][C];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int c = 0; c < C; ++c) acc[t][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int k = 0; k < 4 * NT; ++k) {
    float q[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) q[t] = qs[(4 * k + lane / 16) * ApplyShape<NT, false>::kQRow + 16 * t + (lane & 15)];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const float u = mu_update(m[k][c], g[k].f32(c), p.mu, p.nesterov);
#pragma unroll
      for (int t = 0; t < NT; ++t) acc[t][c] = mfma_f32(q[t], u, acc[t][c]);
    }
  }
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int n = 16 * t + 4 * (lane / 16) + q < s.S ? nj : 0;
#pragma unroll
      for (int c = 0; c < C; ++c) w[t][q][c] = mu_weight(p, w[t][q][c], acc[t][c][q]);
      store_f<VEC, STREAM, C>(p.W + base(16 * t + q), at(16 * t + q, 4 * (lane / 16)), n, w[t][q]);
      store_bf16<VEC, STREAM, C>(p.P + base(16 * t + q), at(16 * t + q, 4 * (lane / 16)), n, w[t][q]);
    }
}

// All steps of one wave (`wave` of `waves`) over a matrix.  scratch: kScratch
// floats of the wave's own.
template <int NT, bool TALL, bool STREAM>
__device__ __forceinline__ void apply_steps(const ApplyArgs& p, const MuShape& s, int64_t mat, int wave, int waves,
                                            int lane, const float* qs, float* scratch) {
  constexpr int kStep = ApplyShape<NT, TALL>::kStep;
  Steps at(s, mat, wave, waves, kStep);
  if constexpr (TALL) {
    const TallLds<NT> x(scratch, s.S, lane);
#pragma unroll 1
    for (; at.valid(); at.i += at.stride) apply_tall<NT, true, STREAM>(p, s, at.j0(at.i), lane, qs, x);
#pragma unroll 1
    for (int64_t j0 = at.rest; j0 < s.L; j0 += (int64_t)at.stride * kStep)
      apply_tall<NT, false, false>(p, s, (int)j0, lane, qs, x);
  } else {
#pragma unroll 1
    for (; at.valid(); at.i += at.stride) apply_wide<NT, true, STREAM>(p, s, at.j0(at.i), lane, qs);
#pragma unroll 1
    for (int64_t j0 = at.rest; j0 < s.L; j0 += (int64_t)at.stride * kStep)
      apply_wide<NT, false, false>(p, s, (int)j0, lane, qs);
  }
}

__device__ __forceinline__ ApplyArgs apply_at(ApplyArgs p, int64_t base) {
  p.G += base;
  p.M += base;
  p.W += base;
  p.P += base;
  return p;
}

// With S <= 16 the iteration takes a wave a few microseconds, less than a
// launch: every work-group runs it for itself, from the partials.
//
// The matrices go from the last to the first, whose m and g pass 1 read or
// wrote longest ago.  STREAM: the stack is larger than half the last-level
// cache; weights and their copy, touched once, then go past it, and more of m
// and g is still there (80 x 64 x 8192: 153 us without STREAM, 116 with it;
// pass 1 of the next call 114 and 91; a stack that fits takes 1 us longer).
//
// Bound by memory: 16 bytes a parameter, 671 MB at 5.8 TB/s there; 32 x 11008 x
// 16, in the cache, 18 us, 90 MB at 5 TB/s with the iteration.
template <int NT, bool TALL, bool STREAM>
__global__ __launch_bounds__(kMuThreads, 2) void k_muon_apply(ApplyArgs args, MuShape s, int splits,
                                                              const float* __restrict__ Qin,
                                                              const double* __restrict__ part, int parts, MuonCoef co,
                                                              float eps) {
  constexpr int N = 16 * NT;
  using Sh = ApplyShape<NT, TALL>;
  __shared__ float qs[N * Sh::kQRow];
  __shared__ __attribute__((aligned(16))) float scratch[TALL ? 4 * Sh::kScratch : 1];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const MuPlace at(s, splits, true);
  if constexpr (NT == 1) {
    __shared__ double red[2 * 256];
    __shared__ float Q[256];
    f64x4 sum[1] = {poly_sum16(part + (size_t)at.mat * parts * 256, wave, parts, lane)};
    gram_reduce<1, 4>(sum, red, wave, lane);
    if (wave == 0) poly_run16(sum[0], co, eps, Q, s.S, lane);
    __syncthreads();
    put_q<1, TALL>(Q, qs, kMuThreads);
  } else {
    put_q<NT, TALL>(Qin + (size_t)at.mat * N * N, qs, kMuThreads);
  }
  __syncthreads();
  apply_steps<NT, TALL, STREAM>(apply_at(args, at.mat * s.rows * s.cols), s, at.mat, at.split * 4 + wave, splits * 4,
                                lane, qs, scratch + wave * Sh::kScratch);
}

// A small matrix of S <= 16 whole: one work-group makes both passes and the
// iteration, in one launch.  The second pass finds m as the first one left it
// (the barriers between order the work-group's own stores and loads).
template <bool TALL>
__global__ __launch_bounds__(512) void k_muon_whole(ApplyArgs args, MuShape s, MuonCoef co, float eps) {
  __shared__ double red[4 * 256];
  using Sh = ApplyShape<1, TALL>;
  __shared__ float Q[256], qs[16 * Sh::kQRow];
  __shared__ __attribute__((aligned(16))) float scratch[TALL ? 8 * Sh::kScratch : 1];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int64_t mat = blockIdx.x;
  const ApplyArgs p = apply_at(args, mat * s.rows * s.cols);
  f64x4 acc[1];
  gram_sums<1, TALL>(p.G, p.M, s, mat, wave, 8, lane, p.mu, p.nesterov, acc);
  gram_reduce<1, 8>(acc, red, wave, lane);
  if (wave == 0) poly_run16(acc[0], co, eps, Q, s.S, lane);
  __syncthreads();
  put_q<1, TALL>(Q, qs, 512);
  __syncthreads();
  apply_steps<1, TALL, false>(p, s, mat, wave, 8, lane, qs, scratch + wave * Sh::kScratch);
}

// ----------------------------------------------------------- launchers ----

static int mu_nt(const MuShape& s) { return (s.S + 15) / 16; }

// Work-groups per matrix: as many as the chip holds at a time (`all`), for one
// more would wait for a whole turn of the others (80 x 64 x 8192, pass 2: 115
// us with 6 a matrix, 143 with 7); each with at least `per` long positions.
static int mu_splits(const MuShape& s, int all, int per) {
  const int64_t most = ((int64_t)s.L + per - 1) / per, n = std::min<int64_t>(all / s.nmat, most);
  return (int)std::max<int64_t>(n, 1);
}
// Splits of pass 1.  The work-group that needs the sum of the partials makes
// it, of up to mu_parts (each costs it 0.3 us at S = 64: 8 x 64 x 8192, pass 1
// and iteration: 62 us with 32, 64 with 16, 55 with 32 that a launch has
// summed; 27 x 32 x 10704: 36 with 28, 38 with 16, 40 summed by a launch).
// More are worth that launch where a split's part of the long axis would take
// longer (1 x 64 x 131072, pass 1 and the sum: 282 us with 16, 30 with 512; 1
// x 32 x 65536: 51 with 32, 37 with 256; even at the lengths of the rule).
static int mu_parts(const MuShape& s) { return s.S > 48 ? 16 : 32; }
static int gram_splits(const MuShape& s) {
  const int n = mu_splits(s, 3 * 256, 256);
  return s.L > (s.S > 48 ? 4096 : s.S > 32 ? 16384 : 32768) ? n : std::min(n, mu_parts(s));
}

static bool mu_whole(const MuShape& s) { return s.S <= 16 && (int64_t)s.S * s.L <= kMuWhole; }

// Partials and, of more than mu_parts, their sums.
static size_t mu_part_bytes(const MuShape& s) {
  const int n = gram_splits(s);
  return (size_t)s.nmat * (n + (n > mu_parts(s))) * mu_tiles(mu_nt(s)) * 256 * sizeof(double);
}

size_t muon_ws_bytes(int64_t nmat, int64_t rows, int64_t cols) {
  const MuShape s = mu_shape(nmat, rows, cols);
  if (mu_whole(s)) return 0;
  const size_t n = 16 * (size_t)mu_nt(s);
  return mu_part_bytes(s) + (n > 16 ? (size_t)nmat * n * n * sizeof(float) : 0);
}

template <int NT, bool TALL>
static void muon_kernels(const ApplyArgs& a, const MuShape& s, float eps, const MuonCoef& co, double* part, float* Q,
                         hipStream_t st) {
  if constexpr (NT == 1)
    if (mu_whole(s)) {
      QLORA_LAUNCH("muon_whole", st, k_muon_whole<TALL>, dim3((unsigned)s.nmat), dim3(512), 0, st, a, s, co, eps);
      return;
    }
  const int gs = gram_splits(s), as = mu_splits(s, 2 * 256, 4 * ApplyShape<NT, TALL>::kStep);
  const dim3 block(kMuThreads);
  QLORA_LAUNCH("muon_gram", st, (k_muon_gram<NT, TALL>), dim3((unsigned)(s.nmat * gs)), block, 0, st, a.G, a.M, s,
               a.mu, a.nesterov, gs, part);
  int parts = gs;
  if (gs > mu_parts(s)) {
    double* sums = part + (size_t)s.nmat * gs * mu_tiles(NT) * 256;
    QLORA_LAUNCH("muon_sum", st, k_muon_sum, dim3((unsigned)(s.nmat * mu_tiles(NT) * 4)), dim3(64 * kSumWaves), 0, st,
                 part, gs, mu_tiles(NT) * 4, sums);
    part = sums;
    parts = 1;
  }
  if constexpr (NT > 1)
    QLORA_LAUNCH("muon_poly", st, (k_muon_poly<NT, TALL>), dim3((unsigned)s.nmat), dim3(64 * kPolyWaves), 0, st, part,
                 parts, s.S, co, eps, Q);
  const dim3 grid((unsigned)(s.nmat * as));
  // m, g, w and p; rows that do not start on a line go through the cache, which
  // puts the lines that steps share together (27 x 52 x 10706: 57 us, past it
  // 101; 80 x 64 x 8192: 153, past it 116)
  if (14 * s.nmat * s.rows * s.cols > ((int64_t)128 << 20) && (TALL || s.L % 32 == 0))
    QLORA_LAUNCH("muon_apply", st, (k_muon_apply<NT, TALL, true>), grid, block, 0, st, a, s, as, Q, part, parts, co, eps);
  else
    QLORA_LAUNCH("muon_apply", st, (k_muon_apply<NT, TALL, false>), grid, block, 0, st, a, s, as, Q, part, parts, co, eps);
}

hipError_t launch_muon(uint16_t* P, float* W, const uint16_t* G, float* m, int64_t nmat, int64_t rows, int64_t cols,
                       float lr, float momentum, int nesterov, float wd, float scale, float eps, const MuonCoef& co,
                       void* ws, hipStream_t st) {
  const MuShape s = mu_shape(nmat, rows, cols);
  double* part = reinterpret_cast<double*>(ws);
  float* Q = reinterpret_cast<float*>(reinterpret_cast<char*>(ws) + mu_part_bytes(s));
  const ApplyArgs a{G, m, W, P, momentum, (float)(1.0 - (double)lr * wd), (float)((double)lr * scale), nesterov};
  using Fn = void (*)(const ApplyArgs&, const MuShape&, float, const MuonCoef&, double*, float*, hipStream_t);
  static const Fn table[2][4] = {
      {muon_kernels<1, false>, muon_kernels<2, false>, muon_kernels<3, false>, muon_kernels<4, false>},
      {muon_kernels<1, true>, muon_kernels<2, true>, muon_kernels<3, true>, muon_kernels<4, true>}};
  table[s.tall][mu_nt(s) - 1](a, s, eps, co, part, Q, st);
  return hipGetLastError();
}

}  // namespace qlora
