// scores.hip -- what a head's logits say of each token: the log-probabilities
// of given tokens, the distribution's entropy and its best words; and the
// gradient of a loss on log-probabilities and entropy.
//
// With t_v = tau (z_v - max z), S = sum exp t_v, p_v = exp(t_v) / S and the
// mean exponent tm = sum p_v t_v:
//
//   logp_j = t_{y_j} - ln S,     H = -sum p_v ln p_v = ln S - tm,
//   d logp_j / d z_v = tau ([v = y_j] - p_v),   d H / d z_v = -tau p_v (t_v - tm)
//
// (p_v ln p_v is 0 for a masked word, p_v = 0).  Exponents are held in units of
// log 2 (rows.hpp) and so is their sum sum_v e_v x_v, in which a masked word's
// -inf counts as -256: times its e_v = 0.  k's rounding moves every x_v and their
// mean alike, so H = ln s - ln 2 (mean x) is free of it.
//
// The n best words.  Every word belongs to one of 64 groups, its 16-byte
// piece's lane.  The n-th largest of the groups' maxima is a bound L that at
// least n words reach, and few more do (n = 20 of independent words: some 25;
// n = 64, where L is the least of the maxima: some 300).  The maxima are formed
// for the row's maximum anyway; words from L on go to a list, whose order by
// (logit, then lowest index) is counted out.  Where equal logits make the list
// too long (a row of one value), the bound comes from counting the digits of
// the whole order instead, in several readings of the row.
#include <type_traits>

#include "launch.hpp"
#include "rows.hpp"

namespace qlora {

constexpr float kFloor = -256.0f;  // exponents of words of probability 0
constexpr float kLowest = -3.4028234663852886e38f;

struct ScoreArgs {
  const void* logits;
  int64_t first, T, ld, ldd;  // rows first to T - 1
  int V;
  const int32_t* tokens;  // T x m
  int m, n;
  float tau;
  Scale c;
  float* logp;     // T x m
  float* entropy;  // T
  int32_t* ids;    // T x n
  float* top;      // T x n
  float* stats;    // (max z, sum of e, mean x) per row
  const float* dlogp;     // T x m
  const float* dentropy;  // T, or nullptr
  void* dlogits;
  bool stream;
};

// Exponents and sums of a row in registers.
struct Sums {
  float s, u;  // of e and of e x
};
template <bool FAR>
__device__ __forceinline__ float exponent(const RowExp& x, float z) {
  return FAR ? x.c.times(z - x.m) : fmaf(z, x.c.lo, fmaf(z, x.c.hi, -x.k));
}
template <typename E, int T, int N, bool FAR>
__device__ __forceinline__ Sums regs_sums_of(const RowRegs<E, T, N>& r, const RowExp& x) {
  constexpr int kPer = Elem<E>::kPer16;
  const float xl = exponent<FAR>(x, r.last), el = exp2_hw(xl);
  float s[2] = {el, 0.0f}, u[2] = {el * fmaxf(xl, kFloor), 0.0f};
#pragma unroll
  for (int j = 0; j < N; ++j) {
    float f[kPer];
    Elem<E>::unpack(anew<1 + FAR>(r.w[j]), f);
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      const float xv = exponent<FAR>(x, f[q]), e = exp2_hw(xv);
      s[q & 1] += e;
      u[q & 1] = fmaf(e, fmaxf(xv, kFloor), u[q & 1]);
    }
  }
  return Sums{s[0] + s[1], u[0] + u[1]};
}

// Running maximum m, sum of e = exp2((z - m) c) and of e x, as Online.
struct OnlineSums {
  float m = kNegInf, s = 0.0f, u = 0.0f;
  __device__ __forceinline__ void rescale(float ref, const Scale& c) {
    const float d = fmaxf(c.times(m - ref), kFloor), f = exp2_hw(d);
    u = f * fmaf(d, s, u);
    s *= f;
  }
  __device__ __forceinline__ void term(float d, const Scale& c) {
    const float x = c.times(d), e = exp2_hw(x);
    s += e;
    u = fmaf(e, fmaxf(x, kFloor), u);
  }
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
    rescale(ref, c);
#pragma unroll
    for (int j = 0; j < N; ++j) {
      Elem<E>::unpack(anew<2>(w[j]), f);
#pragma unroll
      for (int q = 0; q < kPer; ++q) term(f[q] - ref, c);
    }
    m = mx;
  }
  __device__ __forceinline__ void add_one(float f, const Scale& c) {
    const float mx = fmaxf(m, f), ref = mx == kNegInf ? 0.0f : mx;
    rescale(ref, c);
    term(f - ref, c);
    m = mx;
  }
};

template <typename E, int N>
__device__ __forceinline__ void load_pieces(const E* z, const RowSpan& at, int i0, int T, u32x4 (&w)[N]) {
#pragma unroll
  for (int j = 0; j < N; ++j) {
    w[j] = u32x4{Elem<E>::kFill, Elem<E>::kFill, Elem<E>::kFill, Elem<E>::kFill};
    if (i0 + j * T < at.nv) w[j] = *reinterpret_cast<const u32x4*>(z + at.head + (size_t)(i0 + j * T) * Elem<E>::kPer16);
  }
}

// ------------------------------------------------------ the best words ----

// Whole numbers in the order of the floats (-0 as 0; no NaN comes here), and back.
__device__ __forceinline__ uint32_t order_of(float f) {
  const uint32_t b = __float_as_uint(f + 0.0f);
  return (b & 0x80000000u) != 0u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float float_of(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) != 0u ? k & 0x7FFFFFFFu : ~k);
}
// A word's place in the order: by logit, then the lowest index.
__device__ __forceinline__ uint64_t place_of(float f, int i) { return (uint64_t)order_of(f) << 32 | (uint32_t)~i; }

// Largest value of 16 leading bits that at least n of the lanes' maxima reach,
// finite: a masked word is no alternative.
__device__ __forceinline__ float bound_of(float lane_max, int n) {
  const uint32_t key = order_of(lane_max) >> 16;
  uint32_t k = 0u;
#pragma unroll
  for (int b = 15; b >= 0; --b) {
    const uint32_t t = k | (1u << b);
    if (__popcll(__ballot(key >= t)) >= n) k = t;
  }
  return k <= 0x007Fu ? kLowest : float_of(k << 16);
}

constexpr int kList = 1024;  // words that the list holds

struct Best {
  uint64_t list[kList];
  int count;
  int need, above;      // of the counting by digits
  uint64_t prefix;
  int bins[256];
};

__device__ __forceinline__ void best_add(Best& b, float f, int i) {
  const int at = atomicAdd(&b.count, 1);
  if (at < kList) b.list[at] = place_of(f, i);
}

template <typename E>
__device__ __forceinline__ void best_piece(Best& b, const u32x4& w, int i0, float bound) {
  constexpr int kPer = Elem<E>::kPer16;
  float f[kPer];
  Elem<E>::unpack(w, f);
  float mx = f[0];
#pragma unroll
  for (int q = 1; q < kPer; ++q) mx = fmaxf(mx, f[q]);
  if (mx >= bound) {
#pragma unroll
    for (int q = 0; q < kPer; ++q)
      if (f[q] >= bound) best_add(b, f[q], i0 + q);
  }
}

// Every finite word of the row, by whole work-groups' steps: fn(value, index).
template <typename E, int T, typename F>
__device__ __forceinline__ void each_word(const E* z, int V, F fn) {
  for (int i = threadIdx.x; i < V; i += T) {
    const float f = Elem<E>::get(z + i);
    if (f >= kLowest) fn(f, i);
  }
}

// The list of a row with too many words from the bound on: the order's digits
// from the highest down, each counted over the row, until the words from the
// prefix on fit the list.  Ends after eight digits at the latest: places are
// distinct, so that n of them are left.
template <typename E, int T>
__device__ void best_by_digits(const E* z, int V, int n, Best& b) {
  if (threadIdx.x == 0) {
    b.prefix = 0u;
    b.need = n;
  }
  int shift = 64;
  do {
    shift -= 8;
    for (int i = threadIdx.x; i < 256; i += T) b.bins[i] = 0;
    __syncthreads();
    const uint64_t prefix = b.prefix;
    const int need = b.need;
    each_word<E, T>(z, V, [&](float f, int i) {
      const uint64_t p = place_of(f, i);
      if (shift < 56 && (p ^ prefix) >> (shift + 8) != 0u) return;
      const int d = (int)(p >> shift) & 255;
      // equal digits of a wave are counted at once: rows that come here hold many
      const int lead = __builtin_amdgcn_readfirstlane(d);
      const uint64_t same = __ballot(d == lead);
      if (d != lead)
        atomicAdd(&b.bins[d], 1);
      else if ((int)(threadIdx.x & 63) == (int)__ffsll((long long)same) - 1)
        atomicAdd(&b.bins[d], (int)__popcll(same));
    });
    __syncthreads();
    if (threadIdx.x == 0) {
      int above = 0, d = 255;
      while (d > 0 && above + b.bins[d] < need) above += b.bins[d--];
      b.prefix = prefix | (uint64_t)d << shift;
      b.need = need - above;
      b.count = n - need + above + b.bins[d];  // words from the new prefix on
    }
    __syncthreads();
  } while (b.count > kList && shift > 0);
  const uint64_t from = b.prefix;
  __syncthreads();
  if (threadIdx.x == 0) b.count = 0;
  __syncthreads();
  each_word<E, T>(z, V, [&](float f, int i) {
    if (place_of(f, i) >= from) best_add(b, f, i);
  });
  __syncthreads();
}

// ------------------------------------------------------------- forward ----

// A row a work-group, as in the losses: N > 0 pieces a thread in registers, N <
// 0: -N pieces a thread at a time.
template <typename E, int T, int N>
__global__ __launch_bounds__(T) void k_scores(ScoreArgs a) {
  constexpr int W = T / 64;
  __shared__ float maxima[W][64];
  __shared__ float sums[W], means[W];
  __shared__ float bound_sh;
  __shared__ double ln_sh;
  __shared__ Best best;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = a.first + blockIdx.x;
  const int token = lane < a.m ? a.tokens[t * a.m + lane] : -1;
  const bool counted = is_counted(token, a.V);
  if (a.m > 0 && __ballot(counted) == 0u) {
    if ((int)threadIdx.x < a.m) a.logp[t * a.m + threadIdx.x] = 0.0f;
    for (int i = threadIdx.x; i < a.n; i += T) {
      a.ids[t * a.n + i] = -1;
      a.top[t * a.n + i] = kNegInf;
    }
    if (threadIdx.x == 0) {
      a.entropy[t] = 0.0f;
      if (a.stats != nullptr) {
        a.stats[3 * t] = 0.0f;
        a.stats[3 * t + 1] = 1.0f;
        a.stats[3 * t + 2] = 0.0f;
      }
    }
    return;
  }
  const E* z = reinterpret_cast<const E*>(a.logits) + t * a.ld;
  float zy = 0.0f;
  if (wave == 0 && counted) zy = Elem<E>::get(z + token);
  RowRegs<E, T, N < 0 ? 1 : N> r;
  const RowSpan at(z, a.V);
  OnlineSums o;
  float own;  // this thread's largest
  if constexpr (N > 0) {
    r.load(z, a.V, at);
    own = r.max();
  } else {
    for (int i0 = threadIdx.x; i0 < at.nv; i0 += -N * T) {
      u32x4 w[N < 0 ? -N : 1];
      load_pieces<E>(z, at, i0, T, w);
      o.template add<E>(w, a.c);
    }
    if (at.rest < a.V) o.add_one(Elem<E>::get(z + at.rest), a.c);
    own = o.m;
  }
  float group = own;
  if (T > 64) {
    maxima[wave][lane] = own;
    __syncthreads();
    group = maxima[0][lane];
#pragma unroll
    for (int w = 1; w < W; ++w) group = fmaxf(group, maxima[w][lane]);
  }
  const float m = wave_max(group);
  if (a.n > 0 && wave == 0) {
    const float bound = bound_of(group, a.n);
    if (lane == 0) {
      bound_sh = bound;
      best.count = 0;
    }
  }
  const RowExp x(m, a.c);
  Sums sum;
  if constexpr (N > 0) {
    sum = x.far ? regs_sums_of<E, T, N, true>(r, x) : regs_sums_of<E, T, N, false>(r, x);
  } else {
    // from a thread's own maximum to the row's (a row of nothing but -inf has
    // no distribution: NaN)
    const float d = a.c.times(o.m - m), f = exp2_hw(d);
    sum = Sums{o.s * f, f * fmaf(fmaxf(d, kFloor), o.s, o.u)};
  }
  float s = wave_sum(sum.s), u = wave_sum(sum.u);
  if (T > 64) {
    if (lane == 0) {
      sums[wave] = s;
      means[wave] = u;
    }
    __syncthreads();
    s = sums[0];
    u = means[0];
#pragma unroll
    for (int w = 1; w < W; ++w) {
      s += sums[w];
      u += means[w];
    }
  }
  float mean = u / s;
  if constexpr (N < 0) {
    s *= x.shift();
    if (!x.far) mean += (float)((double)m * a.c.c - (double)x.k);
  }
  const bool real = s == s;
  if (wave == 0) {  // fp64, once: one wave
    const double ln_sum = x.ln_sum(s);
    if (lane < a.m)
      a.logp[t * a.m + lane] = counted ? (float)(((double)zy - (double)m) * (double)a.tau - ln_sum) : 0.0f;
    if (lane == 0) {
      const float h = (float)(log((double)s) - kLn2 * (double)mean);
      a.entropy[t] = h < 0.0f ? 0.0f : h;
      if (a.stats != nullptr) {
        a.stats[3 * t] = m;
        a.stats[3 * t + 1] = s;
        a.stats[3 * t + 2] = mean;
      }
      ln_sh = ln_sum;
    }
  }
  if (a.n == 0) return;
  __syncthreads();
  if (real) {
    const float bound = bound_sh;
    if (own >= bound) {
      if constexpr (N > 0) {
#pragma unroll
        for (int j = 0; j < N; ++j)
          best_piece<E>(best, anew<3>(r.w[j]), at.head + (j * T + (int)threadIdx.x) * Elem<E>::kPer16, bound);
      } else {
        for (int i0 = threadIdx.x; i0 < at.nv; i0 += 4 * T) {
          u32x4 w[4];
          load_pieces<E>(z, at, i0, T, w);
#pragma unroll
          for (int j = 0; j < 4; ++j) best_piece<E>(best, w[j], at.head + (i0 + j * T) * Elem<E>::kPer16, bound);
        }
      }
      if (at.rest < a.V) {
        const float f = N > 0 ? r.last : Elem<E>::get(z + at.rest);
        if (f >= bound) best_add(best, f, at.rest);
      }
    }
    __syncthreads();
    if (best.count > kList) best_by_digits<E, T>(z, a.V, a.n, best);
  }
  const int count = real ? best.count : 0;
  const double ln_sum = ln_sh;
  for (int i = threadIdx.x; i < count; i += T) {
    const uint64_t p = best.list[i];
    int rank = 0;
    for (int j = 0; j < count; ++j) rank += best.list[j] > p ? 1 : 0;
    if (rank < a.n) {
      a.ids[t * a.n + rank] = (int)~(uint32_t)p;
      a.top[t * a.n + rank] = (float)(((double)float_of((uint32_t)(p >> 32)) - (double)m) * (double)a.tau - ln_sum);
    }
  }
  for (int i = count + (int)threadIdx.x; i < a.n; i += T) {
    a.ids[t * a.n + i] = -1;
    a.top[t * a.n + i] = real ? kNegInf : s;
  }
}

// ------------------------------------------------------------ gradient ----
//
// d_v = e_v (A + B (x_v - mean)) with A = -tau G / s, G = sum_j g_j over the
// counted tokens, and B = -tau gH ln 2 / s; a token's own element gets tau
// sum g_j over its entries on top.
struct GradOf {
  float A, B, mean;
};
template <typename E, bool FAR, bool ENT>
__device__ __forceinline__ float grad_value(float z, const RowExp& x, const GradOf& g) {
  if (!ENT) return (FAR ? x.far_e(z) : x.template near_g<E>(z)) * g.A;
  const float xv = exponent<FAR>(x, z);
  return exp2_hw(xv) * fmaf(fmaxf(xv, kFloor) - g.mean, g.B, g.A);
}
template <typename E, bool FAR, bool ENT>
__device__ __forceinline__ u32x4 score_grad_piece(const u32x4& w, const RowExp& x, const GradOf& g) {
  constexpr int kPer = Elem<E>::kPer16;
  float f[kPer];
  Elem<E>::unpack(w, f);
#pragma unroll
  for (int q = 0; q < kPer; ++q) f[q] = grad_value<E, FAR, ENT>(f[q], x, g);
  return Elem<E>::pack(f);
}

// One row from memory to memory; where out is z, a thread overwrites only what
// it has read.
template <typename E, int T, int kBatch, bool FAR, bool ENT, bool STREAM>
__device__ __forceinline__ void score_row(const E* z, E* out, int V, const RowSpan& at, const RowExp& x,
                                          const GradOf& g) {
  constexpr int kPer = Elem<E>::kPer16;
  for (int i = threadIdx.x; i < at.nv; i += kBatch * T) {
    u32x4 w[kBatch];
    load_pieces<E>(z, at, i, T, w);
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
      if (i + j * T < at.nv)
        put16<STREAM>(out + at.head + (size_t)(i + j * T) * kPer, score_grad_piece<E, FAR, ENT>(w[j], x, g));
  }
  if (at.rest < V) Elem<E>::put(out + at.rest, grad_value<E, FAR, ENT>(Elem<E>::get(z + at.rest), x, g));
}

template <typename E, int T>
__global__ __launch_bounds__(T) void k_scores_grad(ScoreArgs a) {
  constexpr int B = T == 1024 ? 8 : 4;
  const int lane = threadIdx.x & 63;
  const int64_t t = a.first + gridDim.x - 1 - blockIdx.x;
  const int token = lane < a.m ? a.tokens[t * a.m + lane] : -1;
  const bool counted = is_counted(token, a.V);
  const float g = counted ? a.dlogp[t * a.m + lane] : 0.0f;
  const bool live = a.m == 0 || __ballot(counted) != 0u;
  const float gh = live && a.dentropy != nullptr ? a.dentropy[t] : 0.0f;
  E* out = reinterpret_cast<E*>(a.dlogits) + t * a.ldd;
  if (gh == 0.0f && __ballot(g != 0.0f) == 0u) {
    row_zero<E, T>(out, (int)a.ldd, a.stream);
    return;
  }
  const E* z = reinterpret_cast<const E*>(a.logits) + t * a.ld;
  const float zy = counted ? Elem<E>::get(z + token) : 0.0f;
  // entries of the same token: the first one takes the sum of all of them
  float sum = 0.0f;
  bool first = counted && threadIdx.x < 64;
  if (threadIdx.x < 64)
    for (int i = 0; i < a.m; ++i) {
      const int ti = __builtin_amdgcn_readlane(token, i);
      const float gi = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(g), i));
      if (ti == token) {
        sum += gi;
        if (i < lane) first = false;
      }
    }
  const float G = wave_sum(g);
  const RowExp x(a.stats[3 * t], a.c);
  const float s = a.stats[3 * t + 1];
  const GradOf go{-G * a.tau / s, -gh * a.tau * (float)kLn2 / s, a.stats[3 * t + 2]};
  const RowSpan at(z, a.V);
  // the tokens' logits are in hand before any of the row is written over
  __syncthreads();
  auto row = [&](auto far, auto ent, auto stream) {
    score_row<E, T, B, decltype(far)::value, decltype(ent)::value, decltype(stream)::value>(z, out, a.V, at, x, go);
  };
  const std::true_type yes{};
  const std::false_type no{};
  if (gh != 0.0f)
    x.far ? (a.stream ? row(yes, yes, yes) : row(yes, yes, no)) : (a.stream ? row(no, yes, yes) : row(no, yes, no));
  else
    x.far ? (a.stream ? row(yes, no, yes) : row(yes, no, no)) : (a.stream ? row(no, no, yes) : row(no, no, no));
  for (int i = a.V + (int)threadIdx.x; i < a.ldd; i += T) Elem<E>::put(out + i, 0.0f);
  // the pieces have left before the tokens' elements are stored over them
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  if (first) {
    const float v = x.far ? (gh != 0.0f ? grad_value<E, true, true>(zy, x, go) : grad_value<E, true, false>(zy, x, go))
                          : (gh != 0.0f ? grad_value<E, false, true>(zy, x, go) : grad_value<float, false, false>(zy, x, go));
    Elem<E>::put(out + token, fmaf(sum, a.tau, v));
  }
}

// ---------------------------------------------------------- launchers ----

static dim3 row_grid(const ScoreArgs& a) { return dim3((unsigned)std::min(a.T - a.first, kRowsALaunch)); }

template <typename E, int T, int N>
static void scores_kernel(const ScoreArgs& a, hipStream_t st) {
  ScoreArgs b = a;
  for (; b.first < b.T; b.first += kRowsALaunch)
    QLORA_LAUNCH("scores", st, (k_scores<E, T, N>), row_grid(b), dim3(T), 0, st, b);
}

template <typename E>
static hipError_t launch_scores_of(const ScoreArgs& a, hipStream_t st) {
  const int64_t pieces = ((int64_t)a.V + Elem<E>::kPer16 - 1) / Elem<E>::kPer16;
  if (pieces <= 64 * 4)
    scores_kernel<E, 64, 4>(a, st);
  else if (a.T <= 256 && pieces > 1024 && pieces <= 1024 * 16)
    pieces <= 1024 * 4 ? scores_kernel<E, 1024, 4>(a, st)
                       : (pieces <= 1024 * 8 ? scores_kernel<E, 1024, 8>(a, st) : scores_kernel<E, 1024, 16>(a, st));
  else if (pieces <= 256 * 4)
    scores_kernel<E, 256, 4>(a, st);
  else if (pieces <= 256 * 8)
    scores_kernel<E, 256, 8>(a, st);
  else if (pieces <= 256 * 12)
    scores_kernel<E, 256, 12>(a, st);
  else if (pieces <= 512 * 8)
    scores_kernel<E, 512, 8>(a, st);
  else if (pieces <= 512 * 12)
    scores_kernel<E, 512, 12>(a, st);
  else if (pieces <= 512 * 16)
    scores_kernel<E, 512, 16>(a, st);
  else
    scores_kernel<E, 1024, -4>(a, st);
  return hipGetLastError();
}

template <typename E, int T>
static void scores_grad_kernel(const ScoreArgs& a, hipStream_t st) {
  ScoreArgs b = a;  // the last rows first, which the forward ended with
  for (b.first = (a.T - 1) / kRowsALaunch * kRowsALaunch; b.first >= 0; b.first -= kRowsALaunch)
    QLORA_LAUNCH("scores_grad", st, (k_scores_grad<E, T>), row_grid(b), dim3(T), 0, st, b);
}

template <typename E>
static hipError_t launch_scores_grad_of(const ScoreArgs& a, hipStream_t st) {
  const int64_t pieces = ((int64_t)a.V + Elem<E>::kPer16 - 1) / Elem<E>::kPer16;
  if (pieces <= 64 * 4)
    scores_grad_kernel<E, 64>(a, st);
  else if (pieces <= 256 * 4)
    scores_grad_kernel<E, 256>(a, st);
  else if (pieces <= 4096 && a.T >= 512)
    scores_grad_kernel<E, 512>(a, st);
  else
    scores_grad_kernel<E, 1024>(a, st);
  return hipGetLastError();
}

hipError_t launch_scores(const void* logits, int f32, int64_t T, int V, int64_t ld, const int32_t* tokens, int m, int n,
                         float tau, float* logp, float* entropy, int32_t* ids, float* top, float* stats,
                         hipStream_t st) {
  const ScoreArgs a{logits, 0, T, ld, 0, V, tokens, m, n, tau, exp2_scale(tau), logp, entropy, ids, top, stats,
                    nullptr, nullptr, nullptr, false};
  return f32 ? launch_scores_of<float>(a, st) : launch_scores_of<uint16_t>(a, st);
}

hipError_t launch_scores_grad(const void* logits, int f32, int64_t T, int V, int64_t ld, const int32_t* tokens, int m,
                              float tau, const float* stats, const float* dlogp, const float* dentropy, void* dlogits,
                              int64_t ldd, hipStream_t st) {
  const ScoreArgs a{logits, 0, T, ld, ldd, V, tokens, m, 0, tau, exp2_scale(tau), nullptr, nullptr, nullptr, nullptr,
                    const_cast<float*>(stats), dlogp, dentropy, dlogits, past_cache(T, ldd, f32)};
  return f32 ? launch_scores_grad_of<float>(a, st) : launch_scores_grad_of<uint16_t>(a, st);
}

}  // namespace qlora
