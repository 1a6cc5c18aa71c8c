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
// The n best words.  Every word belongs to one of 128 groups, its 16-byte
// piece's lane and the parity of its wave.  The n-th largest of the groups'
// maxima is a bound L that at least n words reach, and few more do (of
// independent words, n = 20: some 22, n = 64: some 90).  The maxima are formed
// for the row's maximum anyway; words from L on go to a list, whose order by
// (logit, then lowest index) is counted out.  Where that list would be too long
// (a row of equal logits), the n-th largest logit is found by counting digits in
// further readings of the row.
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
  int span;  // gradient: columns of a work-group
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

// Sums are taken with c in one part, c1 = fl(c), and put right afterwards: with
// lo = c - c1 every exponent lacks z lo (below 2^-16), so that to first order (1e-10
// are left)
//
//   s = s1 (1 + ln 2 lo E z),    mean x = mean x1 + lo E z,    E z = (mean x1 + k) / c1
//
// (the change of the mean by lo times the exponents' variance is left out: it is
// 2^-25 of that variance).  An exponent then takes one fused step in place of two.
//
// 0 times a masked word's -inf makes a sum of e x NaN where that of e is none;
// only then are its terms taken again with the exponents held at -256.
struct Sums {
  float s, u;  // of e and of e x
};
template <bool FAR>
__device__ __forceinline__ float exponent1(const Scale& c, float k, float ref, float z) {
  return FAR ? (z - ref) * c.one : fmaf(z, c.one, -k);
}
// A thread's N pieces, unpacked in each pass over them, or (up to 32 words) once:
// for bf16 the second unpacking is a tenth of a row's instructions (4096 x 32000: 52.4
// us with it, 50.8 without).
template <typename E, int N, bool KEEP>
struct Pieces {
  static constexpr int kPer = Elem<E>::kPer16;
  u32x4 w[KEEP ? 1 : N];
  float v[KEEP ? N : 1][kPer];
  __device__ __forceinline__ explicit Pieces(const u32x4 (&from)[N]) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if constexpr (KEEP)
        Elem<E>::unpack(from[j], v[j]);
      else
        w[j] = from[j];
    }
  }
  template <int PASS>
  __device__ __forceinline__ void get(int j, float (&f)[kPer]) const {
    if constexpr (KEEP) {
#pragma unroll
      for (int q = 0; q < kPer; ++q) f[q] = v[j][q];
    } else {
      Elem<E>::unpack(anew<PASS>(w[j]), f);
    }
  }
  __device__ __forceinline__ float max(int j) const {
    float f[kPer];
    get<0>(j, f);
    float mx = f[0];
#pragma unroll
    for (int q = 1; q < kPer; ++q) mx = fmaxf(mx, f[q]);
    return mx;
  }
};

// PART: of the first `have` pieces (the others hold no words).
template <typename E, int N, bool FAR, bool CLAMP, bool PART, bool KEEP>
__device__ __forceinline__ Sums pieces_sums_of(const Pieces<E, N, KEEP>& w, int have, const Scale& c, float k,
                                               float ref) {
  constexpr int kPer = Elem<E>::kPer16;
  float s[2] = {0.0f, 0.0f}, u[2] = {0.0f, 0.0f};
#pragma unroll
  for (int j = 0; j < N; ++j) {
    if (PART && j >= have) break;
    float f[kPer];
    w.template get<1 + PART + 2 * CLAMP>(j, f);
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      const float x = exponent1<FAR>(c, k, ref, f[q]), e = exp2_hw(x);
      s[q & 1] += e;
      u[q & 1] = fmaf(e, CLAMP ? fmaxf(x, kFloor) : x, u[q & 1]);
    }
  }
  return Sums{s[0] + s[1], u[0] + u[1]};
}
template <typename E, int N, bool KEEP>
__device__ __forceinline__ Sums pieces_sums(const Pieces<E, N, KEEP>& w, int have, const Scale& c, float k, float ref,
                                            bool far) {
  if (far) return pieces_sums_of<E, N, true, true, true>(w, have, c, k, ref);
  Sums o = have == N ? pieces_sums_of<E, N, false, false, false>(w, have, c, k, ref)
                     : pieces_sums_of<E, N, false, false, true>(w, have, c, k, ref);
  if (o.u != o.u && o.s == o.s) o = pieces_sums_of<E, N, false, true, true>(w, have, c, k, ref);
  return o;
}
__device__ __forceinline__ Sums one_sum(float z, const Scale& c, float k, float ref, bool far) {
  const float x = far ? exponent1<true>(c, k, ref, z) : exponent1<false>(c, k, ref, z), e = exp2_hw(x);
  return Sums{e, e * fmaxf(x, kFloor)};
}

// Running maximum m of the row's pieces, with the sums of e = 2^(z c1 - K) and of
// e x.  K is the maximum's fl(m c1) (or m c1 itself from 2^9 on).
struct OnlineSums {
  float m = kNegInf;
  double K = 0.0;
  Sums sum{0.0f, 0.0f};
  // the sums so far, relative to another K; of masked words alone they are 0 to any, or
  // a NaN that was among them
  __device__ __forceinline__ Sums at(double to) const {
    const float d = fmaxf((float)(K - to), kFloor), f = exp2_hw(d);
    return m == kNegInf ? sum : Sums{sum.s * f, f * fmaf(d, sum.s, sum.u)};
  }
  // raises the maximum; k, ref and far of the terms to come
  __device__ __forceinline__ void raise(float mx, const Scale& c, float& k, float& ref, bool& far) {
    ref = mx == kNegInf ? 0.0f : mx;
    const double exact = (double)ref * (double)c.one;
    k = (float)exact;
    far = !(fabsf(k) < 512.0f);
    const double to = far ? exact : (double)k;
    sum = at(to);
    m = mx;
    K = to;
  }
  // returns the pieces' own maximum
  template <typename E, int N>
  __device__ __forceinline__ float add(const u32x4 (&from)[N], int have, const Scale& c) {
    const Pieces<E, N, (N * Elem<E>::kPer16 <= 32)> w(from);
    float mx = kNegInf, k, ref;
    bool far;
#pragma unroll
    for (int j = 0; j < N; ++j) mx = fmaxf(mx, w.max(j));
    raise(fmaxf(m, mx), c, k, ref, far);
    const Sums o = pieces_sums(w, have, c, k, ref, far);
    sum.s += o.s;
    sum.u += o.u;
    return mx;
  }
  __device__ __forceinline__ void add_one(float z, const Scale& c) {
    float k, ref;
    bool far;
    raise(fmaxf(m, z), c, k, ref, far);
    const Sums o = one_sum(z, c, k, ref, far);
    sum.s += o.s;
    sum.u += o.u;
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

// How many of a thread's N pieces i0, i0 + T, ... there are.
__device__ __forceinline__ int pieces_there(const RowSpan& at, int i0, int T, int N) {
  return i0 < at.nv ? min(N, (at.nv - 1 - i0) / T + 1) : 0;
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

// Largest value of 16 leading bits that at least n of the 128 maxima (two a lane)
// reach, finite: a masked word is no alternative.
__device__ __forceinline__ float bound_of(float a, float b, int n) {
  const uint32_t ka = order_of(a) >> 16, kb = order_of(b) >> 16;
  uint32_t k = 0u;
#pragma unroll
  for (int i = 15; i >= 0; --i) {
    const uint32_t t = k | (1u << i);
    if (__popcll(__ballot(ka >= t)) + __popcll(__ballot(kb >= t)) >= n) k = t;
  }
  return k <= 0x007Fu ? kLowest : float_of(k << 16);
}

// Words, and parts of a row, that a list holds (fewer than 64 pieces, which may
// leave n = 64 without a bound, have up to 526 words).
constexpr int kList = 640;

struct Best {
  __attribute__((aligned(16))) uint64_t list[kList + 32];
  uint16_t part[kList];  // parts with words from the bound on: step * threads + thread
  int parts, count;
  int need;  // of the counting by digits
  uint32_t prefix;
  int bins[256];
};

__device__ __forceinline__ void best_add(Best& b, float f, int i) {
  const int at = atomicAdd(&b.count, 1);
  if (at < kList) b.list[at] = place_of(f, i);
}

// One piece's words from the bound on, with one addition to the list's length.
template <typename E>
__device__ __forceinline__ void best_piece(Best& b, const u32x4& w, int i0, float bound) {
  constexpr int kPer = Elem<E>::kPer16;
  float f[kPer];
  Elem<E>::unpack(w, f);
  int c = 0;
#pragma unroll
  for (int q = 0; q < kPer; ++q) c += f[q] >= bound ? 1 : 0;
  if (c == 0) return;
  int at = atomicAdd(&b.count, c);
#pragma unroll
  for (int q = 0; q < kPer; ++q)
    if (f[q] >= bound) {
      if (at < kList) b.list[at] = place_of(f[q], i0 + q);
      ++at;
    }
}

// Every finite word of the row, a piece a thread at a time: fn(value, index).
template <typename E, int T, typename F>
__device__ __forceinline__ void each_word(const E* z, int V, const RowSpan& at, F fn) {
  constexpr int kPer = Elem<E>::kPer16;
  for (int i = threadIdx.x; i < at.nv; i += T) {
    float f[kPer];
    Elem<E>::unpack(*reinterpret_cast<const u32x4*>(z + at.head + (size_t)i * kPer), f);
#pragma unroll
    for (int q = 0; q < kPer; ++q)
      if (f[q] >= kLowest) fn(f[q], at.head + i * kPer + q);
  }
  if (at.rest < V) {
    const float f = Elem<E>::get(z + at.rest);
    if (f >= kLowest) fn(f, at.rest);
  }
}

// The list of a row with too many words from the bound on (equal logits, or a
// strong few in one group).  The digits of the n-th largest logit's place among
// the floats, from the highest down, each counted over the row, until the words
// from there on fit the list.  Where they do not even when the logit is known,
// there are more words of that one value: those above it are taken, and of its
// own the first ones by index, in steps of the row that end with enough.  (20
// alternatives where 3 words of 32000 are left above a mask of bf16's lowest value:
// 4 rows 34 us, ordinary ones 11; 4096 rows 363 and 51.)
template <typename E, int T>
__device__ void best_by_digits(const E* z, int V, const RowSpan& at, int n, Best& b) {
  constexpr int kLast = sizeof(E) == 2 ? 16 : 0;  // digits below it follow from those above
  if (threadIdx.x == 0) {
    b.prefix = 0u;
    b.need = n;
  }
  int shift = 32;
  do {
    shift -= 8;
    for (int i = threadIdx.x; i < 256; i += T) b.bins[i] = 0;
    __syncthreads();
    const uint32_t prefix = b.prefix;
    const int need = b.need;
    int digit = 0, run = 0;  // equal digits of a thread are counted at once: rows that come here hold many
    each_word<E, T>(z, V, at, [&](float f, int) {
      const uint32_t p = order_of(f);
      if (shift < 24 && (p ^ prefix) >> (shift + 8) != 0u) return;
      const int d = (int)(p >> shift) & 255;
      if (d != digit) {
        if (run != 0) atomicAdd(&b.bins[digit], run);
        digit = d;
        run = 0;
      }
      ++run;
    });
    if (run != 0) atomicAdd(&b.bins[digit], run);
    __syncthreads();
    if (threadIdx.x < 64) {  // four digits a lane, the highest first: the one that holds the need-th word
      const int top = 255 - 4 * (int)threadIdx.x;
      int c[4], sum = 0;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        c[q] = b.bins[top - q];
        sum += c[q];
      }
      int upto = sum;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int v = __shfl_up(upto, o, 64);
        if ((int)threadIdx.x >= o) upto += v;
      }
      int above = upto - sum;
      if (above < need && upto >= need) {
        int d = top, words = c[0];
#pragma unroll
        for (int q = 1; q < 4; ++q)
          if (d == top - q + 1 && above + words < need) {
            above += words;
            words = c[q];
            --d;
          }
        b.prefix = prefix | (uint32_t)d << shift;
        b.need = need - above;
        b.count = n - need + above + words;  // words from the new prefix on
      }
    }
    __syncthreads();
  } while (b.count > kList && shift > kLast);
  const uint32_t from = b.prefix >> shift;
  const int need = b.need;
  const bool ties = b.count > kList;
  __syncthreads();
  if (threadIdx.x == 0) b.count = 0;
  __syncthreads();
  each_word<E, T>(z, V, at, [&](float f, int i) {
    const uint32_t p = order_of(f) >> shift;
    if (ties ? p > from : p >= from) best_add(b, f, i);
  });
  constexpr int S = T < 256 ? T : 256;
  for (int i0 = 0, found = 0; ties && found < need && i0 < V; i0 += S) {
    const int i = i0 + (int)threadIdx.x;
    bool hit = false;
    if ((int)threadIdx.x < S && i < V) {
      const float f = Elem<E>::get(z + i);
      hit = f >= kLowest && order_of(f) >> shift == from;
      if (hit) best_add(b, f, i);
    }
    found += __syncthreads_count(hit);
  }
  __syncthreads();
}

// ------------------------------------------------------------- forward ----

// The leading half of a float, an order that comparisons of floats imply.
__device__ __forceinline__ uint16_t half_of(float f) { return (uint16_t)(__float_as_uint(f) >> 16); }
__device__ __forceinline__ bool half_reaches(uint16_t h, float bound) {
  return bf16_to_f32(h) >= __uint_as_float(__float_as_uint(bound) & 0xFFFF0000u);
}

// Steps of a row read in pieces whose maxima are kept apart; the last one's stands
// for all that follow.
template <int T>
constexpr int kept_steps() { return T <= 256 ? 4 : 16; }

// A row a work-group, as in the losses: N > 0 pieces a thread in registers, N <
// 0: -N pieces a thread at a time.  The maxima of a row's parts (a thread's pieces,
// or its steps) stay in LDS, so that the words from the bound on are looked for in
// few of them.
//
// Bound by memory and by the exponentials together: a word takes 8.5 issue slots of
// a lane, four of them the exponential's, which is 28 us of 4096 rows of 32000 words
// on all CUs, while their 262 MB take 43 us at 6.1 TB/s; 50.8 us in all.  4096 rows
// of 131072: 182 us, 5.9 TB/s; with 20 alternatives 188, with 64 198.
template <typename E, int T, int N>
__global__ __launch_bounds__(T) void k_scores(ScoreArgs a) {
  constexpr int W = T / 64, P = N < 0 ? -N : N;
  constexpr int Q = N < 0 ? P : 1;  // pieces of a part
  __shared__ float maxima[W][64];
  __shared__ float sums[W], means[W];
  __shared__ float bound_sh;
  __shared__ double ln_sh;
  __shared__ Best best;
  constexpr int kSteps = kept_steps<T>();
  __shared__ uint16_t part_max[N < 0 ? kSteps : N][T];
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
      if (a.stats != nullptr) {  // none: with these a gradient of other tokens is 0 / 0
        a.stats[3 * t] = -kNegInf;
        a.stats[3 * t + 1] = 0.0f;
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
  float own, even, odd = kNegInf;  // this thread's largest, those of its even and its odd pieces
  if constexpr (N > 0) {
    r.load(z, a.V, at);
    even = r.last;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      float f[Elem<E>::kPer16], mx = kNegInf;
      Elem<E>::unpack(anew<0>(r.w[j]), f);
#pragma unroll
      for (int q = 0; q < Elem<E>::kPer16; ++q) mx = fmaxf(mx, f[q]);
      if (a.n > 0) part_max[j][threadIdx.x] = half_of(mx);
      (j % 2 != 0 ? odd : even) = fmaxf(j % 2 != 0 ? odd : even, mx);
    }
    own = fmaxf(even, odd);
  } else {
    float rest = kNegInf;  // of the last steps together
    int step = 0;
    for (int i0 = threadIdx.x; i0 < at.nv; i0 += P * T, ++step) {
      u32x4 w[P];
      load_pieces<E>(z, at, i0, T, w);
      const float mx = o.template add<E>(w, pieces_there(at, i0, T, P), a.c);
      if (step >= kSteps - 1) rest = fmaxf(rest, mx);
      part_max[min(step, kSteps - 1)][threadIdx.x] = half_of(step >= kSteps - 1 ? rest : mx);
    }
    if (at.rest < a.V) o.add_one(Elem<E>::get(z + at.rest), a.c);
    own = o.m;
  }
  // the two groups of this lane: its words in the even and in the odd waves (with
  // one wave, in its even and odd pieces)
  static_assert(N > 0 || T > 64, "one wave holds its row");
  if (T > 64) {
    maxima[wave][lane] = own;
    __syncthreads();
    even = maxima[0][lane];
    odd = maxima[W > 1 ? 1 : 0][lane];
#pragma unroll
    for (int w = 2; w < W; w += 2) {
      even = fmaxf(even, maxima[w][lane]);
      odd = fmaxf(odd, maxima[w + 1][lane]);
    }
  }
  const float m = wave_max(fmaxf(even, odd));
  if (a.n > 0 && wave == 0) {
    const float bound = bound_of(even, odd, a.n);
    if (lane == 0) {
      bound_sh = bound;
      best.count = best.parts = 0;
    }
  }
  const RowExp x(m, a.c);
  Sums sum;
  if constexpr (N > 0) {
    sum = pieces_sums(Pieces<E, N, false>(r.w), pieces_there(at, threadIdx.x, T, N), a.c, x.k, m, x.far);
    const Sums l = one_sum(r.last, a.c, x.k, m, x.far);
    sum.s += l.s;
    sum.u += l.u;
  } else {
    sum = o.at(x.far ? (double)m * (double)a.c.one : (double)x.k);
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
  const bool real = s == s && fabsf(m) < __builtin_inff();  // else no distribution: a NaN, +inf, nothing but -inf
  if (a.n > 0 && real) {
    if (T == 64) __syncthreads();  // the bound (with more waves, before the sums)
    const float bound = bound_sh;
    if (own >= bound) {  // which of this thread's parts
      uint32_t mask = 0u;
      const int parts = N > 0 ? N : min((at.nv - 1 - (int)threadIdx.x) / (P * T) + 1, kSteps);
      if (N > 0 || (int)threadIdx.x < at.nv)
        for (int j = 0; j < parts; ++j) mask |= half_reaches(part_max[j][threadIdx.x], bound) ? 1u << j : 0u;
      if (mask != 0u) {
        int to = atomicAdd(&best.parts, (int)__popc(mask));
        for (; mask != 0u; mask &= mask - 1u, ++to)
          if (to < kList) best.part[to] = (uint16_t)((__ffs(mask) - 1) * T + (int)threadIdx.x);
      }
      if (at.rest < a.V) {
        const float f = N > 0 ? r.last : Elem<E>::get(z + at.rest);
        if (f >= bound) best_add(best, f, at.rest);
      }
    }
  }
  if (wave == 0) {  // fp64, once: one wave
    float mean = u / s;
    {
      const double lo = a.c.c - (double)a.c.one;
      const float off = (float)(lo / (double)a.c.one * ((double)mean + (x.far ? 0.0 : (double)x.k)));
      s = fmaf(s, (float)kLn2 * off, s);
      mean += off;
    }
    if (!real) s = mean = __builtin_nanf("");
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
    // the parts' pieces again, dealt out anew: a piece a thread
    const int units = min(best.parts, kList) * Q;
    const float bound = bound_sh;
    for (int i = threadIdx.x; i < units; i += T) {
      const int part = best.part[i / Q], step = part / T;
      int piece = step * Q * T + part % T + i % Q * T;
      const int last = N < 0 && step == kSteps - 1 ? at.nv : min(at.nv, piece + 1);
      for (; piece < last; piece += Q * T)
        best_piece<E>(best, *reinterpret_cast<const u32x4*>(z + at.head + (size_t)piece * Elem<E>::kPer16),
                      at.head + piece * Elem<E>::kPer16, bound);
    }
    __syncthreads();
    if (best.parts > kList || best.count > kList) best_by_digits<E, T>(z, a.V, at, a.n, best);
  }
  // a word's rank is the number of those before it; four threads count it
  const int count = real ? best.count : 0;
  const double ln_sum = ln_sh;
  for (int i = threadIdx.x; i < 4 * count; i += T) {
    const uint64_t p = best.list[i >> 2];
    int rank = 0;
    for (int j = i & 3; j < count; j += 32) {
#pragma unroll
      for (int q = 0; q < 32; q += 4) rank += best.list[j + q] > p && j + q < count ? 1 : 0;
    }
    rank += __builtin_amdgcn_mov_dpp(rank, 0xB1, 0xF, 0xF, true);  // lanes 1, 0, 3, 2
    rank += __builtin_amdgcn_mov_dpp(rank, 0x4E, 0xF, 0xF, true);  // lanes 2, 3, 0, 1
    if ((i & 3) == 0 && rank < a.n) {
      a.ids[t * a.n + rank] = (int)~(uint32_t)p;
      a.top[t * a.n + rank] = (float)(((double)float_of((uint32_t)(p >> 32)) - (double)m) * (double)a.tau - ln_sum);
    }
  }
  for (int i = count + (int)threadIdx.x; i < a.n; i += T) {
    a.ids[t * a.n + i] = -1;
    a.top[t * a.n + i] = real ? kNegInf : __builtin_nanf("");
  }
}

// ------------------------------------------------------------ gradient ----
//
// d_v = e_v (A + B (x_v - mean)) with A = -tau G / s, G = sum_j g_j over the
// counted tokens, and B = -tau gH ln 2 / s; a token's own element gets tau
// sum g_j over its entries on top.
struct GradOf {
  float A, B, mean, tau;
};
template <typename E, bool FAR, bool ENT>
__device__ __forceinline__ float grad_value(float z, const RowExp& x, const GradOf& g) {
  if (!ENT) return (FAR ? x.far_e(z) : x.template near_g<E>(z)) * g.A;
  // (one part of c for bf16, as in near_g)
  const float xv = FAR ? x.c.times(z - x.m)
                       : (sizeof(E) == 2 ? fmaf(z, x.c.one, -x.k) : fmaf(z, x.c.lo, fmaf(z, x.c.hi, -x.k)));
  return exp2_hw(xv) * fmaf(fmaxf(xv, kFloor) - g.mean, g.B, g.A);
}
// The tokens of a work-group's columns, found by the piece that each lies in: lists
// of entries by the piece's number, so that a thread puts a token's element in
// place in the piece that it stores.  (Stored over the pieces afterwards, the
// elements of 33 tokens a row cost 4096 x 32000 bf16 99 us in place of 79 for one.)
constexpr uint32_t kNoEntry = ~0u;
template <int S>
struct Hits {
  __attribute__((aligned(16))) uint32_t head[S];
  struct __attribute__((aligned(16))) Entry {
    int col;  // of the work-group's columns, -1: none
    float g;
    uint32_t next;
  } of[kMaxScores];
};
// A column's piece; a single element's number is that past the pieces of its thread.
template <typename E>
__device__ __forceinline__ int piece_of(const RowSpan& at, int col) {
  constexpr int kPer = Elem<E>::kPer16;
  if (col < at.head) return at.nv + col;
  const int i = (col - at.head) / kPer;
  return i < at.nv ? i : col - at.nv * (kPer - 1);
}
// By all threads; a lane of the first wave has an entry, those of one column become
// one, which takes the sum of their g in their order.
template <typename E, int T, int S>
__device__ __forceinline__ void hits_fill(Hits<S>& hits, const RowSpan& at, int col, float g) {
  const int lane = threadIdx.x & 63;
  for (int i = threadIdx.x; i < S / 4; i += T)
    reinterpret_cast<u32x4*>(hits.head)[i] = u32x4{kNoEntry, kNoEntry, kNoEntry, kNoEntry};
  __syncthreads();
  if (threadIdx.x < 64) {
    uint32_t next = kNoEntry;
    if (col >= 0) next = atomicExch(&hits.head[piece_of<E>(at, col) & (S - 1)], (uint32_t)lane);
    uint64_t todo = __ballot(next != kNoEntry);  // of columns that may be there twice
    while (todo != 0u) {
      const int c = __builtin_amdgcn_readlane(col, __ffsll((long long)todo) - 1);
      const uint64_t same = __ballot(col == c);
      float sum = 0.0f;
      for (uint64_t left = same; left != 0u; left &= left - 1u)
        sum += __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(g), __ffsll((long long)left) - 1));
      if (col == c) {
        g = sum;
        if (lane != __ffsll((long long)same) - 1) col = -1;
      }
      todo &= ~same;
    }
    hits.of[lane] = {col, g, next};
  }
  __syncthreads();
}

// d of N elements z of the columns from col on; h: the list of their piece.
template <typename E, bool FAR, bool ENT, int N, int S>
__device__ __forceinline__ void grad_values(const float (&z)[N], float (&d)[N], int col, uint32_t h, const Hits<S>& hits,
                                            const RowExp& x, const GradOf& g) {
#pragma unroll
  for (int q = 0; q < N; ++q) d[q] = grad_value<E, FAR, ENT>(z[q], x, g);
  while (h != kNoEntry) {
    const auto e = hits.of[h];
    const int at = e.col - col;
    if ((uint32_t)at < (uint32_t)N) {
      float own = z[0];
#pragma unroll
      for (int q = 1; q < N; ++q) own = q == at ? z[q] : own;
      const float v = fmaf(e.g, g.tau, grad_value<float, FAR, ENT>(own, x, g));
#pragma unroll
      for (int q = 0; q < N; ++q) d[q] = q == at ? v : d[q];
    }
    h = e.next;
  }
}

// One row from memory to memory, w being a thread's first pieces; where out is z, a
// thread overwrites only what it has read.
template <typename E, int T, int kBatch, bool FAR, bool ENT, bool STREAM, int S>
__device__ __forceinline__ void score_row(const E* z, E* out, int V, const RowSpan& at, const Hits<S>& hits,
                                          const RowExp& x, const GradOf& g, u32x4 (&w)[kBatch]) {
  constexpr int kPer = Elem<E>::kPer16;
  for (int i = threadIdx.x; i < at.nv; i += kBatch * T) {
    uint32_t h[kBatch];
    if (i >= T) load_pieces<E>(z, at, i, T, w);
#pragma unroll
    for (int j = 0; j < kBatch; ++j) h[j] = hits.head[(i + j * T) & (S - 1)];
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
      if (i + j * T < at.nv) {
        const int col = at.head + (i + j * T) * kPer;
        float f[kPer], d[kPer];
        Elem<E>::unpack(w[j], f);
        grad_values<E, FAR, ENT>(f, d, col, h[j], hits, x, g);
        put16<STREAM>(out + col, Elem<E>::pack(d));
      }
  }
  if (at.rest < V) {
    const float f[1] = {Elem<E>::get(z + at.rest)};
    float d[1];
    grad_values<E, FAR, ENT>(f, d, at.rest, hits.head[piece_of<E>(at, at.rest) & (S - 1)], hits, x, g);
    Elem<E>::put(out + at.rest, d[0]);
  }
}

// The rows go from the last to the first, which the forward ended with; a
// work-group has a span of columns, and the tokens that lie there.  Bound by
// memory: 4096 rows of 32000 bf16, three tenths uncounted, 33 tokens and an entropy
// term: 74 us (69 at the least), 446 MB at 6.0 TB/s.
template <typename E, int T>
__global__ __launch_bounds__(T) void k_scores_grad(ScoreArgs a) {
  constexpr int B = T == 1024 ? 8 : 4;
  constexpr int S = T == 64 ? 256 : 1024;
  __shared__ Hits<S> hits;
  const int lane = threadIdx.x & 63;
  const int64_t t = a.first + gridDim.x - 1 - blockIdx.x;
  const int c0 = (int)blockIdx.y * a.span;
  const bool last = blockIdx.y == gridDim.y - 1;
  const int V = last ? a.V - c0 : a.span, end = last ? (int)a.ldd - c0 : a.span;
  const int token = lane < a.m ? a.tokens[t * a.m + lane] : -1;
  const bool counted = is_counted(token, a.V);
  const float g = counted ? a.dlogp[t * a.m + lane] : 0.0f;
  const bool live = a.m == 0 || __ballot(counted) != 0u;
  const float gh = live && a.dentropy != nullptr ? a.dentropy[t] : 0.0f;
  E* out = reinterpret_cast<E*>(a.dlogits) + t * a.ldd + c0;
  if (gh == 0.0f && __ballot(g != 0.0f) == 0u) {
    row_zero<E, T>(out, end, a.stream);
    return;
  }
  const E* z = reinterpret_cast<const E*>(a.logits) + t * a.ld + c0;
  const RowSpan at(z, V);
  u32x4 w[B];
  load_pieces<E>(z, at, threadIdx.x, T, w);  // in flight meanwhile
  const float G = wave_sum(g);
  const RowExp x(a.stats[3 * t], a.c);
  const float s = a.stats[3 * t + 1];
  const GradOf go{-G * a.tau / s, -gh * a.tau * (float)kLn2 / s, a.stats[3 * t + 2], a.tau};
  hits_fill<E, T>(hits, at, counted && is_counted(token - c0, V) ? token - c0 : -1, g);
  auto row = [&](auto far, auto ent, auto stream) {
    score_row<E, T, B, decltype(far)::value, decltype(ent)::value, decltype(stream)::value>(z, out, V, at, hits, x, go, w);
  };
  const std::true_type yes{};
  const std::false_type no{};
  if (gh != 0.0f)
    x.far ? (a.stream ? row(yes, yes, yes) : row(yes, yes, no)) : (a.stream ? row(no, yes, yes) : row(no, yes, no));
  else
    x.far ? (a.stream ? row(yes, no, yes) : row(yes, no, no)) : (a.stream ? row(no, no, yes) : row(no, no, no));
  for (int i = V + (int)threadIdx.x; i < end; i += T) Elem<E>::put(out + i, 0.0f);
}

// ---------------------------------------------------------- launchers ----

static dim3 row_grid(const ScoreArgs& a) { return dim3((unsigned)std::min(a.T - a.first, kRowsALaunch)); }

template <typename E, int T, int N>
static void scores_kernel(const ScoreArgs& a, hipStream_t st) {
  ScoreArgs b = a;
  for (; b.first < b.T; b.first += kRowsALaunch)
    QLORA_LAUNCH("scores", st, (k_scores<E, T, N>), row_grid(b), dim3(T), 0, st, b);
}

// Threads a row and what each holds, by the row's number of 16-byte pieces.  One
// wave takes a short row without a barrier.  Up to one row per CU a row's own
// latency counts: the most threads, with eight pieces each in flight.  With more
// rows, 256 or 512 threads and four pieces: several rows a CU, one of which
// computes while others load.  Measured with 20 alternatives (us):
//   1 row, bf16, V = 131072:     1024 x 8 in pieces 13.3, x 4 14.3, x 12 27, 512 x 4
//                                15.3, 1024 x 16 in registers 27.8;
//   200 rows, bf16, V = 32000:   1024 x 4 in registers 9.5, 256 x 4 in pieces 11.4;
//   200 rows, bf16, V = 131072:  1024 x 8 in pieces 17.2, 512 x 4 18.9;
//   400 rows, bf16, V = 32000:   1024 x 4 in registers 13.3, 256 x 4 in pieces 13.2;
//   2048 rows, bf16, V = 32000:  43.7 and 33.3;
//   4096 rows, bf16, V = 64000:  512 x 4 in pieces 97, without alternatives 92, 256 x 4
//                                100; V = 131072: 188 and 182, 256 x 4 192.
template <typename E>
static hipError_t launch_scores_of(const ScoreArgs& a, hipStream_t st) {
  const int64_t pieces = ((int64_t)a.V + Elem<E>::kPer16 - 1) / Elem<E>::kPer16;
  if (pieces <= 64 * 4)
    scores_kernel<E, 64, 4>(a, st);
  else if (a.T <= 256 && pieces > 1024)
    pieces <= 1024 * 4 ? scores_kernel<E, 1024, 4>(a, st) : scores_kernel<E, 1024, -8>(a, st);
  else if (pieces <= 4096)
    scores_kernel<E, 256, -4>(a, st);
  else
    scores_kernel<E, 512, -4>(a, st);
  return hipGetLastError();
}

// span: columns of a work-group.
template <typename E, int T>
static void scores_grad_kernel(const ScoreArgs& a, int span, hipStream_t st) {
  ScoreArgs b = a;  // the last rows first, which the forward ended with
  while ((a.V - 1) / span > 65534) span *= 2;  // a grid's second dimension
  b.span = span;
  const unsigned spans = (unsigned)((a.V - 1) / span + 1);
  for (b.first = (a.T - 1) / kRowsALaunch * kRowsALaunch; b.first >= 0; b.first -= kRowsALaunch) {
    const dim3 rows = row_grid(b);
    QLORA_LAUNCH("scores_grad", st, (k_scores_grad<E, T>), dim3(rows.x, spans), dim3(T), 0, st, b);
  }
}

// A gradient past the cache's half is stored in whole rows, where there are two a
// CU: 2048 x 131072 bf16 197 us, in spans 204.  Any other in spans of four pieces a
// thread: 4 x 131072 bf16 3.9 us, in whole rows 11.8; 96 x 32000 fp32 5.9 and 7.2; 300 x
// 50021 fp32 20.3 and 22.5; 2048 x 32000 bf16 41.0 and 41.5 (two pieces a thread 3.5, 5.8,
// 21.8, 40.8; eight 4.6, 5.8, 20.8, 41.4).
template <typename E>
static hipError_t launch_scores_grad_of(const ScoreArgs& a, hipStream_t st) {
  const int64_t pieces = ((int64_t)a.V + Elem<E>::kPer16 - 1) / Elem<E>::kPer16;
  if (pieces <= 64 * 4)
    scores_grad_kernel<E, 64>(a, a.V, st);
  else if (!a.stream || a.T < 512)
    scores_grad_kernel<E, 256>(a, 256 * 4 * Elem<E>::kPer16, st);
  else if (pieces <= 4096)
    scores_grad_kernel<E, 512>(a, a.V, st);
  else
    scores_grad_kernel<E, 1024>(a, a.V, st);
  return hipGetLastError();
}

hipError_t launch_scores(const void* logits, int f32, int64_t T, int V, int64_t ld, const int32_t* tokens, int m, int n,
                         float tau, float* logp, float* entropy, int32_t* ids, float* top, float* stats,
                         hipStream_t st) {
  const ScoreArgs a{logits, 0, T, ld, 0, V, tokens, m, n, V, tau, exp2_scale(tau), logp, entropy, ids, top, stats,
                    nullptr, nullptr, nullptr, false};
  return f32 ? launch_scores_of<float>(a, st) : launch_scores_of<uint16_t>(a, st);
}

hipError_t launch_scores_grad(const void* logits, int f32, int64_t T, int V, int64_t ld, const int32_t* tokens, int m,
                              float tau, const float* stats, const float* dlogp, const float* dentropy, void* dlogits,
                              int64_t ldd, hipStream_t st) {
  const ScoreArgs a{logits, 0, T, ld, ldd, V, tokens, m, 0, V, tau, exp2_scale(tau), nullptr, nullptr, nullptr, nullptr,
                    const_cast<float*>(stats), dlogp, dentropy, dlogits, past_cache(T, ldd, f32)};
  return f32 ? launch_scores_grad_of<float>(a, st) : launch_scores_grad_of<uint16_t>(a, st);
}

}  // namespace qlora
