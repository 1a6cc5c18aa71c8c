// loss.hip -- from a head's logits to the gradient its backward starts from:
// the log-probability of each token's label, the preference loss of chosen
// and rejected sequences, the clipped policy loss with a KL term, and the
// gradients of all of them in the logits.
//
// One row of logits z (V of them) gives, with tau the inverse temperature,
//
//   t_v = tau (z_v - max z),  S = sum_v exp t_v,  logp = t_y - ln S,
//   d logp / d z_v = tau ([v = y] - exp(t_v) / S).
//
// Exponentials are e_v = 2^(z_v c - k) with c = tau log2 e and k = fl(c max z):
// k's rounding is the same factor in every e_v and in their sum s, so that p_v =
// e_v / s is free of it and only ln S takes it back, ln S = ln s + ln 2 (k - c
// max z), in fp64.  c is held in two parts, hi of 16 bits and lo of 24, and the
// exponent is fma(z, lo, fma(z, hi, -k)).  In one part c's rounding (up to 2^-24
// of it) puts ln S off by ln 2 of it times E_p|x|, some 4e-8, the same way in
// all of a sequence's tokens (4096 of them: 1.5e-4 in its sum, where fp32
// log-probabilities leave 2e-5); the two roundings here fall either way.  From
// |k| = 2^9 on (logits of 355 at tau = 1; and up to where k is infinite, as in a
// row of the type's lowest value) the difference d = z - max z is taken first,
// fma(d, hi, d lo).  The pieces of a bf16 gradient take c in one part, fma(z, fl(c),
// -k): below 2^9 that moves e_v by less than 2^-16 of it, and they are rounded to
// 2^-9 (4096 x 131072, policy loss and gradient: 393 us with one part everywhere,
// 410 with two; fp32 gradients take two).  Sums are fp32 and go through a fixed
// tree, so results do not depend on the schedule.
//
// A row is a work-group's, read 16 bytes a lane.  Where it fits the
// work-group's registers it is read once: all of its loads are in flight
// together, then the maximum, the sum and the gradient follow from the
// registers.  Longer rows are read in pieces with a running maximum, and again
// for the gradient.
#include <algorithm>

#include "common.hpp"
#include "launch.hpp"
#include "rows.hpp"

namespace qlora {

// One 16-byte piece of the gradient: e_v kappa with kappa = -g tau / s.  (The
// label's g tau (1 - p) is stored over it at the row's end: a test for it in
// every piece would keep the loads of the next ones back.)
template <typename E, bool FAR>
__device__ __forceinline__ u32x4 grad_piece(const u32x4& w, const RowExp& x, float kappa) {
  constexpr int kPer = Elem<E>::kPer16;
  float f[kPer];
  Elem<E>::unpack(w, f);
#pragma unroll
  for (int q = 0; q < kPer; ++q) f[q] = (FAR ? x.far_e(f[q]) : x.template near_g<E>(f[q])) * kappa;
  return Elem<E>::pack(f);
}

// What the pieces leave of a row: the single elements, the label's (zy its
// logit; by the thread that stored its piece) and zeros in columns V..cols-1.
template <typename E, int T>
__device__ __forceinline__ void row_end(float last, float zy, E* out, int V, int cols, const RowSpan& at, int label,
                                        const RowExp& x, float kappa, float gt) {
  const int piece = (label - at.head) / Elem<E>::kPer16;
  if (at.rest < V) {
    const float v = x.e(last) * kappa;
    Elem<E>::put(out + at.rest, label == at.rest ? v + gt : v);
  }
  if (label >= at.head && piece < at.nv && piece % T == (int)threadIdx.x)
    Elem<E>::put(out + label, x.e(zy) * kappa + gt);
  for (int i = V + threadIdx.x; i < cols; i += T) Elem<E>::put(out + i, 0.0f);
}

// z -> gradient over one row read from memory.  Where out is z, a thread
// overwrites only what it has read.
template <typename E, int T, int kBatch, bool FAR, bool STREAM>
__device__ __forceinline__ void row_grad_of(const E* z, E* out, const RowSpan& at, const RowExp& x, float kappa) {
  constexpr int kPer = Elem<E>::kPer16;
  int i = threadIdx.x;
  for (; i + (kBatch - 1) * T < at.nv; i += kBatch * T) {
    u32x4 w[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) w[j] = *reinterpret_cast<const u32x4*>(z + at.head + (i + j * T) * kPer);
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
      put16<STREAM>(out + at.head + (i + j * T) * kPer, grad_piece<E, FAR>(w[j], x, kappa));
  }
  u32x4 w[kBatch];
#pragma unroll
  for (int j = 0; j < kBatch; ++j)
    if (i + j * T < at.nv) w[j] = *reinterpret_cast<const u32x4*>(z + at.head + (i + j * T) * kPer);
#pragma unroll
  for (int j = 0; j < kBatch; ++j)
    if (i + j * T < at.nv) put16<STREAM>(out + at.head + (i + j * T) * kPer, grad_piece<E, FAR>(w[j], x, kappa));
}
template <typename E, int T, int B>
__device__ __forceinline__ void row_grad(const E* z, float zy, E* out, int V, int cols, int label, const RowExp& x,
                                         float s, float gt, bool stream) {
  const RowSpan at(z, V);
  const float kappa = -gt / s;
  float last = kNegInf;
  if (at.rest < V) last = Elem<E>::get(z + at.rest);
  if (stream)
    x.far ? row_grad_of<E, T, B, true, true>(z, out, at, x, kappa) : row_grad_of<E, T, B, false, true>(z, out, at, x, kappa);
  else
    x.far ? row_grad_of<E, T, B, true, false>(z, out, at, x, kappa)
          : row_grad_of<E, T, B, false, false>(z, out, at, x, kappa);
  row_end<E, T>(last, zy, out, V, cols, at, label, x, kappa, gt);
}

// The same from the registers.
template <typename E, int T, int N, bool FAR, bool STREAM>
__device__ __forceinline__ void regs_grad_of(const RowRegs<E, T, N>& r, E* out, const RowSpan& at, const RowExp& x,
                                             float kappa) {
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const int i = j * T + threadIdx.x;
    if (i < at.nv)
      put16<STREAM>(out + at.head + i * Elem<E>::kPer16,
                    grad_piece<E, FAR>(anew<1 + FAR + 2 * STREAM>(r.w[j]), x, kappa));
  }
}
template <typename E, int T, int N>
__device__ __forceinline__ void regs_grad(const RowRegs<E, T, N>& r, float zy, E* out, int V, int cols,
                                          const RowSpan& at, int label, const RowExp& x, float s, float gt,
                                          bool stream) {
  const float kappa = -gt / s;
  if (stream)
    x.far ? regs_grad_of<E, T, N, true, true>(r, out, at, x, kappa) : regs_grad_of<E, T, N, false, true>(r, out, at, x, kappa);
  else
    x.far ? regs_grad_of<E, T, N, true, false>(r, out, at, x, kappa)
          : regs_grad_of<E, T, N, false, false>(r, out, at, x, kappa);
  row_end<E, T>(r.last, zy, out, V, cols, at, label, x, kappa, gt);
}

// ------------------------------------------------------- policy loss -----
//
// Per counted token, with ratio r = exp(lp - old), advantage A, clip range
// [lo, hi] = [1 - clip_low, 1 + clip_high] and d = ref - lp:
//
//   loss = -min(r A, clip(r) A) + kl_coef (exp(d) - d - 1)
//   d loss / d lp = -r A (0 where the clip holds) - kl_coef (exp(d) - 1)
//
// lp comes in fp64: the differences with old and ref are small against it.
struct PolicyArgs {
  const float* adv;
  const float* old_logp;  // nullptr: the policy itself (r = 1)
  const float* ref_logp;  // nullptr: no KL term
  const float* weight;    // nullptr: 1
  float lo, hi, kl_coef;
  float* loss;
  float* kl;
};

// exp(d) - 1 - d: below 1/2 in size its series (to d^10 / 10!, 1e-10 of it),
// since exp(d) - 1 and d would cancel; infinite for d = inf.
__device__ __forceinline__ float exp_less_two_terms(float d, float expm1_d) {
  if (!(fabsf(d) < 0.5f)) return d == __builtin_inff() ? d : expm1_d - d;
  float p = 1.0f / 3628800.0f;
  p = fmaf(p, d, 1.0f / 362880.0f);
  p = fmaf(p, d, 1.0f / 40320.0f);
  p = fmaf(p, d, 1.0f / 5040.0f);
  p = fmaf(p, d, 1.0f / 720.0f);
  p = fmaf(p, d, 1.0f / 120.0f);
  p = fmaf(p, d, 1.0f / 24.0f);
  p = fmaf(p, d, 1.0f / 6.0f);
  p = fmaf(p, d, 0.5f);
  return p * d * d;
}

__device__ __forceinline__ float policy_token(const PolicyArgs& a, int64_t t, double lp, float& loss, float& kl) {
  const float A = a.adv[t];
  const float r = a.old_logp != nullptr ? expf((float)(lp - (double)a.old_logp[t])) : (lp == lp ? 1.0f : (float)lp);
  const float rc = fminf(fmaxf(r, a.lo), a.hi);
  const float x = A == 0.0f && r == r ? 0.0f : r * A, y = rc * A;  // (r may be infinite: 0 times it is still 0)
  const bool clipped = y < x;  // the clipped branch is the smaller one, and flat
  loss = -(clipped ? y : x);
  float g = clipped ? 0.0f : -x;
  kl = 0.0f;
  if (a.ref_logp != nullptr) {
    const float d = (float)((double)a.ref_logp[t] - lp);
    const float e = expm1f(d);
    kl = exp_less_two_terms(d, e);
    if (a.kl_coef != 0.0f) {  // a kl that is only watched may be infinite
      loss = fmaf(a.kl_coef, kl, loss);
      g = fmaf(-a.kl_coef, e, g);
    }
  }
  if (a.weight == nullptr) return g;
  const float w = a.weight[t];
  return w == 0.0f ? 0.0f : g * w;  // a token taken out has no gradient, not a NaN either
}

// ------------------------------------------------------- row kernels -----

struct RowArgs {
  const void* logits;
  int64_t first, T, ld, ldd;  // rows first to T - 1
  int V;
  const int32_t* labels;
  float tau;
  Scale c;
  float* logp;
  float* stats;  // (max z, sum of e) per row
  void* dlogits;
  bool stream;  // dlogits past the last-level cache
};

// Log-probabilities, and with POLICY the policy loss and its gradient.  N > 0:
// the row fits N pieces a thread; N < 0: -N pieces a thread at a time.
//
// Bound by memory: the counted rows are read once and the gradient written
// once.  T = 4093, V = 50021, fp32, a tenth uncounted: 119 us, 737 MB at 6.2
// TB/s; T = 4096, V = 32000, bf16, a fifth uncounted, with the gradient: 88
// us, 472 MB at 5.4 TB/s; V = 131071, a tenth uncounted: 409 us, 2.04 GB at
// 5.0 TB/s.
template <typename E, int T, int N, bool POLICY>
__global__ __launch_bounds__(T) void k_rows(RowArgs a, PolicyArgs pa) {
  __shared__ float maxima[T / 64];
  __shared__ float sums[T / 64];
  __shared__ float gsh;
  const E* logits = reinterpret_cast<const E*>(a.logits);
  const int64_t t = a.first + blockIdx.x;
  const int label = a.labels[t];
  E* out = POLICY && a.dlogits != nullptr ? reinterpret_cast<E*>(a.dlogits) + t * a.ldd : nullptr;
  if (!is_counted(label, a.V)) {
    if (out != nullptr) row_zero<E, T>(out, (int)a.ldd, a.stream);
    if (threadIdx.x == 0) {
      a.logp[t] = 0.0f;
      if (a.stats != nullptr) {
        a.stats[2 * t] = 0.0f;
        a.stats[2 * t + 1] = 1.0f;
      }
      if (POLICY) {
        pa.loss[t] = 0.0f;
        if (pa.kl != nullptr) pa.kl[t] = 0.0f;
      }
    }
    return;
  }
  const E* z = logits + t * a.ld;
  // the label's logit is one of the row's: it joins the maximum so that
  // every wave has it in hand before the first barrier, and the row may be
  // written over after that
  const float zy = Elem<E>::get(z + label);
  RowRegs<E, T, N < 0 ? 1 : N> r;
  const RowSpan at(z, a.V);
  Online o;
  float m;
  if constexpr (N > 0) {
    r.load(z, a.V, at);
    m = block_max<T>(fmaxf(r.max(), zy), maxima);
  } else {
    o = row_pieces<E, T, -N>(z, a.V, at, a.c);
    m = block_max<T>(fmaxf(o.m, zy), maxima);
  }
  const RowExp x(m, a.c);
  // (in pieces: a thread without a finite value holds m = -inf and s = 0; a
  // row of nothing but -inf has no distribution and gives NaN)
  float s;
  if constexpr (N > 0)
    s = block_sum<T>(r.sum(x), sums);
  else
    s = block_sum<T>(o.s * x.far_e(o.m), sums) * x.shift();
  float g = 0.0f;
  if (threadIdx.x < 64) {  // fp64, once: one wave
    const double lp = ((double)zy - (double)m) * (double)a.tau - x.ln_sum(s);
    float loss, kl;
    if (POLICY) g = policy_token(pa, t, lp, loss, kl);
    if (threadIdx.x == 0) {
      a.logp[t] = (float)lp;
      if (a.stats != nullptr) {
        a.stats[2 * t] = m;
        a.stats[2 * t + 1] = s;
      }
      if (POLICY) {
        gsh = g;
        pa.loss[t] = loss;
        if (pa.kl != nullptr) pa.kl[t] = kl;
      }
    }
  }
  if (POLICY && out != nullptr) {
    if (T > 64) {
      __syncthreads();
      g = gsh;
    }
    if (g == 0.0f)
      row_zero<E, T>(out, (int)a.ldd, a.stream);
    else if constexpr (N > 0)
      regs_grad<E, T, N>(r, zy, out, a.V, (int)a.ldd, at, label, x, s, g * a.tau, a.stream);
    else
      row_grad<E, T, 4>(z, zy, out, a.V, (int)a.ldd, label, x, s, g * a.tau, a.stream);
  }
}

// The rows go from the last to the first: the forward ended with the last
// ones, and what of them is in the last-level cache is read from there.  Bound
// by memory: T = 4096, V = 131072, bf16, a tenth uncounted: 338 us, 2.04 GB at
// 6.0 TB/s; V = 32000, two fifths uncounted: 64 us, 420 MB at 6.5 TB/s.
template <typename E, int T>
__global__ __launch_bounds__(T) void k_logprob_grad(RowArgs a, const float* __restrict__ dlogp) {
  const int64_t t = a.first + gridDim.x - 1 - blockIdx.x;
  const int label = a.labels[t];
  const float g = dlogp[t];
  E* out = reinterpret_cast<E*>(a.dlogits) + t * a.ldd;
  if (!is_counted(label, a.V) || g == 0.0f) {
    row_zero<E, T>(out, (int)a.ldd, a.stream);
  } else {
    const RowExp x(a.stats[2 * t], a.c);
    const E* z = reinterpret_cast<const E*>(a.logits) + t * a.ld;
    row_grad<E, T, T == 1024 ? 8 : 4>(z, Elem<E>::get(z + label), out, a.V, (int)a.ldd, label, x, a.stats[2 * t + 1],
                                      g * a.tau, a.stream);
  }
}

// --------------------------------------------------- preference loss -----
//
// Sequences 0..P-1 are the chosen ones, P..2P-1 the rejected ones, sequence s
// in tokens cu[s]..cu[s+1]-1.  Over its counted tokens, l_s = sum (logp - ref)
// (divided by their number with `average`), D = l_p - l_{P+p}, h = beta D -
// margin:
//
//   sigmoid  (1-e) softplus(-h) + e softplus(h)
//   hinge    max(0, 1 - h)
//   squared  (D - margin/beta - 1/(2 beta))^2  = ((h - 1/2) / beta)^2
//
// A work-group takes a pair, a half of it a sequence: it sums in fp64
// (thousands of terms, of which a small difference is left) and writes each
// token's d loss / d logp.  Bound by the latency of its few dependent loads
// and barriers (8 pairs of 4096 tokens in all: 6 us, 80 KB).
constexpr int kPrefThreads = 512, kPrefHalf = kPrefThreads / 2;

struct PrefArgs {
  const float* logp;
  const float* ref_logp;
  const int32_t* labels;
  const int32_t* cu;
  const float* weight;
  int64_t T, P;
  int V, kind, average;
  float beta, smoothing, margin;
  float* loss;
  float* reward;
  float* dlogp;
};

__device__ __forceinline__ double softplus(double x) { return fmax(x, 0.0) + log1p(exp(-fabs(x))); }

// Tokens of sequence s, clamped to 0 <= lo <= hi <= T whatever cu holds.
__device__ __forceinline__ void seq_range(const PrefArgs& a, int64_t s, int64_t& lo, int64_t& hi) {
  const int64_t x = a.cu[s], y = a.cu[s + 1];
  lo = x < 0 ? 0 : (x > a.T ? a.T : x);
  hi = y < lo ? lo : (y > a.T ? a.T : y);
}

__global__ __launch_bounds__(kPrefThreads) void k_preference(PrefArgs a) {
  constexpr int W = kPrefHalf / 64;
  __shared__ double sums[2 * W];
  __shared__ int counts[2 * W];
  const int64_t p = blockIdx.x;
  const int k = threadIdx.x / kPrefHalf, i = threadIdx.x % kPrefHalf;  // chosen: 0, rejected: 1
  int64_t lo, hi;
  seq_range(a, k * a.P + p, lo, hi);
  double sum = 0.0;
  int n = 0;
  for (int64_t t0 = lo + i; t0 < hi; t0 += 4 * kPrefHalf) {
    int label[4];
    float lp[4], ref[4];  // in flight
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t t = t0 + j * kPrefHalf;
      label[j] = -1;
      if (t < hi) {
        label[j] = a.labels[t];
        lp[j] = a.logp[t];
        ref[j] = a.ref_logp != nullptr ? a.ref_logp[t] : 0.0f;
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (is_counted(label[j], a.V)) {
        sum += (double)lp[j] - (double)ref[j];
        ++n;
      }
  }
  for (int o = 32; o >= 1; o >>= 1) {
    sum += __shfl_xor(sum, o, 64);
    n += __shfl_xor(n, o, 64);
  }
  if ((threadIdx.x & 63) == 0) {
    sums[threadIdx.x >> 6] = sum;
    counts[threadIdx.x >> 6] = n;
  }
  __syncthreads();
  double l[2], inv[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    l[q] = 0.0;
    int c = 0;
    for (int w = 0; w < W; ++w) {
      l[q] += sums[q * W + w];
      c += counts[q * W + w];
    }
    inv[q] = a.average ? 1.0 / (double)(c > 1 ? c : 1) : 1.0;
    l[q] *= inv[q];
  }
  const double beta = a.beta, e = a.smoothing;
  const double h = beta * (l[0] - l[1]) - a.margin;
  double loss, dh;
  if (a.kind == 0) {
    loss = (1.0 - e) * softplus(-h);
    dh = -(1.0 - e) / (1.0 + exp(h));
    if (e > 0.0) {
      loss += e * softplus(h);
      dh += e / (1.0 + exp(-h));
    }
  } else if (a.kind == 1) {
    loss = fmax(0.0, 1.0 - h);
    dh = h < 1.0 ? -1.0 : 0.0;
    if (h != h) loss = dh = h;
  } else {
    const double x = (h - 0.5) / beta;
    loss = x * x;
    dh = 2.0 * x / beta;
  }
  const double wt = a.weight != nullptr ? (double)a.weight[p] : 1.0;
  const double dl = wt == 0.0 ? 0.0 : dh * beta * wt;  // a pair taken out has no gradient, not a NaN either
  if (threadIdx.x == 0) {
    a.loss[p] = (float)loss;
    if (a.reward != nullptr) {
      a.reward[p] = (float)(beta * l[0]);
      a.reward[a.P + p] = (float)(beta * l[1]);
    }
  }
  if (a.dlogp == nullptr) return;
  const float g = (float)(k == 0 ? dl * inv[0] : -dl * inv[1]);
  for (int64_t t = lo + i; t < hi; t += kPrefHalf) a.dlogp[t] = is_counted(a.labels[t], a.V) ? g : 0.0f;
  // tokens before the first sequence and after the last have no gradient
  if (p == 0 && k == 0)
    for (int64_t t = i; t < lo; t += kPrefHalf) a.dlogp[t] = 0.0f;
  if (p == a.P - 1 && k == 1)
    for (int64_t t = hi + i; t < a.T; t += kPrefHalf) a.dlogp[t] = 0.0f;
}

// ---------------------------------------------------------- launchers ----

static dim3 row_grid(const RowArgs& a) { return dim3((unsigned)std::min(a.T - a.first, kRowsALaunch)); }

template <typename E, int T, int N, bool POLICY>
static void rows_kernel(const char* name, const RowArgs& a, const PolicyArgs& pa, hipStream_t st) {
  RowArgs b = a;
  for (; b.first < b.T; b.first += kRowsALaunch)
    QLORA_LAUNCH(name, st, (k_rows<E, T, N, POLICY>), row_grid(b), dim3(T), 0, st, b, pa);
}

// Threads a row and what each holds, by the row's number of 16-byte pieces.
// One wave takes a short row without a barrier.  Up to one row per CU a row's
// own latency counts: the most threads.  With more rows the row in registers,
// as closely as it fits (pieces that do not exist cost their exponentials all
// the same), as long as a CU holds several rows; beyond that the
// log-probabilities read in pieces, two rows a CU, while the gradient gains
// more from not reading the row again.  Measured on 4096 rows (us,
// log-probabilities / policy loss and gradient):
//   bf16, V = 32000, 4000 pieces:   512 x 8 46 / 94, 256 x 16 48 / 97;
//   bf16, V = 40000, 5000 pieces:   512 x 10 56 / 119, 512 x 16 70 / 120, in
//                                   pieces 1024 x 4 78 / 150;
//   bf16, V = 65536, 8192 pieces:   512 x 16 90 / 196, in pieces 87 / 227;
//   bf16, V = 70000, 8750 pieces:   1024 x 12 - / 255, in pieces 112 / 251;
//   bf16, V = 73000, 9125 pieces:   1024 x 12 - / 266, in pieces 113 / 273;
//   fp32, V = 50000, 12500 pieces:  1024 x 16 - / 312, in pieces 134 / 353;
//   bf16, V = 131072, 16384 pieces: 1024 x 16 220 / 437, 512 x 32 230 / 440,
//                                   in pieces 1024 x 4 176 / 456, 1024 x 8 178
//                                   / -, 512 x 4 183 / 520 (the second reading
//                                   comes from the last-level cache).
template <typename E, bool POLICY>
static hipError_t launch_rows(const char* name, const RowArgs& a, const PolicyArgs& pa, hipStream_t st) {
  const int64_t pieces = ((int64_t)a.V + Elem<E>::kPer16 - 1) / Elem<E>::kPer16;
  if (pieces <= 64 * 4)
    rows_kernel<E, 64, 4, POLICY>(name, a, pa, st);
  else if (a.T <= 256 && pieces > 1024 && pieces <= 1024 * 8)
    pieces <= 1024 * 4 ? rows_kernel<E, 1024, 4, POLICY>(name, a, pa, st)
                       : rows_kernel<E, 1024, 8, POLICY>(name, a, pa, st);
  else if (pieces <= 256 * 4)
    rows_kernel<E, 256, 4, POLICY>(name, a, pa, st);
  else if (pieces <= 256 * 7)
    rows_kernel<E, 256, 7, POLICY>(name, a, pa, st);
  else if (pieces <= 256 * 10)
    rows_kernel<E, 256, 10, POLICY>(name, a, pa, st);
  else if (pieces <= 256 * 12)
    rows_kernel<E, 256, 12, POLICY>(name, a, pa, st);
  else if (pieces <= 512 * 8)
    rows_kernel<E, 512, 8, POLICY>(name, a, pa, st);
  else if (pieces <= 512 * 10)
    rows_kernel<E, 512, 10, POLICY>(name, a, pa, st);
  else if (pieces <= 512 * 12)
    rows_kernel<E, 512, 12, POLICY>(name, a, pa, st);
  else if (pieces <= 512 * 16)
    rows_kernel<E, 512, 16, POLICY>(name, a, pa, st);
  else if (POLICY && pieces > 8960 && pieces <= 1024 * 12)
    rows_kernel<E, 1024, 12, true>(name, a, pa, st);
  else if (POLICY && pieces > 8960 && pieces <= 1024 * 16)
    rows_kernel<E, 1024, 16, true>(name, a, pa, st);
  else
    rows_kernel<E, 1024, -4, POLICY>(name, a, pa, st);
  return hipGetLastError();
}

template <typename E, int T>
static void grad_kernel(const RowArgs& a, const float* dlogp, hipStream_t st) {
  RowArgs b = a;  // the last rows first here too
  for (b.first = (a.T - 1) / kRowsALaunch * kRowsALaunch; b.first >= 0; b.first -= kRowsALaunch)
    QLORA_LAUNCH("logprob_grad", st, (k_logprob_grad<E, T>), row_grid(b), dim3(T), 0, st, b, dlogp);
}

// The same for the gradient alone, in pieces, four of a thread's loads in
// flight, eight with 1024 threads (V = 131072: 1024 threads 338 us, with four
// loads 346, 512 threads 353, 256 375; V = 32000: 512 threads 64, 1024 66, 256
// 69).
template <typename E>
static hipError_t launch_grad(const RowArgs& a, const float* dlogp, hipStream_t st) {
  const int64_t pieces = ((int64_t)a.V + Elem<E>::kPer16 - 1) / Elem<E>::kPer16;
  if (pieces <= 64 * 4)
    grad_kernel<E, 64>(a, dlogp, st);
  else if (pieces <= 256 * 4)
    grad_kernel<E, 256>(a, dlogp, st);
  else if (pieces <= 4096 && a.T >= 512)
    grad_kernel<E, 512>(a, dlogp, st);
  else
    grad_kernel<E, 1024>(a, dlogp, st);
  return hipGetLastError();
}

hipError_t launch_logprob(const void* logits, int f32, int64_t T, int V, int64_t ld, const int32_t* labels, float tau,
                          float* logp, float* stats, hipStream_t st) {
  const RowArgs a{logits, 0, T, ld, 0, V, labels, tau, exp2_scale(tau), logp, stats, nullptr, false};
  return f32 ? launch_rows<float, false>("logprob", a, PolicyArgs{}, st)
             : launch_rows<uint16_t, false>("logprob", a, PolicyArgs{}, st);
}

hipError_t launch_logprob_grad(const void* logits, int f32, int64_t T, int V, int64_t ld, const int32_t* labels,
                               float tau, const float* stats, const float* dlogp, void* dlogits, int64_t ldd,
                               hipStream_t st) {
  const RowArgs a{logits,  0, T, ld, ldd, V, labels, tau, exp2_scale(tau), nullptr,
                  const_cast<float*>(stats), dlogits, past_cache(T, ldd, f32)};
  return f32 ? launch_grad<float>(a, dlogp, st) : launch_grad<uint16_t>(a, dlogp, st);
}

hipError_t launch_policy(const void* logits, int f32, int64_t T, int V, int64_t ld, const int32_t* labels, float tau,
                         const float* adv, const float* old_logp, const float* ref_logp, const float* weight,
                         float clip_low, float clip_high, float kl_coef, float* loss, float* kl, float* logp,
                         void* dlogits, int64_t ldd, hipStream_t st) {
  const PolicyArgs pa{adv, old_logp, ref_logp, weight, 1.0f - clip_low, 1.0f + clip_high, kl_coef, loss, kl};
  const RowArgs a{logits, 0, T, ld, ldd, V, labels, tau, exp2_scale(tau), logp, nullptr, dlogits,
                  past_cache(T, ldd, f32)};
  return f32 ? launch_rows<float, true>("policy", a, pa, st) : launch_rows<uint16_t, true>("policy", a, pa, st);
}

hipError_t launch_preference(const float* logp, const float* ref_logp, const int32_t* labels, int64_t T, int V,
                             const int32_t* cu, int64_t P, int kind, int average, float beta, float smoothing,
                             float margin, const float* weight, float* loss, float* reward, float* dlogp,
                             hipStream_t st) {
  const PrefArgs a{logp, ref_logp, labels, cu, weight, T, P, V, kind, average, beta, smoothing, margin, loss, reward,
                   dlogp};
  QLORA_LAUNCH("preference", st, k_preference, dim3((unsigned)P), dim3(kPrefThreads), 0, st, a);
  return hipGetLastError();
}

}  // namespace qlora
