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
// Subtracting the maximum from z before the product (not fma(z, c, -max c))
// keeps rows of very low finite values, whose scaled maximum is not finite,
// and the label at the maximum exact.  Sums and statistics are fp32 and go
// through a fixed tree, so results do not depend on the schedule.
//
// A row is a work-group's: it is read 16 bytes a lane, at the alignment the
// row happens to have (an odd V or row stride starts rows at any element).
#include <cmath>

#include "common.hpp"
#include "launch.hpp"

namespace qlora {

// 16 bytes at element alignment.
typedef u32x4 __attribute__((aligned(2))) u32x4_any;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNegInf = -__builtin_inff();
constexpr int kRowThreads = 256;

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

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// Maximum and sum over the work-group; every thread gets the result.  `red`
// holds one float per wave and is free again after the next barrier.
__device__ __forceinline__ float block_max(float v, float* red) {
  v = wave_max(v);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  float r = red[0];
  for (int i = 1; i < (int)blockDim.x / 64; ++i) r = fmaxf(r, red[i]);
  return r;
}
__device__ __forceinline__ float block_sum(float v, float* red) {
  v = wave_sum(v);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  float r = red[0];
  for (int i = 1; i < (int)blockDim.x / 64; ++i) r += red[i];
  return r;
}

// Running maximum and sum of exp2((z - m) c).  A maximum of -inf (nothing
// but masked values so far) is read as 0 in the exponents: -inf - (-inf)
// would make a NaN of it.
struct Online {
  float m = kNegInf, s = 0.0f;
  template <int N>
  __device__ __forceinline__ void add(const float (&f)[N], float c) {
    float mx = m;
#pragma unroll
    for (int i = 0; i < N; ++i) mx = fmaxf(mx, f[i]);
    const float ref = mx == kNegInf ? 0.0f : mx;
    float sum = s * exp2_hw((m - ref) * c);
#pragma unroll
    for (int i = 0; i < N; ++i) sum += exp2_hw((f[i] - ref) * c);
    m = mx;
    s = sum;
  }
};

struct RowStats {
  float m, s;  // max z; sum exp(tau (z - m))
};

// zy: the label's logit, one of the row's.  It joins the maximum (which it
// cannot change) so that every wave has it in hand before the first barrier:
// a caller that writes over the row in place may do so after this returns.
template <typename E>
__device__ __forceinline__ RowStats row_stats(const E* z, int V, float zy, float c, float* red) {
  constexpr int N = Elem<E>::kPer16;
  const int nv = V / N;
  Online o;
  for (int i = threadIdx.x; i < nv; i += kRowThreads) {
    float f[N];
    Elem<E>::unpack(*reinterpret_cast<const u32x4_any*>(z + (size_t)i * N), f);
    o.add(f, c);
  }
  const int rest = nv * N + threadIdx.x;
  if (rest < V) {
    const float f[1] = {Elem<E>::get(z + rest)};
    o.add(f, c);
  }
  RowStats r;
  r.m = block_max(fmaxf(o.m, zy), red);
  // a thread without a finite value holds m = -inf and s = 0; a row of
  // nothing but -inf has no distribution and gives NaN
  r.s = block_sum(o.s * exp2_hw((o.m - r.m) * c), red + 16);
  return r;
}

// z -> g tau ([v = y] - exp2((z - m) c - log2 s)) over one row, and zeros in
// the columns V..cols-1.
template <typename E>
__device__ __forceinline__ void row_grad(const E* z, E* out, int V, int cols, int label,
                                         float m, float log2s, float c, float g) {
  constexpr int N = Elem<E>::kPer16;
  const int nv = V / N;
  for (int i = threadIdx.x; i < nv; i += kRowThreads) {
    float f[N];
    Elem<E>::unpack(*reinterpret_cast<const u32x4_any*>(z + (size_t)i * N), f);
#pragma unroll
    for (int q = 0; q < N; ++q) {
      const float p = exp2_hw((f[q] - m) * c - log2s);
      f[q] = (label == i * N + q ? 1.0f - p : -p) * g;
    }
    *reinterpret_cast<u32x4_any*>(out + (size_t)i * N) = Elem<E>::pack(f);
  }
  const int rest = nv * N + threadIdx.x;
  if (rest < V) {
    const float p = exp2_hw((Elem<E>::get(z + rest) - m) * c - log2s);
    Elem<E>::put(out + rest, (label == rest ? 1.0f - p : -p) * g);
  }
  for (int i = V + threadIdx.x; i < cols; i += kRowThreads) Elem<E>::put(out + i, 0.0f);
}

template <typename E>
__device__ __forceinline__ void row_zero(E* __restrict__ out, int cols) {
  constexpr int N = Elem<E>::kPer16;
  const int nv = cols / N;
  for (int i = threadIdx.x; i < nv; i += kRowThreads)
    *reinterpret_cast<u32x4_any*>(out + (size_t)i * N) = u32x4{0u, 0u, 0u, 0u};
  const int rest = nv * N + threadIdx.x;
  if (rest < cols) Elem<E>::put(out + rest, 0.0f);
}

__device__ __forceinline__ bool is_counted(int label, int V) { return (uint32_t)label < (uint32_t)V; }

template <typename E>
__global__ __launch_bounds__(kRowThreads) void k_logprob(const E* __restrict__ logits, int64_t T, int V, int64_t ld,
                                                         const int32_t* __restrict__ labels, float tau,
                                                         float* __restrict__ logp, float* __restrict__ stats) {
  __shared__ float red[32];
  const float c = tau * kLog2e;
  for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
    const int label = labels[t];
    float lp = 0.0f, m = 0.0f, l2 = 0.0f;
    if (is_counted(label, V)) {
      const E* z = logits + t * ld;
      const float zy = Elem<E>::get(z + label);
      const RowStats r = row_stats(z, V, zy, c, red);
      m = r.m;
      l2 = log2f(r.s);
      lp = (zy - m) * tau - logf(r.s);
    }
    if (threadIdx.x == 0) {
      logp[t] = lp;
      if (stats != nullptr) {
        stats[2 * t] = m;
        stats[2 * t + 1] = l2;
      }
    }
    __syncthreads();  // red is written again for the next row
  }
}

template <typename E>
__global__ __launch_bounds__(kRowThreads) void k_logprob_grad(const E* logits, int64_t T, int V, int64_t ld,
                                                              const int32_t* __restrict__ labels, float tau,
                                                              const float* __restrict__ stats,
                                                              const float* __restrict__ dlogp, E* dlogits,
                                                              int64_t ldd) {
  const float c = tau * kLog2e;
  for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
    const int label = labels[t];
    const float g = dlogp[t];
    E* out = dlogits + t * ldd;
    if (!is_counted(label, V) || g == 0.0f)
      row_zero(out, (int)ldd);
    else
      row_grad(logits + t * ld, out, V, (int)ldd, label, stats[2 * t], stats[2 * t + 1], c, g * tau);
  }
}

// ------------------------------------------------------- policy loss -----
//
// Per counted token, with ratio r = exp(lp - old), advantage A, clip range
// [lo, hi] = [1 - clip_low, 1 + clip_high] and d = ref - lp:
//
//   loss = -min(r A, clip(r) A) + kl_coef (exp(d) - d - 1)
//   d loss / d lp = -r A (0 where the clip holds) - kl_coef (exp(d) - 1)
//
// expm1 keeps the KL term's digits where d is small.
struct PolicyArgs {
  const float* adv;
  const float* old_logp;  // nullptr: the policy itself (r = 1)
  const float* ref_logp;  // nullptr: no KL term
  const float* weight;    // nullptr: 1
  float lo, hi, kl_coef;
  float* loss;
  float* kl;
};

__device__ __forceinline__ float policy_token(const PolicyArgs& a, int64_t t, float lp, float& loss, float& kl) {
  const float A = a.adv[t];
  const float r = a.old_logp != nullptr ? expf(lp - a.old_logp[t]) : (lp == lp ? 1.0f : lp);
  const float rc = fminf(fmaxf(r, a.lo), a.hi);
  const float x = r * A, y = rc * A;
  const bool clipped = y < x;  // the clipped branch is the smaller one, and flat
  loss = -(clipped ? y : x);
  float g = clipped ? 0.0f : -x;
  kl = 0.0f;
  if (a.ref_logp != nullptr) {
    const float d = a.ref_logp[t] - lp;
    const float e = expm1f(d);
    kl = e - d;
    loss = fmaf(a.kl_coef, kl, loss);
    g = fmaf(-a.kl_coef, e, g);
  }
  if (a.weight == nullptr) return g;
  const float w = a.weight[t];
  return w == 0.0f ? 0.0f : g * w;  // a token taken out has no gradient, not a NaN either
}

template <typename E>
__global__ __launch_bounds__(kRowThreads) void k_policy(const E* logits, int64_t T, int V, int64_t ld,
                                                        const int32_t* __restrict__ labels, float tau, PolicyArgs a,
                                                        float* __restrict__ logp, E* dlogits, int64_t ldd) {
  __shared__ float red[32];
  const float c = tau * kLog2e;
  for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
    const int label = labels[t];
    E* out = dlogits != nullptr ? dlogits + t * ldd : nullptr;
    float lp = 0.0f, loss = 0.0f, kl = 0.0f;
    if (is_counted(label, V)) {
      const E* z = logits + t * ld;
      const float zy = Elem<E>::get(z + label);
      const RowStats r = row_stats(z, V, zy, c, red);
      lp = (zy - r.m) * tau - logf(r.s);
      const float g = policy_token(a, t, lp, loss, kl);
      if (out != nullptr) {
        if (g == 0.0f)
          row_zero(out, (int)ldd);
        else
          row_grad(z, out, V, (int)ldd, label, r.m, log2f(r.s), c, g * tau);
      }
    } else if (out != nullptr) {
      row_zero(out, (int)ldd);
    }
    if (threadIdx.x == 0) {
      logp[t] = lp;
      a.loss[t] = loss;
      if (a.kl != nullptr) a.kl[t] = kl;
    }
    __syncthreads();
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
// A work-group takes a pair: it sums in fp64 (thousands of terms, of which a
// small difference is left) and writes each token's d loss / d logp.
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

__global__ __launch_bounds__(kRowThreads) void k_preference(PrefArgs a) {
  __shared__ double sums[2][kRowThreads / 64];
  __shared__ int counts[2][kRowThreads / 64];
  const int64_t p = blockIdx.x;
  int64_t lo[2], hi[2];
  seq_range(a, p, lo[0], hi[0]);
  seq_range(a, a.P + p, lo[1], hi[1]);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    double sum = 0.0;
    int n = 0;
    for (int64_t t = lo[k] + threadIdx.x; t < hi[k]; t += kRowThreads) {
      if (is_counted(a.labels[t], a.V)) {
        sum += a.ref_logp != nullptr ? (double)a.logp[t] - (double)a.ref_logp[t] : (double)a.logp[t];
        ++n;
      }
    }
    for (int o = 32; o >= 1; o >>= 1) {
      sum += __shfl_xor(sum, o, 64);
      n += __shfl_xor(n, o, 64);
    }
    if ((threadIdx.x & 63) == 0) {
      sums[k][threadIdx.x >> 6] = sum;
      counts[k][threadIdx.x >> 6] = n;
    }
  }
  __syncthreads();
  double l[2], inv[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    l[k] = 0.0;
    int n = 0;
    for (int w = 0; w < kRowThreads / 64; ++w) {
      l[k] += sums[k][w];
      n += counts[k][w];
    }
    inv[k] = a.average ? 1.0 / (double)(n > 1 ? n : 1) : 1.0;
    l[k] *= inv[k];
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
  const double dl = dh * beta * (a.weight != nullptr ? (double)a.weight[p] : 1.0);
  if (threadIdx.x == 0) {
    a.loss[p] = (float)loss;
    if (a.reward != nullptr) {
      a.reward[p] = (float)(beta * l[0]);
      a.reward[a.P + p] = (float)(beta * l[1]);
    }
  }
  if (a.dlogp == nullptr) return;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const float g = (float)((k == 0 ? dl : -dl) * inv[k]);
    for (int64_t t = lo[k] + threadIdx.x; t < hi[k]; t += kRowThreads)
      a.dlogp[t] = is_counted(a.labels[t], a.V) ? g : 0.0f;
  }
  // tokens before the first sequence and after the last have no gradient
  if (p == 0)
    for (int64_t t = threadIdx.x; t < lo[0]; t += kRowThreads) a.dlogp[t] = 0.0f;
  if (p == a.P - 1)
    for (int64_t t = hi[1] + threadIdx.x; t < a.T; t += kRowThreads) a.dlogp[t] = 0.0f;
}

// ---------------------------------------------------------- launchers ----

// Work-groups of the row kernels: a row each, up to a grid whose thread
// count stays below 2^32.
static dim3 row_grid(int64_t T) { return dim3((unsigned)(T < (1 << 20) ? T : (1 << 20))); }

hipError_t launch_logprob(const void* logits, int f32, int64_t T, int V, int64_t ld, const int32_t* labels, float tau,
                          float* logp, float* stats, hipStream_t st) {
  if (f32)
    QLORA_LAUNCH("logprob", st, k_logprob<float>, row_grid(T), dim3(kRowThreads), 0, st, (const float*)logits, T, V,
                 ld, labels, tau, logp, stats);
  else
    QLORA_LAUNCH("logprob", st, k_logprob<uint16_t>, row_grid(T), dim3(kRowThreads), 0, st, (const uint16_t*)logits,
                 T, V, ld, labels, tau, logp, stats);
  return hipGetLastError();
}

hipError_t launch_logprob_grad(const void* logits, int f32, int64_t T, int V, int64_t ld, const int32_t* labels,
                               float tau, const float* stats, const float* dlogp, void* dlogits, int64_t ldd,
                               hipStream_t st) {
  if (f32)
    QLORA_LAUNCH("logprob_grad", st, k_logprob_grad<float>, row_grid(T), dim3(kRowThreads), 0, st,
                 (const float*)logits, T, V, ld, labels, tau, stats, dlogp, (float*)dlogits, ldd);
  else
    QLORA_LAUNCH("logprob_grad", st, k_logprob_grad<uint16_t>, row_grid(T), dim3(kRowThreads), 0, st,
                 (const uint16_t*)logits, T, V, ld, labels, tau, stats, dlogp, (uint16_t*)dlogits, ldd);
  return hipGetLastError();
}

hipError_t launch_policy(const void* logits, int f32, int64_t T, int V, int64_t ld, const int32_t* labels, float tau,
                         const float* adv, const float* old_logp, const float* ref_logp, const float* weight,
                         float clip_low, float clip_high, float kl_coef, float* loss, float* kl, float* logp,
                         void* dlogits, int64_t ldd, hipStream_t st) {
  const PolicyArgs a{adv, old_logp, ref_logp, weight, 1.0f - clip_low, 1.0f + clip_high, kl_coef, loss, kl};
  if (f32)
    QLORA_LAUNCH("policy", st, k_policy<float>, row_grid(T), dim3(kRowThreads), 0, st, (const float*)logits, T, V, ld,
                 labels, tau, a, logp, (float*)dlogits, ldd);
  else
    QLORA_LAUNCH("policy", st, k_policy<uint16_t>, row_grid(T), dim3(kRowThreads), 0, st, (const uint16_t*)logits, T,
                 V, ld, labels, tau, a, logp, (uint16_t*)dlogits, ldd);
  return hipGetLastError();
}

hipError_t launch_preference(const float* logp, const float* ref_logp, const int32_t* labels, int64_t T, int V,
                             const int32_t* cu, int64_t P, int kind, int average, float beta, float smoothing,
                             float margin, const float* weight, float* loss, float* reward, float* dlogp,
                             hipStream_t st) {
  const PrefArgs a{logp, ref_logp, labels, cu, weight, T, P, V, kind, average, beta, smoothing, margin, loss, reward,
                   dlogp};
  QLORA_LAUNCH("preference", st, k_preference, dim3((unsigned)P), dim3(kRowThreads), 0, st, a);
  return hipGetLastError();
}

}  // namespace qlora
