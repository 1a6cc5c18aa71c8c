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
#include <cmath>

#include "common.hpp"
#include "launch.hpp"

namespace qlora {

constexpr int kMuThreads = 256;
constexpr int kMuTile = 64;  // long positions per LDS tile

struct MuShape {
  int64_t nmat, rows, cols;
  int S, tall;   // short side; rows > cols
  int64_t L;     // long side
};

static MuShape mu_shape(int64_t nmat, int64_t rows, int64_t cols) {
  MuShape s{nmat, rows, cols, 0, rows > cols, 0};
  s.S = (int)(s.tall ? cols : rows);
  s.L = s.tall ? rows : cols;
  return s;
}

__device__ __forceinline__ int64_t mu_at(const MuShape& s, int i, int64_t j) {
  return s.tall ? j * s.S + i : i * s.L + j;
}

__device__ __forceinline__ float mu_momentum(float m, float g, float mu) { return __fadd_rn(__fmul_rn(mu, m), g); }
__device__ __forceinline__ float mu_update(float m, float g, float mu, int nesterov) {
  return nesterov ? __fadd_rn(g, __fmul_rn(mu, m)) : m;
}

// Pass 1: m <- mu m + g, and one fp64 partial of u u^T per (matrix, split).
__global__ __launch_bounds__(kMuThreads) void k_muon_gram(const uint16_t* __restrict__ G, float* __restrict__ M,
                                                          MuShape s, float mu, int nesterov, int splits,
                                                          double* __restrict__ part) {
  __shared__ float tile[kMuTile][65];
  const int64_t mat = blockIdx.x / splits;
  const int split = blockIdx.x % splits;
  const int64_t base = mat * s.rows * s.cols;
  const int S = s.S, SS = S * S;
  double acc[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) acc[e] = 0.0;
  for (int64_t j0 = (int64_t)split * kMuTile; j0 < s.L; j0 += (int64_t)splits * kMuTile) {
    for (int e = threadIdx.x; e < kMuTile * S; e += kMuThreads) {
      const int jj = s.tall ? e / S : e % kMuTile, i = s.tall ? e % S : e / kMuTile;
      float u = 0.0f;
      if (j0 + jj < s.L) {
        const int64_t at = base + mu_at(s, i, j0 + jj);
        const float g = bf16_to_f32(G[at]);
        const float m = mu_momentum(M[at], g, mu);
        M[at] = m;
        u = mu_update(m, g, mu, nesterov);
      }
      tile[jj][i] = u;
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int at = e * kMuThreads + threadIdx.x;
      if (at < SS) {
        const int i = at / S, k = at % S;
        for (int jj = 0; jj < kMuTile; ++jj) acc[e] += (double)tile[jj][i] * (double)tile[jj][k];
      }
    }
    __syncthreads();
  }
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const int at = e * kMuThreads + threadIdx.x;
    if (at < SS) part[(size_t)blockIdx.x * SS + at] = acc[e];
  }
}

// The S x S iteration of one matrix: Q / (|u| + eps), rounded to fp32.
__global__ __launch_bounds__(kMuThreads) void k_muon_poly(const double* __restrict__ part, int splits, int S,
                                                          MuonCoef co, float eps, float* __restrict__ Qout) {
  __shared__ double G[64 * 65], P[64 * 65], Q[64 * 65], R[64 * 65];
  const int SS = S * S, ld = 65;
  const double* src = part + (size_t)blockIdx.x * splits * SS;
  for (int at = threadIdx.x; at < SS; at += kMuThreads) {
    double sum = 0.0;
    for (int k = 0; k < splits; ++k) sum += src[(size_t)k * SS + at];
    G[(at / S) * ld + at % S] = sum;
    Q[(at / S) * ld + at % S] = at / S == at % S ? 1.0 : 0.0;
  }
  __syncthreads();
  double trace = 0.0;
  for (int i = 0; i < S; ++i) trace += G[i * ld + i];
  const double inv = 1.0 / (sqrt(trace) + (double)eps);
  __syncthreads();
  for (int at = threadIdx.x; at < SS; at += kMuThreads) G[(at / S) * ld + at % S] *= inv * inv;
  __syncthreads();
  // out = x y (all of them commute and are symmetric)
  auto mul = [&](const double* x, const double* y, double* out) {
    for (int at = threadIdx.x; at < SS; at += kMuThreads) {
      const int i = at / S, k = at % S;
      double sum = 0.0;
      for (int q = 0; q < S; ++q) sum = fma(x[i * ld + q], y[q * ld + k], sum);
      out[i * ld + k] = sum;
    }
    __syncthreads();
  };
  for (int n = 0; n < co.n; ++n) {
    mul(G, G, P);
    for (int at = threadIdx.x; at < SS; at += kMuThreads) {
      const int i = at / S, k = at % S;
      P[i * ld + k] = (i == k ? co.c[n][0] : 0.0) + co.c[n][1] * G[i * ld + k] + co.c[n][2] * P[i * ld + k];
    }
    __syncthreads();
    mul(P, Q, R);
    for (int at = threadIdx.x; at < SS; at += kMuThreads) Q[(at / S) * ld + at % S] = R[(at / S) * ld + at % S];
    __syncthreads();
    if (n + 1 < co.n) {
      mul(P, G, R);
      mul(R, P, G);
    }
  }
  for (int at = threadIdx.x; at < SS; at += kMuThreads)
    Qout[(size_t)blockIdx.x * SS + at] = (float)(Q[(at / S) * ld + at % S] * inv);
}

// Pass 2: X = Q u, the weights and their bf16 copy.
__global__ __launch_bounds__(kMuThreads) void k_muon_apply(const uint16_t* __restrict__ G,
                                                           const float* __restrict__ M, MuShape s, float mu,
                                                           int nesterov, int splits, const float* __restrict__ Qin,
                                                           float decay, float step, float* __restrict__ W,
                                                           uint16_t* __restrict__ P) {
  __shared__ float tile[kMuTile][65];
  __shared__ float Q[64 * 65];
  const int64_t mat = blockIdx.x / splits;
  const int split = blockIdx.x % splits;
  const int64_t base = mat * s.rows * s.cols;
  const int S = s.S;
  for (int at = threadIdx.x; at < S * S; at += kMuThreads) Q[(at / S) * 65 + at % S] = Qin[(size_t)mat * S * S + at];
  for (int64_t j0 = (int64_t)split * kMuTile; j0 < s.L; j0 += (int64_t)splits * kMuTile) {
    __syncthreads();
    for (int e = threadIdx.x; e < kMuTile * S; e += kMuThreads) {
      const int jj = s.tall ? e / S : e % kMuTile, i = s.tall ? e % S : e / kMuTile;
      float u = 0.0f;
      if (j0 + jj < s.L) {
        const int64_t at = base + mu_at(s, i, j0 + jj);
        u = mu_update(M[at], bf16_to_f32(G[at]), mu, nesterov);
      }
      tile[jj][i] = u;
    }
    __syncthreads();
    for (int e = threadIdx.x; e < kMuTile * S; e += kMuThreads) {
      const int jj = s.tall ? e / S : e % kMuTile, i = s.tall ? e % S : e / kMuTile;
      if (j0 + jj >= s.L) continue;
      float x = 0.0f;
      for (int k = 0; k < S; ++k) x = fmaf(Q[i * 65 + k], tile[jj][k], x);
      const int64_t at = base + mu_at(s, i, j0 + jj);
      const float w = __fsub_rn(__fmul_rn(W[at], decay), __fmul_rn(step, x));
      W[at] = w;
      P[at] = (uint16_t)pack_bf16x2(w, 0.0f);
    }
  }
}

// Work-groups per matrix: about four per CU over the stack, each with at
// least one tile.
static int mu_splits(const MuShape& s) {
  const int64_t tiles = (s.L + kMuTile - 1) / kMuTile;
  int64_t n = (1024 + s.nmat - 1) / s.nmat;
  if (n > tiles) n = tiles;
  return (int)(n < 1 ? 1 : n);
}

static size_t mu_part_bytes(const MuShape& s) {
  return (size_t)align_up((int64_t)((size_t)s.nmat * mu_splits(s) * s.S * s.S * sizeof(double)), 256);
}

size_t muon_ws_bytes(int64_t nmat, int64_t rows, int64_t cols) {
  const MuShape s = mu_shape(nmat, rows, cols);
  return mu_part_bytes(s) + (size_t)nmat * s.S * s.S * sizeof(float);
}

hipError_t launch_muon(uint16_t* P, float* W, const uint16_t* G, float* m, int64_t nmat, int64_t rows, int64_t cols,
                       float lr, float momentum, int nesterov, float wd, float scale, float eps, const MuonCoef& co,
                       void* ws, hipStream_t st) {
  const MuShape s = mu_shape(nmat, rows, cols);
  const int splits = mu_splits(s);
  double* part = reinterpret_cast<double*>(ws);
  float* Q = reinterpret_cast<float*>(reinterpret_cast<char*>(ws) + mu_part_bytes(s));
  const dim3 grid((unsigned)(nmat * splits)), block(kMuThreads);
  QLORA_LAUNCH("muon_gram", st, k_muon_gram, grid, block, 0, st, G, m, s, momentum, nesterov, splits, part);
  QLORA_LAUNCH("muon_poly", st, k_muon_poly, dim3((unsigned)nmat), block, 0, st, part, splits, s.S, co, eps, Q);
  QLORA_LAUNCH("muon_apply", st, k_muon_apply, grid, block, 0, st, G, m, s, momentum, nesterov, splits, Q,
               (float)(1.0 - (double)lr * wd), (float)((double)lr * scale), W, P);
  return hipGetLastError();
}

}  // namespace qlora
