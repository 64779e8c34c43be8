// Orthogonalised update of many small matrices, for gfx950.
//
// For each matrix:  M <- mu M + G,  U = G + mu M (or M without the look-ahead),
//   X_0 = U / max(|U|, eps),  X_{k+1} = X_k p(A_k),  A_k = X_k^T X_k,
//   p(A) = a I + b A + c A^2,  W <- (1 - lr wd) W - lr sqrt(max(1, rows / cols)) X_n.
// With the S columns of X its smaller side (else the transpose is meant), every
// A_k and every product of the p(A_k) is a polynomial in A_0, so
//   A_{k+1} = A_k p(A_k)^2,  X_n = X_0 Q,  Q = p(A_0) p(A_1) ...
// and the long side is passed over twice only: for A_0 and for X_0 Q; what lies
// between are S x S products, and all of them are symmetric and commute.
// An error of A_0 on a small singular value grows by a^2 (about 12) a step, by
// 12^4 until the last p, where the rounding of fp32 would show; so A and Q are
// held in fp64.  |U|^2 is the trace of U^T U.
//
// One work-group takes one matrix from start to end: the S x S work needs one
// CU's LDS and no launch of its own, and the work-groups of a step, which are
// in different phases, share memory and matrix units.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/ttc_block.h"
#include "ttc_device.hpp"
#include "ttc_trace.hpp"

namespace ttc {
namespace {

typedef double f64x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 512;
constexpr int kWaves = kThreads / 64;
constexpr int kMaxSide = 128;
constexpr int kMaxSteps = 32;
constexpr int kLdsSide = 64;  // the S x S matrices of larger ones lie in the scratch

// A matrix as the kernel sees it: element (i, j), i < len along the long side,
// j < side along the short one, is at i * si + j * sj.
struct Mat {
  float* w;
  const float* g;
  float* m;
  int64_t len, si, sj;
  int64_t scratch;  // doubles from the scratch's start on (side > kLdsSide)
  int32_t side;
  float scale;  // sqrt(max(1, rows / cols))
};

struct OrthoArgs {
  const Mat* mats;
  double* scratch;
  double a, b, c;
  float eps, lr, mu, decay;  // decay = 1 - lr wd
  int steps, ahead;
};

constexpr int ld_of(int sp) { return sp + 2; }
constexpr int mat_size(int sp) { return sp * ld_of(sp); }

// One k-step of four: lane l holds row l % 16 of A and column l % 16 of B at
// k = l / 16; element r of the result is row 4 r + l / 16, column l % 16.
__device__ __forceinline__ f64x4 mma64(double x, double y, f64x4 c) {
  return __builtin_amdgcn_mfma_f64_16x16x4f64(x, y, c, 0, 0, 0);
}

// N elements of u of one row of the long side; FIRST also steps the momentum
template <int N, bool FIRST>
__device__ __forceinline__ void load_u(const OrthoArgs& a, const Mat& t, int64_t i, int j, float (&u)[N]) {
#pragma unroll
  for (int e = 0; e < N; ++e) {
    u[e] = 0.f;
    if (i < t.len && j + e < t.side) {
      const int64_t at = i * t.si + (j + e) * t.sj;
      const float g = t.g[at];
      float m = t.m[at];
      if (FIRST) {
        m = a.mu * m + g;
        t.m[at] = m;
      }
      u[e] = a.ahead ? g + a.mu * m : m;
    }
  }
}

// Place of column j in the order that the S x S matrices are kept in: a lane
// reads nt neighbouring columns, one for each of nt tiles, of a block of 16 nt.
__device__ __forceinline__ int place(int j, int nt) {
  const int blk = j / (16 * nt), r = j - blk * 16 * nt;
  return blk * 16 * nt + (r % nt) * 16 + r / nt;
}

// out (NT * 16 square, places) = sum over rows of u[block bi]^T u[block bj], all
// tiles of an off-diagonal block, those on and above the diagonal of a diagonal
// one, written to both sides.  Each wave sums its own rows; the waves' sums are
// added in a fixed order through `lds`.
template <int NT, bool DIAG>
__device__ void gram(const OrthoArgs& a, const Mat& t, int bi, int bj, double* lds, double* out, int ld) {
  constexpr int TILES = DIAG ? NT * (NT + 1) / 2 : NT * NT;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, c = lane & 15, g = lane >> 4;
  f64x4 acc[TILES];
#pragma unroll
  for (int x = 0; x < TILES; ++x) acc[x] = f64x4{0., 0., 0., 0.};
  for (int64_t i0 = 4 * w; i0 < t.len; i0 += 4 * kWaves) {
    float ui[NT], uj[NT];
    load_u<NT, DIAG>(a, t, i0 + g, bi * 16 * NT + c * NT, ui);
    if (!DIAG) load_u<NT, false>(a, t, i0 + g, bj * 16 * NT + c * NT, uj);
    double di[NT], dj[NT];
#pragma unroll
    for (int e = 0; e < NT; ++e) {
      di[e] = ui[e];
      dj[e] = DIAG ? ui[e] : uj[e];
    }
    int x = 0;
#pragma unroll
    for (int p = 0; p < NT; ++p)
#pragma unroll
      for (int q = DIAG ? p : 0; q < NT; ++q, ++x) acc[x] = mma64(di[p], dj[q], acc[x]);
  }
  for (int half = kWaves / 2; half > 0; half >>= 1) {
    __syncthreads();
    if (w >= half && w < 2 * half)
#pragma unroll
      for (int x = 0; x < TILES; ++x)
#pragma unroll
        for (int r = 0; r < 4; ++r) lds[(((w - half) * TILES + x) * 4 + r) * 64 + lane] = acc[x][r];
    __syncthreads();
    if (w < half)
#pragma unroll
      for (int x = 0; x < TILES; ++x)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[x][r] += lds[((w * TILES + x) * 4 + r) * 64 + lane];
  }
  __syncthreads();  // `out` may be what the sums went through
  if (w == 0) {
    int x = 0;
#pragma unroll
    for (int p = 0; p < NT; ++p)
#pragma unroll
      for (int q = DIAG ? p : 0; q < NT; ++q, ++x)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = (bi * NT + p) * 16 + 4 * r + g, col = (bj * NT + q) * 16 + c;
          out[row * ld + col] = acc[x][r];
          out[col * ld + row] = acc[x][r];
        }
  }
  __syncthreads();
}

// Tile x of the nt (nt + 1) / 2 tiles on and above the diagonal.
__device__ __forceinline__ void tile_of(int x, int nt, int& p, int& q) {
  p = 0;
  while (x >= nt - p) x -= nt - p++;
  q = p + x;
}

// Tile (p, q) of the product of two symmetric matrices that commute
__device__ __forceinline__ f64x4 tile_product(const double* x, const double* y, int p, int q, int sp, int ld) {
  const int lane = threadIdx.x & 63;
  const double* rx = x + (p * 16 + (lane & 15)) * ld + (lane >> 4);
  const double* ry = y + (q * 16 + (lane & 15)) * ld + (lane >> 4);
  f64x4 acc = {0., 0., 0., 0.};
#pragma unroll 4
  for (int k = 0; k < sp; k += 4) acc = mma64(rx[k], ry[k], acc);
  return acc;
}

template <typename F>
__device__ __forceinline__ void each_of_tile(int p, int q, int ld, F f) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int row = p * 16 + 4 * r + (lane >> 4), col = q * 16 + (lane & 15);
    f(r, row, col, row * ld + col, col * ld + row);
  }
}

// mats in LDS: at most two tiles a wave (10 tiles of 8 waves); in the scratch 5
constexpr int kTilesPerWave = 5;

// A_0 in `A` -> Q in `Q`, over n steps; P is the third matrix
__device__ void iterate(const OrthoArgs& a, double* A, double* P, double* Q, int nt) {
  const int w = threadIdx.x >> 6, sp = nt * 16, ld = ld_of(sp), tiles = nt * (nt + 1) / 2;
  for (int k = 0; k < a.steps; ++k) {
    const bool last = k + 1 == a.steps;
    for (int x = w; x < tiles; x += kWaves) {
      int p, q;
      tile_of(x, nt, p, q);
      const f64x4 s = tile_product(A, A, p, q, sp, ld);
      each_of_tile(p, q, ld, [&](int r, int row, int col, int at, int mirror) {
        const double v = (row == col ? a.a : 0.) + a.b * A[at] + a.c * s[r];
        P[at] = v;
        P[mirror] = v;
        if (k == 0) {
          Q[at] = v;
          Q[mirror] = v;
        }
      });
    }
    __syncthreads();
    f64x4 fa[kTilesPerWave], fq[kTilesPerWave];
#pragma unroll
    for (int y = 0; y < kTilesPerWave; ++y) {
      const int x = w + y * kWaves;
      if (x >= tiles) break;
      int p, q;
      tile_of(x, nt, p, q);
      if (!last) fa[y] = tile_product(A, P, p, q, sp, ld);
      if (k > 0) fq[y] = tile_product(Q, P, p, q, sp, ld);
    }
    __syncthreads();
#pragma unroll
    for (int y = 0; y < kTilesPerWave; ++y) {
      const int x = w + y * kWaves;
      if (x >= tiles) break;
      int p, q;
      tile_of(x, nt, p, q);
      each_of_tile(p, q, ld, [&](int r, int, int, int at, int mirror) {
        if (!last) A[at] = A[mirror] = fa[y][r];
        if (k > 0) Q[at] = Q[mirror] = fq[y][r];
      });
    }
    __syncthreads();
    if (last) break;
#pragma unroll
    for (int y = 0; y < kTilesPerWave; ++y) {
      const int x = w + y * kWaves;
      if (x >= tiles) break;
      int p, q;
      tile_of(x, nt, p, q);
      fa[y] = tile_product(A, P, p, q, sp, ld);
    }
    __syncthreads();
#pragma unroll
    for (int y = 0; y < kTilesPerWave; ++y) {
      const int x = w + y * kWaves;
      if (x >= tiles) break;
      int p, q;
      tile_of(x, nt, p, q);
      each_of_tile(p, q, ld, [&](int r, int, int, int at, int mirror) { A[at] = A[mirror] = fa[y][r]; });
    }
    __syncthreads();
  }
}

__global__ __launch_bounds__(kThreads) void k_ortho(OrthoArgs a) {
  extern __shared__ __attribute__((aligned(16))) double lds[];
  const Mat t = a.mats[blockIdx.x];
  const int S = t.side, nt = (S + 15) / 16, block = nt <= 4 ? nt : 4;  // tiles of a block of columns
  const int all = nt <= 4 ? nt : 8, sp = all * 16, ld = ld_of(sp);
  double* base = nt <= 4 ? lds : a.scratch + t.scratch;
  double *A = base, *P = base + mat_size(sp), *Q = P + mat_size(sp);
  if (nt == 1) {
    gram<1, true>(a, t, 0, 0, lds, A, ld);
  } else if (nt == 2) {
    gram<2, true>(a, t, 0, 0, lds, A, ld);
  } else if (nt == 3) {
    gram<3, true>(a, t, 0, 0, lds, A, ld);
  } else {
    gram<4, true>(a, t, 0, 0, lds, A, ld);
    if (nt > 4) {
      gram<4, true>(a, t, 1, 1, lds, A, ld);
      gram<4, false>(a, t, 0, 1, lds, A, ld);
    }
  }
  double trace = 0.;
  for (int j = 0; j < sp; ++j) trace += A[j * ld + j];
  // a NaN stays one: the comparison with it is false
  const double norm = sqrt(trace), inv = 1. / (norm < (double)a.eps ? (double)a.eps : norm);
  __syncthreads();
  for (int x = threadIdx.x; x < mat_size(sp); x += kThreads) A[x] *= inv * inv;
  __syncthreads();
  iterate(a, A, P, Q, all);

  // Q in fp32, in the columns' own order, where A and P were
  float* qf = reinterpret_cast<float*>(A);
  const int lq = sp + 4;
  for (int x = threadIdx.x; x < sp * sp; x += kThreads) {
    const int r = x / sp, c = x - r * sp;
    qf[r * lq + c] = (float)Q[place(r, block) * ld + place(c, block)];
  }
  __syncthreads();
  const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
  const float finv = (float)inv, step = a.lr * t.scale;
  for (int64_t i0 = 16 * (threadIdx.x >> 6); i0 < t.len; i0 += 16 * kWaves) {
    const int64_t i = i0 + c;
    f32x4 x[8];
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      if (s >= nt) break;
      float u[4];
      load_u<4, false>(a, t, i, s * 16 + 4 * g, u);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[s][e] = u[e] * finv;
    }
    for (int o = 0; o < nt; ++o) {
      f32x4 acc = zero4();
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        if (s >= nt) break;
        acc = Mma<float>::mma(*reinterpret_cast<const f32x4*>(qf + (o * 16 + c) * lq + s * 16 + 4 * g), x[s], acc);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int j = o * 16 + 4 * g + e;
        if (i < t.len && j < S) {
          float* w = t.w + i * t.si + j * t.sj;
          *w = *w * a.decay - step * acc[e];
        }
      }
    }
  }
}

// ---- host --------------------------------------------------------------------

ttc_status check_mats(int64_t n, const ttc_ortho_mat* mats) {
  if (n < 0 || n > (1 << 24)) return TTC_ERR_SHAPE;
  if (n > 0 && !mats) return TTC_ERR_NULL;
  for (int64_t k = 0; k < n; ++k) {
    const ttc_ortho_mat& m = mats[k];
    if (m.rows < 1 || m.cols < 1 || m.rows > INT32_MAX || m.cols > INT32_MAX) return TTC_ERR_SHAPE;
    if (std::min(m.rows, m.cols) > TTC_ORTHO_MAX_SIDE) return TTC_ERR_SHAPE;
    if (!m.w || !m.g || !m.m) return TTC_ERR_NULL;
    if (((uintptr_t)m.w | (uintptr_t)m.g | (uintptr_t)m.m) & 3) return TTC_ERR_ALIGN;
  }
  return TTC_OK;
}

int padded(int64_t side) { return side <= kLdsSide ? (int)(side + 15) / 16 * 16 : kMaxSide; }

}  // namespace
}  // namespace ttc

using namespace ttc;

extern "C" ttc_status ttc_ortho_workspace(int64_t n, const ttc_ortho_mat* mats, size_t* plan_bytes,
                                          size_t* scratch_bytes) {
  if (!plan_bytes || !scratch_bytes) return TTC_ERR_NULL;
  const ttc_status st = check_mats(n, mats);
  if (st != TTC_OK) return st;
  *plan_bytes = (size_t)n * sizeof(Mat);
  int64_t d = 0;
  for (int64_t k = 0; k < n; ++k)
    if (std::min(mats[k].rows, mats[k].cols) > kLdsSide) d += 3 * mat_size(kMaxSide);
  *scratch_bytes = (size_t)d * sizeof(double);
  return TTC_OK;
}

extern "C" ttc_status ttc_ortho_plan(int64_t n, const ttc_ortho_mat* mats, void* plan, size_t plan_bytes) {
  const ttc_status st = check_mats(n, mats);
  if (st != TTC_OK) return st;
  if (n == 0) return TTC_OK;
  if (!plan) return TTC_ERR_NULL;
  if (plan_bytes < (size_t)n * sizeof(Mat)) return TTC_ERR_WORKSPACE;
  Mat* out = static_cast<Mat*>(plan);
  int64_t d = 0;
  for (int64_t k = 0; k < n; ++k) {
    const ttc_ortho_mat& m = mats[k];
    const bool tall = m.rows >= m.cols;
    Mat t = {};
    t.w = m.w;
    t.g = m.g;
    t.m = m.m;
    t.len = tall ? m.rows : m.cols;
    t.side = (int32_t)(tall ? m.cols : m.rows);
    t.si = tall ? m.cols : 1;
    t.sj = tall ? 1 : m.cols;
    t.scale = (float)sqrt(std::max(1., (double)m.rows / (double)m.cols));
    if (t.side > kLdsSide) {
      t.scratch = d;
      d += 3 * mat_size(kMaxSide);
    }
    out[k] = t;
  }
  // the longest first, so that the last work-groups to start are short ones
  std::stable_sort(out, out + n, [](const Mat& x, const Mat& y) {
    const auto cost = [](const Mat& t) { return (double)(t.len + 8 * t.side) * t.side * t.side; };
    return cost(x) > cost(y);
  });
  return TTC_OK;
}

extern "C" ttc_status ttc_ortho_step(const ttc_ortho_desc* desc, int64_t n, const ttc_ortho_mat* mats, const void* plan,
                                     size_t plan_bytes, void* scratch, size_t scratch_bytes, ttc_stream_t stream) {
  if (!desc) return TTC_ERR_NULL;
  if (desc->steps < 1 || desc->steps > kMaxSteps) return TTC_ERR_SHAPE;
  const float f[] = {desc->a, desc->b, desc->c, desc->eps, desc->lr, desc->mu, desc->weight_decay};
  for (float x : f)
    if (!(fabsf(x) < INFINITY)) return TTC_ERR_SHAPE;
  if (!(desc->eps > 0.f)) return TTC_ERR_SHAPE;
  size_t pb, sb;
  const ttc_status st = ttc_ortho_workspace(n, mats, &pb, &sb);
  if (st != TTC_OK) return st;
  if (n == 0) return TTC_OK;
  if (!plan || (sb && !scratch)) return TTC_ERR_NULL;
  if (((uintptr_t)plan | (uintptr_t)scratch) & 15) return TTC_ERR_ALIGN;
  if (plan_bytes < pb || scratch_bytes < sb) return TTC_ERR_WORKSPACE;
  int64_t side = 1;
  for (int64_t k = 0; k < n; ++k) side = std::max(side, std::min(mats[k].rows, mats[k].cols));
  // the three matrices, or the sums of half the waves on their way to the others
  const int sp = padded(std::min<int64_t>(side, kLdsSide)), nt = sp / 16;
  const int tiles = side > kLdsSide ? 16 : nt * (nt + 1) / 2;
  const size_t lds = sizeof(double) * std::max(3 * mat_size(sp), kWaves / 2 * tiles * 256);
  OrthoArgs a = {};
  a.mats = static_cast<const Mat*>(plan);
  a.scratch = static_cast<double*>(scratch);
  a.a = desc->a;
  a.b = desc->b;
  a.c = desc->c;
  a.eps = desc->eps;
  a.lr = desc->lr;
  a.mu = desc->mu;
  a.decay = 1.f - desc->lr * desc->weight_decay;
  a.steps = desc->steps;
  a.ahead = desc->nesterov != 0;
  hipStream_t s = (hipStream_t)stream;
  (void)hipGetLastError();
  if (lds > 65536)
    (void)hipFuncSetAttribute(reinterpret_cast<const void*>(k_ortho), hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
  TraceScope ts("ortho", s);
  TTC_LAUNCH(k_ortho, dim3((unsigned)n), dim3(kThreads), lds, s, a);
  return hipGetLastError() == hipSuccess ? TTC_OK : TTC_ERR_HIP;
}
