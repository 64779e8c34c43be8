// Attention over a sliding window whose first keys stay visible, for gfx950.
//
// With p = i + (lk - lq) the place of query i among its sequence's keys, key j
// is seen if j <= p + right and (j >= p - left or j < sinks), and
//   o_i = sum_j P_ij v_j,  P_ij = exp(s_ij - lse_i),  s_ij = scale q_i . k_j,
//   lse_i = log sum_j exp(s_ij), sums over the keys that i sees.
// Backward, with delta_i = do_i . o_i and dP_ij = do_i . v_j:
//   dS = P (dP - delta),  dq_i = scale sum_j dS_ij k_j,
//   dk_j = scale sum_i dS_ij q_i,  dv_j = sum_i P_ij do_i.
// Scores are kept in base 2 (scale times log2 e), statistics in fp32.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/ttc_block.h"
#include "ttc_device.hpp"
#include "ttc_trace.hpp"

namespace ttc {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kMaxDim = 128;
constexpr int kMaxHeads = 4096;
constexpr int64_t kMaxTokens = 1 << 28;  // p +- (a window side) stays in 32 bits
constexpr int kNoLimit = 1 << 30;
constexpr int kThreads = 256;
constexpr int64_t kMaxGroups = 1 << 23;

struct AttnArgs {
  const void* q;
  const void* k;
  const void* v;
  const void* o_in;  // backward: the forward's o
  const void* d_o;
  const int32_t* q_off;  // null: every sequence has tq / batch rows
  const int32_t* k_off;
  void* o;
  void* dq;
  void* dk;
  void* dv;
  float* lse;
  float* delta;
  int64_t tq, tk;
  int batch, heads, kv_heads, dim;
  int left, right, sinks;
  float scale, scale2;  // scale2 = scale log2 e
  int tiles;            // tiles of a sequence's rows that the grid has
};

// rows [start, start + len) of sequence b; offsets that do not ascend or pass
// the end are cut, so that no row outside the buffers is touched
struct Span {
  int64_t start;
  int len;
};
__device__ __forceinline__ Span span_of(const int32_t* off, int b, int batch, int64_t t) {
  if (!off) {
    const int len = (int)(t / batch);
    return {(int64_t)b * len, len};
  }
  const int64_t s = min(max((int64_t)off[b], (int64_t)0), t), e = min(max((int64_t)off[b + 1], s), t);
  return {s, (int)(e - s)};
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) v += __shfl_xor(v, m);
  return v;
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) v = fmaxf(v, __shfl_xor(v, m));
  return v;
}
__device__ __forceinline__ float lane_value(float v, int lane) {
  return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), lane));
}

template <typename T>
__device__ __forceinline__ float dot_row(const typename Elem<T>::type* a, const typename Elem<T>::type* b, int dim) {
  typedef typename Mma<T>::frag frag;
  float s = 0.f;
  for (int d = 0; d < dim; d += Mma<T>::EPV) {
    const frag x = *reinterpret_cast<const frag*>(a + d), y = *reinterpret_cast<const frag*>(b + d);
#pragma unroll
    for (int e = 0; e < Mma<T>::EPV; ++e) s += elem_to_f32<T>(x[e]) * elem_to_f32<T>(y[e]);
  }
  return s;
}

// A row at a time, by one wave: the lanes take 64 keys (or queries) for the
// scores, then two of the row's elements each for the products.  Only rows
// that are seen are ever multiplied, so a NaN or an infinity that a row does
// not see cannot reach it.

// o of one query at place p: acc[e] is element lane + 64 e
template <typename T>
__device__ void row_fwd(const AttnArgs& a, const typename Elem<T>::type* q, const typename Elem<T>::type* k,
                        const typename Elem<T>::type* v, int64_t ldk, int p, int lk, float (&acc)[2], float& lse) {
  const int lane = threadIdx.x & 63;
  float m = -INFINITY, l = 0.f;
  acc[0] = acc[1] = 0.f;
  const int end = min(lk, p + a.right + 1), lo = max(0, p - a.left);
  for (int part = 0; part < 2; ++part) {
    const int j1 = part ? end : min(min(a.sinks, lo), end);
    for (int j0 = part ? lo : 0; j0 < j1; j0 += 64) {
      const int n = min(64, j1 - j0);
      const float s = lane < n ? a.scale2 * dot_row<T>(q, k + (j0 + lane) * ldk, a.dim) : -INFINITY;
      const float mn = fmaxf(m, wave_max(s));
      const float keep = m == -INFINITY ? 0.f : exp2f(m - mn);
      const float e = s == -INFINITY ? 0.f : exp2f(s - mn);
      m = mn;
      l = l * keep + wave_sum(e);
      acc[0] *= keep;
      acc[1] *= keep;
      for (int j = 0; j < n; ++j) {
        const float w = lane_value(e, j);
        const typename Elem<T>::type* r = v + (j0 + j) * ldk;
        if (lane < a.dim) acc[0] += w * elem_to_f32<T>(r[lane]);
        if (lane + 64 < a.dim) acc[1] += w * elem_to_f32<T>(r[lane + 64]);
      }
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  acc[0] *= inv;
  acc[1] *= inv;
  // a row that sees nothing weighs nothing in the backward
  lse = l == 0.f ? INFINITY : m + log2f(l);
}

template <typename T>
__device__ __forceinline__ void row_store(typename Elem<T>::type* o, const float (&acc)[2], int dim) {
  const int lane = threadIdx.x & 63;
  if (lane < dim) o[lane] = Mma<T>::from_f32(acc[0]);
  if (lane + 64 < dim) o[lane + 64] = Mma<T>::from_f32(acc[1]);
}

// dq of one query at place p
template <typename T>
__device__ void row_dq(const AttnArgs& a, const typename Elem<T>::type* q, const typename Elem<T>::type* d_o,
                       const typename Elem<T>::type* k, const typename Elem<T>::type* v, int64_t ldk, int p, int lk,
                       float lse, float delta, float (&acc)[2]) {
  const int lane = threadIdx.x & 63;
  acc[0] = acc[1] = 0.f;
  const int end = min(lk, p + a.right + 1), lo = max(0, p - a.left);
  for (int part = 0; part < 2; ++part) {
    const int j1 = part ? end : min(min(a.sinks, lo), end);
    for (int j0 = part ? lo : 0; j0 < j1; j0 += 64) {
      const int n = min(64, j1 - j0);
      float ds = 0.f;
      if (lane < n) {
        const float s = a.scale2 * dot_row<T>(q, k + (j0 + lane) * ldk, a.dim);
        ds = exp2f(s - lse) * (dot_row<T>(d_o, v + (j0 + lane) * ldk, a.dim) - delta) * a.scale;
      }
      for (int j = 0; j < n; ++j) {
        const float w = lane_value(ds, j);
        const typename Elem<T>::type* r = k + (j0 + j) * ldk;
        if (lane < a.dim) acc[0] += w * elem_to_f32<T>(r[lane]);
        if (lane + 64 < a.dim) acc[1] += w * elem_to_f32<T>(r[lane + 64]);
      }
    }
  }
}

// what one query head adds to dk and dv of key j; q, d_o, lse, delta from the
// sequence's first row on
template <typename T>
__device__ void row_dkv(const AttnArgs& a, const typename Elem<T>::type* q, const typename Elem<T>::type* d_o,
                        const float* lse, const float* delta, int64_t ldq, const typename Elem<T>::type* k,
                        const typename Elem<T>::type* v, int j, int lq, int lk, float (&dk)[2], float (&dv)[2]) {
  const int lane = threadIdx.x & 63;
  const int shift = lk - lq;
  const int i_end = j < a.sinks ? lq : min(lq, j + a.left - shift + 1);
  for (int i0 = max(0, j - a.right - shift); i0 < i_end; i0 += 64) {
    const int n = min(64, i_end - i0);
    float ds = 0.f, e = 0.f;
    if (lane < n) {
      const int64_t i = i0 + lane;
      e = exp2f(a.scale2 * dot_row<T>(q + i * ldq, k, a.dim) - lse[i * a.heads]);
      ds = e * (dot_row<T>(d_o + i * ldq, v, a.dim) - delta[i * a.heads]) * a.scale;
    }
    for (int i = 0; i < n; ++i) {
      const float ws = lane_value(ds, i), we = lane_value(e, i);
      const typename Elem<T>::type *rq = q + (i0 + i) * ldq, *rd = d_o + (i0 + i) * ldq;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int c = lane + 64 * x;
        if (c < a.dim) {
          dk[x] += ws * elem_to_f32<T>(rq[c]);
          dv[x] += we * elem_to_f32<T>(rd[c]);
        }
      }
    }
  }
}

// work-group -> (tile, head of `heads`, sequence); the tiles of one head follow each other
struct Place {
  int tile, head, b;
};
__device__ __forceinline__ Place place_of(const AttnArgs& a, int heads) {
  const int g = blockIdx.x, r = g / a.tiles;
  return {g - r * a.tiles, r % heads, r / heads};
}

constexpr int kRows = kThreads / 64;

template <typename T>
__global__ __launch_bounds__(kThreads) void k_attn_fwd(AttnArgs a) {
  typedef typename Elem<T>::type E;
  const Place w = place_of(a, a.heads);
  const Span sq = span_of(a.q_off, w.b, a.batch, a.tq), sk = span_of(a.k_off, w.b, a.batch, a.tk);
  const int64_t ldq = (int64_t)a.heads * a.dim, ldk = (int64_t)a.kv_heads * a.dim;
  const int hk = w.head / (a.heads / a.kv_heads);
  const E* k = static_cast<const E*>(a.k) + sk.start * ldk + (int64_t)hk * a.dim;
  const E* v = static_cast<const E*>(a.v) + sk.start * ldk + (int64_t)hk * a.dim;
  for (int64_t t = w.tile; t * kRows < sq.len; t += a.tiles) {
    const int i = (int)t * kRows + threadIdx.x / 64;
    if (i >= sq.len) continue;
    const int64_t at = (sq.start + i) * ldq + (int64_t)w.head * a.dim;
    float acc[2], lse;
    row_fwd<T>(a, static_cast<const E*>(a.q) + at, k, v, ldk, i + sk.len - sq.len, sk.len, acc, lse);
    row_store<T>(static_cast<E*>(a.o) + at, acc, a.dim);
    if ((threadIdx.x & 63) == 0) a.lse[(sq.start + i) * a.heads + w.head] = lse;
  }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void k_attn_dq(AttnArgs a) {
  typedef typename Elem<T>::type E;
  const Place w = place_of(a, a.heads);
  const Span sq = span_of(a.q_off, w.b, a.batch, a.tq), sk = span_of(a.k_off, w.b, a.batch, a.tk);
  const int64_t ldq = (int64_t)a.heads * a.dim, ldk = (int64_t)a.kv_heads * a.dim;
  const int hk = w.head / (a.heads / a.kv_heads), lane = threadIdx.x & 63;
  const E* k = static_cast<const E*>(a.k) + sk.start * ldk + (int64_t)hk * a.dim;
  const E* v = static_cast<const E*>(a.v) + sk.start * ldk + (int64_t)hk * a.dim;
  for (int64_t t = w.tile; t * kRows < sq.len; t += a.tiles) {
    const int i = (int)t * kRows + threadIdx.x / 64;
    if (i >= sq.len) continue;
    const int64_t at = (sq.start + i) * ldq + (int64_t)w.head * a.dim;
    const E *d_o = static_cast<const E*>(a.d_o) + at, *o = static_cast<const E*>(a.o_in) + at;
    float s = 0.f;
    for (int c = lane; c < a.dim; c += 64) s += elem_to_f32<T>(d_o[c]) * elem_to_f32<T>(o[c]);
    const float delta = wave_sum(s);
    const int64_t st = (sq.start + i) * a.heads + w.head;
    float acc[2];
    row_dq<T>(a, static_cast<const E*>(a.q) + at, d_o, k, v, ldk, i + sk.len - sq.len, sk.len, a.lse[st], delta, acc);
    row_store<T>(static_cast<E*>(a.dq) + at, acc, a.dim);
    if (lane == 0) a.delta[st] = delta;
  }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void k_attn_dkv(AttnArgs a) {
  typedef typename Elem<T>::type E;
  const Place w = place_of(a, a.kv_heads);
  const Span sq = span_of(a.q_off, w.b, a.batch, a.tq), sk = span_of(a.k_off, w.b, a.batch, a.tk);
  const int64_t ldq = (int64_t)a.heads * a.dim, ldk = (int64_t)a.kv_heads * a.dim;
  const int group = a.heads / a.kv_heads;
  for (int64_t t = w.tile; t * kRows < sk.len; t += a.tiles) {
    const int j = (int)t * kRows + threadIdx.x / 64;
    if (j >= sk.len) continue;
    const int64_t at = (sk.start + j) * ldk + (int64_t)w.head * a.dim;
    float dk[2] = {0.f, 0.f}, dv[2] = {0.f, 0.f};
    for (int g = 0; g < group; ++g) {
      const int64_t h = (int64_t)w.head * group + g, row = sq.start * ldq + h * a.dim, st = sq.start * a.heads + h;
      row_dkv<T>(a, static_cast<const E*>(a.q) + row, static_cast<const E*>(a.d_o) + row, a.lse + st, a.delta + st, ldq,
                 static_cast<const E*>(a.k) + at, static_cast<const E*>(a.v) + at, j, sq.len, sk.len, dk, dv);
    }
    row_store<T>(static_cast<E*>(a.dk) + at, dk, a.dim);
    row_store<T>(static_cast<E*>(a.dv) + at, dv, a.dim);
  }
}

struct DecodeArgs {
  AttnArgs a;
  const int32_t* lens;
  int64_t capacity;
};

template <typename T>
__global__ __launch_bounds__(64) void k_attn_decode(DecodeArgs d) {
  typedef typename Elem<T>::type E;
  const AttnArgs& a = d.a;
  const int b = blockIdx.x / a.heads, h = blockIdx.x % a.heads;
  const int n = (int)min(max((int64_t)d.lens[b], (int64_t)0), d.capacity);
  const int64_t ldk = (int64_t)a.kv_heads * a.dim;
  const int64_t at = ((int64_t)b * a.heads + h) * a.dim;
  const int64_t kv = b * d.capacity * ldk + (int64_t)(h / (a.heads / a.kv_heads)) * a.dim;
  float acc[2], lse;
  row_fwd<T>(a, static_cast<const E*>(a.q) + at, static_cast<const E*>(a.k) + kv, static_cast<const E*>(a.v) + kv, ldk,
             n - 1, n, acc, lse);
  row_store<T>(static_cast<E*>(a.o) + at, acc, a.dim);
}

// ---- host --------------------------------------------------------------------

ttc_status check(const ttc_attn_desc* d) {
  if (!d) return TTC_ERR_NULL;
  if (d->heads < 1 || d->kv_heads < 1 || d->heads > kMaxHeads || d->heads % d->kv_heads) return TTC_ERR_SHAPE;
  if (d->dim < 8 || d->dim > kMaxDim || d->dim % 8) return TTC_ERR_SHAPE;
  if (d->sinks < 0) return TTC_ERR_SHAPE;
  if (!(d->scale > -INFINITY && d->scale < INFINITY)) return TTC_ERR_SHAPE;
  if (d->dtype != TTC_F32 && d->dtype != TTC_BF16) return TTC_ERR_DTYPE;
  return TTC_OK;
}

ttc_status check_seqs(const ttc_attn_desc* d, const ttc_attn_seqs* s) {
  const ttc_status st = check(d);
  if (st != TTC_OK) return st;
  if (!s) return TTC_ERR_NULL;
  if (s->batch < 1 || s->tq < 0 || s->tk < 0 || s->tq > kMaxTokens || s->tk > kMaxTokens) return TTC_ERR_SHAPE;
  if (s->max_q < 0 || s->max_k < 0) return TTC_ERR_SHAPE;
  if (!s->q_offsets != !s->k_offsets) return TTC_ERR_NULL;
  if (!s->q_offsets && (s->tq % s->batch || s->tk % s->batch)) return TTC_ERR_SHAPE;
  if ((int64_t)s->batch * d->heads > kMaxGroups) return TTC_ERR_UNSUPPORTED;
  return TTC_OK;
}

bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
size_t stat_bytes(const ttc_attn_desc* d, const ttc_attn_seqs* s) {
  return ((size_t)s->tq * d->heads * sizeof(float) + 15) & ~(size_t)15;
}

AttnArgs make_args(const ttc_attn_desc* d) {
  AttnArgs a = {};
  a.heads = d->heads;
  a.kv_heads = d->kv_heads;
  a.dim = d->dim;
  a.left = d->left < 0 || d->left > kNoLimit ? kNoLimit : d->left;
  a.right = d->right < 0 || d->right > kNoLimit ? kNoLimit : d->right;
  a.sinks = d->sinks;
  a.scale = d->scale;
  a.scale2 = d->scale * kLog2e;
  return a;
}
AttnArgs make_args(const ttc_attn_desc* d, const ttc_attn_seqs* s) {
  AttnArgs a = make_args(d);
  a.q_off = s->q_offsets;
  a.k_off = s->k_offsets;
  a.tq = s->tq;
  a.tk = s->tk;
  a.batch = s->batch;
  return a;
}

// work-groups for tiles of `rows` rows of sequences of at most `longest` rows
// (of `t` rows together), for each of `heads` heads; a work-group takes more
// tiles where the grid has too few
unsigned grid_of(AttnArgs& a, int64_t longest, int64_t t, int rows, int heads) {
  const int64_t most = a.q_off ? (longest < 1 || longest > t ? t : longest) : t / a.batch;
  int64_t tiles = (most + rows - 1) / rows;
  const int64_t cap = kMaxGroups / ((int64_t)a.batch * heads);
  tiles = tiles < 1 ? 1 : tiles > cap ? cap : tiles;
  a.tiles = (int)tiles;
  return (unsigned)(tiles * a.batch * heads);
}

ttc_status launched() { return hipGetLastError() == hipSuccess ? TTC_OK : TTC_ERR_HIP; }

}  // namespace
}  // namespace ttc

using namespace ttc;

extern "C" ttc_status ttc_attn_workspace(const ttc_attn_desc* desc, const ttc_attn_seqs* seqs, size_t* saved_bytes,
                                         size_t* scratch_bytes) {
  if (!saved_bytes || !scratch_bytes) return TTC_ERR_NULL;
  const ttc_status st = check_seqs(desc, seqs);
  if (st != TTC_OK) return st;
  *saved_bytes = stat_bytes(desc, seqs);
  *scratch_bytes = stat_bytes(desc, seqs);
  return TTC_OK;
}

extern "C" ttc_status ttc_attn_fwd(const ttc_attn_desc* desc, const ttc_attn_seqs* seqs, const void* q, const void* k,
                                   const void* v, void* o, void* saved, size_t saved_bytes, ttc_stream_t stream) {
  const ttc_status st = check_seqs(desc, seqs);
  if (st != TTC_OK) return st;
  if (seqs->tq == 0) return TTC_OK;
  if (!q || !o || !saved || (seqs->tk > 0 && (!k || !v))) return TTC_ERR_NULL;
  if (!al16(q) || !al16(k) || !al16(v) || !al16(o) || !al16(saved)) return TTC_ERR_ALIGN;
  if (saved_bytes < stat_bytes(desc, seqs)) return TTC_ERR_WORKSPACE;
  AttnArgs a = make_args(desc, seqs);
  a.q = q;
  a.k = k;
  a.v = v;
  a.o = o;
  a.lse = static_cast<float*>(saved);
  hipStream_t s = (hipStream_t)stream;
  (void)hipGetLastError();
  const unsigned grid = grid_of(a, seqs->max_q, a.tq, kRows, a.heads);
  TraceScope ts("attn_fwd", s);
  auto kern = desc->dtype == TTC_F32 ? k_attn_fwd<float> : k_attn_fwd<bf16_t>;
  TTC_LAUNCH(kern, dim3(grid), dim3(kThreads), 0, s, a);
  return launched();
}

extern "C" ttc_status ttc_attn_bwd(const ttc_attn_desc* desc, const ttc_attn_seqs* seqs, const void* q, const void* k,
                                   const void* v, const void* o, const void* d_o, const void* saved,
                                   size_t saved_bytes, void* dq, void* dk, void* dv, void* scratch,
                                   size_t scratch_bytes, ttc_stream_t stream) {
  const ttc_status st = check_seqs(desc, seqs);
  if (st != TTC_OK) return st;
  if (seqs->tq > 0) {
    if (!q || !o || !d_o || !saved || !dq || !scratch) return TTC_ERR_NULL;
    if (!al16(q) || !al16(o) || !al16(d_o) || !al16(saved) || !al16(dq) || !al16(scratch)) return TTC_ERR_ALIGN;
    if (saved_bytes < stat_bytes(desc, seqs) || scratch_bytes < stat_bytes(desc, seqs)) return TTC_ERR_WORKSPACE;
  }
  if (seqs->tk > 0) {
    if (!k || !v || !dk || !dv) return TTC_ERR_NULL;
    if (!al16(k) || !al16(v) || !al16(dk) || !al16(dv)) return TTC_ERR_ALIGN;
  }
  if (seqs->tq == 0 && seqs->tk == 0) return TTC_OK;
  AttnArgs a = make_args(desc, seqs);
  a.q = q;
  a.k = k;
  a.v = v;
  a.o_in = o;
  a.d_o = d_o;
  a.lse = static_cast<float*>(const_cast<void*>(saved));
  a.delta = static_cast<float*>(scratch);
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  hipStream_t s = (hipStream_t)stream;
  (void)hipGetLastError();
  if (a.tq > 0) {
    const unsigned grid = grid_of(a, seqs->max_q, a.tq, kRows, a.heads);
    TraceScope ts("attn_dq", s);
    auto kern = desc->dtype == TTC_F32 ? k_attn_dq<float> : k_attn_dq<bf16_t>;
    TTC_LAUNCH(kern, dim3(grid), dim3(kThreads), 0, s, a);
  }
  if (a.tk > 0) {
    const unsigned grid = grid_of(a, seqs->max_k, a.tk, kRows, a.kv_heads);
    TraceScope ts("attn_dkv", s);
    auto kern = desc->dtype == TTC_F32 ? k_attn_dkv<float> : k_attn_dkv<bf16_t>;
    TTC_LAUNCH(kern, dim3(grid), dim3(kThreads), 0, s, a);
  }
  return launched();
}

namespace {
ttc_status check_decode(const ttc_attn_desc* d, int64_t batch, int64_t capacity) {
  const ttc_status st = check(d);
  if (st != TTC_OK) return st;
  if (batch < 0 || capacity < 0 || capacity > kMaxTokens) return TTC_ERR_SHAPE;
  if (batch * d->heads > kMaxGroups) return TTC_ERR_UNSUPPORTED;
  return TTC_OK;
}
}  // namespace

extern "C" ttc_status ttc_attn_decode_workspace(const ttc_attn_desc* desc, int64_t batch, int64_t capacity,
                                                size_t* scratch_bytes) {
  if (!scratch_bytes) return TTC_ERR_NULL;
  const ttc_status st = check_decode(desc, batch, capacity);
  if (st != TTC_OK) return st;
  *scratch_bytes = 0;
  return TTC_OK;
}

extern "C" ttc_status ttc_attn_decode(const ttc_attn_desc* desc, int64_t batch, int64_t capacity, const void* q,
                                      const void* k, const void* v, const int32_t* lens, void* o, void* scratch,
                                      size_t scratch_bytes, ttc_stream_t stream) {
  const ttc_status st = check_decode(desc, batch, capacity);
  if (st != TTC_OK) return st;
  if (batch == 0) return TTC_OK;
  if (!q || !lens || !o || (capacity > 0 && (!k || !v))) return TTC_ERR_NULL;
  if (!al16(q) || !al16(k) || !al16(v) || !al16(lens) || !al16(o) || !al16(scratch)) return TTC_ERR_ALIGN;
  (void)scratch_bytes;
  DecodeArgs d = {make_args(desc), lens, capacity};
  d.a.q = q;
  d.a.k = k;
  d.a.v = v;
  d.a.o = o;
  hipStream_t s = (hipStream_t)stream;
  (void)hipGetLastError();
  TraceScope ts("attn_decode", s);
  auto kern = desc->dtype == TTC_F32 ? k_attn_decode<float> : k_attn_decode<bf16_t>;
  TTC_LAUNCH(kern, dim3((unsigned)(batch * desc->heads)), dim3(64), 0, s, d);
  return launched();
}
