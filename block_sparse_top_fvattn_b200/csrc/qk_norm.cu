// Per-head RMS norm of queries and keys with the position rotation in the same pass, from the
// projections' [B, S, H, d] to the attention's [B, H, S, d], and its gradients.
//
// For one head row x of d elements, weights w and the rotation R of its token's position:
//   r = 1 / sqrt(mean(x^2) + eps),   y = R (r x w)
//   R turns the pair (a, b) by the angle t: (a cos t - b sin t, a sin t + b cos t); the pairs are
//   the elements (2i, 2i+1) (interleaved) or (i, i + rot/2); elements from rot on are not turned.
// Gradients, with g = R^T dy:
//   dw = sum over rows of g r x,   dx = r (g w) - x r^3 mean(g w x)
//
// All of it is bound by HBM: every row is read once and written once (the gradients read x and dy
// and write dx). A row is held by d / 8 neighbouring lanes, eight elements each, so one
// 16-byte load (two for fp32) per lane takes a bf16 row and the mean is a few shuffles. A CTA
// takes 16 (d = 128) or 32 (d = 64) tokens and walks over heads: the cosines and sines of a
// token are loaded once and stay in registers for all of its heads, reads of a token's heads are
// neighbours in memory, and so are the writes of neighbouring tokens of one head. kUnroll heads
// are in flight at a time. Measured: 32760 tokens, 40 + 40 heads of 128: 217 us, 97 % of the copy rate;
// 8192 tokens, 12 + 12 heads: 20 us, 79 %; with gradients, 2 x 4099 tokens, 16 + 4 heads of 64: 33 us, 50 %.
#include <cuda_bf16.h>

#include "common.cuh"
#include "qk_norm.cuh"

namespace fv {

namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;          // heads in flight per thread
constexpr int kSms = 148;
constexpr int kBadPosition = 201;   // status detail: a position outside the tables

// Eight elements as loaded, and as fp32.
template <typename T>
struct Raw8;
template <>
struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(p + 4);
  }
  __device__ __forceinline__ void to(float (&x)[8]) const {
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
};
template <>
struct Raw8<__nv_bfloat16> {
  uint4 v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void to(float (&x)[8]) const {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(u[i] << 16);
      x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
};
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&x)[8]) {
  Raw8<T> r;
  r.load(p);
  r.to(x);
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}
// The one rounding to bf16 of a result held in fp32 (to nearest even).
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    u[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}

// Sum over the LPR neighbouring lanes that hold a row.
template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The rotation of one token for the eight elements of a lane.
template <bool INTER>
struct Turn {
  float c[INTER ? 4 : 8], s[INTER ? 4 : 8];
  bool on;            // this lane's elements are turned
  int partner;        // !INTER: lane offset of the pairs' other elements
  bool first;         // !INTER: this lane holds the pairs' first elements

  __device__ __forceinline__ void load(const float* cos, const float* sin, int64_t row, int rot, int l) {
    const int half = rot >> 1;
    on = l * 8 < rot;
    partner = 0;
    first = true;
    int at = l * 4;
    if (!INTER) {
      first = l * 8 < half;
      partner = on ? (first ? half / 8 : -(half / 8)) : 0;
      at = first ? l * 8 : l * 8 - half;
    }
    constexpr int N = INTER ? 4 : 8;
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float4 cv = on ? *reinterpret_cast<const float4*>(cos + row * half + at + i) : make_float4(1, 1, 1, 1);
      const float4 sv = on ? *reinterpret_cast<const float4*>(sin + row * half + at + i) : make_float4(0, 0, 0, 0);
      c[i] = cv.x; c[i + 1] = cv.y; c[i + 2] = cv.z; c[i + 3] = cv.w;
      s[i] = sv.x; s[i + 1] = sv.y; s[i + 2] = sv.z; s[i + 3] = sv.w;
    }
  }

  // x <- R x (SIGN = 1) or R^T x (SIGN = -1). The whole warp takes part.
  template <int SIGN>
  __device__ __forceinline__ void apply(float (&x)[8], int lane) const {
    if (INTER) {
      if (!on) return;       // no shuffles here
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = x[2 * i], b = x[2 * i + 1], t = SIGN * s[i];
        x[2 * i] = a * c[i] - b * t;
        x[2 * i + 1] = a * t + b * c[i];
      }
    } else {
      const float sg = first ? -(float)SIGN : (float)SIGN;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float o = __shfl_sync(0xffffffffu, x[i], lane + partner);
        if (on) x[i] = x[i] * c[i] + sg * (o * s[i]);
      }
    }
  }
};

template <typename T>
__device__ __forceinline__ void load_weight(const void* w, int w_f32, int at, float (&x)[8]) {
  if (w == nullptr) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = 1.f;
  } else if (w_f32) {
    load8(static_cast<const float*>(w) + at, x);
  } else {
    load8(static_cast<const __nv_bfloat16*>(w) + at, x);
  }
}

// The heads [h0, h1) of one tensor that a CTA takes; chunks never mix queries and keys.
struct Chunk {
  bool key;
  int h0, h1, index;
};
__device__ __forceinline__ Chunk chunk_of(int c, int Hq, int Hk, int per) {
  const int nq = (Hq + per - 1) / per;
  Chunk r;
  r.key = c >= nq;
  r.index = r.key ? c - nq : c;
  r.h0 = r.index * per;
  r.h1 = min(r.h0 + per, r.key ? Hk : Hq);
  return r;
}

template <typename T, int D, bool INTER>
__global__ void __launch_bounds__(kThreads) qk_norm_kernel(const QkNormArgs a, const fvattn_qk_shape s, int per) {
  constexpr int LPR = D / 8, TOK = kThreads / LPR;
  const int lane = threadIdx.x & 31, l = threadIdx.x % LPR;
  const Chunk ch = chunk_of(blockIdx.y, (int)s.Hq, (int)s.Hk, per);
  const int64_t ntok = s.B * s.S;
  const int64_t t = (int64_t)blockIdx.x * TOK + threadIdx.x / LPR;
  const bool live = t < ntok;
  const int64_t tt = live ? t : 0;
  const int64_t b = tt / s.S, p = tt - b * s.S;

  const fvattn_strides xs = ch.key ? s.k : s.q, ys = ch.key ? s.ko : s.qo;
  const T* x = static_cast<const T*>(ch.key ? a.k : a.q) + b * xs.b + p * xs.s + l * 8;
  T* y = static_cast<T*>(ch.key ? a.ko : a.qo) + b * ys.b + p * ys.s + l * 8;

  Turn<INTER> turn;
  bool bad = false;
  if (s.rot > 0) {
    int64_t row = p;
    if (a.positions != nullptr) {
      row = a.positions[tt];
      bad = row < 0 || row >= s.table_rows;
      if (bad) row = 0;
    }
    turn.load(a.cos, a.sin, row, s.rot, l);
  }
  float w[8];
  load_weight<T>(ch.key ? a.wk : a.wq, s.weight_dtype == FVATTN_F32, l * 8, w);
  if (bad && live && a.status != nullptr) report_error(a.status, FVATTN_ERR_INVALID, kBadPosition);

  for (int h = ch.h0; h < ch.h1; h += kUnroll) {
    Raw8<T> raw[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (h + u < ch.h1) raw[u].load(x + (int64_t)(h + u) * xs.h);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (h + u >= ch.h1) break;          // the same for the whole CTA
      float v[8];
      raw[u].to(v);
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss += v[i] * v[i];
      const float r = rsqrtf(row_sum<LPR>(ss) * (1.f / D) + s.eps);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = v[i] * r * w[i];
      if (s.rot > 0) turn.template apply<1>(v, lane);
      if (bad) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __int_as_float(0x7fffffff);   // a position outside the tables: NaN
      }
      if (live) store8(y + (int64_t)(h + u) * ys.h, v);
    }
  }
}

template <typename T, int D, bool INTER>
__global__ void __launch_bounds__(kThreads) qk_norm_bwd_kernel(const QkNormArgs a, const fvattn_qk_shape s, int per,
                                                               int walk) {
  constexpr int LPR = D / 8, TOK = kThreads / LPR, U = 4;
  __shared__ float sw[TOK][D];
  allow_next_grid();
  const int lane = threadIdx.x & 31, l = threadIdx.x % LPR, grp = threadIdx.x / LPR;
  const Chunk ch = chunk_of(blockIdx.y, (int)s.Hq, (int)s.Hk, per);
  const int64_t ntok = s.B * s.S;
  const fvattn_strides xs = ch.key ? s.k : s.q, gs = ch.key ? s.ko : s.qo, ds = ch.key ? s.dk : s.dq;
  float w[8], dw[8];
  load_weight<T>(ch.key ? a.wk : a.wq, s.weight_dtype == FVATTN_F32, l * 8, w);
#pragma unroll
  for (int i = 0; i < 8; ++i) dw[i] = 0.f;

  const int64_t t1 = (int64_t)(blockIdx.x + 1) * walk * TOK;
  for (int64_t t0 = (int64_t)blockIdx.x * walk * TOK; t0 < t1 && t0 < ntok; t0 += TOK) {
    const int64_t t = t0 + grp;
    const bool live = t < ntok;
    const int64_t tt = live ? t : 0;
    const int64_t b = tt / s.S, p = tt - b * s.S;
    const T* x = static_cast<const T*>(ch.key ? a.k : a.q) + b * xs.b + p * xs.s + l * 8;
    const T* gy = static_cast<const T*>(ch.key ? a.gk : a.gq) + b * gs.b + p * gs.s + l * 8;
    T* dx = static_cast<T*>(ch.key ? a.ko : a.qo) + b * ds.b + p * ds.s + l * 8;
    Turn<INTER> turn;
    bool bad = false;
    if (s.rot > 0) {
      int64_t row = p;
      if (a.positions != nullptr) {
        row = a.positions[tt];
        bad = row < 0 || row >= s.table_rows;
        if (bad) row = 0;
      }
      turn.load(a.cos, a.sin, row, s.rot, l);
    }
    if (bad && live && a.status != nullptr) report_error(a.status, FVATTN_ERR_INVALID, kBadPosition);
    for (int h = ch.h0; h < ch.h1; h += U) {
      Raw8<T> rx[U], rg[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (h + u >= ch.h1) break;        // the same for the whole CTA
        rx[u].load(x + (int64_t)(h + u) * xs.h);
        rg[u].load(gy + (int64_t)(h + u) * gs.h);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (h + u >= ch.h1) break;
        float v[8], g[8];
        rx[u].to(v);
        rg[u].to(g);
        if (s.rot > 0) turn.template apply<-1>(g, lane);
        float ss = 0.f, sg = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          ss += v[i] * v[i];
          sg += g[i] * w[i] * v[i];
        }
        const float r = rsqrtf(row_sum<LPR>(ss) * (1.f / D) + s.eps);
        const float m = row_sum<LPR>(sg) * (1.f / D) * r * r;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (bad) g[i] = __int_as_float(0x7fffffff);
          if (live) dw[i] += g[i] * (v[i] * r);
          v[i] = r * (g[i] * w[i] - v[i] * m);
        }
        if (live) store8(dx + (int64_t)(h + u) * ds.h, v);
      }
    }
  }
  float* dwo = ch.key ? a.dwk : a.dwq;
  if (dwo == nullptr) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) sw[grp][l * 8 + i] = dw[i];
  __syncthreads();
  // parts: the queries' CTAs first, then the keys', one row of D sums each, in a fixed order
  const int nq = ((int)s.Hq + per - 1) / per;
  const int64_t row = (int64_t)(ch.key ? nq + ch.index : ch.index) * gridDim.x + blockIdx.x;
  for (int c = threadIdx.x; c < D; c += kThreads) {
    float acc = 0.f;
#pragma unroll 4
    for (int k = 0; k < TOK; ++k) acc += sw[k][c];
    a.parts[row * D + c] = acc;
  }
}

// dw[c] = sum over the parts of column c, in 64 bits and in a fixed order. blockIdx.y: queries, keys.
constexpr int kSumThreads = 1024;
__global__ void __launch_bounds__(kSumThreads) qk_norm_sum_kernel(const QkNormArgs a, int D, int64_t parts_q,
                                                                  int64_t parts_k) {
  __shared__ double ss[kSumThreads / 8][8];
  wait_for_previous_grid();
  const int col = blockIdx.x * 8 + (threadIdx.x & 7), k = threadIdx.x >> 3;
  const bool key = blockIdx.y == 1;
  float* out = key ? a.dwk : a.dwq;
  if (out == nullptr) return;
  const float* p = a.parts + (key ? parts_q * D : 0) + col;
  const int64_t n = key ? parts_k : parts_q;
  double acc = 0.0;
#pragma unroll 4
  for (int64_t r = k; r < n; r += kSumThreads / 8) acc += (double)p[r * D];
  ss[k][threadIdx.x & 7] = acc;
  for (int half = kSumThreads / 16; half > 0; half >>= 1) {
    __syncthreads();
    if (k < half) ss[k][threadIdx.x & 7] += ss[k + half][threadIdx.x & 7];
  }
  if (k == 0) out[col] = (float)ss[0][threadIdx.x & 7];
}

// Heads per CTA: all of a tensor's heads when the token tiles alone make several CTAs for every SM (a
// token's cosines and sines are then loaded once for all), in groups of kUnroll fewer otherwise.
int heads_per_cta(const fvattn_qk_shape& s, int64_t tiles) {
  const int64_t want = (int64_t)kSms * 8;
  int per = (int)((imax(s.Hq, s.Hk) + kUnroll - 1) / kUnroll) * kUnroll;
  while (per > kUnroll && tiles * ((s.Hq + per - 1) / per + (s.Hk + per - 1) / per) < want) per -= kUnroll;
  return per;
}

int64_t tok_tiles(const fvattn_qk_shape& s) {
  const int tok = kThreads / (int)(s.d / 8);
  return (s.B * s.S + tok - 1) / tok;
}

// The gradients' CTAs: groups of 4 kUnroll heads, and of `walk` token tiles so that the partial sums of
// the weights' gradients stay few. Fewer heads to a CTA took the gradients of 2 x 4099 tokens, 16 + 4
// heads of 64, from 18 to 21 us.
struct BwdPlan {
  int per, walk, gx;
  int64_t parts_q, parts_k;
};
BwdPlan bwd_plan(const fvattn_qk_shape& s) {
  BwdPlan p;
  const int64_t tiles = tok_tiles(s);
  p.per = 4 * kUnroll;
  while (p.per > 1 && tiles * ((s.Hq + p.per - 1) / p.per + (s.Hk + p.per - 1) / p.per) < (int64_t)kSms * 2) p.per >>= 1;
  const int64_t nq = (s.Hq + p.per - 1) / p.per, nk = (s.Hk + p.per - 1) / p.per;
  p.walk = (int)imax<int64_t>(1, tiles * (nq + nk) / ((int64_t)kSms * 32));
  p.gx = (int)((tiles + p.walk - 1) / p.walk);
  p.parts_q = nq * p.gx;
  p.parts_k = nk * p.gx;
  return p;
}

template <typename T, int D>
cudaError_t fwd_d(const QkNormArgs& a, const fvattn_qk_shape& s, cudaStream_t st) {
  const int64_t tiles = tok_tiles(s);
  const int per = heads_per_cta(s, tiles);
  const dim3 grid((unsigned)tiles, (unsigned)((s.Hq + per - 1) / per + (s.Hk + per - 1) / per));
  if (s.interleaved)
    qk_norm_kernel<T, D, true><<<grid, kThreads, 0, st>>>(a, s, per);
  else
    qk_norm_kernel<T, D, false><<<grid, kThreads, 0, st>>>(a, s, per);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t bwd_d(const QkNormArgs& a, const fvattn_qk_shape& s, cudaStream_t st) {
  const BwdPlan p = bwd_plan(s);
  const dim3 grid((unsigned)p.gx, (unsigned)((p.parts_q + p.parts_k) / p.gx));
  if (s.interleaved)
    qk_norm_bwd_kernel<T, D, true><<<grid, kThreads, 0, st>>>(a, s, p.per, p.walk);
  else
    qk_norm_bwd_kernel<T, D, false><<<grid, kThreads, 0, st>>>(a, s, p.per, p.walk);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || (a.dwq == nullptr && a.dwk == nullptr)) return e;
  return launch_with(qk_norm_sum_kernel, dim3(D / 8, 2), kSumThreads, 0, st, 0, true, a, D, p.parts_q, p.parts_k);
}

}  // namespace

size_t qk_norm_part_bytes(const fvattn_qk_shape& s) {
  const BwdPlan p = bwd_plan(s);
  return (size_t)(p.parts_q + p.parts_k) * (size_t)s.d * sizeof(float);
}

cudaError_t launch_qk_norm(const QkNormArgs& a, const fvattn_qk_shape& s, cudaStream_t st) {
  if (s.dtype == FVATTN_F32) return s.d == 128 ? fwd_d<float, 128>(a, s, st) : fwd_d<float, 64>(a, s, st);
  return s.d == 128 ? fwd_d<__nv_bfloat16, 128>(a, s, st) : fwd_d<__nv_bfloat16, 64>(a, s, st);
}

cudaError_t launch_qk_norm_bwd(const QkNormArgs& a, const fvattn_qk_shape& s, cudaStream_t st) {
  if (s.dtype == FVATTN_F32) return s.d == 128 ? bwd_d<float, 128>(a, s, st) : bwd_d<float, 64>(a, s, st);
  return s.d == 128 ? bwd_d<__nv_bfloat16, 128>(a, s, st) : bwd_d<__nv_bfloat16, 64>(a, s, st);
}

}  // namespace fv
