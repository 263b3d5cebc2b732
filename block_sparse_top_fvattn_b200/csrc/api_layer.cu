// Host side of the operators around the routed attention: the norm and rotation of queries and
// keys, and attention over all keys. Argument validation, workspace layout and launch sequences.
#include <math.h>

#include "common.cuh"
#include "dense.cuh"
#include "qk_norm.cuh"

using namespace fv;

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Strides of a tensor with dims b, h, s and a contiguous last dimension: positive and multiples of
// 16 bytes where the dimension is larger than one (the others are not read; see canonical()).
bool valid_strides(const fvattn_strides& t, int64_t B, int64_t H, int64_t S, int dtype) {
  const int64_t q = dtype == FVATTN_F32 ? 4 : 8;
  const int64_t most = (int64_t)1 << 38;         // 2^40 bytes: what a tensor map can hold
  auto ok = [&](int64_t n, int64_t st) { return n == 1 || (st > 0 && st % q == 0 && st < most); };
  return ok(B, t.b) && ok(H, t.h) && ok(S, t.s);
}

// A stride that is not read, as a value every user of the strides accepts.
fvattn_strides canonical(fvattn_strides t, int64_t B, int64_t H, int64_t S, int64_t d) {
  if (B == 1) t.b = d;
  if (H == 1) t.h = d;
  if (S == 1) t.s = d;
  return t;
}

int validate_qk(const fvattn_qk_shape* s, bool bwd) {
  if (s == nullptr) return FVATTN_ERR_INVALID;
  if (s->B < 1 || s->S < 1 || s->Hq < 1 || s->Hk < 1 || s->d < 1) return FVATTN_ERR_INVALID;
  if (s->dtype != FVATTN_BF16 && s->dtype != FVATTN_F32) return FVATTN_ERR_INVALID;
  if (s->weight_dtype != FVATTN_BF16 && s->weight_dtype != FVATTN_F32) return FVATTN_ERR_INVALID;
  if (s->interleaved != 0 && s->interleaved != 1) return FVATTN_ERR_INVALID;
  if (!(s->eps >= 0.f) || isinf(s->eps)) return FVATTN_ERR_INVALID;
  if (s->rot < 0 || s->rot > s->d) return FVATTN_ERR_INVALID;
  if (s->d != 64 && s->d != 128) return FVATTN_ERR_UNSUPPORTED;
  if (s->rot % 16 != 0) return FVATTN_ERR_UNSUPPORTED;
  if (s->Hq > 65535 / 2 || s->Hk > 65535 / 2) return FVATTN_ERR_UNSUPPORTED;
  if (s->S > (int64_t)1 << 30 || s->B > (int64_t)1 << 30 || s->B * s->S > (int64_t)1 << 31)
    return FVATTN_ERR_UNSUPPORTED;
  if (s->rot > 0 && s->table_rows < 1) return FVATTN_ERR_INVALID;
  if (!valid_strides(s->q, s->B, s->Hq, s->S, s->dtype) || !valid_strides(s->k, s->B, s->Hk, s->S, s->dtype) ||
      !valid_strides(s->qo, s->B, s->Hq, s->S, s->dtype) || !valid_strides(s->ko, s->B, s->Hk, s->S, s->dtype))
    return FVATTN_ERR_INVALID;
  if (bwd && (!valid_strides(s->dq, s->B, s->Hq, s->S, s->dtype) || !valid_strides(s->dk, s->B, s->Hk, s->S, s->dtype)))
    return FVATTN_ERR_INVALID;
  return FVATTN_OK;
}

int check_qk_tables(const fvattn_qk_shape* s, const void* wq, const void* wk, const float* cos, const float* sin,
                    const int32_t* positions, const int32_t* status) {
  if (!aligned(wq, 16) || !aligned(wk, 16) || !aligned(positions, 4) || !aligned(status, 4)) return FVATTN_ERR_INVALID;
  if (s->rot > 0) {
    if (cos == nullptr || sin == nullptr || !aligned(cos, 16) || !aligned(sin, 16)) return FVATTN_ERR_INVALID;
    if (positions == nullptr && s->table_rows < s->S) return FVATTN_ERR_INVALID;
  }
  return FVATTN_OK;
}

int validate_dense(const fvattn_dense_shape* s, const fvattn_dense_mask* m, bool bwd) {
  if (s == nullptr) return FVATTN_ERR_INVALID;
  if (s->B < 1 || s->Hq < 1 || s->Hkv < 1 || s->Sq < 1 || s->Sk < 1 || s->d < 1) return FVATTN_ERR_INVALID;
  if (s->dtype != FVATTN_BF16 && s->dtype != FVATTN_F32) return FVATTN_ERR_INVALID;
  if (isnan(s->scale) || isinf(s->scale)) return FVATTN_ERR_INVALID;
  // a cap's reciprocal and its base-2 exponents have to be numbers
  if (s->softcap != 0.f && !(s->softcap >= 1e-20f && s->softcap <= 1e20f)) return FVATTN_ERR_INVALID;
  if (s->causal != 0 && s->causal != 1) return FVATTN_ERR_INVALID;
  if (s->Hq % s->Hkv != 0) return FVATTN_ERR_INVALID;
  if (s->d != 64 && s->d != 128) return FVATTN_ERR_UNSUPPORTED;
  if (s->Hq / s->Hkv > 64 || s->B > 65535 || s->Hkv > 65535 || s->B * s->Hkv > 65535) return FVATTN_ERR_UNSUPPORTED;
  if (s->Sq > kPosMax || s->Sk > kPosMax || s->Sq * (s->Hq / s->Hkv) > kPosMax) return FVATTN_ERR_UNSUPPORTED;
  if (!valid_strides(s->q, s->B, s->Hq, s->Sq, s->dtype) || !valid_strides(s->k, s->B, s->Hkv, s->Sk, s->dtype) ||
      !valid_strides(s->v, s->B, s->Hkv, s->Sk, s->dtype) || !valid_strides(s->o, s->B, s->Hq, s->Sq, s->dtype))
    return FVATTN_ERR_INVALID;
  if (bwd && (!valid_strides(s->dout, s->B, s->Hq, s->Sq, s->dtype) ||
              !valid_strides(s->dq, s->B, s->Hq, s->Sq, s->dtype) ||
              !valid_strides(s->dk, s->B, s->Hkv, s->Sk, s->dtype) ||
              !valid_strides(s->dv, s->B, s->Hkv, s->Sk, s->dtype)))
    return FVATTN_ERR_INVALID;
  if (m != nullptr) {
    if ((m->doc_q == nullptr) != (m->doc_k == nullptr)) return FVATTN_ERR_INVALID;
    if (m->prefix_len != nullptr && !s->causal) return FVATTN_ERR_INVALID;
    for (const void* p : {(const void*)m->slopes, (const void*)m->q_start, (const void*)m->kv_len,
                          (const void*)m->prefix_len, (const void*)m->doc_q, (const void*)m->doc_k})
      if (!aligned(p, 4)) return FVATTN_ERR_INVALID;
  }
  return FVATTN_OK;
}

DenseArgs dense_args(const fvattn_dense_shape* s, const fvattn_dense_mask* m) {
  DenseArgs a{};
  a.B = (int)s->B;
  a.Hq = (int)s->Hq;
  a.Hkv = (int)s->Hkv;
  a.G = a.Hq / a.Hkv;
  a.Sq = (int)s->Sq;
  a.Sk = (int)s->Sk;
  a.d = (int)s->d;
  a.causal = s->causal;
  a.scale = s->scale > 0.f ? s->scale : (float)(1.0 / sqrt((double)s->d));
  a.cap = s->softcap;
  a.inv_cap = a.cap > 0.f ? 1.f / a.cap : 0.f;
  if (m != nullptr) a.mask = *m;
  a.qs = canonical(s->q, s->B, s->Hq, s->Sq, s->d);
  a.ks = canonical(s->k, s->B, s->Hkv, s->Sk, s->d);
  a.vs = canonical(s->v, s->B, s->Hkv, s->Sk, s->d);
  a.os = canonical(s->o, s->B, s->Hq, s->Sq, s->d);
  a.dos = canonical(s->dout, s->B, s->Hq, s->Sq, s->d);
  a.dqs = canonical(s->dq, s->B, s->Hq, s->Sq, s->d);
  a.dks = canonical(s->dk, s->B, s->Hkv, s->Sk, s->d);
  a.dvs = canonical(s->dv, s->B, s->Hkv, s->Sk, s->d);
  a.splits = a.cluster = a.parts = 1;
  a.split_keys = (a.Sk + kBlock - 1) / kBlock * kBlock;
  return a;
}

// Keys are split over CTAs when the row tiles alone leave the GPU's 148 SMs (two CTAs each) mostly
// idle and each split still has `least_keys` to work on.
constexpr int kSlots = 2 * 148;
constexpr int kMostCluster = 8;
void split_in(DenseArgs& a, int64_t n) {
  const int64_t blocks = ((int64_t)a.Sk + kBlock - 1) / kBlock;
  const int64_t per = (blocks + n - 1) / n;
  a.split_keys = (int)(per * kBlock);
  a.splits = (int)((blocks + per - 1) / per);
}
void plan_splits(DenseArgs& a, int tile_rows_queries, int least_keys) {
  const int64_t tiles = ((int64_t)a.Sq + tile_rows_queries - 1) / tile_rows_queries * a.Hkv * a.B;
  if (tiles * 2 <= kSlots) {
    const int64_t most = ((int64_t)a.Sk + least_keys - 1) / least_keys;
    split_in(a, imax<int64_t>(1, imin(kSlots / tiles, most)));
  }
  a.parts = a.splits;
}
// For few rows: two waves of CTAs (the second evens out sequences of unequal length), of two blocks of keys
// at least; a cluster of a power of two up to its most, and whole clusters beyond. 64 key heads
// over caches of up to 32760 keys: 139 us in 8 splits; 187 us in 5, 156 us in 16.
void plan_few(DenseArgs& a) {
  const int64_t heads = (int64_t)a.B * a.Hkv, blocks = ((int64_t)a.Sk + kBlock - 1) / kBlock;
  const int64_t n = imax<int64_t>(1, imin((2 * kSlots + heads - 1) / heads, (blocks + 1) / 2));
  a.cluster = 1;
  while (a.cluster < kMostCluster && a.cluster < n) a.cluster *= 2;
  split_in(a, n <= kMostCluster ? n : (n + kMostCluster / 2) / kMostCluster * kMostCluster);
  a.splits = (a.splits + a.cluster - 1) / a.cluster * a.cluster;
  a.parts = a.splits / a.cluster;
}
bool few_rows(const DenseArgs& a, int dtype) {
  return dtype == FVATTN_BF16 && (int64_t)a.Sq * a.G <= kFewRows;
}

size_t take(size_t& off, size_t bytes) {
  const size_t o = off;
  off += (bytes + 255) & ~(size_t)255;
  return o;
}

struct DenseWs {
  size_t part_o, part_lse, delta, docs_q, docs_k, total;
};

size_t doc_bytes(int64_t B, int64_t S, int64_t block) { return (size_t)(B * ((S + block - 1) / block)) * sizeof(int2); }

DenseWs fwd_ws(const DenseArgs& a, int dtype) {
  DenseWs w{};
  size_t off = 0;
  const size_t rows = (size_t)a.B * a.Hq * a.Sq;
  if (a.parts > 1) {
    w.part_o = take(off, rows * a.parts * a.d * sizeof(float));
    w.part_lse = take(off, rows * a.parts * sizeof(float));
  }
  if (dtype == FVATTN_BF16 && a.mask.doc_k != nullptr) w.docs_k = take(off, doc_bytes(a.B, a.Sk, kBlock));
  w.total = off;
  return w;
}

constexpr int kBwdKeys = 128, kBwdRows = 64;      // of a tile of dQ's keys, and of dK and dV's rows

DenseWs bwd_ws(const DenseArgs& a, int dtype) {
  DenseWs w{};
  size_t off = 0;
  w.delta = take(off, (size_t)a.B * a.Hq * a.Sq * sizeof(float));
  if (dtype == FVATTN_BF16 && a.mask.doc_k != nullptr) {
    w.docs_q = take(off, doc_bytes(a.B, a.Sq, kBwdRows / a.G));
    w.docs_k = take(off, doc_bytes(a.B, a.Sk, kBwdKeys));
  }
  w.total = off;
  return w;
}

DenseArgs fwd_args(const fvattn_dense_shape* s, const fvattn_dense_mask* m) {
  DenseArgs a = dense_args(s, m);
  if (few_rows(a, s->dtype))
    plan_few(a);
  else if (s->dtype == FVATTN_F32)
    plan_splits(a, imax(1, 64 / a.G), kBlock);         // a tile of 64 keys takes it several microseconds
  else
    plan_splits(a, kTileRows / a.G, 256);
  return a;
}

int dense_attn(const void* q, const void* k, const void* v, const fvattn_dense_shape* shape,
               const fvattn_dense_mask* mask, void* out, void* rest, float* lse, void* workspace, size_t workspace_bytes,
               int32_t* status, fvattn_stream_t stream, uint32_t hold_polls = 0, uint32_t hold_step = 0) {
  const int st = validate_dense(shape, mask, false);
  if (st != FVATTN_OK) return st;
  if (!q || !k || !v || !out) return FVATTN_ERR_INVALID;
  for (const void* p : {q, k, v, (const void*)out, (const void*)rest})
    if (!aligned(p, 16)) return FVATTN_ERR_INVALID;
  if (!aligned(lse, 4) || !aligned(status, 4)) return FVATTN_ERR_INVALID;
  if (rest != nullptr && shape->dtype != FVATTN_BF16) return FVATTN_ERR_INVALID;
  DenseArgs a = fwd_args(shape, mask);
  const DenseWs w = fwd_ws(a, shape->dtype);
  if (w.total > 0 && (workspace == nullptr || !aligned(workspace, 256))) return FVATTN_ERR_INVALID;
  if (workspace_bytes < w.total) return FVATTN_ERR_CAPACITY;
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  a.q = q;
  a.k = k;
  a.v = v;
  a.out = out;
  a.rest = rest;
  a.lse = lse;
  a.status = status;
  a.hold_polls = hold_polls;
  a.hold_step = hold_step;
  if (a.parts > 1) {
    a.part_o = reinterpret_cast<float*>(ws + w.part_o);
    a.part_lse = reinterpret_cast<float*>(ws + w.part_lse);
  }
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (shape->dtype == FVATTN_BF16 && a.mask.doc_k != nullptr) {
    a.doc_blocks_k = reinterpret_cast<int2*>(ws + w.docs_k);
    a.doc_size_k = kBlock;
    e = launch_dense_prepare(a, shape->dtype, s);
  }
  if (e == cudaSuccess)
    e = shape->dtype == FVATTN_F32 ? launch_dense_f32(a, s)
        : few_rows(a, shape->dtype) ? launch_dense_few(a, s)
                                    : launch_dense_tc(a, s);
  if (e == cudaSuccess && a.parts > 1) e = launch_dense_combine(a, shape->dtype, s);
  return cuda_status(e);
}

int dense_attn_bwd(const void* dout, const void* q, const void* k, const void* v, const void* out, const void* rest,
                   const float* lse, const fvattn_dense_shape* shape, const fvattn_dense_mask* mask, void* dq, void* dk,
                   void* dv, void* workspace, size_t workspace_bytes, int32_t* status, fvattn_stream_t stream,
                   uint32_t hold_polls = 0, uint32_t hold_step = 0) {
  const int st = validate_dense(shape, mask, true);
  if (st != FVATTN_OK) return st;
  if (!dout || !q || !k || !v || !out || !lse || !dq || !dk || !dv) return FVATTN_ERR_INVALID;
  for (const void* p : {dout, q, k, v, out, rest, (const void*)dq, (const void*)dk, (const void*)dv})
    if (!aligned(p, 16)) return FVATTN_ERR_INVALID;
  if (!aligned(lse, 4) || !aligned(status, 4)) return FVATTN_ERR_INVALID;
  if (rest != nullptr && shape->dtype != FVATTN_BF16) return FVATTN_ERR_INVALID;
  DenseArgs a = dense_args(shape, mask);
  const DenseWs w = bwd_ws(a, shape->dtype);
  if (workspace == nullptr || !aligned(workspace, 256)) return FVATTN_ERR_INVALID;
  if (workspace_bytes < w.total) return FVATTN_ERR_CAPACITY;
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  a.q = q;
  a.k = k;
  a.v = v;
  a.out = const_cast<void*>(out);
  a.rest = const_cast<void*>(rest);
  a.lse = const_cast<float*>(lse);
  a.dout = dout;
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  a.delta = reinterpret_cast<float*>(ws + w.delta);
  a.status = status;
  a.hold_polls = hold_polls;
  a.hold_step = hold_step;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (shape->dtype == FVATTN_BF16 && a.mask.doc_k != nullptr) {
    a.doc_blocks_q = reinterpret_cast<int2*>(ws + w.docs_q);
    a.doc_blocks_k = reinterpret_cast<int2*>(ws + w.docs_k);
    a.doc_size_q = kBwdRows / a.G;
    a.doc_size_k = kBwdKeys;
  }
  cudaError_t e = launch_dense_prepare(a, shape->dtype, s);
  if (e == cudaSuccess) e = shape->dtype == FVATTN_BF16 ? launch_dense_bwd_tc(a, s) : launch_dense_f32_bwd(a, s);
  return cuda_status(e);
}

}  // namespace

extern "C" {

int fvattn_qk_norm_rope(const void* q, const void* k, const fvattn_qk_shape* shape, const void* wq, const void* wk,
                        const float* cos, const float* sin, const int32_t* positions, void* qo, void* ko,
                        int32_t* status, fvattn_stream_t stream) {
  int st = validate_qk(shape, false);
  if (st != FVATTN_OK) return st;
  if (!q || !k || !qo || !ko) return FVATTN_ERR_INVALID;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(qo, 16) || !aligned(ko, 16)) return FVATTN_ERR_INVALID;
  st = check_qk_tables(shape, wq, wk, cos, sin, positions, status);
  if (st != FVATTN_OK) return st;
  QkNormArgs a{};
  a.q = q;
  a.k = k;
  a.wq = wq;
  a.wk = wk;
  a.cos = cos;
  a.sin = sin;
  a.positions = positions;
  a.qo = qo;
  a.ko = ko;
  a.status = status;
  return cuda_status(launch_qk_norm(a, *shape, reinterpret_cast<cudaStream_t>(stream)));
}

size_t fvattn_qk_norm_rope_workspace_bytes(const fvattn_qk_shape* shape) {
  if (validate_qk(shape, true) != FVATTN_OK) return 0;
  return qk_norm_part_bytes(*shape);
}

int fvattn_qk_norm_rope_bwd(const void* gq, const void* gk, const void* q, const void* k, const fvattn_qk_shape* shape,
                            const void* wq, const void* wk, const float* cos, const float* sin,
                            const int32_t* positions, void* dq, void* dk, float* dwq, float* dwk, void* workspace,
                            size_t workspace_bytes, int32_t* status, fvattn_stream_t stream) {
  int st = validate_qk(shape, true);
  if (st != FVATTN_OK) return st;
  if (!gq || !gk || !q || !k || !dq || !dk) return FVATTN_ERR_INVALID;
  for (const void* p : {gq, gk, q, k, (const void*)dq, (const void*)dk})
    if (!aligned(p, 16)) return FVATTN_ERR_INVALID;
  if (!aligned(dwq, 4) || !aligned(dwk, 4)) return FVATTN_ERR_INVALID;
  st = check_qk_tables(shape, wq, wk, cos, sin, positions, status);
  if (st != FVATTN_OK) return st;
  if (dwq != nullptr || dwk != nullptr) {
    if (workspace == nullptr || !aligned(workspace, 16)) return FVATTN_ERR_INVALID;
    if (workspace_bytes < qk_norm_part_bytes(*shape)) return FVATTN_ERR_CAPACITY;
  }
  QkNormArgs a{};
  a.q = q;
  a.k = k;
  a.wq = wq;
  a.wk = wk;
  a.cos = cos;
  a.sin = sin;
  a.positions = positions;
  a.qo = dq;
  a.ko = dk;
  a.gq = gq;
  a.gk = gk;
  a.dwq = dwq;
  a.dwk = dwk;
  a.parts = static_cast<float*>(workspace);
  a.status = status;
  return cuda_status(launch_qk_norm_bwd(a, *shape, reinterpret_cast<cudaStream_t>(stream)));
}

size_t fvattn_dense_attn_workspace_bytes(const fvattn_dense_shape* shape, const fvattn_dense_mask* mask) {
  if (validate_dense(shape, mask, false) != FVATTN_OK) return (size_t)-1;
  return fwd_ws(fwd_args(shape, mask), shape->dtype).total;
}

int fvattn_dense_attn(const void* q, const void* k, const void* v, const fvattn_dense_shape* shape,
                      const fvattn_dense_mask* mask, void* out, void* rest, float* lse, void* workspace,
                      size_t workspace_bytes, int32_t* status, fvattn_stream_t stream) {
  return dense_attn(q, k, v, shape, mask, out, rest, lse, workspace, workspace_bytes, status, stream);
}

int fvattn_dense_attn_timeout_check(const void* q, const void* k, const void* v, const fvattn_dense_shape* shape,
                                    const fvattn_dense_mask* mask, void* out, void* rest, float* lse, void* workspace,
                                    size_t workspace_bytes, int32_t* status, uint32_t step, uint32_t polls,
                                    fvattn_stream_t stream) {
  if (polls == 0 || status == nullptr) return FVATTN_ERR_INVALID;
  if (shape != nullptr && shape->dtype == FVATTN_F32) return FVATTN_ERR_UNSUPPORTED;
  return dense_attn(q, k, v, shape, mask, out, rest, lse, workspace, workspace_bytes, status, stream, polls, step);
}

size_t fvattn_dense_attn_bwd_workspace_bytes(const fvattn_dense_shape* shape, const fvattn_dense_mask* mask) {
  if (validate_dense(shape, mask, true) != FVATTN_OK) return (size_t)-1;
  return bwd_ws(dense_args(shape, mask), shape->dtype).total;
}

int fvattn_dense_attn_bwd(const void* dout, const void* q, const void* k, const void* v, const void* out,
                          const void* rest, const float* lse, const fvattn_dense_shape* shape,
                          const fvattn_dense_mask* mask, void* dq, void* dk, void* dv, void* workspace,
                          size_t workspace_bytes, int32_t* status, fvattn_stream_t stream) {
  return dense_attn_bwd(dout, q, k, v, out, rest, lse, shape, mask, dq, dk, dv, workspace, workspace_bytes, status,
                        stream);
}

int fvattn_dense_attn_bwd_timeout_check(const void* dout, const void* q, const void* k, const void* v, const void* out,
                                        const void* rest, const float* lse, const fvattn_dense_shape* shape,
                                        const fvattn_dense_mask* mask, void* dq, void* dk, void* dv, void* workspace,
                                        size_t workspace_bytes, int32_t* status, uint32_t step, uint32_t polls,
                                        fvattn_stream_t stream) {
  if (polls == 0 || status == nullptr) return FVATTN_ERR_INVALID;
  if (shape != nullptr && shape->dtype == FVATTN_F32) return FVATTN_ERR_UNSUPPORTED;
  return dense_attn_bwd(dout, q, k, v, out, rest, lse, shape, mask, dq, dk, dv, workspace, workspace_bytes, status,
                        stream, polls, step);
}

}  // extern "C"
