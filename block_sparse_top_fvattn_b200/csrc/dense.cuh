// Attention over all keys with capped, biased and masked scores: what its kernels share
// (dense_tc.cu, dense_bwd_tc.cu: bf16 on the tensor cores; dense_f32.cu: fp32 on the CUDA cores).
//
// The query heads that share a key head are rows of one problem: row i * G + g of key head h is
// query i of query head h * G + g, G = Hq / Hkv. K and V are then read once for all of them, and the
// gradients of a shared key head are sums over its rows.
#pragma once

#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "common.cuh"
#include "fvattn.h"

namespace fv {

struct DenseArgs {
  const void *q, *k, *v;
  void *out, *rest;               // backward: read
  float* lse;                     // backward: read
  const void* dout;
  void *dq, *dk, *dv;
  fvattn_strides qs, ks, vs, os, dos, dqs, dks, dvs;
  fvattn_dense_mask mask;
  int B, Hq, Hkv, G, Sq, Sk, d;
  int causal;
  float scale, cap, inv_cap;
  int splits, split_keys;         // forward: the keys in `splits` ranges of split_keys (a multiple of 64)
  int cluster, parts;             // ranges joined within a cluster; what is left to join through memory
  float *part_o, *part_lse;       // parts > 1: [parts][B][Hq][Sq][d] and [parts][B][Hq][Sq]
  float* delta;                   // backward: [B][Hq][Sq], sum_d out * dout
  // Documents of blocks of tokens (dense_prepare_kernel), null without documents: of the keys in blocks of
  // 64 (forward) or 128 (backward), of the queries in steps of dK and dV (backward).
  int2 *doc_blocks_q, *doc_blocks_k;
  int doc_size_q, doc_size_k;
  int32_t* status;
  uint32_t hold_polls, hold_step; // failure-path check: each loader's wait at this step runs out; 0: none
};

constexpr int kPosMax = (1 << 30) - 1;

// What masks one sequence of the batch.
struct DenseSeq {
  int q0;        // position of the first query
  int kv;        // keys that exist (those that some query may see)
  int prefix;    // keys visible to every query (causal)
};

__device__ __forceinline__ DenseSeq dense_seq(const DenseArgs& a, int b) {
  DenseSeq s;
  s.q0 = a.mask.q_start != nullptr ? min(max(a.mask.q_start[b], -kPosMax), kPosMax) : a.Sk - a.Sq;
  s.kv = a.mask.kv_len != nullptr ? min(max(a.mask.kv_len[b], 0), a.Sk) : a.Sk;
  s.prefix = a.mask.prefix_len != nullptr ? a.mask.prefix_len[b] : 0;
  // under an order nobody sees what is behind the last query (of a cache that is longer): as if it did not exist
  if (a.causal) s.kv = max(0, min(s.kv, max(s.q0 + a.Sq, s.prefix)));
  return s;
}

// Keys [0, limit) are visible to query i as far as length, order and prefix go. Never falls as i grows.
__device__ __forceinline__ int dense_limit(const DenseSeq& s, int causal, int i) {
  return causal ? max(0, min(s.kv, max(s.q0 + i + 1, s.prefix))) : s.kv;
}

// One row's mask, position and slope.
struct DenseRow {
  int limit;     // visible keys are below it
  int doc;       // and of this document (ignored without documents)
  int pos;
  float slope;
};

__device__ __forceinline__ DenseRow dense_row(const DenseArgs& a, const DenseSeq& s, int b, int hq, int i) {
  DenseRow r;
  r.pos = s.q0 + i;
  r.limit = dense_limit(s, a.causal, i);
  r.doc = 0;
  if (a.mask.doc_q != nullptr) {
    r.doc = a.mask.doc_q[(int64_t)b * a.Sq + i];
    if (r.doc < 0) r.limit = 0;
  }
  r.slope = a.mask.slopes != nullptr ? a.mask.slopes[hq] : 0.f;
  return r;
}

// Launchers. Each returns the launch's error.
cudaError_t launch_dense_bwd_tc(const DenseArgs& a, cudaStream_t st);
cudaError_t launch_dense_tc(const DenseArgs& a, cudaStream_t st);
cudaError_t launch_dense_few(const DenseArgs& a, cudaStream_t st);
constexpr int kFewRows = 16;      // the most rows of a key head that launch_dense_few takes
cudaError_t launch_dense_f32(const DenseArgs& a, cudaStream_t st);
cudaError_t launch_dense_combine(const DenseArgs& a, int dtype, cudaStream_t st);
// delta where a.delta is set, the documents of blocks where a.doc_blocks_q and a.doc_blocks_k are.
cudaError_t launch_dense_prepare(const DenseArgs& a, int dtype, cudaStream_t st);
cudaError_t launch_dense_f32_bwd(const DenseArgs& a, cudaStream_t st);

}  // namespace fv
