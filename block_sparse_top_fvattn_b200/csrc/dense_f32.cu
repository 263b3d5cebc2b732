// Attention over all keys in fp32 on the CUDA cores, forward and backward, and the two small
// kernels that the bf16 path shares: the join of split keys, and what the other kernels need first (the row sums
// of out * dout, the documents of blocks of tokens).
//
//   s_ij = cap tanh(scale q_i.k_j / cap) - slope |p_i - j|,  P = softmax over the visible j,
//   out = P V,  lse_i = log sum_j exp(s_ij)
//   dP = dout V^T,  delta_i = sum_d out_id dout_id,  dX = P (dP - delta) (1 - tanh^2) scale
//   dQ = dX K,  dK = dX^T Q,  dV = P^T dout
//
// A CTA takes 64 rows (forward, dQ) or 64 keys (dK, dV) and walks over the other side in tiles of
// 64, operands in shared memory as fp32, a 4 x 4 piece of the 64 x 64 scores and a 4 x d/16 piece
// of each result per thread in registers. Bound by the fp32 pipe and the shared-memory loads that
// feed it. Every sum has a fixed order. Tiles are skipped by limit, not by document. Measured: 1024 tokens, 2
// heads of 64, capped: 31.6 us, 9 TFLOP/s; 2000 tokens, 8 / 2 heads: 313 us, gradients 2098 us.
#include <cuda_bf16.h>

#include "dense.cuh"

namespace fv {

namespace {

constexpr int kT = 64;            // rows and keys of a tile
constexpr int kThreads = 256;

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const float4 a = load4(p), b = load4(p + 4);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&x)[8]) {
  const uint4 v = *reinterpret_cast<const uint4*>(p);
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}

template <int D>
struct Tile {
  static constexpr int kLd = D + 4;        // rows of a tile 16 bytes apart in the banks
  static constexpr int kFloats = kT * kLd;
  static constexpr int kLdP = kT + 4;
  static constexpr int kFloatsP = kT * kLdP;
};

// Rows row0.. of a key head's (query, head of the group) rows into shared memory; others as zeros.
template <int D>
__device__ __forceinline__ void load_rows(float* dst, const float* base, const fvattn_strides& st, int b, int h0, int G,
                                          int row0, int nrows) {
  for (int x = threadIdx.x; x < kT * (D / 4); x += kThreads) {
    const int r = x / (D / 4), c = (x % (D / 4)) * 4;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    const int rho = row0 + r;
    if (rho < nrows) v = load4(base + b * st.b + (h0 + rho % G) * st.h + (int64_t)(rho / G) * st.s + c);
    *reinterpret_cast<float4*>(dst + r * Tile<D>::kLd + c) = v;
  }
}

// Keys j0.. below `end` of one key head; others as zeros (whatever they hold). Padding keys too.
template <int D>
__device__ __forceinline__ void load_keys(float* dst, const float* base, const fvattn_strides& st, int b, int h, int j0,
                                          int end, const int32_t* doc) {
  for (int x = threadIdx.x; x < kT * (D / 4); x += kThreads) {
    const int r = x / (D / 4), c = (x % (D / 4)) * 4;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    const int j = j0 + r;
    if (j < end && (doc == nullptr || doc[j] >= 0)) v = load4(base + b * st.b + h * st.h + (int64_t)j * st.s + c);
    *reinterpret_cast<float4*>(dst + r * Tile<D>::kLd + c) = v;
  }
}

// Pairs of fp32 (one 64-bit register): two products per instruction, and shared memory gives them as
// they are.
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 both(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}

// acc[i][j] = A[ty*4 + i] . B[tx + 16 j] over D (even and odd elements apart until the end).
template <int D>
__device__ __forceinline__ void dot_tile(const float* A, const float* B, int ty, int tx, float (&acc)[4][4]) {
  constexpr int LD = Tile<D>::kLd;
  uint64_t sum[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) sum[i][j] = 0ull;
#pragma unroll 4
  for (int c = 0; c < D; c += 4) {
    ulonglong2 x[4], y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const ulonglong2*>(A + (ty * 4 + i) * LD + c);
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const ulonglong2*>(B + (tx + 16 * j) * LD + c);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) sum[i][j] = fma2(x[i].y, y[j].y, fma2(x[i].x, y[j].x, sum[i][j]));
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 v = both(sum[i][j]);
      acc[i][j] = v.x + v.y;
    }
}

// acc[i] (pairs of columns tx*4 + 64 c ..) += sum_j W[ty*4 + i][j] X[j] over the 64 j of a tile.
template <int D>
__device__ __forceinline__ void add_product(const float* W, const float* X, int ty, int tx, uint64_t (&acc)[4][D / 32]) {
#pragma unroll 2
  for (int j = 0; j < kT; j += 4) {
    float4 w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const float4*>(W + (ty * 4 + i) * Tile<D>::kLdP + j);
#pragma unroll
    for (int jj = 0; jj < 4; ++jj) {
      uint64_t ww[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float v = jj == 0 ? w[i].x : jj == 1 ? w[i].y : jj == 2 ? w[i].z : w[i].w;
        ww[i] = pair(v, v);
      }
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(X + (j + jj) * Tile<D>::kLd + tx * 4 + 64 * c);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc[i][2 * c] = fma2(ww[i], x.x, acc[i][2 * c]);
          acc[i][2 * c + 1] = fma2(ww[i], x.y, acc[i][2 * c + 1]);
        }
      }
    }
  }
}

// Times `by`, to the columns of a row.
template <int D>
__device__ __forceinline__ void store_cols(float* p, int tx, const uint64_t (&acc)[D / 32], float by) {
#pragma unroll
  for (int c = 0; c < D / 64; ++c) {
    const float2 x = both(acc[2 * c]), y = both(acc[2 * c + 1]);
    *reinterpret_cast<float4*>(p + tx * 4 + 64 * c) = make_float4(x.x * by, x.y * by, y.x * by, y.y * by);
  }
}

// The capped and biased score of a product x = q.k, and the derivative of the cap.
__device__ __forceinline__ float score(const DenseArgs& a, const DenseRow& r, float x, int j, float* slope_of_cap) {
  float s = x * a.scale;
  *slope_of_cap = 1.f;
  if (a.cap > 0.f) {
    const float t = tanhf(s * a.inv_cap);
    s = a.cap * t;
    *slope_of_cap = 1.f - t * t;
  }
  if (a.mask.slopes != nullptr) s -= r.slope * (float)abs(r.pos - j);
  return s;
}

__device__ __forceinline__ float half_warp_max(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float half_warp_sum(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Keys j0.. below `end` as load_keys, by asynchronous copies.
template <int D>
__device__ __forceinline__ void copy_keys_async(float* dst, const float* base, const fvattn_strides& st, int b, int h, int j0,
                                                int end, const int32_t* doc) {
  for (int x = threadIdx.x; x < kT * (D / 4); x += kThreads) {
    const int r = x / (D / 4), c = (x % (D / 4)) * 4, j = j0 + r;
    const bool take = j < end && (doc == nullptr || doc[j] >= 0);
    const float* src = base + b * st.b + h * st.h + (take ? (int64_t)j * st.s + c : 0);
    const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(dst + r * Tile<D>::kLd + c));
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(src), "r"(take ? 16 : 0) : "memory");
  }
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

// grid: (row tiles * splits, Hkv, B). The next tile's keys are copied while this one's are worked on; warps
// whose rows are all past the last one (few queries) only copy.
template <int D>
__global__ void __launch_bounds__(kThreads) dense_fwd_kernel(const DenseArgs a) {
  allow_next_grid();
  extern __shared__ float sm[];
  float *sQ = sm, *sKV = sQ + Tile<D>::kFloats, *sP = sKV + 4 * Tile<D>::kFloats;
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  const int split = blockIdx.x % a.splits, tile = gridDim.x / a.splits - 1 - blockIdx.x / a.splits;
  const int h = blockIdx.y, b = blockIdx.z, h0 = h * a.G;
  const int nrows = a.Sq * a.G, row0 = tile * kT;
  const DenseSeq seq = dense_seq(a, b);
  const int32_t* doc_k = a.mask.doc_k != nullptr ? a.mask.doc_k + (int64_t)b * a.Sk : nullptr;
  const int last = min(row0 + kT, nrows) - 1;
  const int begin = split * a.split_keys;
  const int end = (int)imin<int64_t>(dense_limit(seq, a.causal, last / a.G), (int64_t)begin + a.split_keys);
  auto copy = [&](int j0, int buf) {
    float* to = sKV + buf * 2 * Tile<D>::kFloats;
    copy_keys_async<D>(to, static_cast<const float*>(a.k), a.ks, b, h, j0, end, doc_k);
    copy_keys_async<D>(to + Tile<D>::kFloats, static_cast<const float*>(a.v), a.vs, b, h, j0, end, doc_k);
    copies_commit();
  };
  if (begin < end) copy(begin, 0);
  load_rows<D>(sQ, static_cast<const float*>(a.q), a.qs, b, h0, a.G, row0, nrows);

  DenseRow row[4];
  float mx[4], l[4];
  uint64_t o[4][D / 32];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int rho = row0 + ty * 4 + i;
    if (rho < nrows)
      row[i] = dense_row(a, seq, b, h0 + rho % a.G, rho / a.G);
    else
      row[i] = DenseRow{0, 0, 0, 0.f};
    mx[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int c = 0; c < D / 32; ++c) o[i][c] = 0ull;
  }
  const bool live = row0 + (threadIdx.x >> 5) * 8 < nrows;       // the same for a warp
  int buf = 0;
  for (int j0 = begin; j0 < end; j0 += kT, buf ^= 1) {
    __syncthreads();                     // the buffer that the next copies fill has been read
    if (j0 + kT < end) {
      copy(j0 + kT, buf ^ 1);
      copies_wait<1>();
    } else {
      copies_wait<0>();
    }
    __syncthreads();
    if (!live) continue;
    const float *sK = sKV + buf * 2 * Tile<D>::kFloats, *sV = sK + Tile<D>::kFloats;
    float s[4][4];
    dot_tile<D>(sQ, sK, ty, tx, s);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float m = -INFINITY;
#pragma unroll
      for (int jj = 0; jj < 4; ++jj) {
        const int j = j0 + tx + 16 * jj;
        float unused;
        const bool see = j < row[i].limit && (doc_k == nullptr || doc_k[j] == row[i].doc);
        s[i][jj] = see ? score(a, row[i], s[i][jj], j, &unused) : -INFINITY;
        m = fmaxf(m, s[i][jj]);
      }
      const float mn = fmaxf(mx[i], half_warp_max(m));
      const float base = mn == -INFINITY ? 0.f : mn;      // nothing seen so far: weights of 0
      const float f = expf(mx[i] - base);
      float add = 0.f;
#pragma unroll
      for (int jj = 0; jj < 4; ++jj) {
        const float p = expf(s[i][jj] - base);
        add += p;
        sP[(ty * 4 + i) * Tile<D>::kLdP + tx + 16 * jj] = p;
      }
      l[i] = l[i] * f + half_warp_sum(add);
      mx[i] = mn;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) o[i][c] = fma2(o[i][c], pair(f, f), 0ull);
    }
    __syncwarp();                // a row's weights are written and read by one half warp
    add_product<D>(sP, sV, ty, tx, o);
    __syncwarp();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int rho = row0 + ty * 4 + i;
    if (rho >= nrows) continue;
    const int hq = h0 + rho % a.G;
    const int64_t iq = rho / a.G, flat = ((int64_t)b * a.Hq + hq) * a.Sq + iq;
    const float inv = l[i] > 0.f || l[i] != l[i] ? 1.f / l[i] : 0.f;
    const float lse = l[i] == 0.f ? -INFINITY : mx[i] + logf(l[i]);
    const int64_t at = (int64_t)split * a.B * a.Hq * a.Sq + flat;
    float* p = a.parts > 1 ? a.part_o + at * D : static_cast<float*>(a.out) + b * a.os.b + hq * a.os.h + iq * a.os.s;
    store_cols<D>(p, tx, o[i], inv);
    if (tx == 0) {
      if (a.parts > 1)
        a.part_lse[at] = lse;
      else if (a.lse != nullptr)
        a.lse[flat] = lse;
    }
  }
}

// Joins the splits of a row: weights exp(lse_s - max) in a fixed order. One warp per row.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) dense_combine_kernel(const DenseArgs a) {
  wait_for_previous_grid();
  const int64_t rows = (int64_t)a.B * a.Hq * a.Sq;
  const int64_t flat = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (flat >= rows) return;
  float m = -INFINITY;
  for (int s = lane; s < a.parts; s += 32) m = fmaxf(m, a.part_lse[s * rows + flat]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float base = m == -INFINITY ? 0.f : m;
  constexpr int N = D / 32;
  float acc[N], total = 0.f;
#pragma unroll
  for (int c = 0; c < N; ++c) acc[c] = 0.f;
#pragma unroll 4
  for (int s = 0; s < a.parts; ++s) {
    const float w = expf(a.part_lse[s * rows + flat] - base);
    const float* p = a.part_o + (s * rows + flat) * D + lane * N;
    total += w;
#pragma unroll
    for (int c = 0; c < N; ++c) acc[c] = fmaf(w, p[c], acc[c]);
  }
  const int64_t iq = flat % a.Sq, bh = flat / a.Sq, b = bh / a.Hq, hq = bh - b * a.Hq;
  const int64_t at = b * a.os.b + hq * a.os.h + iq * a.os.s + lane * N;
  const float inv = total == 0.f ? 0.f : 1.f / total;
#pragma unroll
  for (int c = 0; c < N; ++c) {
    const float x = acc[c] * inv;
    T* p = static_cast<T*>(a.out) + at + c;
    put(p, x);
    if (a.rest != nullptr) put(static_cast<T*>(a.rest) + at + c, x - to_f32(*p));
  }
  if (lane == 0 && a.lse != nullptr) a.lse[flat] = total == 0.f ? -INFINITY : m + logf(total);
}

// delta = sum_d (out + rest) dout; eight elements per lane, d / 8 lanes per row. Padding queries get 0,
// whatever they hold.
template <typename T, int D>
__device__ __forceinline__ void row_delta(const DenseArgs& a, int64_t block) {
  constexpr int LPR = D / 8;
  const int64_t rows = (int64_t)a.B * a.Hq * a.Sq;
  const int64_t flat = block * (kThreads / LPR) + threadIdx.x / LPR;
  const int l = threadIdx.x % LPR;
  float acc = 0.f;
  if (flat < rows) {
    const int64_t iq = flat % a.Sq, bh = flat / a.Sq, b = bh / a.Hq, hq = bh - b * a.Hq;
    const int64_t at = b * a.os.b + hq * a.os.h + iq * a.os.s + l * 8;
    float o[8], g[8];
    load8(static_cast<const T*>(a.out) + at, o);
    load8(static_cast<const T*>(a.dout) + b * a.dos.b + hq * a.dos.h + iq * a.dos.s + l * 8, g);
    if (a.rest != nullptr) {
      float r[8];
      load8(static_cast<const T*>(a.rest) + at, r);
#pragma unroll
      for (int c = 0; c < 8; ++c) o[c] += r[c];
    }
#pragma unroll
    for (int c = 0; c < 8; ++c) acc = fmaf(o[c], g[c], acc);
    if (a.mask.doc_q != nullptr && a.mask.doc_q[b * a.Sq + iq] < 0) acc = 0.f;
  }
#pragma unroll
  for (int x = LPR / 2; x > 0; x >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, x);
  if (l == 0 && flat < rows) a.delta[flat] = acc;
}

// The documents of each block of `size` tokens of doc [B][S], one warp per block: x = the lowest
// number, with the sign bit set when the block has padding tokens (0x7fffffff without any document),
// y = the highest (-1 without any).
__device__ __forceinline__ void block_docs(const int32_t* doc, int2* blocks, int B, int S, int size, int64_t block) {
  const int nb = (S + size - 1) / size, lane = threadIdx.x & 31;
  const int64_t w = block * (kThreads / 32) + (threadIdx.x >> 5);
  if (w >= (int64_t)B * nb) return;
  const int64_t b = w / nb, j = w - b * nb;
  int lo = 0x7fffffff, hi = -1;
  bool pad = false;
  for (int u = lane; u < size; u += 32) {
    const int64_t t = j * size + u;
    if (t >= S) break;
    const int v = doc[b * S + t];
    if (v < 0) {
      pad = true;
    } else {
      lo = min(lo, v);
      hi = max(hi, v);
    }
  }
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  pad = __any_sync(0xffffffffu, pad);
  if (lane == 0) blocks[w] = make_int2(pad ? (int)((uint32_t)lo | 0x80000000u) : lo, hi);
}

// What the other kernels of a call need first, in one launch: CTAs [0, q0) the rows' delta, [q0, k0) the
// documents of the queries' blocks, the rest those of the keys'.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) dense_prepare_kernel(const DenseArgs a, int64_t q0, int64_t k0) {
  allow_next_grid();
  const int64_t x = blockIdx.x;
  if (x < q0)
    row_delta<T, D>(a, x);
  else if (x < k0)
    block_docs(a.mask.doc_q, a.doc_blocks_q, a.B, a.Sq, a.doc_size_q, x - q0);
  else
    block_docs(a.mask.doc_k, a.doc_blocks_k, a.B, a.Sk, a.doc_size_k, x - k0);
}

// Probability and score gradient of one pair: p = exp(s - lse), ds = p (dp - delta) cap' scale.
__device__ __forceinline__ void pair_grads(const DenseArgs& a, const DenseRow& r, float lse, float delta, float x,
                                           float dp, int j, const int32_t* doc_k, float* p, float* ds) {
  *p = 0.f;
  *ds = 0.f;
  if (j < r.limit && (doc_k == nullptr || doc_k[j] == r.doc)) {
    float dcap;
    const float s = score(a, r, x, j, &dcap);
    *p = expf(s - lse);
    *ds = *p * (dp - delta) * dcap * a.scale;
  }
}

// grid: (row tiles, Hkv, B)
template <int D>
__global__ void __launch_bounds__(kThreads) dense_dq_kernel(const DenseArgs a) {
  extern __shared__ float sm[];
  float *sQ = sm, *sG = sQ + Tile<D>::kFloats, *sK = sG + Tile<D>::kFloats, *sV = sK + Tile<D>::kFloats,
        *sP = sV + Tile<D>::kFloats;
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  const int tile = gridDim.x - 1 - blockIdx.x, h = blockIdx.y, b = blockIdx.z, h0 = h * a.G;
  const int nrows = a.Sq * a.G, row0 = tile * kT;
  const DenseSeq seq = dense_seq(a, b);
  const int32_t* doc_k = a.mask.doc_k != nullptr ? a.mask.doc_k + (int64_t)b * a.Sk : nullptr;
  load_rows<D>(sQ, static_cast<const float*>(a.q), a.qs, b, h0, a.G, row0, nrows);
  load_rows<D>(sG, static_cast<const float*>(a.dout), a.dos, b, h0, a.G, row0, nrows);
  DenseRow row[4];
  float lse[4], delta[4];
  uint64_t dq[4][D / 32];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int rho = row0 + ty * 4 + i;
    row[i] = DenseRow{0, 0, 0, 0.f};
    lse[i] = delta[i] = 0.f;
    if (rho < nrows) {
      const int hq = h0 + rho % a.G;
      const int64_t flat = ((int64_t)b * a.Hq + hq) * a.Sq + rho / a.G;
      row[i] = dense_row(a, seq, b, hq, rho / a.G);
      lse[i] = a.lse[flat];
      delta[i] = a.delta[flat];
    }
#pragma unroll
    for (int c = 0; c < D / 32; ++c) dq[i][c] = 0ull;
  }
  const int last = min(row0 + kT, nrows) - 1;
  const int end = dense_limit(seq, a.causal, last / a.G);
  for (int j0 = 0; j0 < end; j0 += kT) {
    __syncthreads();
    load_keys<D>(sK, static_cast<const float*>(a.k), a.ks, b, h, j0, end, doc_k);
    load_keys<D>(sV, static_cast<const float*>(a.v), a.vs, b, h, j0, end, doc_k);
    __syncthreads();
    float s[4][4], dp[4][4];
    dot_tile<D>(sQ, sK, ty, tx, s);
    dot_tile<D>(sG, sV, ty, tx, dp);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int jj = 0; jj < 4; ++jj) {
        float p, ds;
        pair_grads(a, row[i], lse[i], delta[i], s[i][jj], dp[i][jj], j0 + tx + 16 * jj, doc_k, &p, &ds);
        sP[(ty * 4 + i) * Tile<D>::kLdP + tx + 16 * jj] = ds;
      }
    __syncwarp();
    add_product<D>(sP, sK, ty, tx, dq);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int rho = row0 + ty * 4 + i;
    if (rho >= nrows) continue;
    float* p = static_cast<float*>(a.dq) + b * a.dqs.b + (h0 + rho % a.G) * a.dqs.h + (int64_t)(rho / a.G) * a.dqs.s;
    store_cols<D>(p, tx, dq[i], 1.f);
  }
}

// grid: (key tiles, Hkv, B)
template <int D>
__global__ void __launch_bounds__(kThreads) dense_dkv_kernel(const DenseArgs a) {
  extern __shared__ float sm[];
  float *sK = sm, *sV = sK + Tile<D>::kFloats, *sQ = sV + Tile<D>::kFloats, *sG = sQ + Tile<D>::kFloats,
        *sP = sG + Tile<D>::kFloats, *sS = sP + Tile<D>::kFloatsP;
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  const int j0 = blockIdx.x * kT, h = blockIdx.y, b = blockIdx.z, h0 = h * a.G;
  const int nrows = a.Sq * a.G;
  const DenseSeq seq = dense_seq(a, b);
  const int32_t* doc_k = a.mask.doc_k != nullptr ? a.mask.doc_k + (int64_t)b * a.Sk : nullptr;
  load_keys<D>(sK, static_cast<const float*>(a.k), a.ks, b, h, j0, seq.kv, doc_k);
  load_keys<D>(sV, static_cast<const float*>(a.v), a.vs, b, h, j0, seq.kv, doc_k);
  uint64_t dk[4][D / 32], dv[4][D / 32];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int c = 0; c < D / 32; ++c) dk[i][c] = dv[i][c] = 0ull;
  for (int row0 = 0; row0 < nrows; row0 += kT) {
    const int last = min(row0 + kT, nrows) - 1;
    if (dense_limit(seq, a.causal, last / a.G) <= j0) continue;    // the same for the whole CTA
    __syncthreads();
    load_rows<D>(sQ, static_cast<const float*>(a.q), a.qs, b, h0, a.G, row0, nrows);
    load_rows<D>(sG, static_cast<const float*>(a.dout), a.dos, b, h0, a.G, row0, nrows);
    __syncthreads();
    // scores as [key][row]: this thread's four keys, four rows
    float s[4][4], dp[4][4];
    dot_tile<D>(sK, sQ, ty, tx, s);
    dot_tile<D>(sV, sG, ty, tx, dp);
#pragma unroll
    for (int rr = 0; rr < 4; ++rr) {
      const int rho = row0 + tx + 16 * rr;
      DenseRow row{0, 0, 0, 0.f};
      float lse = 0.f, delta = 0.f;
      if (rho < nrows) {
        const int hq = h0 + rho % a.G;
        const int64_t flat = ((int64_t)b * a.Hq + hq) * a.Sq + rho / a.G;
        row = dense_row(a, seq, b, hq, rho / a.G);
        lse = a.lse[flat];
        delta = a.delta[flat];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float p, ds;
        pair_grads(a, row, lse, delta, s[i][rr], dp[i][rr], j0 + ty * 4 + i, doc_k, &p, &ds);
        sP[(ty * 4 + i) * Tile<D>::kLdP + tx + 16 * rr] = p;
        sS[(ty * 4 + i) * Tile<D>::kLdP + tx + 16 * rr] = ds;
      }
    }
    // a padding query may hold anything: its row must not reach the products below
    if (a.mask.doc_q != nullptr) {
      __syncthreads();
      for (int r = threadIdx.x; r < kT; r += kThreads) {
        const int rho = row0 + r;
        if (rho < nrows && a.mask.doc_q[(int64_t)b * a.Sq + rho / a.G] < 0)
          for (int c = 0; c < D; ++c) sQ[r * Tile<D>::kLd + c] = sG[r * Tile<D>::kLd + c] = 0.f;
      }
      __syncthreads();
    } else {
      __syncwarp();
    }
    add_product<D>(sP, sG, ty, tx, dv);
    add_product<D>(sS, sQ, ty, tx, dk);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int j = j0 + ty * 4 + i;
    if (j >= a.Sk) continue;
    float* pk = static_cast<float*>(a.dk) + b * a.dks.b + h * a.dks.h + (int64_t)j * a.dks.s;
    float* pv = static_cast<float*>(a.dv) + b * a.dvs.b + h * a.dvs.h + (int64_t)j * a.dvs.s;
    store_cols<D>(pk, tx, dk[i], 1.f);
    store_cols<D>(pv, tx, dv[i], 1.f);
  }
}

template <typename K>
cudaError_t run(K kernel, dim3 grid, size_t smem, const DenseArgs& a, cudaStream_t st) {
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  kernel<<<grid, kThreads, smem, st>>>(a);
  return cudaGetLastError();
}

unsigned row_tiles(const DenseArgs& a) { return (unsigned)(((int64_t)a.Sq * a.G + kT - 1) / kT); }

template <int D>
cudaError_t fwd_d(const DenseArgs& a, cudaStream_t st) {
  const size_t smem = (5 * Tile<D>::kFloats + Tile<D>::kFloatsP) * sizeof(float);
  return run(dense_fwd_kernel<D>, dim3(row_tiles(a) * a.splits, a.Hkv, a.B), smem, a, st);
}

template <int D>
cudaError_t bwd_d(const DenseArgs& a, cudaStream_t st) {
  const size_t smem = (4 * Tile<D>::kFloats + 2 * Tile<D>::kFloatsP) * sizeof(float);
  const cudaError_t e = run(dense_dq_kernel<D>, dim3(row_tiles(a), a.Hkv, a.B), smem, a, st);
  if (e != cudaSuccess) return e;
  return run(dense_dkv_kernel<D>, dim3((unsigned)((a.Sk + kT - 1) / kT), a.Hkv, a.B), smem, a, st);
}

unsigned warp_rows(const DenseArgs& a) {
  return (unsigned)(((int64_t)a.B * a.Hq * a.Sq + kThreads / 32 - 1) / (kThreads / 32));
}

}  // namespace

cudaError_t launch_dense_f32(const DenseArgs& a, cudaStream_t st) {
  return a.d == 128 ? fwd_d<128>(a, st) : fwd_d<64>(a, st);
}
cudaError_t launch_dense_f32_bwd(const DenseArgs& a, cudaStream_t st) {
  return a.d == 128 ? bwd_d<128>(a, st) : bwd_d<64>(a, st);
}
cudaError_t launch_dense_prepare(const DenseArgs& a, int dtype, cudaStream_t st) {
  auto warps = [](int64_t B, int64_t S, int64_t size) {
    return (B * ((S + size - 1) / size) + kThreads / 32 - 1) / (kThreads / 32);
  };
  const int64_t per = kThreads / (a.d / 8);
  const int64_t q0 = a.delta != nullptr ? ((int64_t)a.B * a.Hq * a.Sq + per - 1) / per : 0;
  const int64_t k0 = q0 + (a.doc_blocks_q != nullptr ? warps(a.B, a.Sq, a.doc_size_q) : 0);
  const int64_t end = k0 + (a.doc_blocks_k != nullptr ? warps(a.B, a.Sk, a.doc_size_k) : 0);
  if (end > 0x7fffffff) return cudaErrorInvalidValue;
  auto go = [&](auto kernel) {
    kernel<<<(unsigned)end, kThreads, 0, st>>>(a, q0, k0);
    return cudaGetLastError();
  };
  if (dtype == FVATTN_F32) return a.d == 128 ? go(dense_prepare_kernel<float, 128>) : go(dense_prepare_kernel<float, 64>);
  return a.d == 128 ? go(dense_prepare_kernel<__nv_bfloat16, 128>) : go(dense_prepare_kernel<__nv_bfloat16, 64>);
}

cudaError_t launch_dense_combine(const DenseArgs& a, int dtype, cudaStream_t st) {
  auto go = [&](auto kernel) { return launch_with(kernel, dim3(warp_rows(a)), kThreads, 0, st, 0, true, a); };
  if (dtype == FVATTN_F32) return a.d == 128 ? go(dense_combine_kernel<float, 128>) : go(dense_combine_kernel<float, 64>);
  return a.d == 128 ? go(dense_combine_kernel<__nv_bfloat16, 128>) : go(dense_combine_kernel<__nv_bfloat16, 64>);
}

}  // namespace fv
