// Device pieces that the tensor-core kernels of attention over all keys share (forward and backward):
// bounded waits, the walk over key blocks, masks, the score's cap and bias, and the tensor maps.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>

#include "dense.cuh"
#include "tc_ptx.cuh"
#include "tmap.cuh"

namespace fv {

constexpr uint32_t kWaitLimit = 1u << 22;    // polls of a bounded wait (seconds, not minutes)
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ void fail(int* abort, int code) { atomicCAS(abort, 0, code); }

// A bounded wait taken by a whole warp with one outcome for all lanes.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const volatile int* abort) {
  // the blocking poll takes 80 to 100 cycles even for a phase that is complete
  if (__all_sync(0xffffffffu, tc::mbar_test_wait(bar, parity))) return true;
  const bool ok = tc::mbar_wait(bar, parity, abort, kWaitLimit);
  return __all_sync(0xffffffffu, ok);
}

// The failure-path check's wait, at step g of a loader: on a barrier that nothing completes. A whole warp.
__device__ __forceinline__ bool held(const DenseArgs& a, uint64_t* hold, const volatile int* abort, uint32_t g) {
  if (a.hold_polls == 0 || g != a.hold_step) return false;
  return !__all_sync(0xffffffffu, tc::mbar_wait(hold, 0, abort, a.hold_polls));
}

// A barrier among `threads` threads of the CTA (id 0 is __syncthreads').
__device__ __forceinline__ void named_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// 2^x by the ex2.approx instruction (2^-inf = 0), and 1/x by rcp.approx (1/inf = 0).
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Packed pairs of fp32 (one 64-bit register): two operations per instruction.
__device__ __forceinline__ uint64_t f2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void f2_split(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t ffma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t fadd2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t fmul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float max32(const uint32_t (&s)[32]) {
  float m[11];
#pragma unroll
  for (int c = 0; c < 10; ++c)
    m[c] = max3(__uint_as_float(s[3 * c]), __uint_as_float(s[3 * c + 1]), __uint_as_float(s[3 * c + 2]));
  m[10] = fmaxf(__uint_as_float(s[30]), __uint_as_float(s[31]));
  return max3(max3(max3(m[0], m[1], m[2]), m[3], m[4]), max3(m[5], m[6], m[7]), max3(m[8], m[9], m[10]));
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// 32 fp32 results as bf16 (and, with rest, what the rounding leaves) to 16-byte aligned memory.
__device__ __forceinline__ void store_row32(__nv_bfloat16* out, __nv_bfloat16* rest, const uint32_t (&o)[32]) {
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    uint32_t w[4], z[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float x = __uint_as_float(o[8 * v + 2 * e]), y = __uint_as_float(o[8 * v + 2 * e + 1]);
      w[e] = pack_bf16(x, y);
      z[e] = pack_bf16(x - __uint_as_float(w[e] << 16), y - __uint_as_float(w[e] & 0xffff0000u));
    }
    reinterpret_cast<uint4*>(out)[v] = make_uint4(w[0], w[1], w[2], w[3]);
    if (rest != nullptr) reinterpret_cast<uint4*>(rest)[v] = make_uint4(z[0], z[1], z[2], z[3]);
  }
}

// The documents of a sequence's blocks of tokens (dense_prepare_kernel): x = the lowest number, with the
// sign bit set when the block has padding tokens too (0x7fffffff without any document); y = the
// highest (-1 without any).
__device__ __forceinline__ int doc_low(int2 v) { return v.x & 0x7fffffff; }
__device__ __forceinline__ bool doc_uniform(int2 v) { return v.x == v.y; }      // one document, no padding

// Ascending walk over the blocks [j, end) of tokens; with documents, over those whose documents meet the
// range [lo, hi]. Used by whole warps: a warp tests 32 blocks at a time.
template <bool DOCS>
struct BlockWalk {
  int j, end;
  __device__ __forceinline__ BlockWalk(const int2*, int begin, int stop, int, int) : j(begin), end(stop) {}
  __device__ __forceinline__ int next(int) { return j < end ? j++ : -1; }
  __device__ __forceinline__ int2 doc() const { return make_int2(0, 0); }
  __device__ __forceinline__ int count(int) const { return max(0, end - j); }
};
template <>
struct BlockWalk<true> {
  const int2* docs;
  int j, end, lo, hi;
  uint32_t word;          // blocks of the current window that are left
  int base;               // its first block
  int2 held;              // documents of block base + lane
  int at;                 // the last block that next() gave, counted from base

  __device__ __forceinline__ BlockWalk(const int2* docs_, int begin, int stop, int lo_, int hi_)
      : docs(docs_), j(begin), end(stop), lo(lo_), hi(hi_), word(0), base(begin), held(make_int2(0, 0)), at(0) {}
  __device__ __forceinline__ uint32_t window(int first, int lane, int2& v) const {
    v = first + lane < end ? docs[first + lane] : make_int2(0x7fffffff, -1);
    return __ballot_sync(0xffffffffu, doc_low(v) <= hi && v.y >= lo);
  }
  __device__ __forceinline__ int next(int lane) {
    while (word == 0) {
      if (j >= end) return -1;
      base = j;
      word = window(j, lane, held);
      j += 32;
    }
    at = __ffs(word) - 1;
    word &= word - 1;
    return base + at;
  }
  // The documents of the block that next() gave (they are in a lane's registers: no load).
  __device__ __forceinline__ int2 doc() const {
    return make_int2(__shfl_sync(0xffffffffu, held.x, at), __shfl_sync(0xffffffffu, held.y, at));
  }
  __device__ __forceinline__ int count(int lane) const {
    int n = 0;
    int2 v;
    for (int first = j; first < end; first += 32) n += __popc(window(first, lane, v));
    return n;
  }
};

// Bits of the lower n of 64 (n may be negative or above 64).
__device__ __forceinline__ uint64_t low64(int n) { return n >= 64 ? ~0ull : n <= 0 ? 0ull : (1ull << n) - 1ull; }

// For a warp whose lanes hold 64 document numbers (d0, d1: tokens lane and lane + 32) and one of their
// own: bit c of the result says that token c has this lane's. One round per distinct number among
// the lanes, which is one or two where documents are runs of tokens. The whole warp takes part.
__device__ __forceinline__ uint64_t same_document(int d0, int d1, int mine) {
  uint64_t same = 0ull;
  uint32_t left = 0xffffffffu;
  while (left != 0u) {
    const int d = __shfl_sync(0xffffffffu, mine, __ffs(left) - 1);
    const uint32_t lo = __ballot_sync(0xffffffffu, d0 == d), hi = __ballot_sync(0xffffffffu, d1 == d);
    if (mine == d) same = (uint64_t)hi << 32 | lo;
    left &= ~__ballot_sync(0xffffffffu, mine == d);
  }
  return same;
}

// Bit c: key first + c is visible to this lane's row; v: the documents of the block it lies in. The
// whole warp takes part.
template <bool DOCS>
__device__ __forceinline__ uint64_t visible64(const DenseRow& row, const int32_t* doc_k, int2 v, int first, int Sk,
                                              int lane) {
  uint64_t see = low64(row.limit - first);
  if (DOCS) {
    if (doc_uniform(v)) {
      if (v.y != row.doc) see = 0ull;
    } else {
      const int d0 = first + lane < Sk ? doc_k[first + lane] : -1;
      const int d1 = first + 32 + lane < Sk ? doc_k[first + 32 + lane] : -1;
      see &= same_document(d0, d1, row.doc);      // a padding row's limit is 0
    }
  }
  return see;
}

// tanh on pairs: y times a polynomial in y^2, fitted to the least largest error (2e-8 either way; 1e-7
// with fp32 arithmetic), of degree 4 for |y| <= 0.6 and 6 for |y| <= 1. On the FMA pipe: the
// exponentials of the softmax already fill the SFU, and tanh by exponential and reciprocal would triple
// its work.
template <int DEGREE>
__device__ __forceinline__ uint64_t tanh_small2(uint64_t y) {
  constexpr float c4[5] = {0.9999996423721313f, -0.33331209421157837f, 0.13299210369586945f, -0.05169673636555672f,
                           0.01497695129364729f};
  constexpr float c6[7] = {0.9999997019767761f,    -0.33332130312919617f, 0.13319583237171173f, -0.05326582491397858f,
                           0.01997326873242855f, -0.005951268598437309f, 0.0009637684561312199f};
  const uint64_t u = fmul2(y, y);
  uint64_t p = DEGREE == 4 ? f2(c4[4], c4[4]) : f2(c6[6], c6[6]);
#pragma unroll
  for (int k = DEGREE - 1; k >= 0; --k) p = ffma2(p, u, DEGREE == 4 ? f2(c4[k % 5], c4[k % 5]) : f2(c6[k], c6[k]));
  return fmul2(p, y);
}
// tanh(y) = 1 - 2 / (1 + e^2y), off by a few 2^-24; e^2y at inf or 0 gives 1 and -1. For |y| > 1 only: below,
// the difference cancels, and times a cap of 1e6 the 2^-24 would be an error of 0.1 in a small score.
__device__ __forceinline__ float tanh_large(float y) {
  return fmaf(-2.f, rcp(1.f + ex2(y * (2.f * kLog2e))), 1.f);
}
// Two values of any size, each by its own form; all_small: none of the warp's is above 1.
__device__ __forceinline__ void tanh_any2(float y0, float y1, bool all_small, float& t0, float& t1) {
  f2_split(tanh_small2<6>(f2(y0, y1)), t0, t1);
  if (all_small) return;
  if (!(fabsf(y0) <= 1.f)) t0 = tanh_large(y0);
  if (!(fabsf(y1) <= 1.f)) t1 = tanh_large(y1);
}
__device__ __forceinline__ float abs_max32(const uint32_t (&s)[32]) {
  float m = 0.f;
#pragma unroll
  for (int c = 0; c < 32; c += 2)
    m = max3(m, fabsf(__uint_as_float(s[c])), fabsf(__uint_as_float(s[c + 1])));
  return m;
}

template <int DEGREE>
__device__ __forceinline__ void tanh32_small(uint32_t (&s)[32], float in) {
  const uint64_t in2 = f2(in, in);
#pragma unroll
  for (int c = 0; c < 32; c += 2) {
    float a, b;
    f2_split(tanh_small2<DEGREE>(fmul2(f2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), in2)), a, b);
    s[c] = __float_as_uint(a);
    s[c + 1] = __float_as_uint(b);
  }
}
// x[c] stays where bit c of `see` is set and becomes `other` elsewhere.
__device__ __forceinline__ void only32(uint32_t (&x)[32], uint32_t see, float other) {
#pragma unroll
  for (int c = 0; c < 32; ++c)
    if (!((see >> c) & 1u)) x[c] = __float_as_uint(other);
}
// s <- tanh(s * in), by the shortest form that every score of the warp allows. Hidden scores (bits of `see`
// that are not set, where there are any) are left out, or what must not matter (rows that no query fills,
// memory behind the valid keys, padding) would choose the form; a second look does, since most often all of
// them are small (hiding them first took packed training with a cap from 112 to 119 us). The whole warp
// takes part.
__device__ __forceinline__ void tanh32(uint32_t (&s)[32], float in, bool hidden, uint32_t see) {
  float top = abs_max32(s) * in;
  if (hidden && !__all_sync(0xffffffffu, top <= 0.6f)) {
    top = 0.f;
#pragma unroll
    for (int c = 0; c < 32; ++c)
      if ((see >> c) & 1u) top = fmaxf(top, fabsf(__uint_as_float(s[c])));
    top *= in;
  }
  if (__all_sync(0xffffffffu, top <= 0.6f)) {
    tanh32_small<4>(s, in);
  } else if (__all_sync(0xffffffffu, top <= 1.f)) {
    tanh32_small<6>(s, in);
  } else {
#pragma unroll
    for (int c = 0; c < 32; c += 2) {
      float a, b;
      tanh_any2(__uint_as_float(s[c]) * in, __uint_as_float(s[c + 1]) * in, false, a, b);
      s[c] = __float_as_uint(a);
      s[c + 1] = __float_as_uint(b);
    }
  }
}

// The score of a raw product, a row per lane: `apply` leaves values that `after` takes to base-2
// exponents (products, after = scale log2 e; tanh, after = cap log2 e; biased exponents, after = 1).
template <bool CAP, bool BIAS>
struct ScoreMap {
  float in, factor, after, slope2;
  __device__ __forceinline__ ScoreMap(const DenseArgs& a, const DenseRow& row) {
    in = CAP ? a.scale / a.cap : 0.f;
    factor = (CAP ? a.cap : a.scale) * kLog2e;
    after = BIAS ? 1.f : factor;
    slope2 = row.slope * kLog2e;
  }
  // 32 scores in place; far = position of the row minus the first key; hidden, see: as for tanh32, and of
  // hidden scores nothing is said. The whole warp takes part.
  __device__ __forceinline__ void apply(uint32_t (&s)[32], int far, bool hidden, uint32_t see) const {
    if (CAP) tanh32(s, in, hidden, see);
    if (BIAS) bias(s, far);
  }
  __device__ __forceinline__ void bias(uint32_t (&s)[32], int far) const {
    const float f = (float)far;
    const bool past = __all_sync(0xffffffffu, far >= 31), ahead = __all_sync(0xffffffffu, far <= 0);
    if (past || ahead) {
      // all keys on one side of every row: the bias is linear in the key
      const float k1 = past ? slope2 : -slope2, k0 = -k1 * f;
      const uint64_t k12 = f2(k1, k1), k02 = f2(k0, k0), factor2 = f2(factor, factor);
#pragma unroll
      for (int c = 0; c < 32; c += 2) {
        float x, y;
        f2_split(ffma2(f2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), factor2,
                       ffma2(k12, f2((float)c, (float)(c + 1)), k02)), x, y);
        s[c] = __float_as_uint(x);
        s[c + 1] = __float_as_uint(y);
      }
    } else {
#pragma unroll
      for (int c = 0; c < 32; ++c)
        s[c] = __float_as_uint(fmaf(-slope2, fabsf(f - (float)c), __uint_as_float(s[c]) * factor));
    }
  }
};

// p times the cap's derivative 1 - t^2, in pairs.
__device__ __forceinline__ uint64_t times_dcap(uint64_t p, uint64_t t) {
  const uint64_t tt = fmul2(fmul2(t, f2(-1.f, -1.f)), t);
  return ffma2(p, tt, p);
}

// Which tile a CTA takes. Under an order the tiles of a head differ in length and the longest should
// start first, over all heads; but the heads in flight share L2, so heads go in groups whose keys fit
// half of it. Otherwise a head's tiles run next to one another.
struct TileOrder {
  int group;       // key heads (over the batch) per group
  int tiles;       // tiles (or tiles x splits) per key head
  int heads;       // B * Hkv
};
__device__ __forceinline__ void tile_of(const TileOrder& o, int64_t x, int& tile, int& bh) {
  const int64_t per = (int64_t)o.group * o.tiles;
  const int grp = (int)(x / per), rest = (int)(x - grp * per);
  const int n = min(o.group, o.heads - grp * o.group);
  tile = rest / n;
  bh = grp * o.group + rest % n;
}
inline TileOrder tile_order(const DenseArgs& a, int tiles, bool longest_first) {
  const int64_t heads = (int64_t)a.B * a.Hkv, bytes = (int64_t)(longest_first ? a.Sk : 1) * a.d * 4;
  const int64_t fit = imax<int64_t>(1, (int64_t)(60 << 20) / bytes);
  return TileOrder{longest_first ? (int)imin(heads, fit) : 1, tiles, (int)heads};
}

// `rows` tokens from token t0 of a [token][D] matrix into a tile of 128-byte swizzled rows (chunks of 64
// dims), zeros for tokens at or past `end` and for padding documents; lanes `me` of `of`.
template <int D>
__device__ __forceinline__ void copy_keys(unsigned char* dst, const __nv_bfloat16* base, int64_t stride, int t0, int rows,
                                          int end, const int32_t* doc, int me, int of) {
  for (int x = me; x < rows * (D / 8); x += of) {
    const int r = x / (D / 8), c = x % (D / 8);
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (t0 + r < end && (doc == nullptr || doc[t0 + r] >= 0))
      v = *reinterpret_cast<const uint4*>(base + (int64_t)(t0 + r) * stride + c * 8);
    *reinterpret_cast<uint4*>(dst + (c / 8) * rows * 128 + r * 128 + (((c % 8) ^ (r & 7)) << 4)) = v;
  }
}

// The rows of `queries` queries from i0 of a key head's group into a tile of ROWS rows, in the order of
// make_map_rows; zeros for queries at or past Sq and for padding ones.
template <int D, int ROWS>
__device__ __forceinline__ void copy_rows(unsigned char* dst, const __nv_bfloat16* base, const fvattn_strides& s,
                                          const DenseArgs& a, int b, int h, int i0, int queries, const int32_t* doc,
                                          int me, int of) {
  for (int x = me; x < queries * a.G * (D / 8); x += of) {
    const int r = x / (D / 8), c = x % (D / 8), i = i0 + r / a.G;
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (i < a.Sq && (doc == nullptr || doc[i] >= 0))
      v = *reinterpret_cast<const uint4*>(base + (int64_t)b * s.b + (int64_t)(h * a.G + r % a.G) * s.h + (int64_t)i * s.s +
                                          c * 8);
    *reinterpret_cast<uint4*>(dst + (c / 8) * ROWS * 128 + r * 128 + (((c % 8) ^ (r & 7)) << 4)) = v;
  }
}

// ------------------------------------------------------------------ tensor maps (host)

inline bool encode_bf16(CUtensorMap* map, const void* base, int rank, const cuuint64_t* dims, const int64_t* strides,
                        const cuuint32_t* box) {
  EncodeTiledFn enc = encode_fn();
  if (enc == nullptr) return false;
  cuuint64_t bytes[4];
  for (int i = 0; i < rank - 1; ++i) bytes[i] = (cuuint64_t)strides[i] * 2;
  const cuuint32_t one[5] = {1, 1, 1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void*>(base), dims, bytes, box, one,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [B][Hq][Sq][d] seen as [B][Hkv][Sq][G][d], read in boxes of `queries` queries of all G heads and 64
// dims: row i * G + g of the box is query i of head g. Queries past Sq read as zeros.
inline bool make_map_rows(CUtensorMap* map, const void* base, const fvattn_strides& s, const DenseArgs& a, int queries) {
  const cuuint64_t dims[5] = {(cuuint64_t)a.d, (cuuint64_t)a.G, (cuuint64_t)a.Sq, (cuuint64_t)a.Hkv, (cuuint64_t)a.B};
  const int64_t strides[4] = {s.h, s.s, s.h * a.G, s.b};
  const cuuint32_t box[5] = {64, (cuuint32_t)a.G, (cuuint32_t)queries, 1, 1};
  return encode_bf16(map, base, 5, dims, strides, box);
}

// [B][Hkv][Sk][d], read in boxes of `keys` keys and 64 dims; keys past Sk read as zeros.
inline bool make_map_keys(CUtensorMap* map, const void* base, const fvattn_strides& s, const DenseArgs& a, int keys) {
  const cuuint64_t dims[4] = {(cuuint64_t)a.d, (cuuint64_t)a.Sk, (cuuint64_t)a.Hkv, (cuuint64_t)a.B};
  const int64_t strides[3] = {s.s, s.h, s.b};
  const cuuint32_t box[4] = {64, (cuuint32_t)keys, 1, 1};
  return encode_bf16(map, base, 4, dims, strides, box);
}

}  // namespace fv
