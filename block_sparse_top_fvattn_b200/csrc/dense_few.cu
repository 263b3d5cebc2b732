// Attention over all keys for few rows (single tokens over a cache): at most 16 rows, queries times the
// heads that share a key head. bf16 inputs, fp32 scores, softmax statistics and sums.
//
// Bound by reading K and V once from HBM, and by latency where they are short. A tile of 128 rows, as
// the tcgen05 kernel has, would leave one warp of four to do the softmax of a few rows over all keys; here
// four warps take 16 keys each of every block of 64, keep a running maximum, sum and output of
// their own (mma.sync m16n8k16: 16 rows are all it has, 3 % of the tensor rate is all this needs), and
// join them at the end. K and V blocks come by TMA through three stages of 32 KB (d = 128), two CTAs
// per SM: about 190 KB in flight per SM, twice what HBM's latency asks for.
// The keys are split over CTAs until all SMs have work. The splits of a key head form clusters of up to
// eight, which join their results through distributed shared memory; only where eight are not enough
// do partial results go through memory and a second kernel.
//
// P is rounded to bf16 for the second product, and goes in as two bf16 terms with rest: without it outputs are
// off by 0.0018 of their size, where an fp32 computation rounded once is off by 0.0017; the second term always
// would cost 2 us of the 136.
//
// Measured: single tokens over 8 caches of up to 32760, 32 / 8 heads, capped: 136 us, 95 % of the copy rate
// (tiles of 128 rows on tcgen05: 193 us); 4 caches of up to 1000, 8 / 2 heads: 6.7 us (15 us).
//
// Every wait is bounded; one that runs out is reported in the status word and makes the rows NaN.
#include <cooperative_groups.h>
#include <cuda.h>
#include <cuda_bf16.h>

#include "dense.cuh"
#include "dense_tc.cuh"
#include "tc_ptx.cuh"
#include "tmap.cuh"

namespace cg = cooperative_groups;

namespace fv {

namespace {

constexpr int kStages = 3;
constexpr int kWork = 4;                       // warps with keys; one more loads
constexpr int kThreads = (kWork + 1) * 32;
constexpr int kRows = 16;

struct FewBars {
  uint64_t full[kStages], empty[kStages];
  uint64_t hold;                               // never completes (failure-path check)
  float m[kWork][kRows], l[kWork][kRows];      // statistics of the warps
  int doc_lo, doc_hi;
  int abort;
};

template <int D>
struct FewLayout {
  static constexpr int kChunk = kBlock * 128;                // [64 keys x 64 dims] bf16
  static constexpr int kTile = (D / 64) * kChunk;
  static constexpr int kStage = 2 * kTile;                   // K, V
  static constexpr int kOffBar = kStages * kStage;
  static constexpr int kBytes = kOffBar + (int)sizeof(FewBars);
  // at the end, over the stages: the warps' outputs and statistics, then the CTA's
  static constexpr int kOffOut = kWork * kRows * D * 4;
  static_assert(kOffOut + kRows * D * 4 <= kStages * kStage, "the results fit the stages");
};

struct FewStats {
  float m[kRows], l[kRows];                    // of the CTA, for its cluster
};

__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// c[16 x 8] += a[16 x 16] b[16 x 8]
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Byte offset of 16-byte chunk c (of d / 8) of key r in a tile of 64 keys (128-byte swizzle).
__device__ __forceinline__ uint32_t tile_at(int r, int c) {
  return (uint32_t)((c >> 3) * (kBlock * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

// grid: (splits, B * Hkv), clusters of `a.cluster` splits
template <int D, bool CAP, bool BIAS, bool DOCS>
__global__ void __launch_bounds__(kThreads, 2)
    dense_few_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const DenseArgs a) {
  using L = FewLayout<D>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  FewBars* bars = reinterpret_cast<FewBars*>(smem + L::kOffBar);
  __shared__ FewStats cta;
  if (DOCS) wait_for_previous_grid();              // the documents of the blocks
  allow_next_grid();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort = &bars->abort;
  const int split = blockIdx.x, bh = blockIdx.y, b = bh / a.Hkv, h = bh - b * a.Hkv;
  const DenseSeq seq = dense_seq(a, b);
  const int32_t* doc_k = DOCS ? a.mask.doc_k + (int64_t)b * a.Sk : nullptr;
  const int nrows = a.Sq * a.G;
  const int key0 = split * a.split_keys;
  const int key1 = (int)imin<int64_t>(dense_limit(seq, a.causal, a.Sq - 1), (int64_t)key0 + a.split_keys);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      tc::mbar_init(&bars->full[s], 1);
      tc::mbar_init(&bars->empty[s], kWork);
    }
    tc::mbar_init(&bars->hold, 1);
    bars->abort = 0;
    int lo = 0x7fffffff, hi = -1;
    if (DOCS) {
      for (int i = 0; i < a.Sq; ++i) {
        const int d = a.mask.doc_q[(int64_t)b * a.Sq + i];
        if (d >= 0) {
          lo = min(lo, d);
          hi = max(hi, d);
        }
      }
    }
    bars->doc_lo = lo;
    bars->doc_hi = hi;
    tc::fence_mbar_init();
  }
  __syncthreads();
  const int2* docs = DOCS ? a.doc_blocks_k + (int64_t)b * ((a.Sk + kBlock - 1) / kBlock) : nullptr;
  BlockWalk<DOCS> walk(docs, key0 / kBlock, (key1 + kBlock - 1) / kBlock, bars->doc_lo, bars->doc_hi);

  // Thread (lane) of a warp with keys: rows r0 = lane / 4 and r0 + 8; columns 2 (lane % 4) and the next of
  // every eight.
  const int r0 = lane >> 2, c0 = (lane & 3) * 2;
  float o[D / 8][4];
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
  for (int n = 0; n < D / 8; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[n][e] = 0.f;

  if (warp == kWork) {
    // ------------------------------------------------------------ loader
    uint32_t g = 0, armed = 0;
    for (int j; (j = walk.next(lane)) >= 0; ++g) {
      const int s = g % kStages;
      if (held(a, &bars->hold, abort, g)) {
        fail(&bars->abort, 20);
        break;
      }
      if (!warp_wait(&bars->empty[s], ((g / kStages) & 1) ^ 1, abort)) {
        fail(&bars->abort, 1);
        break;
      }
      if (lane == 0) {
        tc::mbar_expect_tx(&bars->full[s], L::kStage);
        for (int c = 0; c < D / 64; ++c) {
          tc::tma_load_4d(smem + s * L::kStage + c * L::kChunk, &tmK, &bars->full[s], c * 64, j * kBlock, h, b);
          tc::tma_load_4d(smem + s * L::kStage + L::kTile + c * L::kChunk, &tmV, &bars->full[s], c * 64, j * kBlock, h, b);
        }
      }
      armed = g + 1;
    }
    // no copy may still be writing shared memory when the CTA goes on to its results
    if (lane == 0)
      for (uint32_t k = armed > kStages ? armed - kStages : 0; k < armed; ++k)
        tc::mbar_wait_drain(&bars->full[k % kStages], (k / kStages) & 1, kWaitLimit);
  } else {
    // ------------------------------------------------------------ 16 keys of every block
    DenseRow row[2];
    uint32_t qf[D / 16][4];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int r = r0 + 8 * u;
      row[u] = DenseRow{0, 0, 0, 0.f};
      const __nv_bfloat16* p = nullptr;
      if (r < nrows) {
        const int i = r / a.G, hq = h * a.G + r % a.G;
        row[u] = dense_row(a, seq, b, hq, i);
        p = static_cast<const __nv_bfloat16*>(a.q) + (int64_t)b * a.qs.b + (int64_t)hq * a.qs.h + (int64_t)i * a.qs.s;
      }
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        qf[k][u] = p != nullptr ? *reinterpret_cast<const uint32_t*>(p + k * 16 + c0) : 0u;
        qf[k][u + 2] = p != nullptr ? *reinterpret_cast<const uint32_t*>(p + k * 16 + 8 + c0) : 0u;
      }
    }
    const float in = CAP ? a.scale / a.cap : 0.f, factor = (CAP ? a.cap : a.scale) * kLog2e;
    uint32_t g = 0;
    for (int j; (j = walk.next(lane)) >= 0; ++g) {
      const int s = g % kStages;
      if (!warp_wait(&bars->full[s], (g / kStages) & 1, abort)) {
        fail(&bars->abort, 2);
        break;
      }
      unsigned char* sv = smem + s * L::kStage + L::kTile;
      const uint32_t ka = tc::smem_u32(smem + s * L::kStage), va = tc::smem_u32(sv);
      const int first = j * kBlock + warp * 16;
      // keys that do not exist although their memory does: zeros, whatever it holds (0 * NaN would reach O)
      const bool dirty = (seq.kv < a.Sk && (j + 1) * kBlock > seq.kv) || (DOCS && walk.doc().x < 0);
      if (dirty) {
        for (int x = lane; x < 16 * (D / 8); x += 32) {
          const int r = x / (D / 8), key = first + r;
          if (key >= seq.kv || (DOCS && doc_k[key] < 0))
            *reinterpret_cast<uint4*>(sv + tile_at(warp * 16 + r, x % (D / 8))) = make_uint4(0u, 0u, 0u, 0u);
        }
        tc::fence_proxy_async_smem();
        __syncwarp();
      }
      float sc[2][4];
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[n][e] = 0.f;
#pragma unroll
      for (int k = 0; k < D / 32; ++k)
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          uint32_t f[4];
          ldmatrix4(ka + tile_at(warp * 16 + n * 8 + (lane & 7), k * 4 + (lane >> 3)), f);
          mma16816(sc[n], qf[2 * k], f[0], f[1]);
          mma16816(sc[n], qf[2 * k + 1], f[2], f[3]);
        }
      float mx[2] = {-INFINITY, -INFINITY};
      if (CAP) {
        float top = 0.f;
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            sc[n][e] *= in;
            top = fmaxf(top, fabsf(sc[n][e]));
          }
        // a value's form does not depend on the others', so hidden ones may be anything
        const bool all_small = __all_sync(0xffffffffu, top <= 1.f);
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; e += 2) tanh_any2(sc[n][e], sc[n][e + 1], all_small, sc[n][e], sc[n][e + 1]);
      }
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int u = e >> 1, key = first + n * 8 + c0 + (e & 1);
          float x = sc[n][e] * factor;
          if (BIAS) x = fmaf(-row[u].slope * kLog2e, (float)abs(row[u].pos - key), x);
          const bool see = key < row[u].limit && (!DOCS || doc_k[key] == row[u].doc);
          sc[n][e] = see ? x : -INFINITY;
          mx[u] = fmaxf(mx[u], sc[n][e]);
        }
      float alpha[2];
      bool grow = false;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        mx[u] = fmaxf(mx[u], __shfl_xor_sync(0xffffffffu, mx[u], 1));
        mx[u] = fmaxf(mx[u], __shfl_xor_sync(0xffffffffu, mx[u], 2));
        const float top = fmaxf(m[u], mx[u]);
        alpha[u] = m[u] == -INFINITY ? 1.f : ex2(m[u] - top);       // nothing seen before: all is zero
        grow = grow || alpha[u] != 1.f;
        m[u] = top;
      }
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[n][e] *= alpha[e >> 1];
        l[0] *= alpha[0];
        l[1] *= alpha[1];
      }
      uint32_t pf[4], left[4];                      // P, and with rest what its rounding left
      const float base[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const float p0 = ex2(sc[n][2 * u] - base[u]), p1 = ex2(sc[n][2 * u + 1] - base[u]);
          l[u] += p0 + p1;
          const uint32_t pk = pack_bf16(p0, p1);
          pf[n * 2 + u] = pk;
          left[n * 2 + u] = pack_bf16(p0 - __uint_as_float(pk << 16), p1 - __uint_as_float(pk & 0xffff0000u));
        }
#pragma unroll
      for (int n = 0; n < D / 16; ++n) {
        uint32_t f[4];
        ldmatrix4_trans(va + tile_at(warp * 16 + ((lane >> 3) & 1) * 8 + (lane & 7), n * 2 + (lane >> 4)), f);
        mma16816(o[2 * n], pf, f[0], f[1]);
        mma16816(o[2 * n + 1], pf, f[2], f[3]);
        if (a.rest != nullptr) {
          mma16816(o[2 * n], left, f[0], f[1]);
          mma16816(o[2 * n + 1], left, f[2], f[3]);
        }
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&bars->empty[s]);
    }
  }
  // ------------------------------------------------------------ the warps' results
  __syncthreads();                                  // every stage has been read, no copy is in flight
  float* part = reinterpret_cast<float*>(smem);     // [warp][row][dim]
  float* mine = part + L::kOffOut / 4;              // the CTA's [row][dim], not divided by its sum
  if (warp < kWork) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      l[u] += __shfl_xor_sync(0xffffffffu, l[u], 1);
      l[u] += __shfl_xor_sync(0xffffffffu, l[u], 2);
      if ((lane & 3) == 0) {
        bars->m[warp][r0 + 8 * u] = m[u];
        bars->l[warp][r0 + 8 * u] = l[u];
      }
#pragma unroll
      for (int n = 0; n < D / 8; ++n)
        *reinterpret_cast<float2*>(part + (warp * kRows + r0 + 8 * u) * D + n * 8 + c0) =
            make_float2(o[n][2 * u], o[n][2 * u + 1]);
    }
  }
  __syncthreads();
  const bool broken = *abort != 0;
  for (int x = threadIdx.x; x < nrows * D; x += kThreads) {
    const int r = x / D, d = x - r * D;
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWork; ++w) top = fmaxf(top, bars->m[w][r]);
    const float base = top == -INFINITY ? 0.f : top;
    float acc = 0.f, sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWork; ++w) {
      const float f = ex2(bars->m[w][r] - base);
      acc = fmaf(f, part[(w * kRows + r) * D + d], acc);
      sum = fmaf(f, bars->l[w][r], sum);
    }
    mine[r * D + d] = acc;
    if (d == 0) {
      cta.m[r] = top;
      cta.l[r] = broken ? __int_as_float(0x7fffffff) : sum;
    }
  }
  // ------------------------------------------------------------ the cluster's
  cg::cluster_group cluster = cg::this_cluster();
  cluster.sync();
  const int ranks = a.cluster, rank = (int)cluster.block_rank();
  const int64_t rows_all = (int64_t)a.B * a.Hq * a.Sq;
  for (int x = rank * kThreads + threadIdx.x; x < nrows * D; x += ranks * kThreads) {
    const int r = x / D, d = x - r * D;
    float top = -INFINITY;
    for (int k = 0; k < ranks; ++k) top = fmaxf(top, cluster.map_shared_rank(&cta, k)->m[r]);
    const float base = top == -INFINITY ? 0.f : top;
    float acc = 0.f, sum = 0.f;
    for (int k = 0; k < ranks; ++k) {
      const FewStats* st = cluster.map_shared_rank(&cta, k);
      const float f = ex2(st->m[r] - base);
      acc = fmaf(f, cluster.map_shared_rank(mine, k)[x], acc);
      sum = fmaf(f, st->l[r], sum);
    }
    const float y = sum == 0.f ? 0.f : acc / sum;
    const float lse = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.69314718055994531f;
    const int i = r / a.G, hq = h * a.G + r % a.G;
    const int64_t flat = ((int64_t)b * a.Hq + hq) * a.Sq + i;
    if (a.parts > 1) {
      const int64_t at = (int64_t)(split / ranks) * rows_all + flat;
      a.part_o[at * D + d] = y;
      if (d == 0) a.part_lse[at] = lse;
    } else {
      const int64_t at = (int64_t)b * a.os.b + (int64_t)hq * a.os.h + (int64_t)i * a.os.s + d;
      const __nv_bfloat16 z = __float2bfloat16_rn(y);
      static_cast<__nv_bfloat16*>(a.out)[at] = z;
      if (a.rest != nullptr) static_cast<__nv_bfloat16*>(a.rest)[at] = __float2bfloat16_rn(y - __bfloat162float(z));
      if (d == 0 && a.lse != nullptr) a.lse[flat] = lse;
    }
  }
  cluster.sync();                                   // a CTA's shared memory is read until here
  if (threadIdx.x == 0 && broken && a.status != nullptr) report_error(a.status, FVATTN_ERR_TIMEOUT, 500 + bars->abort);
}

template <int D, bool CAP, bool BIAS, bool DOCS>
cudaError_t launch(const DenseArgs& a, cudaStream_t st) {
  CUtensorMap mk, mv;
  if (!make_map_keys(&mk, a.k, a.ks, a, kBlock) || !make_map_keys(&mv, a.v, a.vs, a, kBlock)) return cudaErrorInvalidValue;
  const size_t smem = FewLayout<D>::kBytes + 1024;
  auto* kernel = dense_few_kernel<D, CAP, BIAS, DOCS>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_with(kernel, dim3((unsigned)a.splits, (unsigned)(a.B * a.Hkv)), kThreads, smem, st, a.cluster, DOCS, mk, mv,
                     a);
}

template <int D, bool DOCS>
cudaError_t launch_docs(const DenseArgs& a, cudaStream_t st) {
  const bool cap = a.cap > 0.f, bias = a.mask.slopes != nullptr;
  if (cap) return bias ? launch<D, true, true, DOCS>(a, st) : launch<D, true, false, DOCS>(a, st);
  return bias ? launch<D, false, true, DOCS>(a, st) : launch<D, false, false, DOCS>(a, st);
}

template <int D>
cudaError_t launch_d(const DenseArgs& a, cudaStream_t st) {
  return a.mask.doc_k != nullptr ? launch_docs<D, true>(a, st) : launch_docs<D, false>(a, st);
}

}  // namespace

cudaError_t launch_dense_few(const DenseArgs& a, cudaStream_t st) {
  return a.d == 128 ? launch_d<128>(a, st) : launch_d<64>(a, st);
}

}  // namespace fv
