// Attention over all keys on the B200 tensor cores (tcgen05, TMEM, TMA): bf16 inputs, fp32 scores,
// softmax statistics and sums.
//
//   s_ij = cap tanh(scale q_i.k_j / cap) - slope |p_i - j|, out_i = sum_j softmax_j(s_ij) v_j
//
// One CTA takes 128 rows of one key head (row i * G + g: query i of the group's head g, so that shared
// keys are read once) and one range of its keys, in blocks of 64 keys; for each block j
//   S = Q K_j^T          tcgen05.mma M=128 N=64 K=d, fp32 in TMEM, two buffers
//   P = exp2(s - m)      one thread per row: cap, bias and mask of its row, running maximum m that is
//                        raised (with a rescale of O in TMEM) only when it grows by more than 2^8,
//                        P as bf16 over its S buffer. Capped scores, e^-cap to e^cap, would do without a
//                        maximum (prompts: 57.7 instead of 61.1 us), but then large values overflow
//                        and small ones vanish
//   O += P V_j           tcgen05.mma M=128 N=d K=64, P read from TMEM
// Two CTAs share an SM, so one's softmax runs beside the other's products. Blocks that no row of the
// tile can see (behind the limit of its last query, or of other documents) are not visited.
// A few queries over many keys leave most rows empty: the warps of empty rows skip the softmax, the
// keys are split over CTAs, and the partial results are joined by a second kernel.
//
// Rounding P to bf16 is what the second product's operands need; the row sums are of the unrounded P. It leaves
// outputs off by 0.0023 of their size, where an fp32 computation rounded once is off by 0.0017.
// With rest (the output to 16 bits, for the gradients) P goes in as two bf16 terms, the second of them
// what the rounding of the first left, behind it in the S buffer, and the second product is made twice.
//
// Bound by the chain of a softmax warp's step (wait, load, maximum, exponentials, store), not by the SFU
// alone: a polynomial on the FMA pipe for 1/8 to 1/2 of the exponentials gained nothing (packed clips 160 us
// without, 161 to 168 with). Measured, d = 128:
// packed clips of 16380 tokens, 6 heads: 158 us, 633 TFLOP/s; prompts of 2 x 2047 tokens, 16 / 4 heads, capped:
// 61 us; with rest, 8192 causal tokens, 12 heads: 234 us, tensor pipe 72 % active (183 us without rest).
//
// Every wait is bounded; one that runs out stops every role without leaving a copy or product in
// flight, is reported in the status word, and makes the tile's rows NaN.
#include <cuda.h>
#include <cuda_bf16.h>

#include <type_traits>

#include "dense.cuh"
#include "dense_tc.cuh"
#include "tc_ptx.cuh"
#include "tmap.cuh"

namespace fv {

namespace {

constexpr int NS = 2;          // stages of K and of V; the stage of a step is also its S / P buffer
constexpr int kWarps = 6;      // loader, MMA, four softmax warps
constexpr float kRescaleLog2 = 8.0f;

template <int D>
struct FwdLayout {
  static constexpr int kQChunk = kTileRows * 128;     // [128 rows x 64 dims] bf16
  static constexpr int kQBytes = (D / 64) * kQChunk;
  static constexpr int kKVChunk = kBlock * 128;       // [64 keys x 64 dims] bf16
  static constexpr int kKBytes = (D / 64) * kKVChunk;
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = kQBytes;
  static constexpr int kOffV = kOffK + NS * kKBytes;
  static constexpr int kOffBar = kOffV + NS * kKBytes;
  static constexpr int kBytes = kOffBar + 256;
  static constexpr uint32_t kTmemCols = 256;          // S / P buffers at 0 and 64, O at 128
  static constexpr uint32_t kColO = 128;
};

struct FwdBars {
  uint64_t q_full;
  uint64_t k_full[NS];
  uint64_t s_full[2];     // S of a step done: the softmax may read it, its K stage may be refilled
  uint64_t p_full[2];     // P written by the four softmax warps and V landed (the V loader's arrival)
  uint64_t pv_done[2];    // P V done: O is stable, the V stage may be refilled
  uint64_t drain;         // every product of the CTA is done
  uint64_t hold;          // never completes (failure-path check)
  int p_arrived[4];       // per softmax warp: the last step whose P it published
  int v_armed;            // the last step whose V copy was issued
  int doc_lo, doc_hi;     // documents of the tile's rows
  uint32_t tmem_base;
  int abort;
};

static_assert(sizeof(FwdBars) <= 256, "the barriers fit their place");

template <int D, bool CAP, bool BIAS, bool DOCS>
__global__ void __launch_bounds__(kWarps * 32, 2)
    dense_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV, const DenseArgs a, const int qpt,
                    const TileOrder order) {
  using L = FwdLayout<D>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  FwdBars* bars = reinterpret_cast<FwdBars*>(smem + L::kOffBar);
  unsigned char* sQ = smem + L::kOffQ;
  unsigned char* sK = smem + L::kOffK;
  unsigned char* sV = smem + L::kOffV;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort = &bars->abort;
  if (DOCS) wait_for_previous_grid();      // the documents of the blocks
  allow_next_grid();

  int x, bh;
  tile_of(order, blockIdx.x, x, bh);
  const int split = x % a.splits, t = order.tiles / a.splits - 1 - x / a.splits;
  const int b = bh / a.Hkv, h = bh - b * a.Hkv;
  const int i0 = t * qpt, i1 = min(i0 + qpt, a.Sq);                   // this tile's queries
  const DenseSeq seq = dense_seq(a, b);
  const int key0 = split * a.split_keys;
  const int key1 = (int)imin<int64_t>(dense_limit(seq, a.causal, i1 - 1), (int64_t)key0 + a.split_keys);

  if (threadIdx.x == 0) {
    tc::mbar_init(&bars->q_full, 1);
    for (int s = 0; s < 2; ++s) {
      tc::mbar_init(&bars->k_full[s], 1);
      tc::mbar_init(&bars->s_full[s], 1);
      tc::mbar_init(&bars->p_full[s], 5);
      tc::mbar_init(&bars->pv_done[s], 1);
    }
    tc::mbar_init(&bars->drain, 1);
    tc::mbar_init(&bars->hold, 1);
    for (int w = 0; w < 4; ++w) bars->p_arrived[w] = -1;
    bars->v_armed = -1;
    bars->abort = 0;
    bars->doc_lo = 0x7fffffff;
    bars->doc_hi = -1;
    tc::fence_mbar_init();
  }
  if (warp == 1) {
    tc::tmem_alloc(&bars->tmem_base, L::kTmemCols);
    tc::tmem_relinquish();
  }
  if (warp == 0 && lane == 0) {
    tc::prefetch_tmap(&tmQ);
    tc::prefetch_tmap(&tmK);
    tc::prefetch_tmap(&tmV);
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (DOCS) {
    for (int i = i0 + threadIdx.x; i < i1; i += kWarps * 32) {
      const int doc = a.mask.doc_q[(int64_t)b * a.Sq + i];
      if (doc >= 0) {
        atomicMin(&bars->doc_lo, doc);
        atomicMax(&bars->doc_hi, doc);
      }
    }
    __syncthreads();
  }
  const uint32_t tbase = __shfl_sync(0xffffffffu, bars->tmem_base, 0);
  const int2* docs = DOCS ? a.doc_blocks_k + (int64_t)b * ((a.Sk + kBlock - 1) / kBlock) : nullptr;
  BlockWalk<DOCS> walk(docs, key0 / kBlock, (key1 + kBlock - 1) / kBlock, bars->doc_lo, bars->doc_hi);

  if (warp == 0) {
    // ------------------------------------------------------------ loader
    // K_g as soon as the S that read its stage is done, then V_{g-1} once the P V that read its is.
    int k_par[NS] = {-1, -1};
    bool q_armed = false;
    const int32_t* doc_k = DOCS ? a.mask.doc_k + (int64_t)b * a.Sk : nullptr;
    auto load_k = [&](uint32_t g, int j) -> bool {
      const int st = g % NS;
      if (!warp_wait(&bars->s_full[st], ((g / NS) & 1) ^ 1, abort)) return false;
      if (lane == 0) {
        tc::mbar_expect_tx(&bars->k_full[st], L::kKBytes);
        for (int c = 0; c < D / 64; ++c)
          tc::tma_load_4d(sK + st * L::kKBytes + c * L::kKVChunk, &tmK, &bars->k_full[st], c * 64, j * kBlock, h, b);
      }
      k_par[0] = st == 0 ? (int)((g / NS) & 1) : k_par[0];
      k_par[1] = st == 1 ? (int)((g / NS) & 1) : k_par[1];
      return true;
    };
    auto load_v = [&](uint32_t g, int j, bool padded) -> bool {
      const int st = g % NS;
      unsigned char* dst = sV + st * L::kKBytes;
      if (!warp_wait(&bars->pv_done[st], ((g / NS) & 1) ^ 1, abort)) return false;
      // keys that do not exist although their memory does: zeros, whatever it holds (0 * NaN would reach O)
      if ((seq.kv < a.Sk && (j + 1) * kBlock > seq.kv) || padded) {
        copy_keys<D>(dst, static_cast<const __nv_bfloat16*>(a.v) + (int64_t)b * a.vs.b + (int64_t)h * a.vs.h, a.vs.s,
                     j * kBlock, kBlock, seq.kv, doc_k, lane, 32);
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bars->p_full[st]);
      } else if (lane == 0) {
        tc::mbar_expect_tx(&bars->p_full[st], L::kKBytes);
        for (int c = 0; c < D / 64; ++c)
          tc::tma_load_4d(dst + c * L::kKVChunk, &tmV, &bars->p_full[st], c * 64, j * kBlock, h, b);
      }
      if (lane == 0) *reinterpret_cast<volatile int*>(&bars->v_armed) = (int)g;
      return true;
    };
    uint32_t g = 0;
    int before = -1;
    bool padded = false;         // block `before` has padding keys
    bool ok = true;
    for (int j; ok && (j = walk.next(lane)) >= 0; ++g) {
      if (held(a, &bars->hold, abort, g)) {
        fail(&bars->abort, 20);
        ok = false;
        break;
      }
      if (g == 0 && lane == 0) {
        tc::mbar_expect_tx(&bars->q_full, (uint32_t)(qpt * a.G) * 128 * (D / 64));
        q_armed = true;
        for (int c = 0; c < D / 64; ++c) tc::tma_load_5d(sQ + c * L::kQChunk, &tmQ, &bars->q_full, c * 64, 0, i0, h, b);
      }
      ok = load_k(g, j) && (g == 0 || load_v(g - 1, before, padded));
      before = j;
      padded = DOCS && walk.doc().x < 0;
    }
    if (!ok || (g > 0 && !load_v(g - 1, before, padded))) fail(&bars->abort, 3);
    // no copy may still be writing shared memory when the CTA leaves
    if (lane == 0) {
      if (q_armed) tc::mbar_wait_drain(&bars->q_full, 0, kWaitLimit);
      for (int st = 0; st < NS; ++st)
        if (k_par[st] >= 0) tc::mbar_wait_drain(&bars->k_full[st], (uint32_t)k_par[st], kWaitLimit);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    // Order: S_0, [S_1, PV_0], [S_2, PV_1], ..., PV_last. Products of one thread run in issue order,
    // so S_{g+2} (the buffer of S_g and P_g) always follows PV_g.
    // The whole warp keeps step, so that what the products take is the same in all lanes; one lane issues.
    const uint32_t n = (uint32_t)walk.count(lane);
    if (n > 0) {
      constexpr uint32_t idS = tc::idesc_bf16_f32(kTileRows, kBlock, 0, 0);
      constexpr uint32_t idO = tc::idesc_bf16_f32(kTileRows, D, 0, 1);
      const uint64_t qd = tc::smem_desc_sw128(tc::smem_u32(sQ), 16, 1024);
      const uint64_t kd = tc::smem_desc_sw128(tc::smem_u32(sK), 16, 1024);
      const uint64_t vd = tc::smem_desc_sw128(tc::smem_u32(sV), L::kKVChunk, 1024);
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t parity, int code) {
        ok = ok && warp_wait(bar, parity, abort);
        if (!ok) fail(&bars->abort, code);
        tc::fence_after_sync();
        return ok;
      };
      auto pv = [&](uint32_t g) {
        const uint32_t pb = g & 1;
        if (!wait(&bars->p_full[pb], (g >> 1) & 1, 7)) return;
        if (tc::elect_one()) {
          const uint64_t bd = vd + pb * (L::kKBytes >> 4);
#pragma unroll
          for (int kk = 0; kk < kBlock / 16; ++kk)
            tc::mma_f16_tmem_a(tbase + L::kColO, tbase + pb * kBlock + kk * 8, bd + ((kk * 16 * 128) >> 4), idO,
                               kk > 0 ? 1u : (uint32_t)(g > 0));
          if (a.rest != nullptr) {
#pragma unroll
            for (int kk = 0; kk < kBlock / 16; ++kk)
              tc::mma_f16_tmem_a(tbase + L::kColO, tbase + pb * kBlock + 32 + kk * 8, bd + ((kk * 16 * 128) >> 4), idO, 1u);
          }
          tc::mma_commit(&bars->pv_done[pb]);
        }
        __syncwarp();
      };
      wait(&bars->q_full, 0, 5);
      for (uint32_t g = 0; ok && g < n; ++g) {
        const uint32_t st = g % NS;
        if (!wait(&bars->k_full[st], (g / NS) & 1, 6)) break;
        if (tc::elect_one()) {
          const uint64_t bd = kd + st * (L::kKBytes >> 4);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            tc::mma_f16(tbase + st * kBlock, qd + (((kk >> 2) * L::kQChunk + (kk & 3) * 32) >> 4),
                        bd + (((kk >> 2) * L::kKVChunk + (kk & 3) * 32) >> 4), idS, kk > 0 ? 1u : 0u);
          tc::mma_commit(&bars->s_full[st]);        // also frees the K stage
        }
        __syncwarp();
        if (g > 0) pv(g - 1);
      }
      if (ok) pv(n - 1);
      // on every path: the products issued so far are done before TMEM is released
      if (tc::elect_one()) {
        tc::mma_commit(&bars->drain);
        tc::mbar_wait_drain(&bars->drain, 0, kWaitLimit);
      }
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------ softmax and epilogue
    const int q = warp & 3;                  // TMEM lane quarter this warp may access
    const int r = q * 32 + lane;             // tile row == TMEM lane
    const uint32_t lane_off = (uint32_t)(q * 32) << 16;
    const int i = i0 + r / a.G, hq = h * a.G + r % a.G;
    const bool valid = r < qpt * a.G && i < a.Sq;
    DenseRow row{0, 0, 0, 0.f};
    if (valid) row = dense_row(a, seq, b, hq, i);
    const bool live_warp = __any_sync(0xffffffffu, valid);
    const int32_t* doc_k = DOCS ? a.mask.doc_k + (int64_t)b * a.Sk : nullptr;
    const ScoreMap<CAP, BIAS> map(a, row);
    float mrow = -INFINITY;
    uint64_t lsum = f2(0.f, 0.f);
    uint32_t g = 0;
    bool ok = true;
    for (int j; (j = walk.next(lane)) >= 0; ++g) {
      const int sb = g & 1;
      const uint32_t sp = tbase + lane_off + sb * kBlock;     // S_g, then P_g, of this row
      if (!warp_wait(&bars->s_full[sb], (g >> 1) & 1, abort)) {
        fail(&bars->abort, 10);
        ok = false;
        break;
      }
      if (live_warp) {
        tc::fence_after_sync();
        uint32_t lo[32], hi[32];
        tc::tmem_ld32(sp, lo);
        tc::tmem_ld32(sp + 32, hi);
        tc::tmem_ld_wait();
        const uint64_t see = visible64<DOCS>(row, doc_k, walk.doc(), j * kBlock, a.Sk, lane);
        const bool hidden = __any_sync(0xffffffffu, see != ~0ull);
        map.apply(lo, row.pos - j * kBlock, hidden, (uint32_t)see);
        map.apply(hi, row.pos - j * kBlock - 32, hidden, (uint32_t)(see >> 32));
        if (hidden) {
          only32(lo, (uint32_t)see, -INFINITY);
          only32(hi, (uint32_t)(see >> 32), -INFINITY);
        }
        const float mx = fmaxf(max32(lo), max32(hi)) * map.after;
        const bool raise = mrow == -INFINITY || mx > mrow + kRescaleLog2;
        const bool scale_o = raise && g > 0 && mrow != -INFINITY;
        if (__any_sync(0xffffffffu, scale_o)) {
          // tcgen05.ld/st are warp-collective: each lane with its own factor (1 where the max stays)
          const uint32_t gp = g - 1;
          if (!warp_wait(&bars->pv_done[gp & 1], (gp >> 1) & 1, abort)) {
            fail(&bars->abort, 12);
            ok = false;
            break;
          }
          tc::fence_after_sync();
          const float alpha = scale_o ? ex2(mrow - mx) : 1.f;
#pragma unroll 1
          for (int cc = 0; cc < D / 32; ++cc) {
            uint32_t o[32];
            tc::tmem_ld32(tbase + lane_off + L::kColO + cc * 32, o);
            tc::tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tc::tmem_st32(tbase + lane_off + L::kColO + cc * 32, o);
          }
          tc::tmem_st_wait();
          float l0, l1;
          f2_split(lsum, l0, l1);
          lsum = f2(l0 * alpha, l1 * alpha);
        }
        if (raise) mrow = mx;
        // a row that has seen nothing so far keeps -inf; its weights are exp2(-inf) = 0
        const float nm = mrow == -INFINITY ? 0.f : -mrow;
        const uint64_t negm = f2(nm, nm), after2 = f2(map.after, map.after);
        uint64_t acc[4] = {f2(0.f, 0.f), f2(0.f, 0.f), f2(0.f, 0.f), f2(0.f, 0.f)};
        // P of 32 keys over the S buffer, which is in registers; `two`: and what its rounding left behind it
        auto weights = [&](const uint32_t (&x)[32], int at, auto two) {
          uint32_t packed[16], left[16];
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const uint64_t x2 = ffma2(f2(__uint_as_float(x[2 * c]), __uint_as_float(x[2 * c + 1])), after2, negm);
            float x0, x1;
            f2_split(x2, x0, x1);
            const float p0 = ex2(x0), p1 = ex2(x1);
            acc[c & 3] = fadd2(acc[c & 3], f2(p0, p1));
            packed[c] = pack_bf16(p0, p1);
            if (decltype(two)::value)
              left[c] = pack_bf16(p0 - __uint_as_float(packed[c] << 16), p1 - __uint_as_float(packed[c] & 0xffff0000u));
          }
          tc::tmem_st16(sp + at, packed);
          if (decltype(two)::value) tc::tmem_st16(sp + 32 + at, left);
        };
        if (a.rest != nullptr) {
          weights(lo, 0, std::true_type{});
          weights(hi, 16, std::true_type{});
        } else {
          weights(lo, 0, std::false_type{});
          weights(hi, 16, std::false_type{});
        }
        lsum = fadd2(lsum, fadd2(fadd2(acc[0], acc[1]), fadd2(acc[2], acc[3])));
        tc::tmem_st_wait();
        tc::fence_before_sync();
      }
      __syncwarp();
      if (lane == 0) {
        tc::mbar_arrive(&bars->p_full[sb]);
        *reinterpret_cast<volatile int*>(&bars->p_arrived[q]) = (int)g;
      }
    }
    // ------------------------------------------------------------ epilogue
    if (g > 0 && ok) {
      if (!warp_wait(&bars->pv_done[(g - 1) & 1], ((g - 1) >> 1) & 1, abort)) fail(&bars->abort, 13);
      tc::fence_after_sync();
    }
    const bool broken = __any_sync(0xffffffffu, *abort != 0);
    if (live_warp) {
      float l0, l1;
      f2_split(lsum, l0, l1);
      const float lrow = l0 + l1;
      const float nan = __int_as_float(0x7fffffff);
      const float inv = broken ? nan : (lrow == 0.f ? 0.f : 1.f / lrow);
      const float lse = broken ? nan : (lrow == 0.f ? -INFINITY : (mrow + log2f(lrow)) * 0.69314718055994531f);
      const int64_t flat = ((int64_t)b * a.Hq + hq) * a.Sq + i;
      const int64_t part = (int64_t)split * a.B * a.Hq * a.Sq + flat;
      const int64_t at = (int64_t)b * a.os.b + (int64_t)hq * a.os.h + (int64_t)i * a.os.s;
#pragma unroll 1
      for (int cc = 0; cc < D / 32; ++cc) {
        uint32_t o[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = 0u;              // no step: a row that sees nothing
        if (g > 0 && !broken) {
          tc::tmem_ld32(tbase + lane_off + L::kColO + cc * 32, o);
          tc::tmem_ld_wait();
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * inv);
        if (!valid) continue;
        if (a.splits > 1) {
          float4* p = reinterpret_cast<float4*>(a.part_o + part * D + cc * 32);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            p[e] = make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]), __uint_as_float(o[4 * e + 2]),
                               __uint_as_float(o[4 * e + 3]));
        } else {
          store_row32(static_cast<__nv_bfloat16*>(a.out) + at + cc * 32,
                      a.rest != nullptr ? static_cast<__nv_bfloat16*>(a.rest) + at + cc * 32 : nullptr, o);
        }
      }
      if (valid) {
        if (a.splits > 1)
          a.part_lse[part] = lse;
        else if (a.lse != nullptr)
          a.lse[flat] = lse;
      }
    }
  }

  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == 1) tc::tmem_dealloc(tbase, L::kTmemCols);
  if (threadIdx.x == 0 && bars->abort) {
    // A V copy completes the P barrier of its step only together with the four softmax arrivals;
    // after an abort the missing ones are made here, and the copies still in flight are waited for.
    const int va = bars->v_armed;
    for (int gg = va - 1; gg <= va; ++gg) {
      if (gg < 0) continue;
      uint64_t* pb = &bars->p_full[gg & 1];
      const uint32_t par = ((uint32_t)gg >> 1) & 1;
      if (tc::mbar_try_wait(pb, par)) continue;
      for (int w = 0; w < 4; ++w)
        if (bars->p_arrived[w] < gg) tc::mbar_arrive(pb);
      tc::mbar_wait_drain(pb, par, kWaitLimit);
    }
    if (a.status != nullptr) report_error(a.status, FVATTN_ERR_TIMEOUT, bars->abort);
  }
}

template <int D, bool CAP, bool BIAS, bool DOCS>
cudaError_t launch(const DenseArgs& a, cudaStream_t st) {
  const int qpt = kTileRows / a.G;
  CUtensorMap mq, mk, mv;
  if (!make_map_rows(&mq, a.q, a.qs, a, qpt) || !make_map_keys(&mk, a.k, a.ks, a, kBlock) ||
      !make_map_keys(&mv, a.v, a.vs, a, kBlock))
    return cudaErrorInvalidValue;
  const size_t smem = FwdLayout<D>::kBytes + 1024;
  auto* kernel = dense_tc_kernel<D, CAP, BIAS, DOCS>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const TileOrder order = tile_order(a, (a.Sq + qpt - 1) / qpt * a.splits, a.causal);
  const int64_t grid = (int64_t)order.tiles * order.heads;
  if (grid > 0x7fffffff) return cudaErrorInvalidValue;
  return launch_with(kernel, dim3((unsigned)grid), kWarps * 32, smem, st, 0, DOCS, mq, mk, mv, a, qpt, order);
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

cudaError_t launch_dense_tc(const DenseArgs& a, cudaStream_t st) {
  return a.d == 128 ? launch_d<128>(a, st) : launch_d<64>(a, st);
}

}  // namespace fv
