// Gradients of attention over all keys on the B200 tensor cores: bf16 inputs, everything else fp32.
//
//   P = exp(s - lse),  dP = dout V^T,  dS = P (dP - delta) (1 - tanh^2)
//   dV = P^T dout,  dK = scale dS^T Q,  dQ = scale dS K,  delta_i = sum_d out_id dout_id
//
// Two kernels, each of which owns its results: one CTA per 128 keys walks over the row tiles (row
// i * G + g: query i of the group's head g) and keeps dK and dV in TMEM, one CTA per row tile walks over the keys
// and keeps dQ. S and dP are made twice (seven products instead of five), but no result is added to
// by several CTAs, so there are no atomics, equal calls give equal bits, and a shared key head's
// gradient is summed over its query heads in TMEM.
//
// dK, dV: scores transposed (lane = key, column = row), so that P^T and dS^T are written over the
// scores in TMEM as the first operands of their products. Steps of 64 rows alternate between two groups
// of eight warps, each with its own scores and dP in TMEM, so that one group's exponentials run beside
// the other's and beside the products of both:
//   products of slot k    dV(k) S(k+2) dK(k-1) dP(k+1)
//   one group             P(k) from S(k), in slot k-1;      dS(k) from dP(k), in slot k
// dQ: lane = row; S has two buffers, so S(i+1) is ready when dS(i) is done:
//   products   dP(i+1) dQ(i) S(i+2);   warps   P(i+1), then dS(i+1) from dP(i+1)
//
// P and dS are rounded to bf16 as the products' operands: the results are off by 0.0024 of their size, where an
// fp32 computation rounded once is off by 0.0017, and a second term of each would double these products. lse,
// delta and all sums stay in fp32, and the scale is applied once to the sums.
//
// Bound by the chain from products to elementwise work and back. Measured at 8192 tokens, causal, 12 heads,
// d = 128: dK/dV 366 us (tensor pipe 56 % active), dQ 255 us (62 %, SFU 42 %), in a loop at the board's power
// limit, which holds the SMs at 1.61 of 1.97 GHz.
//
// Every wait is bounded; one that runs out stops every role without leaving a copy or product in
// flight, is reported in the status word, and makes the CTA's results NaN.
#include <cooperative_groups.h>
#include <cuda.h>
#include <cuda_bf16.h>

#include <type_traits>

#include "dense.cuh"
#include "dense_tc.cuh"
#include "tc_ptx.cuh"
#include "tmap.cuh"

namespace cg = cooperative_groups;

namespace fv {

namespace {

constexpr int kT = 128;               // rows and keys of a tile
// Loader, sixteen warps for the elementwise work (four per scheduler, which hide one another's waits for
// TMEM and the SFU), and a warp for each kind of product. A wait costs 80 to 100 cycles even for a barrier
// that is complete, and one warp for all products has to take four of them a step. This form, together with
// steps of 64 rows, took dK/dV at 8192 causal tokens, 12 heads, d = 128 from 458 to 387 us.
constexpr int kWarps = 20;
constexpr int kLoader = 16, kMmaS = 17, kMmaOut = 18, kMmaDp = 19;
// Registers: of the 96 per thread at the launch the last four warps give up 56, the sixteen take 8 more
// (128 x 40 + 512 x 104 = 58,368 of the launch's 61,440). With the document code under a template argument: 387
// to 366 us; with 182 bytes of spill stores it had taken 547 us. Left in dK/dV: none to 8 bytes plain and capped,
// 20 with a bias, 70 with a bias and a cap, 44 to 114 with documents.
constexpr int kRegsWork = 104, kRegsOther = 40;
constexpr int kWork = 16;
constexpr int kCols = kT * 4 / kWork; // columns of a score tile per thread
constexpr int kThreads = kWarps * 32;
constexpr uint32_t kColA = 0;         // scores (dQ: their first buffer)
constexpr uint32_t kColB = 128;       // dP (dQ: the scores' second buffer)

template <int D>
struct BwdLayout {
  static constexpr int kChunk = kT * 128;              // [128 tokens x 64 dims] bf16
  static constexpr int kTile = (D / 64) * kChunk;
};

// Shared-memory descriptors of a token-by-dims tile: as the K-major operand of a product over dims, and
// as the MN-major second operand of a product over tokens. Within a tile only the address field (the
// low bits, in units of 16 bytes) changes, so a step costs the issuing thread one addition.
__device__ __forceinline__ uint64_t desc_dims(uint32_t addr) { return tc::smem_desc_sw128(addr, 16, 1024); }
__device__ __forceinline__ uint64_t desc_tokens(uint32_t addr) { return tc::smem_desc_sw128(addr, kT * 128, 1024); }
constexpr uint32_t step_dims(int kk) { return ((kk >> 2) * (kT * 128) + (kk & 3) * 32) >> 4; }
constexpr uint32_t step_tokens(int kk) { return (kk * 16 * 128) >> 4; }

// D[128 x 128] = A B^T over the dims of two tiles.
template <int D>
__device__ __forceinline__ void mma_dims(uint32_t d_tmem, uint64_t a, uint64_t b) {
  constexpr uint32_t id = tc::idesc_bf16_f32(kT, kT, 0, 0);
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) tc::mma_f16(d_tmem, a + step_dims(kk), b + step_dims(kk), id, kk > 0);
}
// D[128 x D] (+)= W B over the 128 tokens of a tile, W (bf16) in TMEM: every kCols tokens over the fp32
// values they were made from.
template <int D>
__device__ __forceinline__ void mma_tokens(uint32_t d_tmem, uint32_t w, uint64_t b, uint32_t add) {
  constexpr uint32_t id = tc::idesc_bf16_f32(kT, D, 0, 1);
#pragma unroll
  for (int kk = 0; kk < kT / 16; ++kk)
    tc::mma_f16_tmem_a(d_tmem, w + (kk / (kCols / 16)) * kCols + (kk % (kCols / 16)) * 8, b + step_tokens(kk), id,
                       kk > 0 ? 1u : add);
}

// 32 fp32 results, times `by`, as bf16.
__device__ __forceinline__ void store32(__nv_bfloat16* p, uint32_t (&o)[32], float by) {
#pragma unroll
  for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * by);
  store_row32(p, nullptr, o);
}

// ------------------------------------------------------------------ dK, dV

constexpr int kR = 64;                // rows of a step
constexpr int kStagesQ = 5;           // S(k+2) is issued before dK(k-1) has released Q(k-1)
constexpr int kStagesG = 4;

// What the rows of a step need, twice per group.
struct RowStats {
  float nlse2[kR];     // - lse log2 e
  float ndelta[kR];    // - delta
  float far[kR];       // position minus the first key of the key tile
  float slope2[kR];    // slope log2 e
  int limit[kR];       // visible keys are below it, counted from the first key of the key tile
  int doc[kR];
};

template <int D>
struct DkvLayout {
  static constexpr int kKeyChunk = kT * 128, kKeyTile = (D / 64) * kKeyChunk;    // [tokens x 64 dims] bf16
  static constexpr int kRowChunk = kR * 128, kRowTile = (D / 64) * kRowChunk;
  static constexpr int kOffK = 0, kOffV = kKeyTile, kOffQ = 2 * kKeyTile, kOffG = kOffQ + kStagesQ * kRowTile;
  static constexpr int kOffStats = kOffG + kStagesG * kRowTile;
  static constexpr int kOffBar = kOffStats + 4 * (int)sizeof(RowStats);
  static constexpr int kBytes = kOffBar + 512;
  // at the end, where a cluster joins its CTAs' results: [dV, dK][key][dim] fp32 over the tiles, rows four
  // floats longer than D (lanes write rows: no two in one bank)
  static constexpr int kLdOut = D + 4;
  static_assert(2 * kT * kLdOut * 4 <= kOffStats, "the results fit the tiles");
  // TMEM: scores of even and odd steps, dP of even and odd steps, the results
  static constexpr uint32_t kColS = 0, kColDp = 128, kColV = 256, kColK = 384;
};

struct DkvBars {
  uint64_t kv_full;
  uint64_t q_full[kStagesQ], q_empty[kStagesQ], g_full[kStagesG], g_empty[kStagesG];     // Q and dout
  uint64_t s_full[2], p_full[2], dp_full[2], ds_full[2];      // by parity of the step
  uint64_t dv_done[2], dk_done[2];
  uint64_t drain;
  uint64_t hold;                      // never completes (failure-path check)
  int doc_lo, doc_hi, doc_pad;        // documents of the keys
  uint32_t tmem_base;
  int abort;
};

static_assert(sizeof(DkvBars) <= 512, "the barriers fit their place");

// One CTA's share of a walk: of its steps every a.cluster-th, from the CTA's rank in the cluster on.
template <bool DOCS>
struct SharedWalk : BlockWalk<DOCS> {
  int skip;      // steps of the others before the next of its own
  __device__ __forceinline__ SharedWalk(const BlockWalk<DOCS>& w, int rank) : BlockWalk<DOCS>(w), skip(rank) {}
  __device__ __forceinline__ int next(int lane, int of) {
    for (; skip > 0; --skip) BlockWalk<DOCS>::next(lane);
    skip = of - 1;
    return BlockWalk<DOCS>::next(lane);
  }
  __device__ __forceinline__ int count(int lane, int of) const {
    return max(0, BlockWalk<DOCS>::count(lane) - skip + of - 1) / of;
  }
};

template <int D, bool CAP, bool BIAS, bool DOCS>
__global__ void __launch_bounds__(kThreads, 1)
    dense_dkv_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmG,
                        const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                        const DenseArgs a, const int qpt, const TileOrder order) {
  using L = DkvLayout<D>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  DkvBars* bars = reinterpret_cast<DkvBars*>(smem + L::kOffBar);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort = &bars->abort;
  wait_for_previous_grid();
  allow_next_grid();
  int x, bh;
  tile_of(order, blockIdx.x / a.cluster, x, bh);      // the first keys are seen by the most rows under an order
  const int b = bh / a.Hkv, h = bh - b * a.Hkv, j0 = x * kT;
  const DenseSeq seq = dense_seq(a, b);
  const int32_t* doc_q = DOCS ? a.mask.doc_q + (int64_t)b * a.Sq : nullptr;
  const int32_t* doc_k = DOCS ? a.mask.doc_k + (int64_t)b * a.Sk : nullptr;
  const int tiles = (a.Sq + qpt - 1) / qpt;

  if (threadIdx.x == 0) {
    tc::mbar_init(&bars->kv_full, 1);
    for (int s = 0; s < kStagesQ; ++s) {
      tc::mbar_init(&bars->q_full[s], 1);
      tc::mbar_init(&bars->q_empty[s], 1);
    }
    for (int s = 0; s < kStagesG; ++s) {
      tc::mbar_init(&bars->g_full[s], 1);
      tc::mbar_init(&bars->g_empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      tc::mbar_init(&bars->dv_done[s], 1);
      tc::mbar_init(&bars->dk_done[s], 1);
      tc::mbar_init(&bars->s_full[s], 1);
      tc::mbar_init(&bars->dp_full[s], 1);
      tc::mbar_init(&bars->p_full[s], kWork / 2);
      tc::mbar_init(&bars->ds_full[s], kWork / 2);
    }
    tc::mbar_init(&bars->drain, 3);
    tc::mbar_init(&bars->hold, 1);
    bars->abort = 0;
    bars->doc_lo = 0x7fffffff;
    bars->doc_hi = -1;
    bars->doc_pad = 0;
    tc::fence_mbar_init();
  }
  if (warp == kMmaS) {
    tc::tmem_alloc(&bars->tmem_base, 512);
    tc::tmem_relinquish();
  }
  // Rows that no copy writes (64 - qpt * G of them) have weights of zero: they must hold numbers.
  if (qpt * a.G < kR) {
    for (int i = threadIdx.x; i < (kStagesQ + kStagesG) * L::kRowTile / 16; i += kThreads)
      reinterpret_cast<uint4*>(smem + L::kOffQ)[i] = make_uint4(0u, 0u, 0u, 0u);
    tc::fence_proxy_async_smem();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (DOCS) {
    if (threadIdx.x < kT && j0 + threadIdx.x < a.Sk) {
      const int doc = doc_k[j0 + threadIdx.x];
      if (doc >= 0) {
        atomicMin(&bars->doc_lo, doc);
        atomicMax(&bars->doc_hi, doc);
      } else {
        bars->doc_pad = 1;
      }
    }
    __syncthreads();
  }
  const uint32_t tbase = __shfl_sync(0xffffffffu, bars->tmem_base, 0);
  // Under an order the rows from the first whose limit passes j0 see the tile (limits never fall).
  int first = 0;
  if (j0 >= seq.kv) {
    first = tiles;
  } else if (a.causal && j0 >= seq.prefix) {
    first = max(0, min(j0 - seq.q0, a.Sq)) / qpt;      // query i sees key j0 when q0 + i >= j0
  }
  const int2* tile_docs = DOCS ? a.doc_blocks_q + (int64_t)b * tiles : nullptr;
  cg::cluster_group cluster = cg::this_cluster();
  const int share = a.cluster;
  SharedWalk<DOCS> walk(BlockWalk<DOCS>(tile_docs, first, tiles, bars->doc_lo, bars->doc_hi), (int)cluster.block_rank());
  const uint32_t n = (uint32_t)walk.count(lane, share);

  if (warp >= kWork) {
    tc::regs_down<kRegsOther>();
    if (warp == kLoader) {
      // ------------------------------------------------------------ loader
      bool kv_armed = false;
      if (lane == 0 && n > 0) {
        tc::mbar_expect_tx(&bars->kv_full, 2 * L::kKeyTile);
        kv_armed = true;
        for (int c = 0; c < D / 64; ++c) {
          tc::tma_load_4d(smem + L::kOffK + c * L::kKeyChunk, &tmK, &bars->kv_full, c * 64, j0, h, b);
          tc::tma_load_4d(smem + L::kOffV + c * L::kKeyChunk, &tmV, &bars->kv_full, c * 64, j0, h, b);
        }
      }
      const uint32_t bytes = (uint32_t)(qpt * a.G) * 128 * (D / 64);
      uint32_t g = 0, q_armed = 0, g_armed = 0;      // steps whose copies were issued
      // One tensor's rows of a step into their stage.
      auto load = [&](const CUtensorMap& map, const void* base, const fvattn_strides& st, uint64_t* full, uint64_t* empty,
                      uint32_t empty_parity, unsigned char* dst, int i0, bool pad) -> bool {
        if (!warp_wait(empty, empty_parity, abort)) return false;
        if (pad) {
          // padding queries may hold anything: copied by hand, with zeros for them
          copy_rows<D, kR>(dst, static_cast<const __nv_bfloat16*>(base), st, a, b, h, i0, qpt, doc_q, lane, 32);
          tc::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(full);
        } else if (lane == 0) {
          tc::mbar_expect_tx(full, bytes);
          for (int c = 0; c < D / 64; ++c) tc::tma_load_5d(dst + c * L::kRowChunk, &map, full, c * 64, 0, i0, h, b);
        }
        return true;
      };
      bool ok = true;
      for (int t; ok && (t = walk.next(lane, share)) >= 0; ++g) {
        if (held(a, &bars->hold, abort, g)) {
          fail(&bars->abort, 20);
          ok = false;
          break;
        }
        const uint32_t sq = g % kStagesQ, sg = g % kStagesG;
        const bool pad = DOCS && walk.doc().x < 0;
        ok = load(tmQ, a.q, a.qs, &bars->q_full[sq], &bars->q_empty[sq], ((g / kStagesQ) & 1) ^ 1,
                  smem + L::kOffQ + sq * L::kRowTile, t * qpt, pad);
        if (ok) q_armed = g + 1;
        ok = ok && load(tmG, a.dout, a.dos, &bars->g_full[sg], &bars->g_empty[sg], ((g / kStagesG) & 1) ^ 1,
                        smem + L::kOffG + sg * L::kRowTile, t * qpt, pad);
        if (ok) g_armed = g + 1;
      }
      if (!ok) fail(&bars->abort, 3);
      if (lane == 0) {
        // no copy may still be writing shared memory when the CTA leaves: the last of each stage
        if (kv_armed) tc::mbar_wait_drain(&bars->kv_full, 0, kWaitLimit);
        for (uint32_t k = q_armed > kStagesQ ? q_armed - kStagesQ : 0; k < q_armed; ++k)
          tc::mbar_wait_drain(&bars->q_full[k % kStagesQ], (k / kStagesQ) & 1, kWaitLimit);
        for (uint32_t k = g_armed > kStagesG ? g_armed - kStagesG : 0; k < g_armed; ++k)
          tc::mbar_wait_drain(&bars->g_full[k % kStagesG], (k / kStagesG) & 1, kWaitLimit);
      }
    } else {
      // ------------------------------------------------------------ MMA issuers
      // Each warp keeps step as a whole, so that what the products take is the same in all lanes; one lane
      // issues.
      if (n > 0) {
        constexpr uint32_t idS = tc::idesc_bf16_f32(kT, kR, 0, 0), idD = tc::idesc_bf16_f32(kT, D, 0, 1);
        constexpr uint32_t kStage = L::kRowTile >> 4;
        bool ok = true;
        auto wait = [&](uint64_t* bar, uint32_t parity, int code) {
          ok = ok && warp_wait(bar, parity, abort);
          if (!ok) fail(&bars->abort, code);
          tc::fence_after_sync();
          return ok;
        };
        // scores^T (K, Q) or dP^T (V, dout): [128 keys x 64 rows] over the dims, for every step
        auto over_dims = [&](int key_off, int row_off, uint32_t stages, uint64_t* full, uint64_t* over, uint32_t col,
                             uint64_t* done, int code) {
          const uint64_t key_tile = tc::smem_desc_sw128(tc::smem_u32(smem + key_off), 16, 1024);
          const uint64_t row_tile = tc::smem_desc_sw128(tc::smem_u32(smem + row_off), 16, 1024);
          wait(&bars->kv_full, 0, code);
          uint32_t st = 0, turn = 0;       // stage of the step and how often it has come round
          for (uint32_t k = 0; ok && k < n; ++k) {
            const uint32_t p = k & 1;
            // what the step before last left in the columns has been read
            if (k >= 2 && !wait(&over[p], ((k >> 1) & 1) ^ 1, code)) break;
            if (!wait(&full[st], turn & 1, code + 10)) break;
            if (tc::elect_one()) {
              const uint64_t rd = row_tile + st * kStage;
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk)
                tc::mma_f16(tbase + col + p * kR, key_tile + (((kk >> 2) * L::kKeyChunk + (kk & 3) * 32) >> 4),
                            rd + (((kk >> 2) * L::kRowChunk + (kk & 3) * 32) >> 4), idS, kk > 0);
              tc::mma_commit(&done[p]);
            }
            __syncwarp();
            if (++st == stages) {
              st = 0;
              ++turn;
            }
          }
        };
        if (warp == kMmaS) {
          over_dims(L::kOffK, L::kOffQ, kStagesQ, bars->q_full, bars->dv_done, L::kColS, bars->s_full, 5);
        } else if (warp == kMmaDp) {
          over_dims(L::kOffV, L::kOffG, kStagesG, bars->g_full, bars->dk_done, L::kColDp, bars->dp_full, 6);
        } else {
          const uint64_t qt = tc::smem_desc_sw128(tc::smem_u32(smem + L::kOffQ), L::kRowChunk, 1024);
          const uint64_t gt = tc::smem_desc_sw128(tc::smem_u32(smem + L::kOffG), L::kRowChunk, 1024);
          // dV or dK += [128 keys x 64 rows] (bf16 in TMEM, every kCols rows over their fp32 values) x [rows x D]
          auto over_rows = [&](uint32_t d_tmem, uint32_t w, uint64_t row_tile, uint32_t add) {
#pragma unroll
            for (int kk = 0; kk < kR / 16; ++kk)
              tc::mma_f16_tmem_a(d_tmem, w + (kk >> 1) * kCols + (kk & 1) * 8, row_tile + ((kk * 16 * 128) >> 4), idD,
                                 kk > 0 ? 1u : add);
          };
          for (uint32_t k = 0; ok && k <= n; ++k) {
            const uint32_t p = k & 1;
            if (k < n) {
              // P(k) says that Q(k) has landed, not that dout(k) has
              if (!wait(&bars->g_full[k % kStagesG], (k / kStagesG) & 1, 7)) break;
              if (!wait(&bars->p_full[p], (k >> 1) & 1, 8)) break;
              if (tc::elect_one()) {
                over_rows(tbase + L::kColV, tbase + L::kColS + p * kR, gt + (k % kStagesG) * kStage, k > 0);
                tc::mma_commit(&bars->dv_done[p]);
              }
              __syncwarp();
            }
            if (k > 0) {
              const uint32_t e = k - 1;
              if (!wait(&bars->ds_full[p ^ 1], (e >> 1) & 1, 9)) break;
              if (tc::elect_one()) {
                over_rows(tbase + L::kColK, tbase + L::kColDp + (p ^ 1) * kR, qt + (e % kStagesQ) * kStage, e > 0);
                tc::mma_commit(&bars->dk_done[p ^ 1]);
                // dS(e) was made from S(e) and dP(e), so with dK(e) all four products of the step are done
                tc::mma_commit(&bars->q_empty[e % kStagesQ]);
                tc::mma_commit(&bars->g_empty[e % kStagesG]);
              }
              __syncwarp();
            }
          }
        }
        // on every path: the products issued so far are done before TMEM is read or released
        if (tc::elect_one()) tc::mma_commit(&bars->drain);
        __syncwarp();
        if (lane == 0) tc::mbar_wait_drain(&bars->drain, 0, kWaitLimit);
        __syncwarp();
      }
    }
    __syncwarp();
    if (share > 1) named_sync(3, kThreads);      // see the results
  } else {
    // ------------------------------------------------------------ elementwise
    tc::regs_up<kRegsWork>();
    // TMEM lane quarter, group (steps of its parity), columns of the step
    const int q = warp & 3, group = warp >> 3, col0 = ((warp >> 2) & 1) * kCols;
    const int r = q * 32 + lane, j = j0 + r;
    const uint32_t lanes = (uint32_t)(q * 32) << 16;
    const uint32_t colS = tbase + lanes + L::kColS + group * kR + col0, colP = tbase + lanes + L::kColDp + group * kR + col0;
    RowStats* stats = reinterpret_cast<RowStats*>(smem + L::kOffStats) + 2 * group;
    const int my_doc = DOCS && j < a.Sk ? doc_k[j] : 0;
    const bool key_ok = j < seq.kv && my_doc >= 0;
    const float in = CAP ? a.scale / a.cap : 0.f, factor = (CAP ? a.cap : a.scale) * kLog2e, fr = (float)r;
    const uint64_t factor2 = f2(factor, factor);
    uint64_t pw[kCols / 2];          // P, then P times the cap's derivative, in pairs
    uint32_t see = 0xffffffffu;      // bit c: row c of this warp's sees this lane's key

    // The row statistics of a step: these threads hold one value each of the group's next step in flight,
    // as loaded (nothing waits for it), and write it at the start of its turn.
    const int tid = threadIdx.x - group * (kWork / 2) * 32;
    const int part = tid / kR, sr = tid % kR, si = sr / a.G, sg = sr - si * a.G;
    float ahead = 0.f;       // lse, delta, document or slope of row sr
    int ahead_limit = 0;     // its limit or position
    auto fetch = [&](int t) {
      const int i0 = t * qpt, i = i0 + si, hq = h * a.G + sg;
      ahead = 0.f;
      ahead_limit = 0;
      if (sr >= min(qpt, a.Sq - i0) * a.G) return;
      const int64_t flat = ((int64_t)b * a.Hq + hq) * a.Sq + i;
      if (part == 0) ahead = a.lse[flat];
      if (part == 1) ahead = a.delta[flat];
      if (part == 2) {
        ahead_limit = dense_limit(seq, a.causal, i);
        if (DOCS) ahead = __int_as_float(doc_q[i]);
      }
      if (BIAS && part == 3) {
        ahead_limit = seq.q0 + i;
        ahead = a.mask.slopes[hq];
      }
    };
    auto put = [&](RowStats& st) {
      if (part == 0) st.nlse2[sr] = -ahead * kLog2e;
      if (part == 1) st.ndelta[sr] = -ahead;
      if (part == 2) {
        const int doc = __float_as_int(ahead);
        st.limit[sr] = (doc < 0 ? 0 : ahead_limit) - j0;
        st.doc[sr] = doc;
      }
      if (BIAS && part == 3) {
        st.far[sr] = (float)(ahead_limit - j0);
        st.slope2[sr] = ahead * kLog2e;
      }
    };

    // P^T of this warp's rows over the scores it is made from, loaded by then
    auto probs = [&](auto masked, const RowStats& st) {
      constexpr bool MASK = decltype(masked)::value;
      uint32_t s[32], packed[16];
      tc::tmem_ld32(colS, s);
      tc::tmem_ld_wait();
      if (CAP) tanh32(s, in, MASK, see);
#pragma unroll
      for (int c = 0; c < 32; c += 4) {
        const ulonglong2 l4 = *reinterpret_cast<const ulonglong2*>(&st.nlse2[col0 + c]);
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
          const uint64_t t2 = f2(__uint_as_float(s[c + e]), __uint_as_float(s[c + e + 1]));
          float y0, y1;
          f2_split(ffma2(t2, factor2, e == 0 ? l4.x : l4.y), y0, y1);
          if (BIAS) {
            const int at = col0 + c + e;
            y0 = fmaf(-st.slope2[at], fabsf(st.far[at] - fr), y0);
            y1 = fmaf(-st.slope2[at + 1], fabsf(st.far[at + 1] - fr), y1);
          }
          float p0 = ex2(y0), p1 = ex2(y1);
          if (MASK) {
            p0 = (see >> (c + e)) & 1u ? p0 : 0.f;
            p1 = (see >> (c + e + 1)) & 1u ? p1 : 0.f;
          }
          packed[(c + e) / 2] = pack_bf16(p0, p1);
          pw[(c + e) / 2] = CAP ? times_dcap(f2(p0, p1), t2) : f2(p0, p1);
        }
      }
      tc::tmem_st16(colS, packed);
    };
    // dS^T over dP^T
    auto grads = [&](auto masked, const RowStats& st) {
      constexpr bool MASK = decltype(masked)::value;
      uint32_t dp[32], packed[16];
      tc::tmem_ld32(colP, dp);
      tc::tmem_ld_wait();
#pragma unroll
      for (int c = 0; c < 32; c += 4) {
        const ulonglong2 d4 = *reinterpret_cast<const ulonglong2*>(&st.ndelta[col0 + c]);
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
          float d0, d1;
          f2_split(fmul2(pw[(c + e) / 2], fadd2(f2(__uint_as_float(dp[c + e]), __uint_as_float(dp[c + e + 1])),
                                                e == 0 ? d4.x : d4.y)), d0, d1);
          if (MASK) {                       // dP of a hidden pair may be anything
            d0 = (see >> (c + e)) & 1u ? d0 : 0.f;
            d1 = (see >> (c + e + 1)) & 1u ? d1 : 0.f;
          }
          packed[(c + e) / 2] = pack_bf16(d0, d1);
        }
      }
      tc::tmem_st16(colP, packed);
    };

    const int jend = min(kT, seq.kv - j0);
    const bool one_doc = bars->doc_lo == bars->doc_hi && !bars->doc_pad;
    bool ok = true;
    int t = walk.next(lane, share);
    if (group == 1) t = walk.next(lane, share);
    int2 docs = t >= 0 ? walk.doc() : make_int2(0, 0);       // of step t
    if (t >= 0) fetch(t);
    for (uint32_t turn = 0; t >= 0; ++turn) {
      RowStats& st = stats[turn & 1];
      const int i0 = t * qpt;
      put(st);
      named_sync(1 + group, kWork / 2 * 32);      // after an abort too: every warp takes all its turns
      walk.next(lane, share);                            // the other group's
      const int next = walk.next(lane, share);
      const int2 next_docs = next >= 0 ? walk.doc() : make_int2(0, 0);
      if (next >= 0) fetch(next);
      see = (uint32_t)(low64(min(qpt, a.Sq - i0) * a.G - col0) & 0xffffffffull);
      // limits never fall along the rows: the first query's is the least
      if (dense_limit(seq, a.causal, i0) - j0 < jend) {
        uint32_t below = 0u;
#pragma unroll 4
        for (int c = 0; c < 32; c += 4) {
          const int4 l = *reinterpret_cast<const int4*>(&st.limit[col0 + c]);
          below |= (uint32_t)((r < l.x) | (r < l.y) << 1 | (r < l.z) << 2 | (r < l.w) << 3) << c;
        }
        see &= below;
      }
      if (DOCS) {
        if (!one_doc || !doc_uniform(docs) || docs.y != bars->doc_lo) {
          see &= (uint32_t)same_document(st.doc[col0 + lane], -1, my_doc);
          if (!key_ok) see = 0u;
        }
      }
      // a key behind the valid ones has no say in the cap's form; else its results alone are left out
      if (CAP && j < a.Sk && !key_ok) see = 0u;
      const bool hidden = __any_sync(0xffffffffu, see != 0xffffffffu);
      if (ok && !warp_wait(&bars->s_full[group], turn & 1, abort)) {
        fail(&bars->abort, 10);
        ok = false;
      }
      if (ok) {
        tc::fence_after_sync();
        if (hidden) probs(std::true_type{}, st); else probs(std::false_type{}, st);
        tc::tmem_st_wait();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bars->p_full[group]);
        if (!warp_wait(&bars->dp_full[group], turn & 1, abort)) {
          fail(&bars->abort, 11);
          ok = false;
        }
      }
      if (ok) {
        tc::fence_after_sync();
        if (hidden) grads(std::true_type{}, st); else grads(std::false_type{}, st);
        tc::tmem_st_wait();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bars->ds_full[group]);
      }
      t = next;
      docs = next_docs;
    }
    // ------------------------------------------------------------ results: one group writes dV, the other dK
    if (n > 0 && ok) {
      if (!warp_wait(&bars->drain, 0, abort)) fail(&bars->abort, 12);
      tc::fence_after_sync();
    }
    // A cluster's results go over the tiles. After an abort copies and products may still be on their way to or
    // from them: the other warps come here once theirs have ended.
    if (share > 1) named_sync(3, kThreads);
    const bool broken = __any_sync(0xffffffffu, *abort != 0);
    const int part_d = (warp >> 2) & 1;
    const float by = broken ? __int_as_float(0x7fffffff) : group == 0 ? 1.f : a.scale;
    const fvattn_strides& ss = group == 0 ? a.dvs : a.dks;
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(group == 0 ? a.dv : a.dk) + (int64_t)b * ss.b + (int64_t)h * ss.h +
                         (int64_t)j * ss.s;
    float* shared_row = reinterpret_cast<float*>(smem) + (group * kT + r) * L::kLdOut;
#pragma unroll 1
    for (int cc = part_d * (D / 64); cc < (part_d + 1) * (D / 64); ++cc) {
      uint32_t o[32];
#pragma unroll
      for (int e = 0; e < 32; ++e) o[e] = 0u;
      if (n > 0 && !broken) {
        tc::tmem_ld32(tbase + lanes + (group == 0 ? L::kColV : L::kColK) + cc * 32, o);
        tc::tmem_ld_wait();
      }
      if (!key_ok && !broken) {
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = 0u;
      }
      if (share == 1) {
        if (j < a.Sk) store32(dst + cc * 32, o, by);
      } else {
#pragma unroll
        for (int e = 0; e < 32; e += 4)
          *reinterpret_cast<float4*>(shared_row + cc * 32 + e) =
              make_float4(__uint_as_float(o[e]) * by, __uint_as_float(o[e + 1]) * by, __uint_as_float(o[e + 2]) * by,
                          __uint_as_float(o[e + 3]) * by);
      }
    }
  }
  if (share > 1) {
    // the cluster's sums, in the order of the ranks; each CTA writes its part of the keys
    cluster.sync();
    const int rows = kT / share, row0 = (int)cluster.block_rank() * rows;
    for (int i = threadIdx.x; i < 2 * rows * (D / 8); i += kThreads) {
      const int which = i / (rows * (D / 8)), k = i % (rows * (D / 8)), row = row0 + k / (D / 8), d = k % (D / 8) * 8;
      float acc[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] = 0.f;
      for (int rank = 0; rank < share; ++rank) {
        const float* p = cluster.map_shared_rank(reinterpret_cast<float*>(smem), rank) + (which * kT + row) * L::kLdOut + d;
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] += p[e];
      }
      if (j0 + row < a.Sk) {
        const fvattn_strides& ss = which == 0 ? a.dvs : a.dks;
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(which == 0 ? a.dv : a.dk) + (int64_t)b * ss.b +
                             (int64_t)h * ss.h + (int64_t)(j0 + row) * ss.s + d;
        *reinterpret_cast<uint4*>(dst) = make_uint4(pack_bf16(acc[0], acc[1]), pack_bf16(acc[2], acc[3]),
                                                    pack_bf16(acc[4], acc[5]), pack_bf16(acc[6], acc[7]));
      }
    }
    cluster.sync();                      // a CTA's shared memory is read until here
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == kMmaS) tc::tmem_dealloc(tbase, 512);
  if (threadIdx.x == 0 && bars->abort && a.status != nullptr)
    report_error(a.status, FVATTN_ERR_TIMEOUT, 300 + bars->abort);
}

// ------------------------------------------------------------------ dQ

template <int D>
struct DqLayout : BwdLayout<D> {
  using B = BwdLayout<D>;
  static constexpr int kStagesK = 3, kStagesV = 2;
  static constexpr int kOffQ = 0, kOffG = B::kTile, kOffK = 2 * B::kTile, kOffV = kOffK + kStagesK * B::kTile;
  static constexpr int kOffBar = kOffV + kStagesV * B::kTile;
  static constexpr int kBytes = kOffBar + 256;
  static constexpr uint32_t kColDp = 256, kColQ = 384;
};

struct DqBars {
  uint64_t q_full;
  uint64_t k_full[3], k_empty[3], v_full[2], v_empty[2];
  uint64_t s_full[2], dq_done[2];      // by parity of the step
  uint64_t dp_full, ds_full;
  uint64_t drain;
  uint64_t hold;                       // never completes (failure-path check)
  int doc_lo, doc_hi;
  uint32_t tmem_base;
  int abort;
};

static_assert(sizeof(DqBars) <= 256, "the barriers fit their place");

template <int D, bool CAP, bool BIAS, bool DOCS>
__global__ void __launch_bounds__(kThreads, 1)
    dense_dq_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmG,
                       const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                       const DenseArgs a, const int qpt,
                       const TileOrder order) {
  using L = DqLayout<D>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  DqBars* bars = reinterpret_cast<DqBars*>(smem + L::kOffBar);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort = &bars->abort;
  wait_for_previous_grid();
  allow_next_grid();
  int x, bh;
  tile_of(order, blockIdx.x, x, bh);
  const int t = order.tiles - 1 - x, b = bh / a.Hkv, h = bh - b * a.Hkv;      // the longest tiles first
  const int i0 = t * qpt, i1 = min(i0 + qpt, a.Sq);
  const DenseSeq seq = dense_seq(a, b);
  const int32_t* doc_q = DOCS ? a.mask.doc_q + (int64_t)b * a.Sq : nullptr;
  const int32_t* doc_k = DOCS ? a.mask.doc_k + (int64_t)b * a.Sk : nullptr;
  const int blocks = (a.Sk + kT - 1) / kT;

  if (threadIdx.x == 0) {
    tc::mbar_init(&bars->q_full, 1);
    for (int s = 0; s < 3; ++s) {
      tc::mbar_init(&bars->k_full[s], 1);
      tc::mbar_init(&bars->k_empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      tc::mbar_init(&bars->v_full[s], 1);
      tc::mbar_init(&bars->v_empty[s], 1);
      tc::mbar_init(&bars->s_full[s], 1);
      tc::mbar_init(&bars->dq_done[s], 1);
    }
    tc::mbar_init(&bars->dp_full, 1);
    tc::mbar_init(&bars->ds_full, kWork);
    tc::mbar_init(&bars->drain, 2);
    tc::mbar_init(&bars->hold, 1);
    bars->abort = 0;
    bars->doc_lo = 0x7fffffff;
    bars->doc_hi = -1;
    tc::fence_mbar_init();
  }
  if (warp == kMmaS) {
    tc::tmem_alloc(&bars->tmem_base, 512);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (DOCS) {
    for (int i = i0 + threadIdx.x; i < i1; i += kThreads) {
      const int doc = doc_q[i];
      if (doc >= 0) {
        atomicMin(&bars->doc_lo, doc);
        atomicMax(&bars->doc_hi, doc);
      }
    }
    __syncthreads();
  }
  const uint32_t tbase = __shfl_sync(0xffffffffu, bars->tmem_base, 0);
  const int key1 = dense_limit(seq, a.causal, i1 - 1);
  BlockWalk<DOCS> walk(DOCS ? a.doc_blocks_k + (int64_t)b * blocks : nullptr, 0, (key1 + kT - 1) / kT,
                 bars->doc_lo, bars->doc_hi);
  const uint32_t n = (uint32_t)walk.count(lane);

  if (warp >= kWork) {
    tc::regs_down<kRegsOther>();
    if (warp == kLoader) {
      // ------------------------------------------------------------ loader
      uint32_t g = 0, k_armed = 0, v_armed = 0;      // steps whose copies were issued
      bool q_armed = false, ok = true;
      for (int j; ok && (j = walk.next(lane)) >= 0; ++g) {
        if (held(a, &bars->hold, abort, g)) {
          fail(&bars->abort, 20);
          ok = false;
          break;
        }
        const uint32_t sk = g % 3, sv = g & 1;
        unsigned char* dk = smem + L::kOffK + sk * L::kTile;
        if (g == 0) {
          if (lane == 0) {
            tc::mbar_expect_tx(&bars->q_full, 2 * (uint32_t)(qpt * a.G) * 128 * (D / 64));
            for (int c = 0; c < D / 64; ++c) {
              tc::tma_load_5d(smem + L::kOffQ + c * L::kChunk, &tmQ, &bars->q_full, c * 64, 0, i0, h, b);
              tc::tma_load_5d(smem + L::kOffG + c * L::kChunk, &tmG, &bars->q_full, c * 64, 0, i0, h, b);
            }
          }
          q_armed = true;
        }
        ok = warp_wait(&bars->k_empty[sk], ((g / 3) & 1) ^ 1, abort);
        if (!ok) break;
        // keys that do not exist: zeros, whatever their memory holds (0 * NaN would reach dQ)
        const bool dirty = (seq.kv < a.Sk && (j + 1) * kT > seq.kv) || (DOCS && walk.doc().x < 0);
        if (dirty) {
          copy_keys<D>(dk, static_cast<const __nv_bfloat16*>(a.k) + (int64_t)b * a.ks.b + (int64_t)h * a.ks.h, a.ks.s, j * kT,
                       kT, seq.kv, doc_k, lane, 32);
          tc::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&bars->k_full[sk]);
        } else if (lane == 0) {
          tc::mbar_expect_tx(&bars->k_full[sk], L::kTile);
          for (int c = 0; c < D / 64; ++c)
            tc::tma_load_4d(dk + c * L::kChunk, &tmK, &bars->k_full[sk], c * 64, j * kT, h, b);
        }
        k_armed = g + 1;
        ok = warp_wait(&bars->v_empty[sv], ((g >> 1) & 1) ^ 1, abort);
        if (!ok) break;
        if (lane == 0) {
          tc::mbar_expect_tx(&bars->v_full[sv], L::kTile);
          for (int c = 0; c < D / 64; ++c)
            tc::tma_load_4d(smem + L::kOffV + sv * L::kTile + c * L::kChunk, &tmV, &bars->v_full[sv], c * 64, j * kT, h, b);
        }
        v_armed = g + 1;
      }
      if (!ok) fail(&bars->abort, 3);
      if (lane == 0) {
        // no copy may still be writing shared memory when the CTA leaves: the last of each stage
        if (q_armed) tc::mbar_wait_drain(&bars->q_full, 0, kWaitLimit);
        for (uint32_t k = k_armed > 3 ? k_armed - 3 : 0; k < k_armed; ++k)
          tc::mbar_wait_drain(&bars->k_full[k % 3], (k / 3) & 1, kWaitLimit);
        for (uint32_t k = v_armed > 2 ? v_armed - 2 : 0; k < v_armed; ++k)
          tc::mbar_wait_drain(&bars->v_full[k & 1], (k >> 1) & 1, kWaitLimit);
      }
    } else {
      // ------------------------------------------------------------ MMA issuers
      // Each warp keeps step as a whole, so that what the products take is the same in all lanes; one lane
      // issues. One warp makes dP and dQ, in this order: dS(g+1) waits for dP(g+1).
      if (n > 0 && warp != kMmaDp) {
        constexpr uint32_t kStage = L::kTile >> 4;
        bool ok = true;
        auto wait = [&](uint64_t* bar, uint32_t parity, int code) {
          ok = ok && warp_wait(bar, parity, abort);
          if (!ok) fail(&bars->abort, code);
          tc::fence_after_sync();
          return ok;
        };
        wait(&bars->q_full, 0, 7);
        uint32_t st = 0, turn = 0;       // K's stage of the step and how often it has come round
        auto advance = [&] {
          if (++st == L::kStagesK) {
            st = 0;
            ++turn;
          }
        };
        if (warp == kMmaS) {
          const uint64_t qa = desc_dims(tc::smem_u32(smem + L::kOffQ)), kd = desc_dims(tc::smem_u32(smem + L::kOffK));
          for (uint32_t g = 0; ok && g < n; ++g) {
            // dS of the step before last has been read
            if (g >= 2 && !wait(&bars->dq_done[g & 1], ((g >> 1) & 1) ^ 1, 4)) break;
            if (!wait(&bars->k_full[st], turn & 1, 5)) break;
            if (tc::elect_one()) {
              mma_dims<D>(tbase + (g & 1 ? kColB : kColA), qa, kd + st * kStage);
              tc::mma_commit(&bars->s_full[g & 1]);
            }
            __syncwarp();
            advance();
          }
        } else {
          const uint64_t ga = desc_dims(tc::smem_u32(smem + L::kOffG)), vd = desc_dims(tc::smem_u32(smem + L::kOffV));
          const uint64_t kt = desc_tokens(tc::smem_u32(smem + L::kOffK));
          for (uint32_t g = 0; ok && g <= n; ++g) {
            if (g < n && !wait(&bars->v_full[g & 1], (g >> 1) & 1, 6)) break;
            // dP(g) may overwrite dP(g-1) once dS(g-1) has been made from it
            if (g > 0 && !wait(&bars->ds_full, (g - 1) & 1, 8)) break;
            if (g < n) {
              if (tc::elect_one()) {
                mma_dims<D>(tbase + L::kColDp, ga, vd + (g & 1) * kStage);
                tc::mma_commit(&bars->dp_full);
                tc::mma_commit(&bars->v_empty[g & 1]);
              }
              __syncwarp();
            }
            if (g > 0) {
              const uint32_t e = g - 1;
              if (tc::elect_one()) {
                mma_tokens<D>(tbase + L::kColQ, tbase + (e & 1 ? kColB : kColA), kt + st * kStage, e > 0);
                tc::mma_commit(&bars->dq_done[e & 1]);
                tc::mma_commit(&bars->k_empty[st]);
              }
              __syncwarp();
              advance();
            }
          }
        }
        if (tc::elect_one()) tc::mma_commit(&bars->drain);
        __syncwarp();
        if (lane == 0) tc::mbar_wait_drain(&bars->drain, 0, kWaitLimit);
        __syncwarp();
      }
    }
  } else {
    // ------------------------------------------------------------ elementwise
    tc::regs_up<kRegsWork>();
    const int q = warp & 3, cg = warp >> 2, col0 = cg * kCols;      // TMEM lane quarter, keys of a tile
    const int r = q * 32 + lane, i = i0 + r / a.G, hq = h * a.G + r % a.G;
    const uint32_t lanes = (uint32_t)(q * 32) << 16;
    const bool valid = r < qpt * a.G && i < a.Sq;
    DenseRow row{0, 0, 0, 0.f};
    float lse2 = 0.f, delta = 0.f;
    if (valid) {
      row = dense_row(a, seq, b, hq, i);
      const int64_t flat = ((int64_t)b * a.Hq + hq) * a.Sq + i;
      lse2 = a.lse[flat] * kLog2e;
      delta = a.delta[flat];
    }
    const ScoreMap<CAP, BIAS> map(a, row);
    const uint64_t after2 = f2(map.after, map.after), nlse2 = f2(-lse2, -lse2), ndelta2 = f2(-delta, -delta);
    uint64_t pw[kCols / 2];          // P, then P times the cap's derivative, in pairs
    uint32_t see = 0xffffffffu;      // bit c: this lane's row sees key c of this warp's
    uint32_t g = 0;
    const uint32_t colP = tbase + lanes + L::kColDp + col0;

    auto probs = [&](auto masked, uint32_t colS, int far) {
      constexpr bool MASK = decltype(masked)::value;
      uint32_t s[32];
      tc::tmem_ld32(colS, s);
      tc::tmem_ld_wait();
      if (CAP) {
        tanh32(s, map.in, MASK, see);
        if (BIAS) {                         // kept for the derivative: the bias takes its place
#pragma unroll
          for (int c = 0; c < 32; c += 2) pw[c / 2] = f2(__uint_as_float(s[c]), __uint_as_float(s[c + 1]));
        }
      }
      if (BIAS) map.bias(s, far);
#pragma unroll
      for (int c = 0; c < 32; c += 2) {
        const uint64_t t2 = f2(__uint_as_float(s[c]), __uint_as_float(s[c + 1]));
        float y0, y1;
        f2_split(ffma2(t2, after2, nlse2), y0, y1);
        float p0 = ex2(y0), p1 = ex2(y1);
        if (MASK) {
          p0 = (see >> c) & 1u ? p0 : 0.f;
          p1 = (see >> (c + 1)) & 1u ? p1 : 0.f;
        }
        pw[c / 2] = CAP ? times_dcap(f2(p0, p1), BIAS ? pw[c / 2] : t2) : f2(p0, p1);
      }
    };
    // dS over the scores of this warp, which are in registers
    auto grads = [&](auto masked, uint32_t colS) {
      constexpr bool MASK = decltype(masked)::value;
      uint32_t dp[32], packed[16];
      tc::tmem_ld32(colP, dp);
      tc::tmem_ld_wait();
#pragma unroll
      for (int c = 0; c < 32; c += 2) {
        float d0, d1;
        f2_split(fmul2(pw[c / 2], fadd2(f2(__uint_as_float(dp[c]), __uint_as_float(dp[c + 1])), ndelta2)), d0, d1);
        if (MASK) {                         // dP of a hidden pair may be anything
          d0 = (see >> c) & 1u ? d0 : 0.f;
          d1 = (see >> (c + 1)) & 1u ? d1 : 0.f;
        }
        packed[c / 2] = pack_bf16(d0, d1);
      }
      tc::tmem_st16(colS, packed);
    };

    bool ok = true;
    for (int j; (j = walk.next(lane)) >= 0; ++g) {
      const uint32_t colS = tbase + lanes + (g & 1 ? kColB : kColA) + col0;
      const int first = j * kT + col0;
      see = (uint32_t)visible64<DOCS>(row, doc_k, walk.doc(), first, a.Sk, lane);
      const bool hidden = __any_sync(0xffffffffu, see != 0xffffffffu);
      if (!warp_wait(&bars->s_full[g & 1], (g >> 1) & 1, abort)) {
        fail(&bars->abort, 10);
        ok = false;
        break;
      }
      tc::fence_after_sync();
      if (hidden) probs(std::true_type{}, colS, row.pos - first); else probs(std::false_type{}, colS, row.pos - first);
      if (!warp_wait(&bars->dp_full, g & 1, abort)) {
        fail(&bars->abort, 11);
        ok = false;
        break;
      }
      tc::fence_after_sync();
      if (hidden) grads(std::true_type{}, colS); else grads(std::false_type{}, colS);
      tc::tmem_st_wait();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&bars->ds_full);
    }
    if (n > 0 && ok) {
      if (!warp_wait(&bars->drain, 0, abort)) fail(&bars->abort, 12);
      tc::fence_after_sync();
    }
    const bool broken = __any_sync(0xffffffffu, *abort != 0);
    const float by = broken ? __int_as_float(0x7fffffff) : a.scale;
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.dq) + (int64_t)b * a.dqs.b + (int64_t)hq * a.dqs.h +
                         (int64_t)i * a.dqs.s;
    // each column group of warps writes 32 dims
#pragma unroll 1
    for (int cc = cg; cc < D / 32; cc += kWork / 4) {
      uint32_t o[32];
#pragma unroll
      for (int e = 0; e < 32; ++e) o[e] = 0u;
      if (n > 0 && !broken) {
        tc::tmem_ld32(tbase + lanes + L::kColQ + cc * 32, o);
        tc::tmem_ld_wait();
      }
      if (valid) store32(dst + cc * 32, o, by);
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == kMmaS) tc::tmem_dealloc(tbase, 512);
  if (threadIdx.x == 0 && bars->abort && a.status != nullptr)
    report_error(a.status, FVATTN_ERR_TIMEOUT, 400 + bars->abort);
}

// All of TMEM is one CTA's, so no second one may share the SM: it would wait for the first to leave.
constexpr size_t kAloneBytes = 120 * 1024;

template <int D, bool CAP, bool BIAS, bool DOCS>
cudaError_t launch(const DenseArgs& a, cudaStream_t st) {
  const int qpt = kTileRows / a.G;
  const int qpr = kR / a.G;
  CUtensorMap mq, mg, mqr, mgr, mk, mv;
  if (!make_map_rows(&mq, a.q, a.qs, a, qpt) || !make_map_rows(&mg, a.dout, a.dos, a, qpt) ||
      !make_map_rows(&mqr, a.q, a.qs, a, qpr) || !make_map_rows(&mgr, a.dout, a.dos, a, qpr) ||
      !make_map_keys(&mk, a.k, a.ks, a, kT) || !make_map_keys(&mv, a.v, a.vs, a, kT))
    return cudaErrorInvalidValue;
  {
    auto* kernel = dense_dkv_tc_kernel<D, CAP, BIAS, DOCS>;
    const size_t smem = imax<size_t>(DkvLayout<D>::kBytes + 1024, kAloneBytes);
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    const TileOrder order = tile_order(a, (a.Sk + kT - 1) / kT, a.causal);
    // Where the key tiles leave half of the 148 SMs idle, a cluster shares a tile's steps, four each at least
    // (2 x 1999 packed tokens, 8 / 2 heads of 64: 64 tiles, 60 us in clusters of two, 84 us without).
    const int64_t grid = (int64_t)order.tiles * order.heads, steps = (a.Sq + qpr - 1) / qpr;
    if (grid > 0x7fffffff) return cudaErrorInvalidValue;
    DenseArgs c = a;
    c.cluster = 1;
    while (c.cluster < 8 && grid * c.cluster * 2 <= 148 && steps >= c.cluster * 8) c.cluster *= 2;
    e = launch_with(kernel, dim3((unsigned)(grid * c.cluster)), kThreads, smem, st, c.cluster, true, mqr, mgr, mk, mv, c, qpr,
                    order);
    if (e != cudaSuccess) return e;
  }
  auto* kernel = dense_dq_tc_kernel<D, CAP, BIAS, DOCS>;
  const size_t smem = imax<size_t>(DqLayout<D>::kBytes + 1024, kAloneBytes);
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const TileOrder order = tile_order(a, (a.Sq + qpt - 1) / qpt, a.causal);
  if ((int64_t)order.tiles * order.heads > 0x7fffffff) return cudaErrorInvalidValue;
  return launch_with(kernel, dim3((unsigned)(order.tiles * order.heads)), kThreads, smem, st, 0, true, mq, mg, mk, mv, a, qpt,
                     order);
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

cudaError_t launch_dense_bwd_tc(const DenseArgs& a, cudaStream_t st) {
  return a.d == 128 ? launch_d<128>(a, st) : launch_d<64>(a, st);
}

}  // namespace fv
