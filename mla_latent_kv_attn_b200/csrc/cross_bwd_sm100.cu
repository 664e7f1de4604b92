// cross_bwd_sm100.cu - the gradients of the cross attention on the sm_100a tensor cores, for bf16
// with head widths 64 and 128 (the mathematics are in cross_simt.cu).  Three launches:
//
//   stats   per query row lse log2(e) and delta = g . o, in arrays padded to whole 128-row tiles (a
//           padding row's lse is +infinity, so that its probabilities are zero)
//   dK, dV  a 128-row tile of states per block, streaming the query tiles of the heads that share
//           it:  S^T = K Q_i^T, dP^T = V G_i^T, dV += P^T G_i, dK += dS^T Q_i
//   dQ      a 128-row query tile per item, streaming the states' tiles:
//             S = Q K_j^T, dP = G V_j^T, dS = P o (dP - delta) scale, dQ += dS K_j
//           and, where several blocks share a tile of states, the sums of their dK and dV, added in a
//           fixed order and rounded once
//
// The launches overlap: each grid starts while the one before it ends and waits for it where it needs
// its results (stats -> dK, dV: the statistics; dK, dV -> dQ: only the sums) and once more at its end,
// so that the end of the last says that all have ended.  One after the other, and with the sums in a
// launch of their own, the call took 69 us instead of 63.
// S and dP are computed twice (7 products where 5 would do): a single pass has to add dQ over the
// blocks of the state tiles, through atomics in an order that changes from run to run, or in fp32 copies
// that cost more memory traffic than the two products (115 MB for 4680 queries, 12 heads and 512
// states).  A cluster per set of up to 8 state tiles could add them in order through shared memory, and
// up to 128 states need no sum; that kernel is not built.
// (The statistics inside the dQ kernel, by warps of their own, made that call 75 us instead of 70: the
// first tiles wait for rows from DRAM.)
// Measured: 4680 queries, 512 states, 12 heads of 128: 62.3 us a call with three inputs in turn (part of
// them in L2), 591 TFLOP/s over the five products of the formula and 828 over the seven computed (0.50
// of the measured peak), 68.3 us where every call finds its inputs in memory; batch 4 of these, three
// inputs in turn, 170 to 216 us by how mixed the lengths are and 242 at full ones; batch 2, 1333 queries,
// up to 333 states, 16 heads of 64 on 4: 34 us.
// P and dS are rounded to bf16 as operands (in TMEM), the type that the products with bf16 K, Q and G
// take; every product accumulates in fp32 in TMEM.  The gradients are then off by 2.4e-3 of themselves
// (root mean square), where rounding the results alone gives 1.7e-3.
// Every wait is bounded; one that runs out writes MLA_ERR_DEVICE_TIMEOUT to dev_status.
#include "cross_tc.cuh"

namespace mla {

namespace {

using namespace sm100;

constexpr int kT = kCrossTile;            // rows of every tile
constexpr int kSoftmaxThreads = 256;      // two threads per row, each with half of the columns
constexpr int kProducerWarp = 8;
constexpr int kIssuerA = 9, kIssuerB = 10;
constexpr int kSumWarp = 11;
constexpr int kThreads = 384;
constexpr uint32_t kTmemCols = 512;

struct CrossBwdParams {
  int B, H, Hkv, rep, n_q, n_kv, n_pad;   // n_pad: n_q rounded up to whole tiles of both kinds
  int q_tiles, items;                     // dQ: items of one query tile
  int kv_tiles, splits;                   // dK, dV: blocks that share a tile's queries,
  int qn_tiles;                           // query tiles of 80
  float scale, scale_log2;
  const int32_t* kv_len;
  const float* lse2;                      // [B, H, n_pad]
  const float* delta;                     // [B, H, n_pad]
  float* partial;                         // [2, splits, B, Hkv, kv_tiles, D/4, 128, 4]
  int* next_item;                         // dQ: the next item that no block has
  int32_t* dev_status;
};

// p = 2^(s scale - l) of kN columns of a row, in place; l is the row's (dQ, l_step 0) or the column's
// (dK, dV: neg_l2 holds kN / 2 pairs).
template <int kN>
__device__ __forceinline__ void probabilities(uint32_t* s, uint64_t scale2, const uint64_t* neg_l2,
                                              int l_step) {
#pragma unroll
  for (int k = 0; k < kN / 2; ++k) {
    float x0, x1;
    f2_unpack(f2_fma(f2_pack(__uint_as_float(s[2 * k]), __uint_as_float(s[2 * k + 1])), scale2,
                     neg_l2[k * l_step]),
              x0, x1);
    s[2 * k] = __float_as_uint(fast_exp2(x0));
    s[2 * k + 1] = __float_as_uint(fast_exp2(x1));
  }
}

// dS = p (dP scale - delta scale) of kN columns, as bf16 pairs.
template <int kN>
__device__ __forceinline__ void score_gradients(const uint32_t (&dp)[kN], const uint32_t* p,
                                                uint64_t scale2, const uint64_t* neg_d2, int d_step,
                                                uint32_t (&w)[kN / 2]) {
#pragma unroll
  for (int k = 0; k < kN / 2; ++k) {
    float d0, d1;
    f2_unpack(f2_mul(f2_fma(f2_pack(__uint_as_float(dp[2 * k]), __uint_as_float(dp[2 * k + 1])),
                            scale2, neg_d2[k * d_step]),
                     f2_pack(__uint_as_float(p[2 * k]), __uint_as_float(p[2 * k + 1]))),
              d0, d1);
    w[k] = pack_bf16x2(d0, d1);
  }
}

// acc (+)= A B with A [128, 128] as bf16 pairs in TMEM, each half of its columns in the first 32 of
// 64 columns from `a` on, and B [128, D] a tile read MN-major.
template <int D>
__device__ __forceinline__ void mma_pairs_by_tile(uint32_t acc, uint32_t a, uint32_t tile,
                                                  bool accumulate) {
  constexpr uint32_t idesc = idesc_bf16_f32(kT, D, 0, 1);
  const uint64_t b = smem_desc(tile, kT * 128, 1024, kSwizzle128B);
#pragma unroll
  for (int kk = 0; kk < kT / 16; ++kk)
    mma_ts(acc, a + 64 * (kk >> 2) + 8 * (kk & 3), b + 128 * kk, idesc,
           (accumulate || kk) ? 1u : 0u);
}

// d = A B^T of two K-major tiles in shared memory, A [128, D] and B [kN, D].
template <int D, int kN = kT>
__device__ __forceinline__ void mma_tiles(uint32_t d, uint32_t a_tile, uint32_t b_tile) {
  constexpr uint32_t idesc = idesc_bf16_f32(kT, kN, 0, 0);
  const uint64_t a = smem_desc(a_tile, 16, 1024, kSwizzle128B);
  const uint64_t b = smem_desc(b_tile, 16, 1024, kSwizzle128B);
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk)
    mma_ss(d, a + (((kk >> 2) * kT * 128 >> 4) + 2 * (kk & 3)),
           b + (((kk >> 2) * kN * 128 >> 4) + 2 * (kk & 3)), idesc, kk ? 1u : 0u);
}

// acc (+)= A B with A [128, kN] as bf16 pairs in kN / 2 columns of TMEM from `a` on, and B [kN, D] a
// tile read MN-major.
template <int D, int kN>
__device__ __forceinline__ void mma_pairs_by_rows(uint32_t acc, uint32_t a, uint32_t tile,
                                                  bool accumulate) {
  constexpr uint32_t idesc = idesc_bf16_f32(kT, D, 0, 1);
  const uint64_t b = smem_desc(tile, kN * 128, 1024, kSwizzle128B);
#pragma unroll
  for (int kk = 0; kk < kN / 16; ++kk)
    mma_ts(acc, a + 8 * kk, b + 128 * kk, idesc, (accumulate || kk) ? 1u : 0u);
}

// One thread: the tile of rows [row, row + kN) of head h of sample b.
template <int D, int kN = kT>
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap* map, uint32_t bar, int h,
                                          int row, int b) {
#pragma unroll
  for (int k = 0; k < D / 64; ++k)
    tma_load_4d(dst + k * kN * 128, map, bar, 64 * k, h, row, b);
}

// ------------------------------------------------------------------------------------- stats

// One block per 64 rows of one head: 16 lanes read a row (8 or 4 values each).
constexpr int kStatRows = 64;

template <int D>
__global__ void __launch_bounds__(256)
    cross_stats_kernel(const bf16* __restrict__ out, const bf16* __restrict__ g,
                       const float* __restrict__ lse, float* __restrict__ lse2,
                       float* __restrict__ delta, int* next_item, int first_item, int H, int n_q,
                       int n_pad) {
  grid_dep_wait();
  grid_dep_launch();
  if ((threadIdx.x | blockIdx.x | blockIdx.y | blockIdx.z) == 0) *next_item = first_item;
  constexpr int kPer = D / 16;
  const int h = blockIdx.y, b = blockIdx.z;
  const int64_t bh = static_cast<int64_t>(b) * H + h;
  const int l16 = threadIdx.x % 16, i0 = blockIdx.x * kStatRows + threadIdx.x / 16;
  constexpr int kRows = kStatRows / 16;
  // every row's loads are on their way before the first is used
  uint32_t x[kRows][kPer / 2], y[kRows][kPer / 2];
  float l[kRows];
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    const int i = i0 + 16 * k;
    const int64_t at = ((static_cast<int64_t>(b) * n_q + min(i, n_q - 1)) * H + h) * D + l16 * kPer;
    if constexpr (D == 128) {
      *reinterpret_cast<uint4*>(x[k]) = *reinterpret_cast<const uint4*>(out + at);
      *reinterpret_cast<uint4*>(y[k]) = *reinterpret_cast<const uint4*>(g + at);
    } else {
      *reinterpret_cast<uint2*>(x[k]) = *reinterpret_cast<const uint2*>(out + at);
      *reinterpret_cast<uint2*>(y[k]) = *reinterpret_cast<const uint2*>(g + at);
    }
    l[k] = i < n_q ? lse[bh * n_q + i] * kLog2e : INFINITY;
  }
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    const int i = i0 + 16 * k;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < kPer / 2; ++e) {
      // a bf16 is the upper half of its float
      s = fmaf(__uint_as_float(x[k][e] << 16), __uint_as_float(y[k][e] << 16), s);
      s = fmaf(__uint_as_float(x[k][e] & 0xffff0000u), __uint_as_float(y[k][e] & 0xffff0000u), s);
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (l16 == 0) {
      lse2[bh * n_pad + i] = l[k];
      delta[bh * n_pad + i] = i < n_q ? s : 0.f;
    }
  }
}

// ---------------------------------------------------------------------------------------- dQ

// dK and dV where several blocks share a tile of states: the sums over them, in order.  A warp takes
// 32 columns of 32 rows, a row per thread; rows of masked states are 0.  The block's next piece is
// number `*next`; false when there is none.
template <int D>
__device__ __forceinline__ bool sum_piece(const CrossBwdParams& p, bf16* d_k, bf16* d_v, int* next,
                                          int lane) {
  constexpr int kRowParts = kT / 32, kColParts = D / 32;
  int e = lane == 0 ? atomicAdd(next, 1) : 0;
  e = blockIdx.x + gridDim.x * __shfl_sync(0xffffffffu, e, 0);
  const int bt = e / (2 * kRowParts * kColParts);
  if (bt >= p.B * p.Hkv * p.kv_tiles) return false;
  const int row = e % kRowParts * 32 + lane, c = e / kRowParts % kColParts * 32;
  const int which = e / (kRowParts * kColParts) % 2;
  const int tile = bt % p.kv_tiles, kh = bt / p.kv_tiles % p.Hkv, b = bt / p.kv_tiles / p.Hkv;
  const int j = tile * kT + row;
  if (j >= p.n_kv) return true;
  float4 a[8] = {};
  if (j < cross_len(p.kv_len, b, p.n_kv)) {
    const int64_t step = static_cast<int64_t>(p.B) * p.Hkv * p.kv_tiles * (kT * D);
    const float4* src = reinterpret_cast<const float4*>(
        p.partial + which * p.splits * step + static_cast<int64_t>(bt) * (kT * D)) + c / 4 * kT + row;
#pragma unroll 2
    for (int s = 0; s < p.splits; ++s, src += step / 4) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float4 v = __ldcg(src + k * kT);
        a[k].x += v.x; a[k].y += v.y; a[k].z += v.z; a[k].w += v.w;
      }
    }
  }
  uint4* dst = reinterpret_cast<uint4*>(
      (which ? d_v : d_k) + ((static_cast<int64_t>(b) * p.n_kv + j) * p.Hkv + kh) * D + c);
#pragma unroll
  for (int k = 0; k < 8; k += 2)
    dst[k / 2] = make_uint4(pack_bf16x2(a[k].x, a[k].y), pack_bf16x2(a[k].z, a[k].w),
                            pack_bf16x2(a[k + 1].x, a[k + 1].y), pack_bf16x2(a[k + 1].z, a[k + 1].w));
  return true;
}

template <int D_>
struct DqShape {
  static constexpr int D = D_;
  static constexpr int kTile = kT * D * 2;
  // K_j is held from S(j) to the product with dS(j), almost two steps; V_j for one product
  static constexpr int kKStages = D == 128 ? 3 : 4;
  static constexpr int kVStages = D == 128 ? 1 : 3;
  static constexpr int kTiles = 3 + kKStages + kVStages;      // Q, G, dQ, then the rings
  static constexpr int kSmem = kTiles * kTile + 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory");
};
constexpr uint32_t kDqColS = 0, kDqColDP = 128, kDqColAcc = 384;    // dP twice

struct DqItem {
  int b, h, q0, len;
  __device__ __forceinline__ int tiles() const { return ceil_div(len, kT); }
};
constexpr int kItems = 4;                 // ring of items

template <int kKStages, int kVStages>
struct DqShared {
  uint64_t item_full[kItems], item_empty[kItems];
  uint64_t q_full, q_empty;               // the item's Q, read by its last S
  uint64_t g_full, g_empty;               // the item's G, read by its last dP
  uint64_t k_full[kKStages], k_empty[kKStages];
  uint64_t v_full[kVStages], v_empty[kVStages];
  uint64_t s_full, s_free;                // S(j) complete; read
  uint64_t dp_full[2], dq_done[2];        // dP(j) complete; the product with dS(j) complete
  uint64_t ds_full[2];                    // dS(j) in TMEM: by parity, for dS(j+1) may come before
                                          // the issuer has seen dS(j)
  uint64_t acc_free;                      // the item's dQ is in registers
  uint64_t staged, stage_free;            // and in shared memory; stored from there
  uint32_t tmem_base;
  int abort_flag;
  int next_sum;                           // pieces of the sums that warps have taken
  DqItem item[kItems];                    // q0 < 0: there are no more
};

// Item `it`; its length comes from global memory, some 700 cycles away.
__device__ __forceinline__ DqItem dq_item(const CrossBwdParams& p, int it) {
  DqItem w{0, 0, -1, 0};
  if (it >= p.items) return w;
  w.q0 = (it % p.q_tiles) * kT;
  const int bh = it / p.q_tiles;
  w.h = bh % p.H;
  w.b = bh / p.H;
  w.len = cross_len(p.kv_len, w.b, p.n_kv);
  return w;
}

// Roles (384 threads): warps 0-7 softmax (warps w and w + 4 share 32 rows, each half of the
// columns), 8 TMA producer, 9 issuer of S, 10 issuer of dP and dQ, 11 sums of dK and dV, which
// the softmax warps end after their items.  The two dP buffers let dP(j+1) run under the softmax of
// j, and S(j+1) runs once S(j) has been read.
// The producer draws the block's items after its first from a counter that the statistics reset, an
// item ahead of its loads, and hands them to the other roles; these take an item ahead of their work
// (the softmax reads its rows' statistics then).  Blocks start as the dK, dV kernel's end and lengths
// differ: with a fixed share for each block, the call of four samples took 216 us.
// (Three more warps for the sums would leave each thread 128 registers, too few for the softmax.)
// This grid starts block by block as the dK, dV kernel's blocks end: only the sums need its results.
// (It starts when every block of that kernel runs and has seen the end of the statistics.  What it
// reads before its own wait comes from L2, where everything written before the statistics ended is:
// this SM's L1 may hold lines from before.)
template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    cross_dq_tc_kernel(const __grid_constant__ CUtensorMap tm_q,
                       const __grid_constant__ CUtensorMap tm_g,
                       const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v,
                       const __grid_constant__ CUtensorMap tm_dq, bf16* __restrict__ d_q,
                       bf16* __restrict__ d_k, bf16* __restrict__ d_v, CrossBwdParams p) {
  using Sh = DqShape<D>;
  constexpr int kTile = Sh::kTile, kKStages = Sh::kKStages, kVStages = Sh::kVStages;
  static_assert(sizeof(DqShared<kKStages, kVStages>) <= 1024, "shared memory");
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t sQ = smem_u32(smem_raw), sG = sQ + kTile, sOut = sG + kTile, sK = sOut + kTile;
  const uint32_t sV = sK + kKStages * kTile;
  auto& sh = *reinterpret_cast<DqShared<kKStages, kVStages>*>(smem_raw + Sh::kTiles * kTile);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  volatile int* abort_flag = &sh.abort_flag;

  if (threadIdx.x == 0) {
    sh.abort_flag = 0;
    sh.next_sum = 0;
    mbar_init(smem_u32(&sh.q_full), 1);
    mbar_init(smem_u32(&sh.q_empty), 1);
    mbar_init(smem_u32(&sh.g_full), 1);
    mbar_init(smem_u32(&sh.g_empty), 1);
    mbar_init(smem_u32(&sh.stage_free), 1);
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&sh.dp_full[b]), 1);
      mbar_init(smem_u32(&sh.dq_done[b]), 1);
      mbar_init(smem_u32(&sh.ds_full[b]), kSoftmaxThreads);
    }
    for (int s = 0; s < kItems; ++s) {
      mbar_init(smem_u32(&sh.item_full[s]), 1);
      mbar_init(smem_u32(&sh.item_empty[s]), 2 + kSoftmaxThreads / 32);   // issuers, softmax warps
    }
    for (int s = 0; s < kKStages; ++s) {
      mbar_init(smem_u32(&sh.k_full[s]), 1);
      mbar_init(smem_u32(&sh.k_empty[s]), 1);
    }
    for (int s = 0; s < kVStages; ++s) {
      mbar_init(smem_u32(&sh.v_full[s]), 1);
      mbar_init(smem_u32(&sh.v_empty[s]), 1);
    }
    mbar_init(smem_u32(&sh.s_full), 1);
    mbar_init(smem_u32(&sh.s_free), kSoftmaxThreads);
    mbar_init(smem_u32(&sh.acc_free), kSoftmaxThreads);
    mbar_init(smem_u32(&sh.staged), kSoftmaxThreads);
    fence_barrier_init();
  }
  if (warp == kIssuerA) {
    tmem_alloc(smem_u32(&sh.tmem_base), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem_base;
  grid_dep_launch();

  const auto wait = [&](uint64_t& bar, uint32_t phase) {
    return mbar_wait_or_abort(smem_u32(&bar), phase & 1, abort_flag, p.dev_status);
  };
  DqItem next = dq_item(p, blockIdx.x);       // every role finds the first item itself
  // The next item, for a thread that others do not follow.
  uint32_t n_items = 0;
  const auto take = [&]() {
    const int slot = n_items % kItems;
    DqItem w{0, 0, -1, 0};
    if (wait(sh.item_full[slot], n_items / kItems)) {
      w = sh.item[slot];
      mbar_arrive(smem_u32(&sh.item_empty[slot]));
    }
    ++n_items;
    return w;
  };
  // The same for a warp.
  const auto take_warp = [&]() {
    const int slot = n_items % kItems;
    DqItem w{0, 0, -1, 0};
    if (__all_sync(0xffffffffu, wait(sh.item_full[slot], n_items / kItems))) w = sh.item[slot];
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&sh.item_empty[slot]));
    ++n_items;
    return w;
  };

  if (warp == kProducerWarp) {
    if (lane == 0) {
      uint32_t n = 0, t = 0;              // items with loads, tiles
      bool ok = true;
      const auto publish = [&](const DqItem& w) {
        const int slot = n_items % kItems;
        if (!wait(sh.item_empty[slot], n_items / kItems + 1)) return false;
        sh.item[slot] = w;
        mbar_arrive(smem_u32(&sh.item_full[slot]));
        ++n_items;
        return true;
      };
      while (ok && next.q0 >= 0) {
        const DqItem w = next;
        const int id = atomicAdd(p.next_item, 1), nt = w.tiles();
        if (nt > 0) {
          ok = wait(sh.q_empty, n + 1);
          if (!ok) break;
          const uint32_t qb = smem_u32(&sh.q_full);
          mbar_arrive_expect_tx(qb, kTile);
          load_tile<D>(sQ, &tm_q, qb, w.h, w.q0, w.b);
        }
        for (int j = 0; j < nt && ok; ++j, ++t) {
          const int ks = t % kKStages, vs = t % kVStages;
          ok = wait(sh.k_empty[ks], t / kKStages + 1);
          if (!ok) break;
          const uint32_t kb = smem_u32(&sh.k_full[ks]);
          mbar_arrive_expect_tx(kb, kTile);
          load_tile<D>(sK + ks * kTile, &tm_k, kb, w.h / p.rep, j * kT, w.b);
          if (j == 0) {
            ok = wait(sh.g_empty, n + 1);
            if (!ok) break;
            const uint32_t gb = smem_u32(&sh.g_full);
            mbar_arrive_expect_tx(gb, kTile);
            load_tile<D>(sG, &tm_g, gb, w.h, w.q0, w.b);
          }
          ok = wait(sh.v_empty[vs], t / kVStages + 1);
          if (!ok) break;
          const uint32_t vb = smem_u32(&sh.v_full[vs]);
          mbar_arrive_expect_tx(vb, kTile);
          load_tile<D>(sV + vs * kTile, &tm_v, vb, w.h / p.rep, j * kT, w.b);
          if (j == 0) {
            next = dq_item(p, id);
            ok = publish(next);
          }
        }
        if (nt == 0) {
          next = dq_item(p, id);
          ok = publish(next);
        } else {
          ++n;
        }
      }
    }
  } else if (warp == kIssuerA) {
    if (lane == 0) {
      uint32_t n = 0, t = 0;
      bool ok = true;
      while (ok && next.q0 >= 0) {
        const DqItem w = next;
        next = take();
        const int nt = w.tiles();
        if (nt == 0) continue;
        ok = wait(sh.q_full, n);
        for (int j = 0; j < nt && ok; ++j, ++t) {
          ok = wait(sh.k_full[t % kKStages], t / kKStages) && (t == 0 || wait(sh.s_free, t - 1));
          if (!ok) break;
          tc_fence_after();
          mma_tiles<D>(tmem + kDqColS, sQ, sK + (t % kKStages) * kTile);
          mma_commit(smem_u32(&sh.s_full));
          if (j == nt - 1) mma_commit(smem_u32(&sh.q_empty));
        }
        ++n;
      }
    }
  } else if (warp == kIssuerB) {
    if (lane == 0) {
      uint32_t n = 0, t = 0;
      bool ok = true;
      // dP of tile u into buffer u & 1, which the product with dS(u-2) has read
      const auto issue_dp = [&](uint32_t u, bool last) {
        if (!wait(sh.v_full[u % kVStages], u / kVStages) ||
            (u >= 2 && !wait(sh.dq_done[u & 1], (u >> 1) - 1)))
          return false;
        tc_fence_after();
        mma_tiles<D>(tmem + kDqColDP + 128 * (u & 1), sG, sV + (u % kVStages) * kTile);
        mma_commit(smem_u32(&sh.v_empty[u % kVStages]));
        mma_commit(smem_u32(&sh.dp_full[u & 1]));
        if (last) mma_commit(smem_u32(&sh.g_empty));
        return true;
      };
      while (ok && next.q0 >= 0) {
        const DqItem w = next;
        next = take();
        const int nt = w.tiles();
        if (nt == 0) continue;
        ok = wait(sh.g_full, n) && issue_dp(t, nt == 1);
        for (int j = 0; j < nt && ok; ++j, ++t) {
          if (j + 1 < nt) ok = issue_dp(t + 1, j + 2 == nt);
          ok = ok && wait(sh.ds_full[t & 1], t >> 1) && (j > 0 || n == 0 || wait(sh.acc_free, n - 1));
          if (!ok) break;
          tc_fence_after();
          mma_pairs_by_tile<D>(tmem + kDqColAcc, tmem + kDqColDP + 128 * (t & 1),
                               sK + (t % kKStages) * kTile, j > 0);
          mma_commit(smem_u32(&sh.k_empty[t % kKStages]));
          mma_commit(smem_u32(&sh.dq_done[t & 1]));
        }
        ++n;
      }
    }
  } else if (warp == kSumWarp) {
    if (p.splits > 1) {
      grid_dep_wait();
      while (sum_piece<D>(p, d_k, d_v, &sh.next_sum, lane)) {
      }
    }
  } else {
    const int ch = warp / 4, row = (warp % 4) * 32 + lane;
    const uint32_t tl = tmem + (static_cast<uint32_t>((warp % 4) * 32) << 16);
    const uint32_t ts = tl + kDqColS + 64 * ch;
    const uint64_t sl2 = f2_pack(p.scale_log2, p.scale_log2);
    const auto wait_all = [&](uint64_t& bar, uint32_t phase) {
      return __all_sync(0xffffffffu, wait(bar, phase)) != 0;
    };
    uint32_t n = 0, t = 0;
    bool ok = true;
    float next_l = 0.f, next_d = 0.f;
    const auto read_stats = [&]() {
      if (next.q0 < 0) return;
      const int64_t at = (static_cast<int64_t>(next.b) * p.H + next.h) * p.n_pad + next.q0 + row;
      next_l = __ldcg(p.lse2 + at);
      next_d = __ldcg(p.delta + at);
    };
    read_stats();
    while (ok && next.q0 >= 0) {
      const DqItem w = next;
      const float nl = -next_l, row_delta = next_d;
      next = take_warp();
      read_stats();
      const int nt = w.tiles();
      if (nt == 0) {
        const int i = w.q0 + row;
        if (i < p.n_q) {
          uint4* o4 = reinterpret_cast<uint4*>(
              d_q + ((static_cast<int64_t>(w.b) * p.n_q + i) * p.H + w.h) * D + D / 2 * ch);
          for (int c = 0; c < D / 16; ++c) o4[c] = make_uint4(0u, 0u, 0u, 0u);
        }
        continue;
      }
      // a single state's softmax is constant: its dS is zero
      const float sc = w.len == 1 ? 0.f : p.scale, nd = -row_delta * sc;
      const uint64_t nl2 = f2_pack(nl, nl), sc2 = f2_pack(sc, sc), nd2 = f2_pack(nd, nd);
      for (int j = 0; j < nt; ++j, ++t) {
        ok = wait_all(sh.s_full, t);
        if (!ok) break;
        tc_fence_after();
        const int valid = w.len - j * kT - 64 * ch;
        uint32_t pr[64];                 // S, then P
        tmem_ld64_wait(ts, pr);
        tc_fence_before();
        mbar_arrive(smem_u32(&sh.s_free));
        probabilities<64>(pr, sl2, &nl2, 0);
        ok = wait_all(sh.dp_full[t & 1], t >> 1);
        if (!ok) break;
        tc_fence_after();
        const uint32_t td = tl + kDqColDP + 128 * (t & 1) + 64 * ch;
#pragma unroll
        for (int c = 0; c < 64; c += 32) {
          uint32_t dp[32], ds[16];
          tmem_ld32_wait(td + c, dp);
          score_gradients<32>(dp, pr + c, sc2, &nd2, 0, ds);
          if (valid < c + 32) {
            // masked states, whatever their scores and dP hold
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              if (c + 2 * k >= valid) ds[k] = 0u;
              else if (c + 2 * k + 1 >= valid) ds[k] &= 0xffffu;
            }
          }
          tmem_st16(td + c / 2, ds);
        }
        if (w.len - j * kT < kT && w.len < p.n_kv) {
          // the product reads the keys of masked states: this half's rows become zeros
          zero_rows<D / 64, kT>(sK + (t % kKStages) * kTile, 64 * ch + max(valid, 0), 64 * ch + 64,
                            threadIdx.x % 128, 128);
          fence_proxy_async_smem();
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(smem_u32(&sh.ds_full[t & 1]));
      }
      if (!ok) break;
      if (threadIdx.x == 0 && n > 0) {       // its copy out of shared memory, an item ago
        bulk_wait_group_read<0>();
        mbar_arrive(smem_u32(&sh.stage_free));
      }
      ok = wait_all(sh.dq_done[(t - 1) & 1], (t - 1) >> 1) &&
           (n == 0 || wait_all(sh.stage_free, n - 1));
      if (!ok) break;
      tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < D / 2; c += 32) {
        uint32_t r[32];
        const int col = D / 2 * ch + c;
        tmem_ld32_wait(tl + kDqColAcc + col, r);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            v[e] = pack_bf16x2(__uint_as_float(r[8 * k + 2 * e]), __uint_as_float(r[8 * k + 2 * e + 1]));
          store_shared16(swizzled_piece(sOut + (col / 64) * kT * 128, row, (col % 64) / 8 + k), v);
        }
      }
      tc_fence_before();
      mbar_arrive(smem_u32(&sh.acc_free));
      fence_proxy_async_smem();
      mbar_arrive(smem_u32(&sh.staged));
      if (threadIdx.x == 0 && wait(sh.staged, n)) {
        for (int k = 0; k < D / 64; ++k)           // (rows past n_q are not written)
          tma_store_4d(&tm_dq, sOut + k * kT * 128, 64 * k, w.h, w.q0, w.b);
        bulk_commit_group();
      }
      __syncwarp();
      ++n;
    }
    if (threadIdx.x == 0) bulk_wait_group_all();
    __syncwarp();
    if (ok && p.splits > 1) {
      grid_dep_wait();
      while (sum_piece<D>(p, d_k, d_v, &sh.next_sum, lane)) {
      }
    }
  }
  settle_after_abort(abort_flag);
  tc_fence_before();
  __syncthreads();
  if (warp == kIssuerA) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  grid_dep_wait();      // the end of this grid says that those before it have ended
}

// ------------------------------------------------------------------------------------- dK, dV

constexpr int kQN = 80;            // queries of a streamed tile (64: the call 4 % slower)
constexpr int kQH = kQN / 2;       // columns that a thread holds at a time

template <int D_>
struct DkvShape {
  static constexpr int D = D_;
  static constexpr int kTile = kT * D * 2;                    // K, V
  static constexpr int kQTile = kQN * D * 2;                  // Q_i, G_i
  static constexpr int kStages = D == 128 ? 3 : 4;
  static constexpr int kStatBytes = 2 * kQN * 4;              // lse2 and delta of a query tile
  static constexpr int kStat = 2 * kTile + 2 * kStages * kQTile;
  static constexpr int kSync = kStat + kStages * kStatBytes;
  static constexpr int kSmem = kSync + 1024;
  static_assert(kSync % 8 == 0 && kSmem <= 227 * 1024, "shared memory");
};
// TMEM columns: dK and dV (D each) from 0, then
constexpr uint32_t kColS = 256, kColP = kColS + kQN, kColDP = 384, kColDS = kColDP + kQN;

// Arrays of two: by the parity of the tile.
template <int kStages>
struct DkvShared {
  uint64_t k_full, v_full;
  uint64_t q_full[kStages], q_empty[kStages];    // Q_i and its statistics
  uint64_t g_full[kStages], g_empty[kStages];
  uint64_t s_full[2], s_free[2];                 // S^T complete; read
  uint64_t dp_full[2], dp_free[2];               // dP^T complete; read
  uint64_t p_full[2], ds_full[2];                // P^T, dS^T in TMEM
  uint64_t dv_done[2], dk_done[2];               // the products that read them complete
  uint32_t tmem_base;
  int abort_flag;
};

// A block per split, state tile, key head and sample.  Roles (352 threads): warps 0-3 and 4-7 softmax
// of the even and of the odd query tiles, one state (TMEM lane) per thread, 8 TMA producer, 9 issuer
// of S^T and dV, 10 issuer of dP^T and dK.  With tiles of 80 queries S^T, P^T, dP^T and dS^T have
// columns of their own beside dK and dV, so every product runs as soon as its operands are there and
// two tiles are in the softmax at a time.  (With 128 queries P^T has to take the place of S^T and
// dS^T that of dP^T, and a step is a chain of products and exponentials: 3240 cycles for 128 queries,
// against 2048 of products.)
// Rows of masked states hold whatever their scores gave; they reach no other row and are not used.
constexpr int kThreadsKV = 352;

template <int D>
__global__ void __launch_bounds__(kThreadsKV, 1)
    cross_dkv_tc_kernel(const __grid_constant__ CUtensorMap tm_q,
                        const __grid_constant__ CUtensorMap tm_g,
                        const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v, bf16* __restrict__ d_k,
                        bf16* __restrict__ d_v, CrossBwdParams p) {
  using Sh = DkvShape<D>;
  constexpr int kTile = Sh::kTile, kQTile = Sh::kQTile, kStages = Sh::kStages;
  constexpr uint32_t kColDK = 0, kColDV = D;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t sK = smem_u32(smem_raw), sV = sK + kTile, sQ = sV + kTile;
  const uint32_t sG = sQ + kStages * kQTile, sStat = sK + Sh::kStat;
  const float* stats = reinterpret_cast<const float*>(smem_raw + Sh::kStat);
  auto& sh = *reinterpret_cast<DkvShared<kStages>*>(smem_raw + Sh::kSync);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int split = blockIdx.x % p.splits, bt = blockIdx.x / p.splits;
  const int tile = bt % p.kv_tiles, kh = bt / p.kv_tiles % p.Hkv, b = bt / p.kv_tiles / p.Hkv;
  volatile int* abort_flag = &sh.abort_flag;

  if (threadIdx.x == 0) {
    sh.abort_flag = 0;
    mbar_init(smem_u32(&sh.k_full), 1);
    mbar_init(smem_u32(&sh.v_full), 1);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_u32(&sh.q_full[s]), 1);
      mbar_init(smem_u32(&sh.q_empty[s]), 1);
      mbar_init(smem_u32(&sh.g_full[s]), 1);
      mbar_init(smem_u32(&sh.g_empty[s]), 2);      // dP^T and dV
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sh.s_full[i]), 1);
      mbar_init(smem_u32(&sh.s_free[i]), kT);
      mbar_init(smem_u32(&sh.dp_full[i]), 1);
      mbar_init(smem_u32(&sh.dp_free[i]), kT);
      mbar_init(smem_u32(&sh.p_full[i]), kT);
      mbar_init(smem_u32(&sh.ds_full[i]), kT);
      mbar_init(smem_u32(&sh.dv_done[i]), 1);
      mbar_init(smem_u32(&sh.dk_done[i]), 1);
    }
    fence_barrier_init();
  }
  if (warp == kIssuerA) {
    tmem_alloc(smem_u32(&sh.tmem_base), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem_base;

  const auto wait = [&](uint64_t& bar, uint32_t phase) {
    return mbar_wait_or_abort(smem_u32(&bar), phase & 1, abort_flag, p.dev_status);
  };
  const auto wait2 = [&](uint64_t (&bar)[2], int i) { return wait(bar[i & 1], i >> 1); };
  const int len = cross_len(p.kv_len, b, p.n_kv);
  // this block's share of the (head, query tile) pairs: none for a tile of masked states
  const int work = p.rep * p.qn_tiles;
  const int first = static_cast<int>(static_cast<int64_t>(work) * split / p.splits);
  const int n = tile * kT < len
                    ? static_cast<int>(static_cast<int64_t>(work) * (split + 1) / p.splits) - first
                    : 0;

  // row `row` of the tile's dK (0) or dV (1)
  const auto grad_row = [&](int which, int row) {
    return (which ? d_v : d_k) +
           ((static_cast<int64_t>(b) * p.n_kv + tile * kT + row) * p.Hkv + kh) * D;
  };

  if (n == 0) {
    // a tile of masked states: zeros, here or from the sum
    if (p.splits == 1 && threadIdx.x < 2 * kT) {
      const int row = threadIdx.x % kT;
      if (tile * kT + row < p.n_kv) {
        uint4* dst = reinterpret_cast<uint4*>(grad_row(threadIdx.x / kT, row));
        for (int c = 0; c < D / 8; ++c) dst[c] = make_uint4(0u, 0u, 0u, 0u);
      }
    }
  } else if (warp == kProducerWarp) {
    if (lane == 0) {
      const uint32_t kb = smem_u32(&sh.k_full), vb = smem_u32(&sh.v_full);
      mbar_arrive_expect_tx(kb, kTile);
      load_tile<D>(sK, &tm_k, kb, kh, tile * kT, b);
      bool ok = true;
      for (int i = 0; i < n && ok; ++i) {
        const int s = i % kStages;
        const int h = kh * p.rep + (first + i) / p.qn_tiles, q0 = (first + i) % p.qn_tiles * kQN;
        ok = wait(sh.q_empty[s], i / kStages + 1);
        if (!ok) break;
        const uint32_t qb = smem_u32(&sh.q_full[s]);
        const uint32_t st = sStat + s * Sh::kStatBytes;
        const int64_t so = (static_cast<int64_t>(b) * p.H + h) * p.n_pad + q0;
        mbar_arrive_expect_tx(qb, kQTile + Sh::kStatBytes);
        load_tile<D, kQN>(sQ + s * kQTile, &tm_q, qb, h, q0, b);
        if (i == 0) {
          mbar_arrive_expect_tx(vb, kTile);
          load_tile<D>(sV, &tm_v, vb, kh, tile * kT, b);
        }
        ok = wait(sh.g_empty[s], i / kStages + 1);
        if (!ok) break;
        const uint32_t gb = smem_u32(&sh.g_full[s]);
        mbar_arrive_expect_tx(gb, kQTile);
        load_tile<D, kQN>(sG + s * kQTile, &tm_g, gb, h, q0, b);
        if (i == 0) {
          grid_dep_wait();          // the statistics
          grid_dep_launch();
        }
        bulk_load(st, p.lse2 + so, kQN * 4, qb);
        bulk_load(st + kQN * 4, p.delta + so, kQN * 4, qb);
      }
    }
  } else if (warp == kIssuerA) {
    if (lane == 0) {
      const auto issue_s = [&](int i) {
        const int s = i % kStages;
        if (!wait(sh.q_full[s], i / kStages) || (i > 0 && !wait2(sh.s_free, i - 1))) return false;
        tc_fence_after();
        mma_tiles<D, kQN>(tmem + kColS, sK, sQ + s * kQTile);
        mma_commit(smem_u32(&sh.s_full[i & 1]));
        return true;
      };
      bool ok = wait(sh.k_full, 0) && issue_s(0);
      for (int i = 0; i < n && ok; ++i) {
        const int s = i % kStages;
        ok = (i + 1 == n || issue_s(i + 1)) && wait(sh.g_full[s], i / kStages) &&
             wait2(sh.p_full, i);
        if (!ok) break;
        tc_fence_after();
        mma_pairs_by_rows<D, kQN>(tmem + kColDV, tmem + kColP, sG + s * kQTile, i > 0);
        mma_commit(smem_u32(&sh.g_empty[s]));
        mma_commit(smem_u32(&sh.dv_done[i & 1]));
      }
    }
  } else if (warp == kIssuerB) {
    if (lane == 0) {
      const auto issue_dp = [&](int i) {
        const int s = i % kStages;
        if (!wait(sh.g_full[s], i / kStages) || (i > 0 && !wait2(sh.dp_free, i - 1))) return false;
        tc_fence_after();
        mma_tiles<D, kQN>(tmem + kColDP, sV, sG + s * kQTile);
        mma_commit(smem_u32(&sh.g_empty[s]));
        mma_commit(smem_u32(&sh.dp_full[i & 1]));
        return true;
      };
      bool ok = wait(sh.v_full, 0) && issue_dp(0);
      for (int i = 0; i < n && ok; ++i) {
        const int s = i % kStages;
        ok = (i + 1 == n || issue_dp(i + 1)) && wait2(sh.ds_full, i);
        if (!ok) break;
        tc_fence_after();
        mma_pairs_by_rows<D, kQN>(tmem + kColDK, tmem + kColDS, sQ + s * kQTile, i > 0);
        mma_commit(smem_u32(&sh.q_empty[s]));
        mma_commit(smem_u32(&sh.dk_done[i & 1]));
      }
    }
  } else {
    const int grp = warp / 4, row = (warp % 4) * 32 + lane;
    const uint32_t tl = tmem + (static_cast<uint32_t>((warp % 4) * 32) << 16);
    // a single state's softmax is constant: its dS is zero
    const float sc = len == 1 ? 0.f : p.scale;
    const uint64_t sl2 = f2_pack(p.scale_log2, p.scale_log2), sc2 = f2_pack(sc, sc);
    const uint64_t neg2 = f2_pack(-1.f, -1.f), nsc2 = f2_pack(-sc, -sc);
    const auto all = [&](bool ok) { return __all_sync(0xffffffffu, ok) != 0; };
    bool ok = true;
    for (int i = grp; i < n; i += 2) {
      const int s = i % kStages;
      // S^T(i); the statistics came with the loads of q_full, complete since
      ok = all(wait2(sh.s_full, i) && wait(sh.q_full[s], i / kStages));
      if (!ok) break;
      tc_fence_after();
      const float4* lse4 = reinterpret_cast<const float4*>(stats + s * (Sh::kStatBytes / 4));
      const float4* del4 = lse4 + kQN / 4;
      uint32_t pr[kQN];                // S^T, then P^T
      uint32_t w[2][kQH / 2];
      tmem_ld80_wait(tl + kColS, pr);
      tc_fence_before();
      mbar_arrive(smem_u32(&sh.s_free[i & 1]));
#pragma unroll
      for (int c = 0; c < kQN; c += kQH) {
        uint64_t nl2[kQH / 2];
#pragma unroll
        for (int k = 0; k < kQH / 4; ++k) {
          const float4 l = lse4[c / 4 + k];
          nl2[2 * k] = f2_mul(f2_pack(l.x, l.y), neg2);
          nl2[2 * k + 1] = f2_mul(f2_pack(l.z, l.w), neg2);
        }
        probabilities<kQH>(pr + c, sl2, nl2, 1);
#pragma unroll
        for (int k = 0; k < kQH / 2; ++k)
          w[c / kQH][k] = pack_bf16x2(__uint_as_float(pr[c + 2 * k]), __uint_as_float(pr[c + 2 * k + 1]));
      }
      // dV(i-1) has read P^T(i-1)
      if (i > 0) ok = all(wait2(sh.dv_done, i - 1));
      if (!ok) break;
      tc_fence_after();
      tmem_st20(tl + kColP, w[0]);
      tmem_st20(tl + kColP + kQH / 2, w[1]);
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(smem_u32(&sh.p_full[i & 1]));
      ok = all(wait2(sh.dp_full, i));
      if (!ok) break;
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < kQN; c += kQH) {
        uint32_t dp[kQH];
        uint64_t nd2[kQH / 2];
        tmem_ld40_wait(tl + kColDP + c, dp);
        if (c + kQH == kQN) {
          tc_fence_before();
          mbar_arrive(smem_u32(&sh.dp_free[i & 1]));
        }
#pragma unroll
        for (int k = 0; k < kQH / 4; ++k) {
          const float4 d = del4[c / 4 + k];
          nd2[2 * k] = f2_mul(f2_pack(d.x, d.y), nsc2);
          nd2[2 * k + 1] = f2_mul(f2_pack(d.z, d.w), nsc2);
        }
        score_gradients<kQH>(dp, pr + c, sc2, nd2, 1, w[c / kQH]);
      }
      // dK(i-1) has read dS^T(i-1)
      if (i > 0) ok = all(wait2(sh.dk_done, i - 1));
      if (!ok) break;
      tc_fence_after();
      tmem_st20(tl + kColDS, w[0]);
      tmem_st20(tl + kColDS + kQH / 2, w[1]);
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(smem_u32(&sh.ds_full[i & 1]));
    }
    if (ok) ok = all(wait2(sh.dv_done, n - 1) && wait2(sh.dk_done, n - 1));
    if (ok) {
      tc_fence_after();
      if (p.splits == 1) {
        // the gradients themselves; rows of masked states are zero
        const int j = tile * kT + row;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t r[32];
          tmem_ld32_wait(tl + (grp == 0 ? kColDK : kColDV) + c, r);
          uint32_t v[16];
#pragma unroll
          for (int e = 0; e < 16; ++e)
            v[e] = j < len ? pack_bf16x2(__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1])) : 0u;
          if (j < p.n_kv) {
            uint4* dst = reinterpret_cast<uint4*>(grad_row(grp, row) + c);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              dst[k] = make_uint4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
          }
        }
      } else {
        // four columns of 32 rows are 512 consecutive bytes
        const int64_t tile_at =
            (((static_cast<int64_t>(split) * p.B + b) * p.Hkv + kh) * p.kv_tiles + tile) * (kT * D);
        const int64_t half = static_cast<int64_t>(p.splits) * p.B * p.Hkv * p.kv_tiles * (kT * D);
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t r[32];
          tmem_ld32_wait(tl + (grp == 0 ? kColDK : kColDV) + c, r);
          float4* dst = reinterpret_cast<float4*>(p.partial + grp * half + tile_at) + (c / 4) * kT + row;
#pragma unroll
          for (int k = 0; k < 8; ++k)
            dst[k * kT] = make_float4(__uint_as_float(r[4 * k]), __uint_as_float(r[4 * k + 1]),
                                      __uint_as_float(r[4 * k + 2]), __uint_as_float(r[4 * k + 3]));
        }
      }
    }
  }
  settle_after_abort(abort_flag);
  tc_fence_before();
  __syncthreads();
  if (warp == kIssuerA) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  grid_dep_wait();      // (a block without work)
}

// Blocks per tile of states.  With a tile for every SM none is shared: dQ fills the SMs that the last
// tiles leave.  That gains at mixed lengths (4 samples of 4680 queries, 12 heads, 512 states: 178 us
// against 192 with three blocks per tile) and where tiles fill whole rounds (2 samples of 2000 queries,
// 40 heads: 169 against 195), and loses at full lengths in between (247 against 233: 192 tiles on 148
// SMs); the host does not know the lengths.  Otherwise, of the counts that give every block at least one
// query tile, the one whose waves of 148 blocks take the fewest steps (a block costs about three steps
// beside its query tiles), the smallest on a tie: each more adds sums to write and read.  (Fewer blocks
// that leave SMs to dQ from the start: 88 us against 63 in one sample; loads of dQ slow the block on the
// SM beside it.)
int dkv_splits(int tiles, int work) {
  if (tiles >= 148) return 1;
  int best = 1;
  int64_t best_cost = INT64_MAX;
  for (int s = 1; s <= std::min(work, 16); ++s) {
    const int64_t waves = (static_cast<int64_t>(tiles) * s + 147) / 148;
    const int64_t cost = waves * (ceil_div(work, s) + 3);
    if (cost < best_cost) {
      best_cost = cost;
      best = s;
    }
  }
  return best;
}

struct BwdLayout {
  int n_pad, q_tiles, qn_tiles, kv_tiles, splits;
  size_t lse2, delta, partial, next_item, bytes;      // offsets of the arrays, and their end
};

BwdLayout bwd_layout(const CrossDims& d) {
  BwdLayout l;
  l.q_tiles = ceil_div(d.n_q, kT);
  l.qn_tiles = ceil_div(d.n_q, kQN);
  l.n_pad = round_up(std::max(l.q_tiles * kT, l.qn_tiles * kQN), kStatRows);
  l.kv_tiles = ceil_div(d.n_kv, kT);
  l.splits = dkv_splits(d.B * d.Hkv * l.kv_tiles, d.H / d.Hkv * l.qn_tiles);
  const size_t stat = static_cast<size_t>(d.B) * d.H * l.n_pad * sizeof(float);   // 256-byte rows
  l.lse2 = 0;
  l.delta = stat;
  l.partial = 2 * stat;
  const int sums = l.splits == 1 ? 0 : l.splits;
  l.next_item = l.partial +
            2 * static_cast<size_t>(sums) * d.B * d.Hkv * l.kv_tiles * kT * d.d * sizeof(float);
  l.bytes = l.next_item + sizeof(int);
  return l;
}

template <int D>
mla_status bwd_impl(const CrossDims& d, const CrossBwdArgs& a, void* workspace, cudaStream_t s) {
  const BwdLayout l = bwd_layout(d);
  char* ws = static_cast<char*>(workspace);
  CUtensorMap tq, tg, tk, tv, tdq, tqn, tgn;
  mla_status st;
  if ((st = cross_tmap(&tq, a.q, d.B, d.n_q, d.H, D, d.q_row, kT)) != MLA_OK) return st;
  if ((st = cross_tmap(&tg, a.d_out, d.B, d.n_q, d.H, D, d.H * D, kT)) != MLA_OK) return st;
  if ((st = cross_tmap(&tk, a.k, d.B, d.n_kv, d.Hkv, D, d.k_row, kT)) != MLA_OK) return st;
  if ((st = cross_tmap(&tv, a.v, d.B, d.n_kv, d.Hkv, D, d.v_row, kT)) != MLA_OK) return st;
  if ((st = cross_tmap(&tqn, a.q, d.B, d.n_q, d.H, D, d.q_row, kQN)) != MLA_OK) return st;
  if ((st = cross_tmap(&tgn, a.d_out, d.B, d.n_q, d.H, D, d.H * D, kQN)) != MLA_OK) return st;
  if ((st = cross_tmap(&tdq, a.d_q, d.B, d.n_q, d.H, D, d.H * D, kT)) != MLA_OK) return st;
  CrossBwdParams p;
  p.B = d.B; p.H = d.H; p.Hkv = d.Hkv; p.rep = d.H / d.Hkv; p.n_q = d.n_q; p.n_kv = d.n_kv;
  p.n_pad = l.n_pad;
  p.q_tiles = l.q_tiles; p.qn_tiles = l.qn_tiles;
  p.items = p.q_tiles * d.H * d.B;      // fewer than 2^31: every item has at least one query row
  p.kv_tiles = l.kv_tiles; p.splits = l.splits;
  p.scale = d.scale; p.scale_log2 = d.scale * kLog2e;
  p.kv_len = a.kv_len;
  float* lse2 = reinterpret_cast<float*>(ws + l.lse2);
  float* delta = reinterpret_cast<float*>(ws + l.delta);
  p.lse2 = lse2; p.delta = delta; p.partial = reinterpret_cast<float*>(ws + l.partial);
  p.next_item = reinterpret_cast<int*>(ws + l.next_item);
  p.dev_status = a.dev_status;
  const int tiles = d.B * d.Hkv * l.kv_tiles;      // at most 2^25: a tile has a state of 64 elements
  const int blocks = l.splits > 1 ? 148 : std::min(p.items, 148);       // (every SM takes sums)
  MLA_CUDA_TRY(cudaFuncSetAttribute(cross_dq_tc_kernel<D>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize, DqShape<D>::kSmem));
  MLA_CUDA_TRY(cudaFuncSetAttribute(cross_dkv_tc_kernel<D>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize, DkvShape<D>::kSmem));
  MLA_CUDA_TRY(launch_pdl(cross_stats_kernel<D>, dim3(l.n_pad / kStatRows, d.H, d.B), dim3(256), 0, s,
                          static_cast<const bf16*>(a.out), static_cast<const bf16*>(a.d_out), a.lse,
                          lse2, delta, p.next_item, blocks, d.H, d.n_q, l.n_pad));
  MLA_CUDA_TRY(launch_pdl(cross_dkv_tc_kernel<D>, dim3(tiles * l.splits),
                          dim3(kThreadsKV), DkvShape<D>::kSmem, s, tqn, tgn, tk, tv,
                          static_cast<bf16*>(a.d_k), static_cast<bf16*>(a.d_v), p));
  MLA_CUDA_TRY(launch_pdl(cross_dq_tc_kernel<D>, dim3(blocks), dim3(kThreads), DqShape<D>::kSmem, s,
                          tq, tg, tk, tv, tdq, static_cast<bf16*>(a.d_q), static_cast<bf16*>(a.d_k),
                          static_cast<bf16*>(a.d_v), p));
  return MLA_OK;
}

}  // namespace

size_t cross_bwd_tc_workspace(const CrossDims& d) { return bwd_layout(d).bytes; }

mla_status cross_bwd_tc(const CrossDims& d, const CrossBwdArgs& a, void* workspace,
                        cudaStream_t s) {
  return d.d == 128 ? bwd_impl<128>(d, a, workspace, s) : bwd_impl<64>(d, a, workspace, s);
}

}  // namespace mla
