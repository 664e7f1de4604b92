// cross_sm100.cu - cross attention to an encoder's states on the sm_100a tensor cores: the forward
// for bf16 with head widths 64 and 128 (the mathematics are in cross_simt.cu).
//
// One persistent CTA per SM takes work items of 256 query rows of one head of one sample, as two
// streams of 128 rows that share every key and value tile: while one stream's softmax runs on the
// CUDA cores, the other's products run on the tensor cores.  (With 128 rows per item the keys and
// values would cross L2 -> SM twice as often, 114 MB in the call of 4680 queries, 12 heads and 512
// states, whose products take 9 us.)  Roles (384 threads):
//   warps 0-3, 4-7  softmax of stream 0, 1, one TMEM lane (query row) per thread: online softmax in
//                 the log2 domain, O rescaled only when a row's maximum grows by more than 2^8; P
//                 rounded to bf16 (the type that the product with bf16 V takes: O is off by 2.3e-3 of
//                 itself, 1.7e-3 by its own rounding; the row sum l is taken from the unrounded values
//                 in fp32); O / l into shared memory, lse
//   warp 8        TMA producer: the item's two Q tiles (into the buffer that the item before last
//                 left), then K_0, V_0, K_1, V_1, ... through a ring of stages
//   warps 9, 10   MMA issuer of stream 0, 1: S = Q K_j^T (both in shared memory) and
//                 O += P_j V_j (P in TMEM, V read MN-major)
//   warp 11       TMA stores of O from the item's Q buffer.  (Stored by the softmax threads, 16
//                 bytes of 32 rows at a time, O took 9000 cycles an item.)
// A tile has 128 states for d 64 and 80 for d 128: S (80 columns) and P (40) of a stream then fit
// beside an O of 128, all of TMEM with two streams, and QK(j+1) runs under the softmax of j.  With 128
// states P would have to take the place of S, and a step is the chain QK, softmax, PV: 4900 cycles a
// pair of tiles of 128, against 2048 of products.
// An item's first QK of stream 1 waits for that of stream 0: streams in step would load the tensor
// and the CUDA cores in turn (6000 cycles a pair of tiles, against 2048 of products and 4500 as it is).
// States past a sample's length are masked: their scores become -infinity by selection, and their
// value rows are overwritten with zeros in shared memory (0 * NaN would reach O).
// Measured: 4680 queries, 512 states, 12 heads of 128: 24.8 us a call, 594 TFLOP/s (0.36 of the measured
// peak): two rounds of items, one of 148 pairs and one of 148 single tiles; the products' hand-overs
// bound them, and a pair's round in the steady state takes 11 us.  Batch 8 of these: 139 us at full
// lengths, 87 to 123 at mixed ones.  Batch 2, 1333 queries, up to 1501 states, 16 heads of 64 on 4:
// 42 us whatever the shorter sample's length: a round of 148 pairs takes 21 us in the steady state (13
// of them exponentials, 16 a cycle and SM; XU 51 % and tensor pipe 25 % active over the call), and the
// 56 single tiles left over, of the longest sample, the rest.  One query: 9.3 us, the host's side of the
// call.
#include <cfloat>

#include "cross_tc.cuh"

namespace mla {

namespace {

using namespace sm100;

constexpr int kBM = kCrossTile;      // query rows of a stream
constexpr int kStreamThreads = 128;
constexpr int kProducerWarp = 8;
constexpr int kIssuerWarp = 9;       // and 10; warp 9 also allocates TMEM
constexpr int kStoreWarp = 11;
constexpr int kThreads = 384;
constexpr int kSms = 148;
constexpr int kMaxSplits = 8;         // CTAs of a cluster
constexpr uint32_t kTmemCols = 512;
constexpr float kLn2 = 0.69314718055994530942f;

template <int D_>
struct FwdShape {
  static constexpr int D = D_;
  static_assert(D == 64 || D == 128, "head width");
  static constexpr int kBN = D == 128 ? 80 : 128;         // states of a tile
  static constexpr int kBlocks = D / 64;                  // 64-column blocks, 128B swizzle
  static constexpr int kBlk = kBM * 128;                  // 16 KB
  static constexpr int kTile = kBlocks * kBlk;            // Q, O
  static constexpr int kKvBlk = kBN * 128;                // 10 KB
  static constexpr int kKvTile = kBlocks * kKvBlk;
  static constexpr int kStages = D == 128 ? 4 : 8;
  static constexpr int kTileBytes = 4 * kTile + kStages * kKvTile;
  static constexpr int kSmem = kTileBytes + 2048;         // tiles, then FwdShared
  static_assert(kSmem <= 227 * 1024, "shared memory");
  // TMEM columns of stream i
  static constexpr uint32_t s_col(int i) { return 128u * i; }
  static constexpr uint32_t p_col(int i) { return D == 128 ? 128u * i + kBN : 256u + 64u * i; }
  static constexpr uint32_t o_col(int i) { return D == 128 ? 256u + 128u * i : 384u + 64u * i; }
};

struct CrossFwdParams {
  int n_q, H, rep, n_kv;
  // Items: `wide` ones of two query tiles (pairs per sample and head: of its tiles, in order), then
  // `halves` of one tile each that the pairs from `wide` on fall into, then the odd last tiles.
  int pairs, wide, halves, items;
  int splits;                        // CTAs (a cluster) that share an item's states
  float scale_log2;
  const int32_t* kv_len;
  bf16* out;
  float* lse;
  int32_t* dev_status;
};

// Barriers and small data behind the tiles.
template <int kStages>
struct FwdShared {
  uint64_t q_full[2][2], q_empty[2][2];     // [stream][buffer]
  uint64_t kv_full[kStages], kv_empty[kStages];
  uint64_t s_full[2];        // S(j) complete
  uint64_t s_free[2];        // S(j) has been read
  uint64_t p_full[2][2];     // each half of the states of P(j) is in TMEM
  uint64_t pv_done[2];       // PV(j) complete
  uint64_t o_free[2];        // the item's O is in registers
  uint64_t o_staged[2][2];   // and in the item's Q buffer: by buffer, for the next item's O may come
                             // before the store warp has seen this one's
  uint64_t first_qk[2];      // stream 0's first S of an item (by parity)
  uint32_t tmem_base;
  int abort_flag;
  float part_m[kBM], part_l[kBM];      // a split item's share of the row maxima and sums
};
static_assert(sizeof(FwdShared<8>) <= 2048, "shared memory");

struct Item {
  int b, h, q0, streams, len;
  int j0, nt;                // first tile of states, and how many
};

// Item `it` (the last one when there is none).  Every role decodes an item ahead of its work: the
// length comes from global memory, some 700 cycles away.
__device__ __forceinline__ Item item_of(const CrossFwdParams& p, int it, int bn) {
  it = min(it, p.items - 1);
  Item w;
  int bh;
  if (it < p.wide) {
    bh = it / p.pairs;
    w.q0 = (it % p.pairs) * 2 * kBM;
    w.streams = 2;
  } else {
    it -= p.wide;
    if (it < p.halves) {
      const int pair = p.wide + it / 2;
      bh = pair / p.pairs;
      w.q0 = (pair % p.pairs * 2 + it % 2) * kBM;
    } else {
      bh = it - p.halves;
      w.q0 = p.pairs * 2 * kBM;
    }
    w.streams = 1;
  }
  w.h = bh % p.H;
  w.b = bh / p.H;
  w.len = cross_len(p.kv_len, w.b, p.n_kv);
  w.j0 = 0;
  w.nt = ceil_div(w.len, bn);
  return w;
}

__device__ __forceinline__ void load_scores(uint32_t t, uint32_t (&s)[80]) { tmem_ld80_wait(t, s); }
__device__ __forceinline__ void load_scores(uint32_t t, uint32_t (&s)[128]) { tmem_ld128_wait(t, s); }
__device__ __forceinline__ void store_pairs(uint32_t t, const uint32_t (&w)[20]) { tmem_st20(t, w); }
__device__ __forceinline__ void store_pairs(uint32_t t, const uint32_t (&w)[32]) { tmem_st32(t, w); }

// The largest of a row's scores; those from `valid` on become -infinity.
template <int kBN>
__device__ __forceinline__ float masked_max(uint32_t (&s)[kBN], int valid) {
  if (valid < kBN) {
#pragma unroll
    for (int c = 0; c < kBN; ++c)
      if (c >= valid) s[c] = 0xff800000u;
  }
  float m8[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    float a = __uint_as_float(s[k]);
#pragma unroll
    for (int c = 8; c + 8 < kBN; c += 16)
      a = fmax3(a, __uint_as_float(s[c + k]), __uint_as_float(s[c + 8 + k]));
    m8[k] = kBN / 8 % 2 ? a : fmaxf(a, __uint_as_float(s[kBN - 8 + k]));
  }
  return fmaxf(fmax3(fmax3(m8[0], m8[1], m8[2]), m8[3], m8[4]), fmax3(m8[5], m8[6], m8[7]));
}

// p = 2^(s scale - m) of 2 kPairs consecutive scores of a row, packed to bf16 pairs; returns their
// sum.  (Taking every fourth or more of them from a polynomial on the FMA pipe made the call 4 to 7 %
// slower.)
template <int kPairs>
__device__ __forceinline__ float exp_pairs(const uint32_t* s, float scale_log2, float m,
                                           uint32_t (&w)[kPairs]) {
  const uint64_t sc2 = f2_pack(scale_log2, scale_log2), nm2 = f2_pack(-m, -m);
  uint64_t sum2[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    float x0, x1;
    f2_unpack(f2_fma(f2_pack(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), sc2, nm2),
              x0, x1);
    const float p0 = fast_exp2(x0), p1 = fast_exp2(x1);
    sum2[i & 3] = f2_add(sum2[i & 3], f2_pack(p0, p1));
    w[i] = pack_bf16x2(p0, p1);
  }
  float l0, l1;
  f2_unpack(f2_add(f2_add(sum2[0], sum2[1]), f2_add(sum2[2], sum2[3])), l0, l1);
  return l0 + l1;
}

// kSplit: a cluster of p.splits CTAs takes one item of one query tile, each a share of its states;
// their O, m and l meet in shared memory at the end.
template <int D, bool kSplit>
__global__ void __launch_bounds__(kThreads, 1)
    cross_fwd_tc_kernel(const __grid_constant__ CUtensorMap tm_q,
                        const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v,
                        const __grid_constant__ CUtensorMap tm_o, CrossFwdParams p) {
  using Sh = FwdShape<D>;
  constexpr int kStages = Sh::kStages, kTile = Sh::kTile, kBlk = Sh::kBlk;
  constexpr int kKvTile = Sh::kKvTile, kKvBlk = Sh::kKvBlk, kBN = Sh::kBN, kHalf = kBN / 2;
  // (the declared alignment is the swizzle's; there is no shared memory beside this)
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t sQ = smem_u32(smem_raw), sKV = sQ + 4 * kTile;  // Q buffer b of stream i: 2 i + b
  FwdShared<kStages>& sh = *reinterpret_cast<FwdShared<kStages>*>(smem_raw + Sh::kTileBytes);
  auto& q_full = sh.q_full;
  auto& q_empty = sh.q_empty;
  auto& kv_full = sh.kv_full;
  auto& kv_empty = sh.kv_empty;
  auto& s_full = sh.s_full;
  auto& s_free = sh.s_free;
  auto& p_full = sh.p_full;
  auto& pv_done = sh.pv_done;
  auto& o_free = sh.o_free;
  auto& o_staged = sh.o_staged;
  auto& first_qk = sh.first_qk;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  volatile int* abort_flag = &sh.abort_flag;

  if (kSplit && threadIdx.x < kBM) {
    sh.part_m[threadIdx.x] = -INFINITY;
    sh.part_l[threadIdx.x] = 0.f;
  }
  if (threadIdx.x == 0) {
    sh.abort_flag = 0;
    for (int i = 0; i < 2; ++i) {
      for (int b = 0; b < 2; ++b) {
        mbar_init(smem_u32(&q_full[i][b]), 1);
        mbar_init(smem_u32(&q_empty[i][b]), 1);
        mbar_init(smem_u32(&p_full[i][b]), kStreamThreads);
        mbar_init(smem_u32(&o_staged[i][b]), kStreamThreads);
      }
      mbar_init(smem_u32(&s_full[i]), 1);
      mbar_init(smem_u32(&s_free[i]), kStreamThreads);
      mbar_init(smem_u32(&pv_done[i]), 1);
      mbar_init(smem_u32(&o_free[i]), kStreamThreads);
      mbar_init(smem_u32(&first_qk[i]), 1);
    }
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_u32(&kv_full[s]), 1);
      mbar_init(smem_u32(&kv_empty[s]), 2);       // one arrival per stream
    }
    fence_barrier_init();
  }
  if (warp == kIssuerWarp) {
    tmem_alloc(smem_u32(&sh.tmem_base), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem_base;
  grid_dep_wait();
  grid_dep_launch();

  const auto wait = [&](uint64_t& bar, uint32_t phase) {
    return mbar_wait_or_abort(smem_u32(&bar), phase & 1, abort_flag, p.dev_status);
  };
  const int first_item = kSplit ? blockIdx.x / p.splits : blockIdx.x;
  const int item_step = kSplit ? p.items : gridDim.x;           // (a cluster has one item)
  const auto decode = [&](int it) {
    Item w = item_of(p, it, kBN);
    if constexpr (kSplit) {
      const int rank = blockIdx.x % p.splits, nt = w.nt;
      w.j0 = nt * rank / p.splits;
      w.nt = nt * (rank + 1) / p.splits - w.j0;
    }
    return w;
  };
  Item next = decode(first_item);

  if (warp == kProducerWarp) {
    if (lane == 0) {
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
      uint32_t n_item[2] = {0, 0}, u = 0;          // items of the streams, uses of the ring
      bool ok = true;
      for (int it = first_item; it < p.items && ok; it += item_step) {
        const Item w = next;
        next = decode(it + item_step);
        if (w.nt == 0) continue;
        for (int i = 0; i < w.streams && ok; ++i) {
          const int b = n_item[i] & 1;
          ok = wait(q_empty[i][b], (n_item[i] >> 1) + 1);
          if (!ok) break;
          ++n_item[i];
          const uint32_t fb = smem_u32(&q_full[i][b]);
          mbar_arrive_expect_tx(fb, kTile);
          for (int k = 0; k < Sh::kBlocks; ++k)
            tma_load_4d(sQ + (2 * i + b) * kTile + k * kBlk, &tm_q, fb, 64 * k, w.h,
                        w.q0 + i * kBM, w.b);
        }
        for (int j = 0; j < 2 * w.nt && ok; ++j, ++u) {
          const int s = u % kStages;
          ok = wait(kv_empty[s], u / kStages + 1);
          if (!ok) break;
          const uint32_t fb = smem_u32(&kv_full[s]);
          mbar_arrive_expect_tx(fb, kKvTile);
          for (int k = 0; k < Sh::kBlocks; ++k)
            tma_load_4d(sKV + s * kKvTile + k * kKvBlk, j & 1 ? &tm_v : &tm_k, fb, 64 * k, w.h / p.rep,
                        (w.j0 + (j >> 1)) * kBN, w.b);
        }
      }
    }
  } else if (warp == kStoreWarp) {
    if (!kSplit && lane == 0) {
      tma_prefetch_desc(&tm_o);
      uint32_t n_item[2] = {0, 0};
      bool ok = true;
      for (int it = first_item; it < p.items && ok; it += item_step) {
        const Item w = next;
        next = decode(it + item_step);
        if (w.nt == 0) continue;
        for (int i = 0; i < w.streams; ++i) {
          const int b = n_item[i] & 1;
          ok = wait(o_staged[i][b], n_item[i]++ >> 1);
          if (!ok) break;
          for (int k = 0; k < Sh::kBlocks; ++k)     // (rows past n_q are not written)
            tma_store_4d(&tm_o, sQ + (2 * i + b) * kTile + k * kBlk, 64 * k, w.h, w.q0 + i * kBM,
                         w.b);
          bulk_commit_group();
          bulk_wait_group_read<0>();
          mbar_arrive(smem_u32(&q_empty[i][b]));
        }
      }
      bulk_wait_group_all();
    }
  } else if (warp >= kIssuerWarp) {
    const int i = warp - kIssuerWarp;
    if (lane == 0) {
      constexpr uint32_t idesc_qk = idesc_bf16_f32(kBM, kBN, 0, 0);
      constexpr uint32_t idesc_pv = idesc_bf16_f32(kBM, D, 0, 1);
      const uint64_t qd0 = smem_desc(sQ + 2 * i * kTile, 16, 1024, kSwizzle128B);
      const uint64_t kd0 = smem_desc(sKV, 16, 1024, kSwizzle128B);
      const uint64_t vd0 = smem_desc(sKV, kKvBlk, 1024, kSwizzle128B);
      const uint32_t ts = tmem + Sh::s_col(i), tp = tmem + Sh::p_col(i), to = tmem + Sh::o_col(i);
      uint32_t n_item = 0, t = 0, u0 = 0;   // items and tiles of this stream, uses of the ring
      uint32_t n_both = 0;                  // items in which both streams have rows
      bool ok = true;
      const auto issue_qk = [&](uint32_t u) {
        const uint64_t qd = qd0 + ((n_item & 1) * kTile >> 4);
        const uint64_t kd = kd0 + ((u % kStages) * kKvTile >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_ss(ts, qd + (((kk >> 2) * kBlk >> 4) + 2 * (kk & 3)),
                 kd + (((kk >> 2) * kKvBlk >> 4) + 2 * (kk & 3)), idesc_qk, kk ? 1u : 0u);
        mma_commit(smem_u32(&kv_empty[u % kStages]));
        mma_commit(smem_u32(&s_full[i]));
      };
      for (int it = first_item; it < p.items && ok; it += item_step) {
        const Item w = next;
        next = decode(it + item_step);
        if (w.nt == 0) continue;
        if (i >= w.streams) {              // no rows for this stream: release what it would read
          for (int j = 0; j < 2 * w.nt && ok; ++j, ++u0) {
            ok = wait(kv_full[u0 % kStages], u0 / kStages);
            if (ok) mbar_arrive(smem_u32(&kv_empty[u0 % kStages]));
          }
          continue;
        }
        const bool both = w.streams == 2;
        ok = wait(q_full[i][n_item & 1], n_item >> 1);
        // Stream 0 cannot be two such items ahead of stream 1 (whose Q buffers would have to be
        // free again), so a barrier for each parity tells the items apart.
        if (i == 1) ok = ok && wait(first_qk[n_both & 1], n_both >> 1);
        for (int j = 0; j < w.nt && ok; ++j) {
          const uint32_t uk = u0 + 2 * j, uv = uk + 1;
          if (j == 0) {
            ok = wait(kv_full[uk % kStages], uk / kStages) && (t == 0 || wait(s_free[i], t - 1));
            if (!ok) break;
            tc_fence_after();
            issue_qk(uk);
            if (i == 0 && both) mma_commit(smem_u32(&first_qk[n_both & 1]));
          }
          if (j + 1 < w.nt) {
            const uint32_t un = uk + 2;
            ok = wait(kv_full[un % kStages], un / kStages) && wait(s_free[i], t);
            if (!ok) break;
            tc_fence_after();
            issue_qk(un);
          }
          ok = wait(kv_full[uv % kStages], uv / kStages) &&
               (j > 0 || n_item == 0 || wait(o_free[i], n_item - 1));
          const uint64_t vd = vd0 + ((uv % kStages) * kKvTile >> 4);
          for (int half = 0; half < 2 && ok; ++half) {
            ok = wait(p_full[i][half], t);
            if (!ok) break;
            tc_fence_after();
            // (the states of a k-step that spans the halves come with the second)
#pragma unroll
            for (int kk = 0; kk < kBN / 16; ++kk)
              if ((16 * kk + 15 >= kHalf) == (half == 1))
                mma_ts(to, tp + 8 * kk, vd + 128 * kk, idesc_pv, (j | kk) != 0 ? 1u : 0u);
          }
          if (!ok) break;
          mma_commit(smem_u32(&kv_empty[uv % kStages]));
          mma_commit(smem_u32(&pv_done[i]));
          ++t;
        }
        u0 += 2 * w.nt;
        ++n_item;
        n_both += both;
      }
    }
  } else {
    // ------------------------------------------------------------------ softmax
    const int i = warp / 4;                              // stream
    const int row = (warp % 4) * 32 + lane;              // TMEM lane
    const uint32_t tl = tmem + (static_cast<uint32_t>((warp % 4) * 32) << 16);
    const uint32_t ts = tl + Sh::s_col(i), tp = tl + Sh::p_col(i), to = tl + Sh::o_col(i);
    const auto wait_all = [&](uint64_t& bar, uint32_t phase) {
      return __all_sync(0xffffffffu, wait(bar, phase)) != 0;
    };
    uint32_t t = 0, u0 = 0, n_item = 0;
    bool ok = true;
    for (int it = first_item; it < p.items && ok; it += item_step) {
      const Item w = next;
      next = decode(it + item_step);
      if (w.nt == 0) {
        if constexpr (kSplit) break;
        const int n = w.q0 + i * kBM + row;
        if (i < w.streams && n < p.n_q) {
          uint4* o4 = reinterpret_cast<uint4*>(
              p.out + ((static_cast<int64_t>(w.b) * p.n_q + n) * p.H + w.h) * D);
          for (int c = 0; c < D / 8; ++c) o4[c] = make_uint4(0u, 0u, 0u, 0u);
          if (p.lse != nullptr)
            p.lse[(static_cast<int64_t>(w.b) * p.H + w.h) * p.n_q + n] = -INFINITY;
        }
        continue;
      }
      if (i >= w.streams) {
        u0 += 2 * w.nt;
        continue;
      }
      float m = 0.f, l = 0.f;
      for (int j = 0; j < w.nt; ++j, ++t) {
        ok = wait_all(s_full[i], t);
        if (!ok) break;
        tc_fence_after();
        const int valid = w.len - (w.j0 + j) * kBN;
        uint32_t s[kBN];
        load_scores(ts, s);
        tc_fence_before();
        mbar_arrive(smem_u32(&s_free[i]));
        const float mx = masked_max(s, valid) * p.scale_log2;
        float alpha = 1.f;
        bool rescale = false;
        if (j == 0) {
          m = fmaxf(mx, -FLT_MAX);      // scores of -infinity weigh nothing, also in the first tile
        } else if (__any_sync(0xffffffffu, mx > m + 8.f)) {
          const float m_new = fmaxf(m, mx);
          alpha = fast_exp2(m - m_new);
          l *= alpha;
          m = m_new;
          rescale = true;
        }
        uint32_t pw[kHalf / 2];
        l += exp_pairs(s, p.scale_log2, m, pw);
        // O and P's buffer are free once PV(j-1) is complete
        if (t > 0) {
          ok = wait_all(pv_done[i], t - 1);
          if (!ok) break;
          tc_fence_after();
        }
        if (rescale) {
#pragma unroll 1
          for (int c = 0; c < D; c += 16) {
            uint32_t r[16];
            tmem_ld16_wait(to + c, r);
#pragma unroll
            for (int k = 0; k < 16; ++k) r[k] = __float_as_uint(__uint_as_float(r[k]) * alpha);
            tmem_st16(to + c, r);
          }
        }
        if (valid < kBN && w.len < p.n_kv) {
          // the value rows of masked states (both streams write the same zeros)
          const uint32_t uv = u0 + 2 * j + 1;
          ok = wait_all(kv_full[uv % kStages], uv / kStages);
          if (!ok) break;
          zero_rows<Sh::kBlocks, kBN>(sKV + (uv % kStages) * kKvTile, valid, kBN, row, kBM);
          fence_proxy_async_smem();
        }
        store_pairs(tp, pw);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(smem_u32(&p_full[i][0]));
        l += exp_pairs(s + kHalf, p.scale_log2, m, pw);
        store_pairs(tp + kHalf / 2, pw);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(smem_u32(&p_full[i][1]));
      }
      if (!ok) break;
      u0 += 2 * w.nt;
      ok = wait_all(pv_done[i], t - 1);
      if (!ok) break;
      tc_fence_after();
      if constexpr (kSplit) {
        // O as it is, 16-byte pieces of a row in an order that spreads them over the banks
        sh.part_m[row] = m;
        sh.part_l[row] = l;
#pragma unroll 1
        for (int c = 0; c < D; c += 16) {
          uint32_t r[16];
          tmem_ld16_wait(to + c, r);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t v[4] = {r[4 * k], r[4 * k + 1], r[4 * k + 2], r[4 * k + 3]};
            store_shared16(sQ + row * (4 * D) + ((c / 4 + k) ^ (row % (D / 4))) * 16, v);
          }
        }
        break;
      }
      const float inv_l = 1.f / l;
      const int n = w.q0 + i * kBM + row;
      if (p.lse != nullptr && n < p.n_q)
        p.lse[(static_cast<int64_t>(w.b) * p.H + w.h) * p.n_q + n] = (m + log2f(l)) * kLn2;
      // O / l over the item's Q tile, which its last product has read: 16-byte pieces of this row
      // where a TMA copy with the 128-byte swizzle expects them
      const uint32_t stage = sQ + (2 * i + (n_item & 1)) * kTile;
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        uint32_t r[32];
        tmem_ld32_wait(to + c, r);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            v[e] = pack_bf16x2(__uint_as_float(r[8 * k + 2 * e]) * inv_l,
                               __uint_as_float(r[8 * k + 2 * e + 1]) * inv_l);
          store_shared16(swizzled_piece(stage + (c / 64) * kBlk, row, (c % 64) / 8 + k), v);
        }
      }
      tc_fence_before();
      mbar_arrive(smem_u32(&o_free[i]));
      fence_proxy_async_smem();
      mbar_arrive(smem_u32(&o_staged[i][n_item & 1]));
      ++n_item;
    }
  }
  settle_after_abort(abort_flag);
  tc_fence_before();
  __syncthreads();
  if (warp == kIssuerWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  if constexpr (kSplit) {
    // Every thread of the cluster comes here, also behind a wait that ran out (its rows then still
    // say m = -infinity).  O = sum_r 2^(m_r - m) O_r / sum_r 2^(m_r - m) l_r over the CTAs in order;
    // a thread takes four columns of a row.
    cluster_sync_all();
    const Item w = item_of(p, first_item, kBN);
    const int rows = min(kBM, p.n_q - w.q0);
    for (int e = (blockIdx.x % p.splits) * kThreads + threadIdx.x; e < rows * (D / 4);
         e += p.splits * kThreads) {
      const int r = e / (D / 4), piece = e % (D / 4);
      const uint32_t at_m = smem_u32(&sh.part_m[r]), at_l = smem_u32(&sh.part_l[r]);
      const uint32_t at_o = sQ + r * (4 * D) + (piece ^ (r % (D / 4))) * 16;
      // every load is on its way before the first is used
      float mc[kMaxSplits], lc[kMaxSplits];
      float4 oc[kMaxSplits];
#pragma unroll
      for (int c = 0; c < kMaxSplits; ++c) {
        const bool in = c < p.splits;
        mc[c] = in ? load_cluster_f(map_to_cta(at_m, c)) : -INFINITY;
        lc[c] = in ? load_cluster_f(map_to_cta(at_l, c)) : 0.f;
        oc[c] = in ? load_cluster_f4(map_to_cta(at_o, c)) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      float m = mc[0], l = 0.f;
#pragma unroll
      for (int c = 1; c < kMaxSplits; ++c) m = fmaxf(m, mc[c]);
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int c = 0; c < kMaxSplits; ++c) {
        if (mc[c] == -INFINITY) continue;        // no states
        const float f = fast_exp2(mc[c] - m);
        l = fmaf(f, lc[c], l);
        o.x = fmaf(f, oc[c].x, o.x);
        o.y = fmaf(f, oc[c].y, o.y);
        o.z = fmaf(f, oc[c].z, o.z);
        o.w = fmaf(f, oc[c].w, o.w);
      }
      const float inv = w.len > 0 ? 1.f / l : 0.f;
      const int64_t n = w.q0 + r;
      *reinterpret_cast<uint2*>(p.out + ((w.b * static_cast<int64_t>(p.n_q) + n) * p.H + w.h) * D +
                                4 * piece) =
          make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
      if (piece == 0 && p.lse != nullptr)
        p.lse[(static_cast<int64_t>(w.b) * p.H + w.h) * p.n_q + n] = (m + log2f(l)) * kLn2;
    }
    cluster_sync_all();       // the others have read this CTA's part
  }
}

template <int D>
mla_status fwd_impl(const CrossDims& d, const CrossArgs& a, cudaStream_t s) {
  using Sh = FwdShape<D>;
  CUtensorMap tq, tk, tv, to;
  mla_status st;
  if ((st = cross_tmap(&tq, a.q, d.B, d.n_q, d.H, D, d.q_row, kBM)) != MLA_OK) return st;
  if ((st = cross_tmap(&tk, a.k, d.B, d.n_kv, d.Hkv, D, d.k_row, Sh::kBN)) != MLA_OK) return st;
  if ((st = cross_tmap(&tv, a.v, d.B, d.n_kv, d.Hkv, D, d.v_row, Sh::kBN)) != MLA_OK) return st;
  if ((st = cross_tmap(&to, a.out, d.B, d.n_q, d.H, D, d.H * D, kBM)) != MLA_OK) return st;
  CrossFwdParams p;
  p.n_q = d.n_q; p.H = d.H; p.rep = d.H / d.Hkv; p.n_kv = d.n_kv;
  // fewer than 2^31 of each: every item has at least one query row
  const int tiles = ceil_div(d.n_q, kBM), heads = d.B * d.H, odd = tiles % 2 * heads;
  const int pairs = tiles / 2 * heads;
  p.pairs = tiles / 2;
  p.splits = 1;
  // Whole rounds of the SMs take pairs.  The pairs of the last, partial round become single tiles if
  // those fit in one round: a tile alone takes two thirds of a pair's time.
  p.wide = pairs / kSms * kSms;
  if (2 * (pairs - p.wide) + odd > kSms) p.wide = pairs;
  p.halves = 2 * (pairs - p.wide);
  p.items = p.wide + p.halves + odd;
  p.scale_log2 = d.scale * kLog2e;
  p.kv_len = a.kv_len; p.out = static_cast<bf16*>(a.out); p.lse = a.lse;
  p.dev_status = a.dev_status;
  // With at least three SMs for every single tile, several share its states.  In a graph, one query
  // against 512 and 2048 states: 12 tiles, 8 CTAs each, 6.5 and 9.4 us; 36 tiles, 4 each, 13.9 and 25.0;
  // 48, 3 each, 15.9 and 29.4; 50, unsplit, 11.2 and 31.4.  So sharing gains at many states and, where
  // clusters of 3 to 6 do not all find room at once, loses up to 5 us at few.  Two CTAs each for 50 to 74
  // tiles: 9.5 and 19.6 us, not taken up here.
  if (p.wide == 0 && 3 * p.items <= kSms)
    p.splits = std::min(std::min(kMaxSplits, kSms / p.items), ceil_div(d.n_kv, Sh::kBN));
  if (p.splits > 1) {
    MLA_CUDA_TRY(cudaFuncSetAttribute(cross_fwd_tc_kernel<D, true>,
                                      cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::kSmem));
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(p.items * p.splits);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Sh::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = p.splits;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled() ? 2 : 1;
    MLA_CUDA_TRY(cudaLaunchKernelEx(&cfg, cross_fwd_tc_kernel<D, true>, tq, tk, tv, to, p));
    return MLA_OK;
  }
  MLA_CUDA_TRY(cudaFuncSetAttribute(cross_fwd_tc_kernel<D, false>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::kSmem));
  MLA_CUDA_TRY(launch_pdl(cross_fwd_tc_kernel<D, false>, dim3(std::min(p.items, kSms)),
                          dim3(kThreads), Sh::kSmem, s, tq, tk, tv, to, p));
  return MLA_OK;
}

}  // namespace

bool cross_tc_supported(const CrossDims& d) {
  return d.dtype == MLA_BF16 && d.path == MLA_PATH_AUTO && (d.d == 64 || d.d == 128);
}

mla_status cross_fwd_tc(const CrossDims& d, const CrossArgs& a, cudaStream_t s) {
  return d.d == 128 ? fwd_impl<128>(d, a, s) : fwd_impl<64>(d, a, s);
}

}  // namespace mla
