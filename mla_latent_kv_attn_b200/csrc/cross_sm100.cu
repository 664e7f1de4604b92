// cross_sm100.cu - cross attention to an encoder's states on the sm_100a tensor cores: the forward
// for bf16 with head widths 64 and 128 (the mathematics are in cross_simt.cu).
//
// One persistent CTA per SM takes work items of 256 query rows of one head of one sample, as two
// streams of 128 rows that share every key and value tile: while one stream's softmax runs on the
// CUDA cores, the other's products run on the tensor cores.  (With 128 rows per item the keys and
// values would cross L2 -> SM twice as often, 114 MB in the call of 4680 queries, 12 heads and 512
// states, whose products take 9 us.)  Roles (352 threads):
//   warps 0-3, 4-7  softmax of stream 0, 1: one TMEM lane (query row) per thread; online softmax in
//                   the log2 domain, O rescaled only when a row's maximum grows by more than 2^8;
//                   P rounded to bf16 (the tensor cores' operand type; the row sum l is taken from
//                   the unrounded values in fp32); O / l, lse
//   warp 8          TMA producer: the item's two Q tiles, then K_0, V_0, K_1, V_1, ... (128 states
//                   each) through a ring of shared-memory stages
//   warps 9, 10     MMA issuer of stream 0, 1: S = Q K_j^T (both in shared memory) and
//                   O += P_j V_j (P in TMEM, V read MN-major)
// TMEM, 512 columns: two S buffers, two O accumulators and, for d 64, two P buffers.  For d 128
// nothing is left for P: it takes the second half of its S buffer, and QK(j+1) waits for PV(j).
// P becomes visible to PV in two halves of 64 states, so PV starts while the second half of the
// exponentials is still being computed.
// States past a sample's length are masked: their scores become -infinity by selection, and their
// value rows are overwritten with zeros in shared memory (0 * NaN would reach O).
#include "cross.h"
#include "exp2.cuh"
#include "kernels.h"
#include "sm100.cuh"

namespace mla {

namespace {

using namespace sm100;

constexpr int kBM = 128;             // query rows of a stream
constexpr int kBN = 128;             // states of a tile
constexpr int kProducerWarp = 8;
constexpr int kIssuerWarp = 9;       // and 10; warp 9 also allocates TMEM
constexpr int kThreads = 352;
constexpr uint32_t kTmemCols = 512;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kLog2e = 1.4426950408889634f;

template <int D_>
struct FwdShape {
  static constexpr int D = D_;
  static_assert(D == 64 || D == 128, "head width");
  static constexpr int kBlocks = D / 64;                  // 64-column blocks, 128B swizzle
  static constexpr int kBlk = kBM * 128;                  // 16 KB
  static constexpr int kTile = kBlocks * kBlk;
  static constexpr int kStages = D == 128 ? 5 : 8;
  static constexpr int kSmem = (2 + kStages) * kTile + 1024;
  static_assert(kSmem + 512 <= 227 * 1024, "shared memory");
  static constexpr bool kAliasP = D == 128;
  // Pairs (out of every 8) whose exponentials take the FMA-pipe polynomial instead of the SFU.
  static constexpr int kPolyPairs = 2;
  static constexpr uint32_t s_col(int i) { return 128u * i; }
  static constexpr uint32_t p_col(int i) { return kAliasP ? 128u * i + 64u : 256u + 64u * i; }
  static constexpr uint32_t o_col(int i) { return kAliasP ? 256u + 128u * i : 384u + 64u * i; }
};

struct CrossFwdParams {
  int n_q, H, rep, n_kv, pairs;      // pairs: items per (sample, head)
  int items;
  float scale_log2;
  const int32_t* kv_len;
  bf16* out;
  float* lse;
  int32_t* dev_status;
};

struct Item {
  int b, h, q0, len, nt;
};

__device__ __forceinline__ Item item_of(const CrossFwdParams& p, int it) {
  Item w;
  w.q0 = (it % p.pairs) * 2 * kBM;
  const int bh = it / p.pairs;
  w.h = bh % p.H;
  w.b = bh / p.H;
  w.len = cross_len(p.kv_len, w.b, p.n_kv);
  w.nt = ceil_div(w.len, kBN);
  return w;
}

// Zeros rows [from, 128) of a tile of kBlocks blocks of 128-byte rows (whatever the swizzle: it
// permutes within a row), `threads` threads of index t.
template <int kBlocks>
__device__ __forceinline__ void zero_rows(uint32_t tile, int from, int t, int threads) {
  const int n = (128 - from) * 8 * kBlocks;
  for (int i = t; i < n; i += threads) {
    const int blk = i / ((128 - from) * 8), o = i % ((128 - from) * 8);
    asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(tile + blk * 128 * 128 +
                                                                  from * 128 + o * 16),
                 "r"(0)
                 : "memory");
  }
}

// p = 2^(s scale - m) of kN consecutive scores of a row, packed to bf16 pairs; returns their sum.
template <int kN, int kPolyPairs>
__device__ __forceinline__ float exp_pairs(const uint32_t* s, float scale_log2, float m,
                                           uint32_t* w) {
  const uint64_t sc2 = f2_pack(scale_log2, scale_log2), nm2 = f2_pack(-m, -m);
  uint64_t sum2[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
  for (int i = 0; i < kN / 2; ++i) {
    float x0, x1, p0, p1;
    f2_unpack(f2_fma(f2_pack(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), sc2, nm2),
              x0, x1);
    if ((i & 7) < kPolyPairs) {
      exp2_poly_pair(x0, x1, p0, p1);
    } else {
      p0 = fast_exp2(x0);
      p1 = fast_exp2(x1);
    }
    sum2[i & 3] = f2_add(sum2[i & 3], f2_pack(p0, p1));
    w[i] = pack_bf16x2(p0, p1);
  }
  float l0, l1;
  f2_unpack(f2_add(f2_add(sum2[0], sum2[1]), f2_add(sum2[2], sum2[3])), l0, l1);
  return l0 + l1;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    cross_fwd_tc_kernel(const __grid_constant__ CUtensorMap tm_q,
                        const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v, CrossFwdParams p) {
  using Sh = FwdShape<D>;
  constexpr int kStages = Sh::kStages, kTile = Sh::kTile, kBlk = Sh::kBlk;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t q_full[2], q_empty[2];
  __shared__ __align__(8) uint64_t kv_full[kStages], kv_empty[kStages];
  __shared__ __align__(8) uint64_t s_full[2];      // S(j) complete
  __shared__ __align__(8) uint64_t s_free[2];      // S(j) is in registers (P in its own columns)
  __shared__ __align__(8) uint64_t p_half[2][2];   // states 0-63, 64-127 of P(j) are in TMEM
  __shared__ __align__(8) uint64_t pv_done[2];     // PV(j) complete
  __shared__ __align__(8) uint64_t o_free[2];      // the item's O is in registers
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_sh;

  const uint32_t sbase = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t sQ = sbase, sKV = sbase + 2 * kTile;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  volatile int* abort_flag = &abort_sh;

  if (threadIdx.x == 0) {
    abort_sh = 0;
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&q_full[i]), 1);
      mbar_init(smem_u32(&q_empty[i]), 1);
      mbar_init(smem_u32(&s_full[i]), 1);
      mbar_init(smem_u32(&s_free[i]), kBM);
      mbar_init(smem_u32(&p_half[i][0]), kBM);
      mbar_init(smem_u32(&p_half[i][1]), kBM);
      mbar_init(smem_u32(&pv_done[i]), 1);
      mbar_init(smem_u32(&o_free[i]), kBM);
    }
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_u32(&kv_full[s]), 1);
      mbar_init(smem_u32(&kv_empty[s]), 2);       // one arrival per stream
    }
    fence_barrier_init();
  }
  if (warp == kIssuerWarp) {
    tmem_alloc(smem_u32(&tmem_base_sh), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base_sh;
  grid_dep_wait();
  grid_dep_launch();

  const auto wait = [&](uint64_t& bar, uint32_t phase) {
    return mbar_wait_or_abort(smem_u32(&bar), phase & 1, abort_flag, p.dev_status);
  };

  if (warp == kProducerWarp) {
    if (lane == 0) {
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
      uint32_t n_item[2] = {0, 0}, u = 0;          // uses of the Q tiles and of the ring
      bool ok = true;
      for (int it = blockIdx.x; it < p.items && ok; it += gridDim.x) {
        const Item w = item_of(p, it);
        if (w.nt == 0) continue;
        for (int i = 0; i < 2 && ok; ++i) {
          if (w.q0 + i * kBM >= p.n_q) break;
          ok = wait(q_empty[i], n_item[i] + 1);
          if (!ok) break;
          ++n_item[i];
          const uint32_t fb = smem_u32(&q_full[i]);
          mbar_arrive_expect_tx(fb, kTile);
          for (int k = 0; k < Sh::kBlocks; ++k)
            tma_load_4d(sQ + i * kTile + k * kBlk, &tm_q, fb, 64 * k, w.h, w.q0 + i * kBM, w.b);
        }
        for (int j = 0; j < 2 * w.nt && ok; ++j, ++u) {
          const int s = u % kStages;
          ok = wait(kv_empty[s], u / kStages + 1);
          if (!ok) break;
          const uint32_t fb = smem_u32(&kv_full[s]);
          mbar_arrive_expect_tx(fb, kTile);
          for (int k = 0; k < Sh::kBlocks; ++k)
            tma_load_4d(sKV + s * kTile + k * kBlk, j & 1 ? &tm_v : &tm_k, fb, 64 * k, w.h / p.rep,
                        (j >> 1) * kBN, w.b);
        }
      }
    }
  } else if (warp >= kIssuerWarp) {
    const int i = warp - kIssuerWarp;
    if (lane == 0) {
      constexpr uint32_t idesc_qk = idesc_bf16_f32(kBM, kBN, 0, 0);
      constexpr uint32_t idesc_pv = idesc_bf16_f32(kBM, D, 0, 1);
      const uint64_t qd = smem_desc(sQ + i * kTile, 16, 1024, kSwizzle128B);
      const uint64_t kd0 = smem_desc(sKV, 16, 1024, kSwizzle128B);
      const uint64_t vd0 = smem_desc(sKV, kBlk, 1024, kSwizzle128B);
      const uint32_t ts = tmem + Sh::s_col(i), tp = tmem + Sh::p_col(i), to = tmem + Sh::o_col(i);
      uint32_t n_item = 0, t = 0, u0 = 0;   // items and tiles of this stream, uses of the ring
      bool ok = true;
      const auto issue_qk = [&](uint32_t u) {
        const uint64_t kd = kd0 + ((u % kStages) * kTile >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * kBlk >> 4) + 2 * (kk & 3);
          mma_ss(ts, qd + off, kd + off, idesc_qk, kk ? 1u : 0u);
        }
        mma_commit(smem_u32(&kv_empty[u % kStages]));
        mma_commit(smem_u32(&s_full[i]));
      };
      for (int it = blockIdx.x; it < p.items && ok; it += gridDim.x) {
        const Item w = item_of(p, it);
        if (w.nt == 0) continue;
        if (w.q0 + i * kBM >= p.n_q) {     // no rows for this stream: release what it would read
          for (int j = 0; j < 2 * w.nt && ok; ++j, ++u0) {
            ok = wait(kv_full[u0 % kStages], u0 / kStages);
            if (ok) mbar_arrive(smem_u32(&kv_empty[u0 % kStages]));
          }
          continue;
        }
        ok = wait(q_full[i], n_item);
        for (int j = 0; j < w.nt && ok; ++j) {
          const uint32_t uk = u0 + 2 * j, uv = uk + 1;
          if (Sh::kAliasP || j == 0) {
            // the S buffer: PV of the last tile has read P out of it, or (P in its own columns)
            // the softmax has loaded that tile's S
            ok = wait(kv_full[uk % kStages], uk / kStages) &&
                 (t == 0 || wait(Sh::kAliasP ? pv_done[i] : s_free[i], t - 1));
            if (!ok) break;
            tc_fence_after();
            issue_qk(uk);
            if (j == w.nt - 1) mma_commit(smem_u32(&q_empty[i]));
          }
          if (!Sh::kAliasP && j + 1 < w.nt) {      // QK(j+1) runs under the softmax of j
            const uint32_t un = uk + 2;
            ok = wait(kv_full[un % kStages], un / kStages) && wait(s_free[i], t);
            if (!ok) break;
            tc_fence_after();
            issue_qk(un);
            if (j + 1 == w.nt - 1) mma_commit(smem_u32(&q_empty[i]));
          }
          ok = wait(kv_full[uv % kStages], uv / kStages) &&
               (j > 0 || n_item == 0 || wait(o_free[i], n_item - 1));
          const uint64_t vd = vd0 + ((uv % kStages) * kTile >> 4);
          for (int half = 0; half < 2 && ok; ++half) {
            ok = wait(p_half[i][half], t);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int k4 = 0; k4 < 4; ++k4) {
              const int kk = 4 * half + k4;
              mma_ts(to, tp + 8 * kk, vd + 128 * kk, idesc_pv, (j | kk) != 0 ? 1u : 0u);
            }
          }
          if (!ok) break;
          mma_commit(smem_u32(&kv_empty[uv % kStages]));
          mma_commit(smem_u32(&pv_done[i]));
          ++t;
        }
        u0 += 2 * w.nt;
        ++n_item;
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
    uint32_t t = 0, u0 = 0;
    bool ok = true;
    for (int it = blockIdx.x; it < p.items && ok; it += gridDim.x) {
      const Item w = item_of(p, it);
      const int n = w.q0 + i * kBM + row;
      const int64_t sr = (static_cast<int64_t>(w.b) * p.H + w.h) * p.n_q + n;
      bf16* orow = p.out + ((static_cast<int64_t>(w.b) * p.n_q + n) * p.H + w.h) * D;
      if (w.nt == 0) {
        if (n < p.n_q) {
          for (int c = 0; c < D / 8; ++c)
            reinterpret_cast<uint4*>(orow)[c] = make_uint4(0u, 0u, 0u, 0u);
          if (p.lse != nullptr) p.lse[sr] = -INFINITY;
        }
        continue;
      }
      if (w.q0 + i * kBM >= p.n_q) {
        u0 += 2 * w.nt;
        continue;
      }
      float m = 0.f, l = 0.f;
      for (int j = 0; j < w.nt; ++j, ++t) {
        ok = wait_all(s_full[i], t);
        if (!ok) break;
        tc_fence_after();
        uint32_t s[kBN];
        tmem_ld128_wait(ts, s);
        const int valid = w.len - j * kBN;
        if (valid < kBN) {
#pragma unroll
          for (int c = 0; c < kBN; ++c)
            if (c >= valid) s[c] = 0xff800000u;        // -infinity
        }
        float mx;
        {
          float m8[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            float a = fmax3(__uint_as_float(s[k]), __uint_as_float(s[k + 8]),
                            __uint_as_float(s[k + 16]));
#pragma unroll
            for (int c = 24; c < kBN - 8; c += 16)
              a = fmax3(a, __uint_as_float(s[c + k]), __uint_as_float(s[c + 8 + k]));
            m8[k] = fmaxf(a, __uint_as_float(s[kBN - 8 + k]));
          }
          mx = fmax3(fmax3(m8[0], m8[1], m8[2]), fmax3(m8[3], m8[4], m8[5]),
                     fmaxf(m8[6], m8[7])) * p.scale_log2;
        }
        if constexpr (!Sh::kAliasP) {
          tc_fence_before();
          mbar_arrive(smem_u32(&s_free[i]));
        }
        float alpha = 1.f;
        bool rescale = false;
        if (j == 0) {
          m = mx;
        } else if (__any_sync(0xffffffffu, mx > m + 8.f)) {
          const float m_new = fmaxf(m, mx);
          alpha = fast_exp2(m - m_new);
          l *= alpha;
          m = m_new;
          rescale = true;
        }
        // with P in S's columns, S(j) came after PV(j-1); otherwise wait for that product before
        // P's buffer or O is written
        if (!Sh::kAliasP && t > 0) {
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
          zero_rows<Sh::kBlocks>(sKV + (uv % kStages) * kTile, valid, row, kBM);
          fence_proxy_async_smem();
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t pw[32];
          l += valid >= kBN ? exp_pairs<64, Sh::kPolyPairs>(s + 64 * half, p.scale_log2, m, pw)
                            : exp_pairs<64, 0>(s + 64 * half, p.scale_log2, m, pw);
#pragma unroll
          for (int c = 0; c < 32; c += 16) {
            uint32_t w16[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) w16[k] = pw[c + k];
            tmem_st16(tp + 32 * half + c, w16);
          }
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(smem_u32(&p_half[i][half]));
        }
      }
      if (!ok) break;
      u0 += 2 * w.nt;
      ok = wait_all(pv_done[i], t - 1);
      if (!ok) break;
      tc_fence_after();
      const float inv_l = 1.f / l;
      if (p.lse != nullptr && n < p.n_q) p.lse[sr] = (m + log2f(l)) * kLn2;
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        uint32_t r[32];
        tmem_ld32_wait(to + c, r);
        uint32_t v[16];
#pragma unroll
        for (int k = 0; k < 16; ++k)
          v[k] = pack_bf16x2(__uint_as_float(r[2 * k]) * inv_l, __uint_as_float(r[2 * k + 1]) * inv_l);
        if (n < p.n_q) {
          uint4* d4 = reinterpret_cast<uint4*>(orow + c);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            d4[k] = make_uint4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
        }
      }
      tc_fence_before();
      mbar_arrive(smem_u32(&o_free[i]));
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kIssuerWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Tensor map of [B, n, heads, d] rows with 64-column, `rows`-row boxes, 128-byte swizzle.
mla_status cross_tmap(CUtensorMap* m, const void* base, int B, int n, int heads, int d, int64_t row,
                      uint32_t rows) {
  const uint64_t dims[4] = {static_cast<uint64_t>(d), static_cast<uint64_t>(heads),
                            static_cast<uint64_t>(n), static_cast<uint64_t>(B)};
  const uint64_t strides[3] = {d * 2ull, static_cast<uint64_t>(row) * 2,
                               static_cast<uint64_t>(n) * static_cast<uint64_t>(row) * 2};
  const uint32_t box[4] = {64, 1, rows, 1};
  return make_tmap_bf16(m, base, 4, dims, strides, box, 128);
}

template <int D>
mla_status fwd_impl(const CrossDims& d, const CrossArgs& a, cudaStream_t s) {
  using Sh = FwdShape<D>;
  CUtensorMap tq, tk, tv;
  mla_status st;
  if ((st = cross_tmap(&tq, a.q, d.B, d.n_q, d.H, D, d.q_row, kBM)) != MLA_OK) return st;
  if ((st = cross_tmap(&tk, a.k, d.B, d.n_kv, d.Hkv, D, d.k_row, kBN)) != MLA_OK) return st;
  if ((st = cross_tmap(&tv, a.v, d.B, d.n_kv, d.Hkv, D, d.v_row, kBN)) != MLA_OK) return st;
  CrossFwdParams p;
  p.n_q = d.n_q; p.H = d.H; p.rep = d.H / d.Hkv; p.n_kv = d.n_kv;
  p.pairs = ceil_div(d.n_q, 2 * kBM);
  p.items = p.pairs * d.H * d.B;      // fewer than 2^31: every item has at least one query row
  p.scale_log2 = d.scale * kLog2e;
  p.kv_len = a.kv_len; p.out = static_cast<bf16*>(a.out); p.lse = a.lse;
  p.dev_status = a.dev_status;
  MLA_CUDA_TRY(cudaFuncSetAttribute(cross_fwd_tc_kernel<D>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::kSmem));
  MLA_CUDA_TRY(launch_pdl(cross_fwd_tc_kernel<D>, dim3(std::min(p.items, 148)), dim3(kThreads),
                          Sh::kSmem, s, tq, tk, tv, p));
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
