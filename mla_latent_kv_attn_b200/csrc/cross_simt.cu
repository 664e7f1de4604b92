// cross_simt.cu - cross attention to an encoder's states on CUDA cores: every dtype and any head
// width up to 256.  It serves fp32, the head widths the tensor-core kernels do not cover, and
// cross-checks of those kernels.
//
//   x_ij = scale q_i . k_j over the sample's valid states j < len, p = softmax_j(x),
//   o_i = sum_j p_ij v_j, lse_i = log sum_j exp(x_ij);  len = 0 gives o = 0 and lse = -inf
//   dP_ij = g_i . v_j, dS_ij = scale p_ij (dP_ij - delta_i), delta_i = g_i . o_i,
//   dq_i = sum_j dS_ij k_j, dk_j = sum_i dS_ij q_i, dv_j = sum_i p_ij g_i
// with the key and value gradients summed over the query heads that share the key head.
//
// One warp owns one row (a query row, or a key row in the key kernel), its values spread over the
// lanes (lane l holds elements l, l + 32, ...).  Every dot product is a lane-wise sum and a
// butterfly reduction, which bounds these kernels; four rows of the other side are in flight at a
// time so that the reductions overlap.  All sums are fp32 and run in a fixed order.
#include "cross.h"

namespace mla {

namespace {

constexpr int kPer = kCrossMaxD / 32;   // elements per lane
constexpr int kRows = 4;                // rows of the other side in flight
constexpr int kWarps = 4;
constexpr float kLog2e = 1.4426950408889634f;

template <typename T>
__device__ __forceinline__ void load_row(const T* p, int d, int lane, float (&x)[kPer]) {
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = lane + 32 * i;
    x[i] = e < d ? Elem<T>::to_f(p[e]) : 0.f;
  }
}

template <typename T>
__device__ __forceinline__ void store_row(T* p, int d, int lane, const float (&x)[kPer], float f) {
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = lane + 32 * i;
    if (e < d) p[e] = Elem<T>::from_f(x[i] * f);
  }
}

__device__ __forceinline__ float dot(const float (&a)[kPer], const float (&b)[kPer]) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) s = fmaf(a[i], b[i], s);
  return s;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <typename T>
__global__ void __launch_bounds__(32 * kWarps)
    cross_fwd_simt_kernel(CrossDims d, CrossArgs a, float scale_log2) {
  const int lane = threadIdx.x % 32;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + threadIdx.x / 32;   // (b, i, h)
  if (row >= static_cast<int64_t>(d.B) * d.n_q * d.H) return;
  const int h = static_cast<int>(row % d.H);
  const int64_t bi = row / d.H;
  const int b = static_cast<int>(bi / d.n_q), i = static_cast<int>(bi % d.n_q);
  const int kh = h / (d.H / d.Hkv);
  const int len = cross_len(a.kv_len, b, d.n_kv);
  float q[kPer], o[kPer] = {};
  load_row(static_cast<const T*>(a.q) + bi * d.q_row + static_cast<int64_t>(h) * d.d, d.d, lane, q);
  const T* k0 = static_cast<const T*>(a.k) + static_cast<int64_t>(b) * d.n_kv * d.k_row +
                static_cast<int64_t>(kh) * d.d;
  const T* v0 = static_cast<const T*>(a.v) + static_cast<int64_t>(b) * d.n_kv * d.v_row +
                static_cast<int64_t>(kh) * d.d;
  float m = -INFINITY, l = 0.f;
  for (int j0 = 0; j0 < len; j0 += kRows) {
    float x[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      float k[kPer];
      const int j = min(j0 + r, len - 1);
      load_row(k0 + j * d.k_row, d.d, lane, k);
      x[r] = dot(q, k);
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) x[r] = j0 + r < len ? warp_sum(x[r]) * scale_log2 : -INFINITY;
    // at least one of the scores is finite, so the new maximum is
    const float mn = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), m);
    const float alpha = exp2f(m - mn);
    m = mn;
    l *= alpha;
#pragma unroll
    for (int e = 0; e < kPer; ++e) o[e] *= alpha;
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      if (j0 + r >= len) break;
      const float p = exp2f(x[r] - m);
      l += p;
      float v[kPer];
      load_row(v0 + (j0 + r) * d.v_row, d.d, lane, v);
#pragma unroll
      for (int e = 0; e < kPer; ++e) o[e] = fmaf(p, v[e], o[e]);
    }
  }
  store_row(static_cast<T*>(a.out) + row * d.d, d.d, lane, o, len > 0 ? 1.f / l : 0.f);
  if (a.lse != nullptr && lane == 0)
    a.lse[(static_cast<int64_t>(b) * d.H + h) * d.n_q + i] =
        len > 0 ? (m + log2f(l)) * 0.69314718055994530942f : -INFINITY;
}

// One warp per (b, i, h): rows are dense, so the warp reads d consecutive elements of each.
template <typename T>
__global__ void __launch_bounds__(32 * kWarps)
    cross_delta_kernel(const T* __restrict__ out, const T* __restrict__ g, float* __restrict__ delta,
                       int B, int n_q, int H, int d) {
  const int lane = threadIdx.x % 32;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + threadIdx.x / 32;
  if (row >= static_cast<int64_t>(B) * n_q * H) return;
  float x[kPer], y[kPer];
  load_row(out + row * d, d, lane, x);
  load_row(g + row * d, d, lane, y);
  const float s = warp_sum(dot(x, y));
  const int h = static_cast<int>(row % H);
  const int64_t bi = row / H;
  if (lane == 0)
    delta[((bi / n_q) * H + h) * n_q + bi % n_q] = s;
}

// A sample with a single valid state has p = 1 whatever its score: the gradients of its query
// and key are exactly zero, which dP - delta, computed from two roundings of one number, is not.
__device__ __forceinline__ float d_score(float p, float dp, float delta, float scale, int len) {
  return len == 1 ? 0.f : p * (dp - delta) * scale;
}

template <typename T>
__global__ void __launch_bounds__(32 * kWarps)
    cross_dq_simt_kernel(CrossDims d, CrossBwdArgs a, const float* delta) {
  const int lane = threadIdx.x % 32;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + threadIdx.x / 32;
  if (row >= static_cast<int64_t>(d.B) * d.n_q * d.H) return;
  const int h = static_cast<int>(row % d.H);
  const int64_t bi = row / d.H;
  const int b = static_cast<int>(bi / d.n_q), i = static_cast<int>(bi % d.n_q);
  const int kh = h / (d.H / d.Hkv);
  const int len = cross_len(a.kv_len, b, d.n_kv);
  const int64_t sr = (static_cast<int64_t>(b) * d.H + h) * d.n_q + i;
  float q[kPer], g[kPer], dq[kPer] = {};
  load_row(static_cast<const T*>(a.q) + bi * d.q_row + static_cast<int64_t>(h) * d.d, d.d, lane, q);
  load_row(static_cast<const T*>(a.d_out) + row * d.d, d.d, lane, g);
  const T* k0 = static_cast<const T*>(a.k) + static_cast<int64_t>(b) * d.n_kv * d.k_row +
                static_cast<int64_t>(kh) * d.d;
  const T* v0 = static_cast<const T*>(a.v) + static_cast<int64_t>(b) * d.n_kv * d.v_row +
                static_cast<int64_t>(kh) * d.d;
  const float lse = a.lse[sr], dl = delta[sr];
  for (int j0 = 0; j0 < len; j0 += kRows) {
    float x[kRows], dp[kRows], k[kRows][kPer];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      float v[kPer];
      const int j = min(j0 + r, len - 1);
      load_row(k0 + j * d.k_row, d.d, lane, k[r]);
      load_row(v0 + j * d.v_row, d.d, lane, v);
      x[r] = dot(q, k[r]);
      dp[r] = dot(g, v);
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      x[r] = warp_sum(x[r]);
      dp[r] = warp_sum(dp[r]);
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      if (j0 + r >= len) break;
      const float p = exp2f((x[r] * d.scale - lse) * kLog2e);
      const float ds = d_score(p, dp[r], dl, d.scale, len);
#pragma unroll
      for (int e = 0; e < kPer; ++e) dq[e] = fmaf(ds, k[r][e], dq[e]);
    }
  }
  store_row(static_cast<T*>(a.d_q) + row * d.d, d.d, lane, dq, 1.f);
}

template <typename T>
__global__ void __launch_bounds__(32 * kWarps)
    cross_dkv_simt_kernel(CrossDims d, CrossBwdArgs a, const float* delta) {
  const int lane = threadIdx.x % 32;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + threadIdx.x / 32;   // (b, j, kh)
  if (row >= static_cast<int64_t>(d.B) * d.n_kv * d.Hkv) return;
  const int kh = static_cast<int>(row % d.Hkv);
  const int64_t bj = row / d.Hkv;
  const int b = static_cast<int>(bj / d.n_kv), j = static_cast<int>(bj % d.n_kv);
  const int len = cross_len(a.kv_len, b, d.n_kv);
  float dk[kPer] = {}, dv[kPer] = {};
  if (j < len) {
    float k[kPer], v[kPer];
    load_row(static_cast<const T*>(a.k) + bj * d.k_row + static_cast<int64_t>(kh) * d.d, d.d, lane, k);
    load_row(static_cast<const T*>(a.v) + bj * d.v_row + static_cast<int64_t>(kh) * d.d, d.d, lane, v);
    const int rep = d.H / d.Hkv;
    for (int h = kh * rep; h < (kh + 1) * rep; ++h) {
      const T* q0 = static_cast<const T*>(a.q) + static_cast<int64_t>(b) * d.n_q * d.q_row +
                    static_cast<int64_t>(h) * d.d;
      const T* g0 = static_cast<const T*>(a.d_out) +
                    (static_cast<int64_t>(b) * d.n_q * d.H + h) * d.d;
      const int64_t sr = (static_cast<int64_t>(b) * d.H + h) * d.n_q;
      for (int i0 = 0; i0 < d.n_q; i0 += kRows) {
        float x[kRows], dp[kRows], q[kRows][kPer], g[kRows][kPer];
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          const int i = min(i0 + r, d.n_q - 1);
          load_row(q0 + i * d.q_row, d.d, lane, q[r]);
          load_row(g0 + static_cast<int64_t>(i) * d.H * d.d, d.d, lane, g[r]);
          x[r] = dot(q[r], k);
          dp[r] = dot(g[r], v);
        }
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          x[r] = warp_sum(x[r]);
          dp[r] = warp_sum(dp[r]);
        }
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          const int i = i0 + r;
          if (i >= d.n_q) break;
          const float p = exp2f((x[r] * d.scale - a.lse[sr + i]) * kLog2e);
          const float ds = d_score(p, dp[r], delta[sr + i], d.scale, len);
#pragma unroll
          for (int e = 0; e < kPer; ++e) {
            dk[e] = fmaf(ds, q[r][e], dk[e]);
            dv[e] = fmaf(p, g[r][e], dv[e]);
          }
        }
      }
    }
  }
  store_row(static_cast<T*>(a.d_k) + row * d.d, d.d, lane, dk, 1.f);
  store_row(static_cast<T*>(a.d_v) + row * d.d, d.d, lane, dv, 1.f);
}

// Blocks for `rows` warps; fewer than 2^31 rows (each row has at least one element, and every
// array holds fewer than 2^31).
unsigned blocks_for(int64_t rows) { return static_cast<unsigned>((rows + kWarps - 1) / kWarps); }

}  // namespace

mla_status cross_fwd_simt(const CrossDims& d, const CrossArgs& a, cudaStream_t s) {
  const unsigned blocks = blocks_for(static_cast<int64_t>(d.B) * d.n_q * d.H);
  if (d.dtype == MLA_FP32)
    cross_fwd_simt_kernel<float><<<blocks, 32 * kWarps, 0, s>>>(d, a, d.scale * kLog2e);
  else
    cross_fwd_simt_kernel<bf16><<<blocks, 32 * kWarps, 0, s>>>(d, a, d.scale * kLog2e);
  MLA_LAUNCH_CHECK("cross_fwd_simt");
  return MLA_OK;
}

mla_status cross_delta(const CrossDims& d, const void* out, const void* d_out, float* delta,
                       cudaStream_t s) {
  const unsigned blocks = blocks_for(static_cast<int64_t>(d.B) * d.n_q * d.H);
  if (d.dtype == MLA_FP32)
    cross_delta_kernel<float><<<blocks, 32 * kWarps, 0, s>>>(
        static_cast<const float*>(out), static_cast<const float*>(d_out), delta, d.B, d.n_q, d.H, d.d);
  else
    cross_delta_kernel<bf16><<<blocks, 32 * kWarps, 0, s>>>(
        static_cast<const bf16*>(out), static_cast<const bf16*>(d_out), delta, d.B, d.n_q, d.H, d.d);
  MLA_LAUNCH_CHECK("cross_delta");
  return MLA_OK;
}

mla_status cross_bwd_simt(const CrossDims& d, const CrossBwdArgs& a, float* delta, cudaStream_t s) {
  mla_status st = cross_delta(d, a.out, a.d_out, delta, s);
  if (st != MLA_OK) return st;
  const unsigned qb = blocks_for(static_cast<int64_t>(d.B) * d.n_q * d.H);
  const unsigned kb = blocks_for(static_cast<int64_t>(d.B) * d.n_kv * d.Hkv);
  if (d.dtype == MLA_FP32) {
    cross_dq_simt_kernel<float><<<qb, 32 * kWarps, 0, s>>>(d, a, delta);
    MLA_LAUNCH_CHECK("cross_dq_simt");
    cross_dkv_simt_kernel<float><<<kb, 32 * kWarps, 0, s>>>(d, a, delta);
  } else {
    cross_dq_simt_kernel<bf16><<<qb, 32 * kWarps, 0, s>>>(d, a, delta);
    MLA_LAUNCH_CHECK("cross_dq_simt");
    cross_dkv_simt_kernel<bf16><<<kb, 32 * kWarps, 0, s>>>(d, a, delta);
  }
  MLA_LAUNCH_CHECK("cross_dkv_simt");
  return MLA_OK;
}

}  // namespace mla
