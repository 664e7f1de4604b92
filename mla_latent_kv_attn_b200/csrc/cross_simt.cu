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
// One warp owns one row (a query row, or a key row in the key kernel) and takes 32 rows of the other
// side at a time, in two ways: for the dot products a lane takes one of the 32 rows whole (its own
// row comes from shared memory), for the weighted sums the lanes share each row's elements (lane l
// has l, l + 32, ...) and the weights come by shuffles.  A step of 32 rows then waits for memory
// twice; with the elements over the lanes in both, a butterfly sum per row and four rows in flight
// bounded these kernels (16 queries against 24 states in fp32: 14.3 us a call, now bound by the
// launch).  All sums are fp32 and run in a fixed order.  Every warp reads the other side's rows itself,
// which costs at a layer's size: 4680 queries, 512 states, 12 heads of 128 in fp32 4.2 ms forward and 18.1
// ms backward (29 GB of keys and values through L2 a forward, whose multiply-adds are 0.2 ms at the CUDA
// cores' peak); 96 in bf16 2.1 and 8.9 ms, 256 in bf16 6.3 and 26 ms.
#include <cfloat>

#include "cross.h"

namespace mla {

namespace {

constexpr int kWarps = 4;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// The warp's own row, as floats, into its shared memory.
template <typename T>
__device__ __forceinline__ void stage_row(const T* row, int d, int lane, float* to) {
  for (int e = lane; e < d; e += 32) to[e] = Elem<T>::to_f(row[e]);
}

// row . mine; kVec: rows start on 16 bytes and hold whole 16-byte pieces.
template <typename T, bool kVec>
__device__ __forceinline__ float dot_row(const T* __restrict__ row, const float* mine, int d) {
  float s = 0.f;
  if constexpr (kVec) {
    constexpr int kPiece = 16 / sizeof(T);
#pragma unroll 4
    for (int e = 0; e < d; e += kPiece) {
      const uint4 raw = *reinterpret_cast<const uint4*>(row + e);
      const T* t = reinterpret_cast<const T*>(&raw);
#pragma unroll
      for (int k = 0; k < kPiece; ++k) s = fmaf(Elem<T>::to_f(t[k]), mine[e + k], s);
    }
  } else {
#pragma unroll 4
    for (int e = 0; e < d; ++e) s = fmaf(Elem<T>::to_f(row[e]), mine[e], s);
  }
  return s;
}

// acc += sum over r < n of weight_r row_r, row r at rows + r * stride, weight_r that of lane r.
template <typename T, int kPer>
__device__ __forceinline__ void add_rows(const T* __restrict__ rows, int64_t stride, int n,
                                         float weight, int d, int lane, float (&acc)[kPer]) {
#pragma unroll 8
  for (int r = 0; r < n; ++r) {
    const float w = __shfl_sync(0xffffffffu, weight, r);
    const T* row = rows + r * stride;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = lane + 32 * i;
      if (e < d) acc[i] = fmaf(w, Elem<T>::to_f(row[e]), acc[i]);
    }
  }
}

template <typename T, int kPer>
__device__ __forceinline__ void store_row(T* p, int d, int lane, const float (&x)[kPer], float f) {
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = lane + 32 * i;
    if (e < d) p[e] = Elem<T>::from_f(x[i] * f);
  }
}

// kPer: elements per lane, d <= 32 kPer.
template <typename T, int kPer, bool kVec>
__global__ void __launch_bounds__(32 * kWarps)
    cross_fwd_simt_kernel(CrossDims d, CrossArgs a, float scale_log2) {
  __shared__ float mine_sh[kWarps][32 * kPer];
  const int lane = threadIdx.x % 32;
  float* mine = mine_sh[threadIdx.x / 32];
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + threadIdx.x / 32;   // (b, i, h)
  if (row >= static_cast<int64_t>(d.B) * d.n_q * d.H) return;
  const int h = static_cast<int>(row % d.H);
  const int64_t bi = row / d.H;
  const int b = static_cast<int>(bi / d.n_q), i = static_cast<int>(bi % d.n_q);
  const int kh = h / (d.H / d.Hkv);
  const int len = cross_len(a.kv_len, b, d.n_kv);
  stage_row(static_cast<const T*>(a.q) + bi * d.q_row + static_cast<int64_t>(h) * d.d, d.d, lane, mine);
  __syncwarp();
  const T* k0 = static_cast<const T*>(a.k) + static_cast<int64_t>(b) * d.n_kv * d.k_row +
                static_cast<int64_t>(kh) * d.d;
  const T* v0 = static_cast<const T*>(a.v) + static_cast<int64_t>(b) * d.n_kv * d.v_row +
                static_cast<int64_t>(kh) * d.d;
  float o[kPer] = {};
  float m = -FLT_MAX, l = 0.f;          // (finite: scores of -infinity weigh nothing)
  for (int j0 = 0; j0 < len; j0 += 32) {
    const int n = min(32, len - j0);
    const float x = lane < n ? dot_row<T, kVec>(k0 + (j0 + lane) * d.k_row, mine, d.d) * scale_log2
                             : -INFINITY;
    const float mn = fmaxf(m, warp_max(x));
    const float alpha = exp2f(m - mn), p = exp2f(x - mn);
    m = mn;
    l = l * alpha + warp_sum(p);
#pragma unroll
    for (int e = 0; e < kPer; ++e) o[e] *= alpha;
    add_rows(v0 + j0 * d.v_row, d.v_row, n, p, d.d, lane, o);
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
  float s = 0.f;
  for (int e = lane; e < d; e += 32)
    s = fmaf(Elem<T>::to_f(out[row * d + e]), Elem<T>::to_f(g[row * d + e]), s);
  s = warp_sum(s);
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

template <typename T, int kPer, bool kVec>
__global__ void __launch_bounds__(32 * kWarps)
    cross_dq_simt_kernel(CrossDims d, CrossBwdArgs a, const float* delta) {
  __shared__ float mine_sh[kWarps][2][32 * kPer];
  const int lane = threadIdx.x % 32;
  float* q = mine_sh[threadIdx.x / 32][0];
  float* g = mine_sh[threadIdx.x / 32][1];
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + threadIdx.x / 32;
  if (row >= static_cast<int64_t>(d.B) * d.n_q * d.H) return;
  const int h = static_cast<int>(row % d.H);
  const int64_t bi = row / d.H;
  const int b = static_cast<int>(bi / d.n_q), i = static_cast<int>(bi % d.n_q);
  const int kh = h / (d.H / d.Hkv);
  const int len = cross_len(a.kv_len, b, d.n_kv);
  const int64_t sr = (static_cast<int64_t>(b) * d.H + h) * d.n_q + i;
  stage_row(static_cast<const T*>(a.q) + bi * d.q_row + static_cast<int64_t>(h) * d.d, d.d, lane, q);
  stage_row(static_cast<const T*>(a.d_out) + row * d.d, d.d, lane, g);
  __syncwarp();
  const T* k0 = static_cast<const T*>(a.k) + static_cast<int64_t>(b) * d.n_kv * d.k_row +
                static_cast<int64_t>(kh) * d.d;
  const T* v0 = static_cast<const T*>(a.v) + static_cast<int64_t>(b) * d.n_kv * d.v_row +
                static_cast<int64_t>(kh) * d.d;
  const float lse = a.lse[sr], dl = delta[sr];
  float dq[kPer] = {};
  for (int j0 = 0; j0 < len; j0 += 32) {
    const int n = min(32, len - j0);
    float ds = 0.f;
    if (lane < n) {
      const float x = dot_row<T, kVec>(k0 + (j0 + lane) * d.k_row, q, d.d);
      const float dp = dot_row<T, kVec>(v0 + (j0 + lane) * d.v_row, g, d.d);
      ds = d_score(exp2f((x * d.scale - lse) * kLog2e), dp, dl, d.scale, len);
    }
    add_rows(k0 + j0 * d.k_row, d.k_row, n, ds, d.d, lane, dq);
  }
  store_row(static_cast<T*>(a.d_q) + row * d.d, d.d, lane, dq, 1.f);
}

template <typename T, int kPer, bool kVec>
__global__ void __launch_bounds__(32 * kWarps)
    cross_dkv_simt_kernel(CrossDims d, CrossBwdArgs a, const float* delta) {
  __shared__ float mine_sh[kWarps][2][32 * kPer];
  const int lane = threadIdx.x % 32;
  float* k = mine_sh[threadIdx.x / 32][0];
  float* v = mine_sh[threadIdx.x / 32][1];
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + threadIdx.x / 32;   // (b, j, kh)
  if (row >= static_cast<int64_t>(d.B) * d.n_kv * d.Hkv) return;
  const int kh = static_cast<int>(row % d.Hkv);
  const int64_t bj = row / d.Hkv;
  const int b = static_cast<int>(bj / d.n_kv), j = static_cast<int>(bj % d.n_kv);
  const int len = cross_len(a.kv_len, b, d.n_kv);
  float dk[kPer] = {}, dv[kPer] = {};
  if (j < len) {
    stage_row(static_cast<const T*>(a.k) + bj * d.k_row + static_cast<int64_t>(kh) * d.d, d.d, lane, k);
    stage_row(static_cast<const T*>(a.v) + bj * d.v_row + static_cast<int64_t>(kh) * d.d, d.d, lane, v);
    __syncwarp();
    const int rep = d.H / d.Hkv;
    const int64_t g_row = static_cast<int64_t>(d.H) * d.d;
    for (int h = kh * rep; h < (kh + 1) * rep; ++h) {
      const T* q0 = static_cast<const T*>(a.q) + static_cast<int64_t>(b) * d.n_q * d.q_row +
                    static_cast<int64_t>(h) * d.d;
      const T* g0 = static_cast<const T*>(a.d_out) +
                    (static_cast<int64_t>(b) * d.n_q * d.H + h) * d.d;
      const int64_t sr = (static_cast<int64_t>(b) * d.H + h) * d.n_q;
      for (int i0 = 0; i0 < d.n_q; i0 += 32) {
        const int n = min(32, d.n_q - i0);
        float p = 0.f, ds = 0.f;
        if (lane < n) {
          const int64_t i = i0 + lane;
          const float x = dot_row<T, kVec>(q0 + i * d.q_row, k, d.d);
          const float dp = dot_row<T, kVec>(g0 + i * g_row, v, d.d);
          p = exp2f((x * d.scale - a.lse[sr + i]) * kLog2e);
          ds = d_score(p, dp, delta[sr + i], d.scale, len);
        }
        add_rows(q0 + i0 * d.q_row, d.q_row, n, ds, d.d, lane, dk);
        add_rows(g0 + i0 * g_row, g_row, n, p, d.d, lane, dv);
      }
    }
  }
  store_row(static_cast<T*>(a.d_k) + row * d.d, d.d, lane, dk, 1.f);
  store_row(static_cast<T*>(a.d_v) + row * d.d, d.d, lane, dv, 1.f);
}

// Blocks for `rows` warps; fewer than 2^31 rows (each row has at least one element, and every
// array holds fewer than 2^31).
unsigned blocks_for(int64_t rows) { return static_cast<unsigned>((rows + kWarps - 1) / kWarps); }

template <typename T, int kPer, bool kVec>
mla_status fwd(const CrossDims& d, const CrossArgs& a, cudaStream_t s) {
  cross_fwd_simt_kernel<T, kPer, kVec>
      <<<blocks_for(static_cast<int64_t>(d.B) * d.n_q * d.H), 32 * kWarps, 0, s>>>(
          d, a, d.scale * kLog2e);
  MLA_LAUNCH_CHECK("cross_fwd_simt");
  return MLA_OK;
}

template <typename T, int kPer, bool kVec>
mla_status bwd(const CrossDims& d, const CrossBwdArgs& a, float* delta, cudaStream_t s) {
  const unsigned qb = blocks_for(static_cast<int64_t>(d.B) * d.n_q * d.H);
  cross_delta_kernel<T><<<qb, 32 * kWarps, 0, s>>>(static_cast<const T*>(a.out),
                                                   static_cast<const T*>(a.d_out), delta, d.B, d.n_q,
                                                   d.H, d.d);
  MLA_LAUNCH_CHECK("cross_delta");
  cross_dq_simt_kernel<T, kPer, kVec><<<qb, 32 * kWarps, 0, s>>>(d, a, delta);
  MLA_LAUNCH_CHECK("cross_dq_simt");
  cross_dkv_simt_kernel<T, kPer, kVec>
      <<<blocks_for(static_cast<int64_t>(d.B) * d.n_kv * d.Hkv), 32 * kWarps, 0, s>>>(d, a, delta);
  MLA_LAUNCH_CHECK("cross_dkv_simt");
  return MLA_OK;
}

// Rows hold whole 16-byte pieces when d elements do: the arrays start on 16 bytes, dense strides are
// then multiples of 16 bytes and given ones are checked to be.
template <typename F>
mla_status by_shape(const CrossDims& d, const F& f) {
  const bool vec = d.d * dtype_size(d.dtype) % 16 == 0;
#define MLA_CROSS_CASE(PER)                                                       \
  if (d.d <= 32 * PER) {                                                          \
    if (d.dtype == MLA_FP32)                                                      \
      return vec ? f.template operator()<float, PER, true>()                      \
                 : f.template operator()<float, PER, false>();                    \
    return vec ? f.template operator()<bf16, PER, true>()                         \
               : f.template operator()<bf16, PER, false>();                       \
  }
  MLA_CROSS_CASE(1) MLA_CROSS_CASE(2) MLA_CROSS_CASE(4) MLA_CROSS_CASE(8)
#undef MLA_CROSS_CASE
  MLA_FAIL(MLA_ERR_UNSUPPORTED, "d_head (%d) above %d", d.d, kCrossMaxD);
}

struct Fwd {
  const CrossDims& d;
  const CrossArgs& a;
  cudaStream_t s;
  template <typename T, int kPer, bool kVec>
  mla_status operator()() const { return fwd<T, kPer, kVec>(d, a, s); }
};

struct Bwd {
  const CrossDims& d;
  const CrossBwdArgs& a;
  float* delta;
  cudaStream_t s;
  template <typename T, int kPer, bool kVec>
  mla_status operator()() const { return bwd<T, kPer, kVec>(d, a, delta, s); }
};

}  // namespace

mla_status cross_fwd_simt(const CrossDims& d, const CrossArgs& a, cudaStream_t s) {
  return by_shape(d, Fwd{d, a, s});
}

mla_status cross_bwd_simt(const CrossDims& d, const CrossBwdArgs& a, float* delta, cudaStream_t s) {
  return by_shape(d, Bwd{d, a, delta, s});
}

}  // namespace mla
