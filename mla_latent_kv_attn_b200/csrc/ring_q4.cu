// ring_q4.cu - the latent ring held in 4 bits: append (quantise), read back, and the pass that
// decodes an attention call's ring keys.
//
// Format.  The D latents of a token fall into groups of 16 (d_c and d_rope are multiples of 16, so
// no group mixes content and positional values).  A group has one scale byte with 5 exponent and
// 3 mantissa bits, s = 2^(E - 20) (1 + M / 8), and 16 codes c in [-7, 7], two to a byte (the even
// column in the low half), each stored as c + 8.  The value is c s: 4.5 bits per value.
//   encode: s = the smallest scale >= max|x| / 7, c = rint(x / s), so that |x - c s| <= s / 2
//   (a group beyond 7 times the largest scale saturates; a NaN is stored as 0).
// Why this scale: c has 3 significant bits and s has 4, so c s has at most 7 and is exact in bf16
// (8 bits) and in fp16 (11 bits; the least value, 2^-20, is a multiple of fp16's least step 2^-24,
// the largest, 26880, is below its limit).  The attention kernels then read the very values the
// ring stands for, and the only loss is that of the codes.  The tensor-core attention reads them as
// fp16, whose three bits more make the query's, the rotated keys' and P's rounding 8 times
// smaller.  Groups of 16 with a scale byte cost the same as groups of 32 with a
// 16-bit scale and follow the values' range twice as closely.
//
// The bits work out without a table: a float's exponent and top three mantissa bits, rounded up,
// minus a bias are the scale byte.  All three passes are bound by memory, or by latency where they
// move a few megabytes: one thread per group, 16- and 8-byte accesses, no shared memory.
#include <cuda_fp16.h>

#include "kernels.h"
#include "ring_q4.h"

namespace mla {

namespace {

constexpr int kThreads = 256;
constexpr int kScaleBias = 107 * 8;     // (fp32 exponent bias 127 - 20) on top of 3 mantissa bits

__device__ __forceinline__ float scale_of(uint32_t byte) {
  return __uint_as_float((byte + kScaleBias) << 20);
}

// Smallest scale byte whose scale is at least r >= 0: the 20 mantissa bits below the third are
// rounded up by a carry into the bits above; clamped to the range of a byte.
__device__ __forceinline__ uint32_t scale_byte(float r) {
  const int b = static_cast<int>((__float_as_uint(r) + 0xFFFFFu) >> 20) - kScaleBias;
  return static_cast<uint32_t>(min(max(b, 0), 255));
}

// 16 values of T to or from 16-byte pieces.
template <typename T>
__device__ __forceinline__ void load16(const T* p, float (&x)[kQ4Group]) {
  constexpr int kPieces = kQ4Group * sizeof(T) / 16;
  uint4 raw[kPieces];
#pragma unroll
  for (int i = 0; i < kPieces; ++i) raw[i] = reinterpret_cast<const uint4*>(p)[i];
  const T* t = reinterpret_cast<const T*>(raw);
#pragma unroll
  for (int i = 0; i < kQ4Group; ++i) x[i] = Elem<T>::to_f(t[i]);
}

// Values to U: T itself, or fp16 with what lies past its range held at its limits (only a chunk
// latent can; the ring itself ends at 26880).
template <typename U>
struct To {
  static __device__ __forceinline__ U from(float v) { return Elem<U>::from_f(v); }
};
template <>
struct To<__half> {
  static __device__ __forceinline__ __half from(float v) {
    if (isfinite(v)) v = fminf(fmaxf(v, -65504.f), 65504.f);
    return __float2half_rn(v);
  }
};

template <typename U>
__device__ __forceinline__ void store16(U* p, const float (&x)[kQ4Group]) {
  constexpr int kPieces = kQ4Group * sizeof(U) / 16;
  uint4 raw[kPieces];
  U* t = reinterpret_cast<U*>(raw);
#pragma unroll
  for (int i = 0; i < kQ4Group; ++i) t[i] = To<U>::from(x[i]);
#pragma unroll
  for (int i = 0; i < kPieces; ++i) reinterpret_cast<uint4*>(p)[i] = raw[i];
}

// Values of one group: (code - 8) * scale, exact in fp32 and in bf16.
__device__ __forceinline__ void decode16(uint2 codes, uint32_t byte, float (&x)[kQ4Group]) {
  const float s = scale_of(byte);
#pragma unroll
  for (int i = 0; i < kQ4Group; ++i) {
    const uint32_t w = i < 8 ? codes.x : codes.y;
    x[i] = static_cast<float>(static_cast<int>((w >> (4 * (i & 7))) & 15u) - 8) * s;
  }
}

// One thread per group of the chunk: token j of sample b, group g, goes to ring slot
// (first_frame + j / tpf) mod W.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    q4_append_kernel(const T* __restrict__ lat, uint8_t* __restrict__ codes,
                     uint8_t* __restrict__ scales, int32_t* __restrict__ slot_frame, int B, int n_q,
                     int tpf, int W, int groups, int first_frame) {
  grid_dep_wait();
  grid_dep_launch();
  const int64_t total = static_cast<int64_t>(B) * n_q * groups;
  for (int64_t e = blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x; e < total;
       e += static_cast<int64_t>(gridDim.x) * kThreads) {
    const int g = static_cast<int>(e % groups);
    const int64_t bj = e / groups;
    const int b = static_cast<int>(bj / n_q), j = static_cast<int>(bj % n_q);
    const int f = first_frame + j / tpf, slot = f % W;
    float x[kQ4Group];
    load16(lat + e * kQ4Group, x);
    float mx = 0.f;
#pragma unroll
    for (int i = 0; i < kQ4Group; ++i) mx = fmaxf(mx, fabsf(x[i]));   // (a NaN is passed over)
    const uint32_t byte = scale_byte(__fdiv_rn(mx, 7.f));
    const float s = scale_of(byte);
    uint2 c = make_uint2(0u, 0u);
#pragma unroll
    for (int i = 0; i < kQ4Group; ++i) {
      // division, not a product with 1/s: a quotient that is a tie must stay one
      const float r = x[i] == x[i] ? fminf(fmaxf(rintf(__fdiv_rn(x[i], s)), -7.f), 7.f) : 0.f;
      const uint32_t u = static_cast<uint32_t>(static_cast<int>(r) + 8) << (4 * (i & 7));
      if (i < 8) c.x |= u;
      else c.y |= u;
    }
    const int64_t row = (static_cast<int64_t>(b) * W + slot) * tpf + j % tpf;
    reinterpret_cast<uint2*>(codes)[row * groups + g] = c;
    scales[row * groups + g] = static_cast<uint8_t>(byte);
    if (g == 0 && j % tpf == 0) slot_frame[static_cast<int64_t>(b) * W + slot] = f;
  }
}

// One thread per group: rows [0, rows) of each sample's ring into out [B, rows, 16 groups].
template <typename T>
__global__ void __launch_bounds__(kThreads)
    q4_read_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                   T* __restrict__ out, int B, int rows, int ring_rows, int groups) {
  grid_dep_wait();
  grid_dep_launch();
  const int64_t per = static_cast<int64_t>(rows) * groups;
  const int64_t total = B * per;
  for (int64_t e = blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x; e < total;
       e += static_cast<int64_t>(gridDim.x) * kThreads) {
    const int64_t src = (e / per) * ring_rows * groups + e % per;
    float x[kQ4Group];
    decode16(reinterpret_cast<const uint2*>(codes)[src], scales[src], x);
    store16(out + e * kQ4Group, x);
  }
}

// What an attention call over the 4-bit ring reads, in one launch and one thread per 16 values:
//   e < n_ring               content group of ring row r -> ring[b, r, :] (rows ring_width wide; the
//                            attention takes positional keys from ws)
//   e < n_ring + n_chunk     content group of chunk row r -> chunk[b, r, :]  (fp16 only)
//   else                     16 positional values of key-workspace row r: ring slot r decoded, or
//                            chunk token r - nc_pad, rotated at its position and rounded once;
//                            zeros in the padding rows (the layout of key_workspace_layout)
// The content is decoded once per call and not inside the attention kernel: there every CTA (one
// per head and 128 query rows, 444 in the Wan preset's call) reads the whole ring, so it would
// decode it 444 times over, on the threads that the softmax already keeps busy.
template <typename T, typename U>
__global__ void __launch_bounds__(kThreads)
    q4_prepare_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                      const T* __restrict__ chunk_lat, const int32_t* __restrict__ slot_frame,
                      U* __restrict__ ring, U* __restrict__ chunk, U* __restrict__ ws, int B, int W,
                      int D, int d_c, int ring_width, int n_q, int nc, int nc_pad, int rows_ws,
                      int first_frame, RopeGeom geom, int32_t* dev_status) {
  grid_dep_wait();
  grid_dep_launch();
  const int groups = D / kQ4Group, cg = d_c / kQ4Group, rg = groups - cg;
  const int64_t ring_rows = static_cast<int64_t>(W) * geom.tpf;
  const int64_t n_ring = static_cast<int64_t>(B) * nc * cg;
  const int64_t n_content = n_ring + (chunk != nullptr ? static_cast<int64_t>(B) * n_q * cg : 0);
  const int64_t total = n_content + static_cast<int64_t>(B) * rows_ws * rg;
  for (int64_t e = blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x; e < total;
       e += static_cast<int64_t>(gridDim.x) * kThreads) {
    float x[kQ4Group];
    if (e < n_ring) {
      const int g = static_cast<int>(e % cg);
      const int64_t br = e / cg;
      const int64_t src = ((br / nc) * ring_rows + br % nc) * groups + g;
      decode16(reinterpret_cast<const uint2*>(codes)[src], scales[src], x);
      store16(ring + br * ring_width + g * kQ4Group, x);
      continue;
    }
    if (e < n_content) {
      const int g = static_cast<int>((e - n_ring) % cg);
      const int64_t br = (e - n_ring) / cg;
      load16(chunk_lat + br * D + g * kQ4Group, x);
      store16(chunk + br * d_c + g * kQ4Group, x);
      continue;
    }
    const int64_t p = e - n_content;
    const int g = static_cast<int>(p % rg);
    const int64_t br = p / rg;
    const int b = static_cast<int>(br / rows_ws), r = static_cast<int>(br % rows_ws);
    const bool from_ring = r < nc, from_chunk = r >= nc_pad && r - nc_pad < n_q;
    if (from_ring) {
      const int64_t src = (b * ring_rows + r) * groups + cg + g;
      decode16(reinterpret_cast<const uint2*>(codes)[src], scales[src], x);
    } else if (from_chunk) {
      load16(chunk_lat + (static_cast<int64_t>(b) * n_q + (r - nc_pad)) * D + d_c + g * kQ4Group, x);
    } else {
#pragma unroll
      for (int i = 0; i < kQ4Group; ++i) x[i] = 0.f;
    }
    if (from_ring || from_chunk) {
      int t, h, w;
      key_position(slot_frame, b, W, geom.tpf, geom.frame_w, nc, first_frame,
                   from_ring ? r : nc + (r - nc_pad), t, h, w);
      if (from_ring) debug_check(t >= 0 && t < first_frame && t >= first_frame - W, dev_status);
#pragma unroll
      for (int i = 0; i < kQ4Group; i += 2)
        rope_rotate(x[i], x[i + 1], rope_angle(geom, (g * kQ4Group + i) / 2, t, h, w));
    }
    store16(ws + br * (rg * kQ4Group) + g * kQ4Group, x);
  }
}

int blocks_for(int64_t total) {
  return static_cast<int>(std::min<int64_t>((total + kThreads - 1) / kThreads, 148 * 8));
}

}  // namespace

mla_status q4_append(const Dims& d, const void* chunk_lat, uint8_t* codes, uint8_t* scales,
                     int32_t* slot_frame, int first_frame, cudaStream_t s) {
  const int groups = d.D / kQ4Group;
  const dim3 grid(blocks_for(static_cast<int64_t>(d.B) * d.n_q * groups));
  if (d.dtype == MLA_FP32)
    MLA_CUDA_TRY(launch_pdl(q4_append_kernel<float>, grid, dim3(kThreads), 0, s,
                            static_cast<const float*>(chunk_lat), codes, scales, slot_frame, d.B,
                            d.n_q, d.tpf, d.W, groups, first_frame));
  else
    MLA_CUDA_TRY(launch_pdl(q4_append_kernel<bf16>, grid, dim3(kThreads), 0, s,
                            static_cast<const bf16*>(chunk_lat), codes, scales, slot_frame, d.B,
                            d.n_q, d.tpf, d.W, groups, first_frame));
  return MLA_OK;
}

mla_status q4_read(const Dims& d, const uint8_t* codes, const uint8_t* scales, int rows, void* out,
                   cudaStream_t s) {
  if (rows == 0) return MLA_OK;
  const int groups = d.D / kQ4Group;
  const dim3 grid(blocks_for(static_cast<int64_t>(d.B) * rows * groups));
  if (d.dtype == MLA_FP32)
    MLA_CUDA_TRY(launch_pdl(q4_read_kernel<float>, grid, dim3(kThreads), 0, s, codes, scales,
                            static_cast<float*>(out), d.B, rows, d.W * d.tpf, groups));
  else
    MLA_CUDA_TRY(launch_pdl(q4_read_kernel<bf16>, grid, dim3(kThreads), 0, s, codes, scales,
                            static_cast<bf16*>(out), d.B, rows, d.W * d.tpf, groups));
  return MLA_OK;
}

namespace {

template <typename T, typename U>
mla_status prepare(const Dims& d, const uint8_t* codes, const uint8_t* scales,
                   const void* chunk_lat, const int32_t* slot_frame, int n_valid, int first_frame,
                   void* workspace, bool f16, int32_t* dev_status, cudaStream_t s) {
  const KeyWorkspace kw = key_workspace_layout(d, n_valid);
  const Q4Workspace w = q4_workspace_layout(d, n_valid, f16);
  char* base = static_cast<char*>(workspace);
  const int64_t rows = static_cast<int64_t>(kw.nc) + (f16 ? d.n_q : 0);
  const int64_t total = d.B * (rows * (d.d_c / kQ4Group) +
                               static_cast<int64_t>(kw.rows) * (d.d_rope / kQ4Group));
  MLA_CUDA_TRY(launch_pdl(
      q4_prepare_kernel<T, U>, dim3(blocks_for(total)), dim3(kThreads), 0, s, codes, scales,
      static_cast<const T*>(chunk_lat), slot_frame, reinterpret_cast<U*>(base + w.key_bytes),
      f16 ? reinterpret_cast<U*>(base + w.key_bytes + w.ring_bytes) : static_cast<U*>(nullptr),
      reinterpret_cast<U*>(base), d.B, d.W, d.D, d.d_c, f16 ? d.d_c : d.D, d.n_q, kw.nc, kw.nc_pad,
      kw.rows, first_frame, rope_geom(d), dev_status));
  return MLA_OK;
}

}  // namespace

mla_status q4_prepare(const Dims& d, const uint8_t* codes, const uint8_t* scales,
                      const void* chunk_lat, const int32_t* slot_frame, int n_valid,
                      int first_frame, void* workspace, bool f16, int32_t* dev_status,
                      cudaStream_t s) {
  if (f16)
    return prepare<bf16, __half>(d, codes, scales, chunk_lat, slot_frame, n_valid, first_frame,
                                 workspace, true, dev_status, s);
  if (d.dtype == MLA_FP32)
    return prepare<float, float>(d, codes, scales, chunk_lat, slot_frame, n_valid, first_frame,
                                 workspace, false, dev_status, s);
  return prepare<bf16, bf16>(d, codes, scales, chunk_lat, slot_frame, n_valid, first_frame,
                             workspace, false, dev_status, s);
}

Q4Workspace q4_workspace_layout(const Dims& d, int n_valid, bool f16) {
  const KeyWorkspace kw = key_workspace_layout(d, n_valid);
  const auto round256 = [](size_t n) { return (n + 255) / 256 * 256; };
  Q4Workspace w;
  w.key_bytes = round256(kw.bytes);
  w.ring_bytes = round256(static_cast<size_t>(d.B) * kw.nc *
                          (f16 ? d.d_c * sizeof(__half) : d.D * dtype_size(d.dtype)));
  w.chunk_bytes = f16 ? round256(static_cast<size_t>(d.B) * d.n_q * d.d_c * sizeof(__half)) : 0;
  w.bytes = w.key_bytes + w.ring_bytes + w.chunk_bytes;
  return w;
}

}  // namespace mla
