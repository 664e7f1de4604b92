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
// minus a bias are the scale byte.  All three passes move few bytes, so what bounds them is latency and
// the instructions: a thread per group or half group, no shared memory, and few instructions a
// value (no division, no conversion between integers and floats).
// Measured (Wan widths): appending 37,440 tokens and reading 112,320 back 24 us for both, 13 us of
// bytes (cold and alone: the append 12.7 us for 3.3 of bytes, its issue slots 73 % busy with the encoding;
// the read 17 us for 9.9, 57 % busy); 4680 and 9360 tokens 12.7 us, the host's side of two calls; the pass
// before the attention over 21 frames of 252 tokens in two samples 7.8 us cold.
#include <cuda_fp16.h>

#include "kernels.h"
#include "ring_q4.h"

namespace mla {

namespace {

constexpr int kThreads = 256;
constexpr int kScaleBias = 107 * 8;     // (fp32 exponent bias 127 - 20) on top of 3 mantissa bits
constexpr float kRound = 12582912.f;    // 1.5 * 2^23: x + this holds the integer nearest x in its low bits

__device__ __forceinline__ float scale_of(uint32_t byte) {
  return __uint_as_float((byte + kScaleBias) << 20);
}

// Byte of the smallest scale s with 7 s >= mx >= 0 (255 if there is none): the 20 mantissa bits of
// mx / 7 below the third are rounded up by a carry into the bits above.  The quotient may have been
// rounded down to a scale that is a hair too small; 7 s is exact and tells.
__device__ __forceinline__ uint32_t scale_byte(float mx) {
  const float r = __fdiv_rn(mx, 7.f);
  int b = static_cast<int>((__float_as_uint(r) + 0xFFFFFu) >> 20) - kScaleBias;
  b = min(max(b, 0), 255);
  if (b < 255 && 7.f * scale_of(b) < mx) ++b;
  return static_cast<uint32_t>(b);
}

// x / s to the nearest integer, ties to even, within +-7 (a NaN gives 0): a product with 1/s, put
// right by the exact remainder x - c s.  (A division each would take several times the
// instructions, and they bound the pass.)  kShort: x has 8 significant bits, so a quotient that is
// not a tie lies 2^-13 or more from one, beyond the product's error, and only ties can be wrong.
template <bool kShort>
__device__ __forceinline__ float nearest_code(float x, float s, float rcp) {
  x = x == x ? fminf(fmaxf(x, -7.f * s), 7.f * s) : 0.f;
  const float t = fmaf(x, rcp, kRound);        // kRound + integer
  float c = t - kRound;
  const float rem = fmaf(-c, s, x), h = 0.5f * s;
  const bool odd = (__float_as_uint(t) & 1u) != 0;
  if ((fabsf(rem) == h && odd) || (!kShort && fabsf(rem) > h)) c += copysignf(1.f, rem);
  return c;
}

// Eight codes, each plus 8, in four bits each (the first lowest): four at a time in the low bits of
// a float.
template <bool kShort>
__device__ __forceinline__ uint32_t encode8(const float* x, float s, float rcp) {
  uint32_t half[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float f = nearest_code<kShort>(x[4 * i + 3], s, rcp);
#pragma unroll
    for (int k = 2; k >= 0; --k) f = fmaf(f, 16.f, nearest_code<kShort>(x[4 * i + k], s, rcp));
    half[i] = __float_as_uint(f + (8388608.f + 8.f * 4369.f));       // 4369 = 1 + 16 + 256 + 4096
  }
  return __byte_perm(half[0], half[1], 0x5410);                     // their low 16 bits
}

// kN values of T from 16-byte pieces.
template <int kN, typename T>
__device__ __forceinline__ void load_values(const T* p, float (&x)[kN]) {
  constexpr int kPieces = kN * sizeof(T) / 16;
  uint4 raw[kPieces];
#pragma unroll
  for (int i = 0; i < kPieces; ++i) raw[i] = reinterpret_cast<const uint4*>(p)[i];
  const T* t = reinterpret_cast<const T*>(raw);
#pragma unroll
  for (int i = 0; i < kN; ++i) x[i] = Elem<T>::to_f(t[i]);
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

// kN values as U to 16-byte pieces.
template <int kN, typename U>
__device__ __forceinline__ void store_values(U* p, const float (&x)[kN]) {
  constexpr int kPieces = kN * sizeof(U) / 16;
  uint4 raw[kPieces];
  U* t = reinterpret_cast<U*>(raw);
#pragma unroll
  for (int i = 0; i < kN; ++i) t[i] = To<U>::from(x[i]);
#pragma unroll
  for (int i = 0; i < kPieces; ++i) reinterpret_cast<uint4*>(p)[i] = raw[i];
}

// Eight values: (code - 8) * scale, exact in fp32 and in bf16.  A code in the low bits of 2^23 is
// that float plus the code: no conversion, which the SFU would do.
__device__ __forceinline__ void decode8(uint32_t codes, uint32_t byte, float (&x)[8]) {
  const float s = scale_of(byte);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    x[i] = (__uint_as_float(0x4B000000u | ((codes >> (4 * i)) & 15u)) - 8388616.f) * s;
}

// In the append and the preparation gridDim.y samples take turns, and a sample's pieces are spread
// over gridDim.x blocks, one per thread at a time.  Ring and chunk hold fewer than 2^31 values each,
// so the append has fewer than 2^27 pieces, and the preparation, whose pieces are those of both and of
// up to 254 padding rows of keys, fewer than 2^29 + 2^14: 32-bit index arithmetic.

// Token j of the chunk, group g, goes to ring slot (first_frame + j / tpf) mod W.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    q4_append_kernel(const T* __restrict__ lat, uint8_t* __restrict__ codes,
                     uint8_t* __restrict__ scales, int32_t* __restrict__ slot_frame, int B, int n_q,
                     int tpf, int W, int groups, int first_frame) {
  grid_dep_wait();
  grid_dep_launch();
  const int total = n_q * groups;
  for (int b = blockIdx.y; b < B; b += gridDim.y) {
    for (int e = blockIdx.x * kThreads + threadIdx.x; e < total; e += gridDim.x * kThreads) {
      const int j = e / groups, g = e - j * groups;
      const int fj = j / tpf, i = j - fj * tpf;
      const int f = first_frame + fj, slot = f % W;
      float x[kQ4Group];
      load_values<kQ4Group>(lat + (static_cast<int64_t>(b) * total + e) * kQ4Group, x);
      float mx = 0.f;
#pragma unroll
      for (int k = 0; k < kQ4Group; ++k) mx = fmaxf(mx, fabsf(x[k]));   // (a NaN is passed over)
      const uint32_t byte = scale_byte(mx);
      const float s = scale_of(byte), rcp = __frcp_rn(s);
      constexpr bool kShort = sizeof(T) == 2;
      const uint2 c = make_uint2(encode8<kShort>(x, s, rcp), encode8<kShort>(x + 8, s, rcp));
      const int64_t to = ((static_cast<int64_t>(b) * W + slot) * tpf + i) * groups + g;
      reinterpret_cast<uint2*>(codes)[to] = c;
      scales[to] = static_cast<uint8_t>(byte);
      if (g == 0 && i == 0) slot_frame[static_cast<int64_t>(b) * W + slot] = f;
    }
  }
}

// Every row of each sample's ring into out, eight values (half a group) at a time: a warp's stores
// are 512 consecutive bytes of bf16.  Four loads are on their way before the first is used.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    q4_read_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                   T* __restrict__ out, int64_t total) {
  grid_dep_wait();
  grid_dep_launch();
  const int64_t step = static_cast<int64_t>(gridDim.x) * kThreads;
  for (int64_t e0 = blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x; e0 < total;
       e0 += 4 * step) {
    uint32_t c[4], s[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t e = min(e0 + k * step, total - 1);
      c[k] = reinterpret_cast<const uint32_t*>(codes)[e];
      s[k] = scales[e / 2];
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (e0 + k * step >= total) break;
      float x[8];
      decode8(c[k], s[k], x);
      store_values<8>(out + (e0 + k * step) * 8, x);
    }
  }
}

// What an attention call over the 4-bit ring reads, in one launch; piece e of a sample is
//   e < n_ring               8 content values of ring row r -> ring[b, r, :] (rows ring_width wide; the
//                            attention takes positional keys from ws)
//   e < n_content            8 content values of chunk row r -> chunk[b, r, :]  (fp16 only)
//   else                     8 positional values of key-workspace row r: ring slot r decoded, or
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
  // pieces of 8 values per row: all, content, positional
  const int pieces = D / 8, cp = d_c / 8, rp = pieces - cp;
  const int n_ring = nc * cp, n_content = n_ring + (chunk != nullptr ? n_q * cp : 0);
  const int total = n_content + rows_ws * rp;
  const uint32_t* codes32 = reinterpret_cast<const uint32_t*>(codes);
  for (int b = blockIdx.y; b < B; b += gridDim.y) {
    const int64_t ring_row0 = static_cast<int64_t>(b) * W * geom.tpf;
    for (int e = blockIdx.x * kThreads + threadIdx.x; e < total; e += gridDim.x * kThreads) {
      float x[8];
      if (e < n_ring) {
        const int r = e / cp, g = e - r * cp;
        const int64_t src = (ring_row0 + r) * pieces + g;
        decode8(codes32[src], scales[src / 2], x);
        store_values<8>(ring + (static_cast<int64_t>(b) * nc + r) * ring_width + g * 8, x);
        continue;
      }
      if (e < n_content) {
        const int r = (e - n_ring) / cp, g = (e - n_ring) - r * cp;
        const int64_t row = static_cast<int64_t>(b) * n_q + r;
        load_values<8>(chunk_lat + row * D + g * 8, x);
        store_values<8>(chunk + row * d_c + g * 8, x);
        continue;
      }
      const int p = e - n_content, r = p / rp, g = p - r * rp;
      const bool from_ring = r < nc, from_chunk = r >= nc_pad && r - nc_pad < n_q;
      if (from_ring) {
        const int64_t src = (ring_row0 + r) * pieces + cp + g;
        decode8(codes32[src], scales[src / 2], x);
      } else if (from_chunk) {
        load_values<8>(chunk_lat + (static_cast<int64_t>(b) * n_q + (r - nc_pad)) * D + d_c + g * 8, x);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = 0.f;
      }
      if (from_ring || from_chunk) {
        int t, h, w;
        key_position(slot_frame, b, W, geom.tpf, geom.frame_w, nc, first_frame,
                     from_ring ? r : nc + (r - nc_pad), t, h, w);
        if (from_ring) debug_check(t >= 0 && t < first_frame && t >= first_frame - W, dev_status);
#pragma unroll
        for (int i = 0; i < 8; i += 2)
          rope_rotate(x[i], x[i + 1], rope_angle(geom, (g * 8 + i) / 2, t, h, w));
      }
      store_values<8>(ws + (static_cast<int64_t>(b) * rows_ws + r) * (rp * 8) + g * 8, x);
    }
  }
}

// Blocks for B samples of `total` pieces each: up to sixteen blocks per SM in all.
dim3 grid_for(int B, int64_t total) {
  const int y = std::min(B, 65535);
  const int64_t x = std::min<int64_t>((total + kThreads - 1) / kThreads, std::max(148 * 16 / y, 1));
  return dim3(static_cast<unsigned>(x), static_cast<unsigned>(y));
}

}  // namespace

mla_status q4_append(const Dims& d, const void* chunk_lat, uint8_t* codes, uint8_t* scales,
                     int32_t* slot_frame, int first_frame, cudaStream_t s) {
  const int groups = d.D / kQ4Group;
  const dim3 grid = grid_for(d.B, static_cast<int64_t>(d.n_q) * groups);
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

mla_status q4_read(const Dims& d, const uint8_t* codes, const uint8_t* scales, void* out,
                   cudaStream_t s) {
  const int64_t total = static_cast<int64_t>(d.B) * d.W * d.tpf * (d.D / 8);
  const dim3 grid = grid_for(1, total);
  if (d.dtype == MLA_FP32)
    MLA_CUDA_TRY(launch_pdl(q4_read_kernel<float>, grid, dim3(kThreads), 0, s, codes, scales,
                            static_cast<float*>(out), total));
  else
    MLA_CUDA_TRY(launch_pdl(q4_read_kernel<bf16>, grid, dim3(kThreads), 0, s, codes, scales,
                            static_cast<bf16*>(out), total));
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
  const int64_t total = rows * (d.d_c / 8) + static_cast<int64_t>(kw.rows) * (d.d_rope / 8);
  MLA_CUDA_TRY(launch_pdl(
      q4_prepare_kernel<T, U>, grid_for(d.B, total), dim3(kThreads), 0, s, codes, scales,
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
