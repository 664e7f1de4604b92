// cross_tc.cuh - pieces shared by the tensor-core kernels of the cross attention.
#pragma once

#include "cross.h"
#include "exp2.cuh"
#include "kernels.h"
#include "sm100.cuh"

namespace mla {

constexpr int kCrossTile = 128;          // rows of every operand tile
constexpr float kLog2e = 1.4426950408889634f;

// Zeros rows [from, to) of a tile of kBlocks blocks of kRows 128-byte rows (whatever the swizzle: it
// permutes within a row), `threads` threads of index t.
template <int kBlocks, int kRows>
__device__ __forceinline__ void zero_rows(uint32_t tile, int from, int to, int t, int threads) {
  const int n = (to - from) * 8;
  for (int i = t; i < n; i += threads) {
#pragma unroll
    for (int blk = 0; blk < kBlocks; ++blk)
      asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(tile + blk * kRows * 128 +
                                                                    from * 128 + i * 16),
                   "r"(0)
                   : "memory");
  }
}

// 2^x of a pair on the FMA pipe, as exp2_poly_pair but by the polynomial of degree 4 that takes 2^f at
// the five Chebyshev nodes of [-1/2, 1/2] (relative error below 3.6e-6 with these fp32
// coefficients): the row sum, and with it the fp32 lse, is taken from these values.
__device__ __forceinline__ void exp2_poly4_pair(float x0, float x1, float& y0, float& y1) {
  using namespace sm100;
  const uint64_t x = f2_pack(fmaxf(x0, -125.f), fmaxf(x1, -125.f));
  const uint64_t magic = f2_pack(kRoundMagic, kRoundMagic);
  const uint64_t t = f2_add(x, magic);                              // magic + n, exactly
  const uint64_t f = f2_add(x, f2_fma(t, f2_pack(-1.f, -1.f), magic));    // x - n
  uint64_t q = f2_fma(f, f2_pack(0.009666368515386919f, 0.009666368515386919f),
                      f2_pack(0.05592197584225607f, 0.05592197584225607f));
  q = f2_fma(q, f, f2_pack(0.24022349038020357f, 0.24022349038020357f));
  q = f2_fma(q, f, f2_pack(0.6931210452034271f, 0.6931210452034271f));
  q = f2_fma(q, f, f2_pack(1.f, 1.f));
  float q0, q1, t0, t1;
  f2_unpack(q, q0, q1);
  f2_unpack(t, t0, t1);
  // the low bits of t hold n: shifted into the exponent field they scale q by 2^n
  y0 = __uint_as_float(__float_as_uint(q0) + (__float_as_uint(t0) << 23));
  y1 = __uint_as_float(__float_as_uint(q1) + (__float_as_uint(t1) << 23));
}

// 16-byte piece `piece` (0-7) of row `row` of a block of 128-byte rows, where a TMA copy with the
// 128-byte swizzle places it.
__device__ __forceinline__ uint32_t swizzled_piece(uint32_t block, int row, int piece) {
  return block + row * 128 + ((piece ^ (row & 7)) << 4);
}

__device__ __forceinline__ void store_shared16(uint32_t at, const uint32_t (&v)[4]) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3])
               : "memory");
}

// Tensor map of [B, n, heads, d] rows with 64-column, `rows`-row boxes, 128-byte swizzle.
inline mla_status cross_tmap(CUtensorMap* m, const void* base, int B, int n, int heads, int d, int64_t row,
                      uint32_t rows) {
  const uint64_t dims[4] = {static_cast<uint64_t>(d), static_cast<uint64_t>(heads),
                            static_cast<uint64_t>(n), static_cast<uint64_t>(B)};
  const uint64_t strides[3] = {d * 2ull, static_cast<uint64_t>(row) * 2,
                               static_cast<uint64_t>(n) * static_cast<uint64_t>(row) * 2};
  const uint32_t box[4] = {64, 1, rows, 1};
  return make_tmap_bf16(m, base, 4, dims, strides, box, 128);
}

}  // namespace mla
