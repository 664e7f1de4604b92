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
