// cross.h - internal launchers of the cross attention to an encoder's states (mla_abi.cu calls
// them; cross_simt.cu and cross_sm100.cu implement them).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace mla {

// Sizes of a cross-attention call; the row strides are in elements from one token to the next
// (a token's heads are dense, a sample's tokens follow one another).
struct CrossDims {
  int B, H, Hkv, d, n_q, n_kv;
  float scale;
  int dtype, path;
  int64_t q_row, k_row, v_row;
};

struct CrossArgs {
  const void* q;           // [B, n_q, H, d]
  const void* k;           // [B, n_kv, Hkv, d]
  const void* v;           // [B, n_kv, Hkv, d]
  const int32_t* kv_len;   // [B] or null (every state valid)
  void* out;               // [B, n_q, H, d]
  float* lse;              // [B, H, n_q] or null
  int32_t* dev_status;     // or null
};

struct CrossBwdArgs {
  const void* q;
  const void* k;
  const void* v;
  const int32_t* kv_len;
  const void* out;         // the forward's output
  const float* lse;        // and statistics
  const void* d_out;       // [B, n_q, H, d]
  void* d_q;               // dense, as q
  void* d_k;               // dense, as k
  void* d_v;
  int32_t* dev_status;
};

// Valid states of sample b: kv_len[b] clamped to [0, n_kv].  (From L2: some kernels read it before they
// wait for the grid in front of them.)
__device__ __forceinline__ int cross_len(const int32_t* kv_len, int b, int n_kv) {
  if (kv_len == nullptr) return n_kv;
  const int n = __ldcg(kv_len + b);
  return n < 0 ? 0 : (n > n_kv ? n_kv : n);
}

// CUDA-core kernels: every dtype and any d up to kCrossMaxD (cross_simt.cu).
constexpr int kCrossMaxD = 256;
mla_status cross_fwd_simt(const CrossDims& d, const CrossArgs& a, cudaStream_t s);
mla_status cross_bwd_simt(const CrossDims& d, const CrossBwdArgs& a, float* delta, cudaStream_t s);

// Tensor-core kernels: bf16 with d 64 or 128 (cross_sm100.cu, cross_bwd_sm100.cu).
bool cross_tc_supported(const CrossDims& d);
mla_status cross_fwd_tc(const CrossDims& d, const CrossArgs& a, cudaStream_t s);
size_t cross_bwd_tc_workspace(const CrossDims& d);
mla_status cross_bwd_tc(const CrossDims& d, const CrossBwdArgs& a, void* workspace, cudaStream_t s);

}  // namespace mla
