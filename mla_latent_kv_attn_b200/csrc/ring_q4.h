// ring_q4.h - internal launchers of the 4-bit latent ring (ring_q4.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace mla {

constexpr int kQ4Group = 16;   // values that share a scale

// Workspace of an attention call over the 4-bit ring: the rotated keys (as the attention over a
// T ring has them), then what the kernel reads the latents from.  On the tensor cores (f16) that is
// the contents in fp16, ring [B, n_valid * tpf, d_c] and chunk [B, n_q, d_c]; elsewhere the decoded
// ring rows in T, [B, n_valid * tpf, D], beside the caller's chunk.
struct Q4Workspace {
  size_t key_bytes, ring_bytes, chunk_bytes, bytes;
};
Q4Workspace q4_workspace_layout(const Dims& d, int n_valid, bool f16);

// chunk_lat [B, n_q, D] into the slots of frames first_frame .. first_frame + C - 1.
mla_status q4_append(const Dims& d, const void* chunk_lat, uint8_t* codes, uint8_t* scales,
                     int32_t* slot_frame, int first_frame, cudaStream_t s);
// Every sample's ring as T values, out [B, W * tpf, D].
mla_status q4_read(const Dims& d, const uint8_t* codes, const uint8_t* scales, void* out,
                   cudaStream_t s);
// Writes an attention call's workspace (f16 as above).
mla_status q4_prepare(const Dims& d, const uint8_t* codes, const uint8_t* scales,
                      const void* chunk_lat, const int32_t* slot_frame, int n_valid,
                      int first_frame, void* workspace, bool f16, int32_t* dev_status,
                      cudaStream_t s);

}  // namespace mla
