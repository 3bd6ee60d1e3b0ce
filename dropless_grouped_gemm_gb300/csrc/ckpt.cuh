// ckpt.cuh - host-side interface of the 8-bit checkpoint kernels (ckpt.cu).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace moe {

// n values in whole 32-blocks
cudaError_t launch_ckpt_pack(const uint16_t* src, long long n, uint8_t* q, uint8_t* sc,
                             cudaStream_t s);
cudaError_t launch_ckpt_unpack(const uint8_t* q, const uint8_t* sc, long long n, uint16_t* dst,
                               cudaStream_t s);
// the packed rows of [T, d] in expert-major order, in bf16 (row_of_pair may
// be NULL: row order)
cudaError_t launch_ckpt_gather(const uint8_t* q, const uint8_t* sc, const int32_t* row_of_pair,
                               const int32_t* pair_of_row, int T, int k, int d, int M_cap,
                               uint16_t* dst, int num_sms, cudaStream_t s);

}  // namespace moe
