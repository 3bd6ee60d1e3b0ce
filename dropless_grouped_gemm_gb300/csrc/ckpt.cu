// ckpt.cu - activations kept in 8 bits between the forward and the backward:
// E4M3 codes with one E8M0 scale per 32 values of a row (the block rule of
// mx.cuh), 1.03 bytes a value against bf16's 2.
//
// Rows are whole numbers of blocks, so packing and unpacking are flat passes
// over rows * cols / 32 blocks; the gather walks tokens and writes each
// token's rows of the expert-major buffer.  All are HBM-bound: 16-byte
// accesses to the bf16 side, several in flight per thread.
#include <cuda_runtime.h>

#include "ckpt.cuh"
#include "mx.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;

// one thread: 8 values (16 bytes of bf16, 8 bytes of codes); four lanes
// share a block
__global__ void __launch_bounds__(kThreads)
    pack_kernel(const uint4* __restrict__ src, long long n8, uint2* __restrict__ q,
                uint8_t* __restrict__ s) {
  const long long base = static_cast<long long>(blockIdx.x) * (kThreads * kUnroll) + threadIdx.x;
  uint4 v[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const long long i = base + u * kThreads;
    v[u] = i < n8 ? src[i] : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const long long i = base + u * kThreads;
    const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
    float amax = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(w[j])), fabsf(bf16_hi(w[j]))));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    const uint32_t code = mx_scale_code(amax);
    const float inv = mx_inv_scale(code);
    uint32_t o[2];
#pragma unroll
    for (int j = 0; j < 2; ++j)
      o[j] = e4m3x2(bf16_lo(w[2 * j]) * inv, bf16_hi(w[2 * j]) * inv) |
             (e4m3x2(bf16_lo(w[2 * j + 1]) * inv, bf16_hi(w[2 * j + 1]) * inv) << 16);
    if (i < n8) {
      q[i] = make_uint2(o[0], o[1]);
      if ((threadIdx.x & 3) == 0) s[i >> 2] = static_cast<uint8_t>(code);
    }
  }
}

__global__ void __launch_bounds__(kThreads)
    unpack_kernel(const uint2* __restrict__ q, const uint8_t* __restrict__ s, long long n8,
                  uint4* __restrict__ dst) {
  const long long base = static_cast<long long>(blockIdx.x) * (kThreads * kUnroll) + threadIdx.x;
  uint2 c[kUnroll];
  float sc[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const long long i = base + u * kThreads;
    c[u] = i < n8 ? q[i] : make_uint2(0, 0);
    sc[u] = i < n8 ? mx_scale(s[i >> 2]) : 0.f;
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const long long i = base + u * kThreads;
    uint32_t o[4];
    mx_decode8(c[u].x, c[u].y, sc[u], o);
    if (i < n8) dst[i] = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

// Gather of the packed token rows into expert-major bf16 rows.  Token order
// (row_of_pair given): a warp decodes a 1,024-value segment of a token's row
// once and writes it to each of the token's rows; the items after the tokens
// are the rows, of which those without a valid pair are zeroed.  Row order
// (row_of_pair NULL): a warp takes a segment of one row.
constexpr int kWarps = kThreads / 32;
constexpr int kSeg = 128;   // groups of 8 values per segment

__device__ __forceinline__ void load_seg(const uint2* q, const uint8_t* s, int v0, int dv,
                                         int lane, uint4 (&x)[kSeg / 32]) {
  uint2 c[kSeg / 32];
  float sc[kSeg / 32];
#pragma unroll
  for (int i = 0; i < kSeg / 32; ++i) {
    const int v = v0 + lane + 32 * i;
    c[i] = v < dv ? __ldg(q + v) : make_uint2(0, 0);
    sc[i] = v < dv ? mx_scale(__ldg(s + (v >> 2))) : 0.f;
  }
#pragma unroll
  for (int i = 0; i < kSeg / 32; ++i) {
    uint32_t o[4];
    mx_decode8(c[i].x, c[i].y, sc[i], o);
    x[i] = make_uint4(o[0], o[1], o[2], o[3]);
  }
}
__device__ __forceinline__ void store_seg(uint4* out, int v0, int dv, int lane,
                                          const uint4 (&x)[kSeg / 32]) {
#pragma unroll
  for (int i = 0; i < kSeg / 32; ++i) {
    const int v = v0 + lane + 32 * i;
    if (v < dv) __stcs(out + v, x[i]);
  }
}

template <bool TOKENS>
__global__ void __launch_bounds__(kThreads)
    gather_kernel(const uint2* __restrict__ q, const uint8_t* __restrict__ s,
                  const int32_t* __restrict__ row_of_pair, const int32_t* __restrict__ pair_of_row,
                  int T, int k, int dv, int M_cap, uint4* __restrict__ dst) {
  const int lane = threadIdx.x & 31;
  const long long P = static_cast<long long>(T) * k;
  const int nseg = (dv + kSeg - 1) / kSeg;
  const long long head = static_cast<long long>(TOKENS ? T : M_cap) * nseg;
  const long long items = head + (TOKENS ? M_cap : 0);
  for (long long it = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
       it < items; it += static_cast<long long>(gridDim.x) * kWarps) {
    if (it < head) {
      const int r0 = static_cast<int>(it / nseg);
      const int v0 = static_cast<int>(it - static_cast<long long>(r0) * nseg) * kSeg;
      uint4 x[kSeg / 32];
      if constexpr (TOKENS) {
        const long long t = r0;
        load_seg(q + t * dv, s + t * (dv / 4), v0, dv, lane, x);
        for (int j = 0; j < k; ++j) {
          const long long p = t * k + j;
          const int r = row_of_pair[p];
          if (r < 0 || r >= M_cap || pair_of_row[r] != p) continue;
          store_seg(dst + static_cast<long long>(r) * dv, v0, dv, lane, x);
        }
      } else {
        const int p = pair_of_row[r0];
        if (p >= 0 && p < P) {
          const long long t = p / k;
          load_seg(q + t * dv, s + t * (dv / 4), v0, dv, lane, x);
        } else {
#pragma unroll
          for (int i = 0; i < kSeg / 32; ++i) x[i] = make_uint4(0, 0, 0, 0);
        }
        store_seg(dst + static_cast<long long>(r0) * dv, v0, dv, lane, x);
      }
    } else {
      const int r = static_cast<int>(it - head);
      const int p = pair_of_row[r];
      if (p < 0 || p >= P) {
        uint4* out = dst + static_cast<long long>(r) * dv;
        for (int v = lane; v < dv; v += 32) __stcs(out + v, make_uint4(0, 0, 0, 0));
      }
    }
  }
}

}  // namespace

cudaError_t launch_ckpt_pack(const uint16_t* src, long long n, uint8_t* q, uint8_t* sc,
                             cudaStream_t s) {
  const long long n8 = n / 8;
  const long long blocks = (n8 + kThreads * kUnroll - 1) / (kThreads * kUnroll);
  pack_kernel<<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(
      reinterpret_cast<const uint4*>(src), n8, reinterpret_cast<uint2*>(q), sc);
  return cudaGetLastError();
}

cudaError_t launch_ckpt_unpack(const uint8_t* q, const uint8_t* sc, long long n, uint16_t* dst,
                               cudaStream_t s) {
  const long long n8 = n / 8;
  const long long blocks = (n8 + kThreads * kUnroll - 1) / (kThreads * kUnroll);
  unpack_kernel<<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(
      reinterpret_cast<const uint2*>(q), sc, n8, reinterpret_cast<uint4*>(dst));
  return cudaGetLastError();
}

cudaError_t launch_ckpt_gather(const uint8_t* q, const uint8_t* sc, const int32_t* row_of_pair,
                               const int32_t* pair_of_row, int T, int k, int d, int M_cap,
                               uint16_t* dst, int num_sms, cudaStream_t s) {
  const int dv = d / 8;
  const long long nseg = (dv + kSeg - 1) / kSeg;
  const long long items = row_of_pair ? static_cast<long long>(T) * nseg + M_cap
                                      : static_cast<long long>(M_cap) * nseg;
  const long long want = (items + kWarps - 1) / kWarps;
  const long long most = 8LL * num_sms;
  const int grid = static_cast<int>(want < most ? want : most);
  const uint2* qv = reinterpret_cast<const uint2*>(q);
  uint4* out = reinterpret_cast<uint4*>(dst);
  if (row_of_pair)
    gather_kernel<true><<<grid, kThreads, 0, s>>>(qv, sc, row_of_pair, pair_of_row, T, k, dv, M_cap, out);
  else
    gather_kernel<false><<<grid, kThreads, 0, s>>>(qv, sc, nullptr, pair_of_row, T, k, dv, M_cap, out);
  return cudaGetLastError();
}

}  // namespace moe
