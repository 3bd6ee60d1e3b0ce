// fp4_mma.cuh - what the two product kernels of the 4-bit formats share: the
// block-scaled MMA, and the output of consecutive columns of a row.
#pragma once

#include "act.cuh"
#include "fp4_dev.cuh"

namespace moe {

constexpr int kFp4StageK = 256;                   // values of K a stage: one 128-byte swizzle row
constexpr int kFp4StepK = 64;                     // of an MMA
template <bool NV>
struct Fp4Sf {
  static constexpr int chunks = NV ? 4 : 2;       // scale chunks of a 128-row operand a stage
  static constexpr int bytes = chunks * kFp4ChunkBytes;
  static constexpr int cols = chunks * 4;         // TMEM columns of one operand's
};

// Instruction descriptor, kind::mxf4nvf4: A and B E2M1 (bits 7-9, 10-11: 1),
// K-major, bits 17-22 N >> 3, bit 23 scale type (0 E4M3, 1 E8M0), bits 24-28
// M >> 4, scale-factor byte selectors B bits 4-5, A bits 29-30, bit 31 0: K = 64.
template <bool NV>
__device__ __forceinline__ constexpr uint32_t fp4_idesc(int M, int N) {
  return (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) | (NV ? 0u : 1u << 23) |
         (static_cast<uint32_t>(M >> 4) << 24);
}
// step kk of a stage: NV takes chunk kk whole; MX chunk kk / 2, of which bytes
// 0-1 or 2-3
template <bool NV>
__device__ __forceinline__ constexpr uint32_t fp4_select(int kk) {
  return NV ? 0u : ((static_cast<uint32_t>(2 * (kk & 1)) << 29) | (static_cast<uint32_t>(2 * (kk & 1)) << 4));
}
template <bool NV>
__device__ __forceinline__ constexpr int fp4_step_chunk(int kk) { return NV ? kk : kk / 2; }

template <bool NV, bool PAIR>
__device__ __forceinline__ void umma_fp4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                         uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                         uint32_t accumulate) {
#define MOE_FP4_MMA(CTAS, VEC)                                                              \
  asm volatile(                                                                             \
      "{\n\t.reg .pred p;\n\t"                                                              \
      "setp.ne.b32 p, %6, 0;\n\t"                                                           \
      "tcgen05.mma.cta_group::" CTAS ".kind::mxf4nvf4.block_scale.scale_vec::" VEC          \
      " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),                               \
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)             \
      : "memory")
  if constexpr (PAIR) {
    if constexpr (NV) MOE_FP4_MMA("2", "4X");
    else MOE_FP4_MMA("2", "2X");
  } else {
    if constexpr (NV) MOE_FP4_MMA("1", "4X");
    else MOE_FP4_MMA("1", "2X");
  }
#undef MOE_FP4_MMA
}

// no-swizzle descriptor of a 512-byte scale chunk (32 rows x 16 bytes, 8-row
// core matrices 128 bytes apart)
__device__ __forceinline__ uint64_t fp4_sf_desc(uint32_t saddr) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(512 >> 4) << 16) |
         (static_cast<uint64_t>(128 >> 4) << 32) | (static_cast<uint64_t>(1) << 46);
}
__device__ __forceinline__ void fp4_sf_copy(uint32_t taddr, uint64_t sdesc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc)
               : "memory");
}

// The experts' rows in shared memory: offsets made safe (clamped to [0, M_cap],
// by their running maximum, from 0) and the first unit of each expert, by one
// warp; units(rows) is how many an expert of so many rows has.
template <class Units>
__device__ __forceinline__ void fp4_schedule(const int32_t* offsets, int E, int M_cap, int* s_off,
                                             int* s_ts, int32_t* err, Units units) {
  const int lane = threadIdx.x & 31;
  if (offsets == nullptr) {
    if (lane == 0) {
      s_off[0] = 0;
      s_off[1] = M_cap;
      s_ts[0] = 0;
      s_ts[1] = units(M_cap);
    }
    return;
  }
  bool bad = false;
  int top = 0, carry = 0;
  for (int base = 0; base <= E; base += 128) {        // four loads in flight
    int raw[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const int i = base + 32 * b + lane;
      raw[b] = i <= E ? offsets[i] : 0;
    }
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const int i = base + 32 * b + lane;
      if (base + 32 * b > E) break;
      int m = max(min(max(raw[b], 0), M_cap), top);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, m, o);
        if (lane >= o) m = max(m, y);
      }
      if (i <= E) {
        if (m != raw[b] || (i == 0 && m != 0)) bad = true;
        s_off[i] = m;
      }
      // expert i - 1 ends at m
      int prev = __shfl_up_sync(0xffffffffu, m, 1);
      if (lane == 0) prev = top;
      int c = (i >= 1 && i <= E) ? units(m - prev) : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, c, o);
        if (lane >= o) c += y;
      }
      if (i <= E) s_ts[i] = carry + c;
      top = __shfl_sync(0xffffffffu, m, 31);
      carry += __shfl_sync(0xffffffffu, c, 31);
    }
  }
  if (__any_sync(0xffffffffu, bad) && lane == 0 && blockIdx.x == 0) set_err(err, MOE_DEV_BAD_OFFSETS);
}

// the expert that unit u belongs to
__device__ __forceinline__ int fp4_expert_of(const int* s_ts, int E, int u) {
  int lo = 0, hi = E - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (s_ts[mid + 1] <= u) lo = mid + 1;
    else hi = mid;
  }
  return lo;
}

// t_a t_e of an expert
__device__ __forceinline__ float fp4_alpha(const Fp4GemmArgs& g, int e) {
  const float a = g.a_t ? *g.a_t : 1.f, w = g.w_t ? g.w_t[e] : 1.f;
  return a * w;
}

}  // namespace moe
