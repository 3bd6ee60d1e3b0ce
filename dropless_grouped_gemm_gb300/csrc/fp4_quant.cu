// fp4_quant.cu - quantisation to 4 bits and back (formats and scale layout in
// fp4.cuh).
//
// All are bound by HBM: rows are read once (2 bytes a value) and written once
// (0.5 bytes and the scale).  A thread takes 16 consecutive values (two 16-byte
// loads), so a warp takes 512 of a row; NV's block is a thread's, MX's a pair
// of threads'.  Four lanes join their scale bytes into one store.  With the
// routing maps (a permute) a token's values are quantised once and written to
// each of its k rows.  Weights with blocks along the outer index: a warp takes
// 64 x 64 values, a lane two columns of 64 (64 loads of 4 bytes, 128 bytes a
// warp), so the transposition needs no shared memory and the codes leave in
// whole 32-byte sectors.
#include <cuda_runtime.h>

#include "fp4_dev.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr unsigned kAll = 0xffffffffu;

// The offsets made safe (clamped to [0, rows], by their running maximum) in
// shared memory, by the whole block; bad ones are reported by block 0.
__device__ __forceinline__ void load_offsets(const Fp4Rows& r, int* s_off, int32_t* err) {
  if (r.offsets == nullptr) return;
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    bool bad = false;
    int top = 0;
    for (int base = 0; base <= r.E; base += 32) {
      const int i = base + lane;
      const int raw = i <= r.E ? r.offsets[i] : 0;
      int m = max(min(max(raw, 0), static_cast<int>(r.rows)), top);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kAll, m, o);
        if (lane >= o) m = max(m, y);
      }
      if (i <= r.E) {
        if (m != raw || (i == 0 && m != 0)) bad = true;
        s_off[i] = m;
      }
      top = __shfl_sync(kAll, m, 31);
    }
    if (__any_sync(kAll, bad) && lane == 0 && blockIdx.x == 0) set_err(err, MOE_DEV_BAD_OFFSETS);
  }
  __syncthreads();
}

// the expert of a row; false: the row is outside every expert
__device__ __forceinline__ bool place_of(const Fp4Rows& r, const int* s_off, long long row,
                                         Fp4Place& p) {
  if (r.offsets == nullptr) {
    p.e = r.E == 1 ? 0 : static_cast<int>(row / r.rows_per_e);
    p.off = p.e * r.rows_per_e;
  } else {
    if (row < s_off[0] || row >= s_off[r.E]) return false;
    int lo = 0, hi = r.E - 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (s_off[mid + 1] <= row) lo = mid + 1;
      else hi = mid;
    }
    p.e = lo;
    p.off = s_off[lo];
  }
  p.tile0 = fp4_tile0(p.off, p.e);
  return true;
}

__device__ __forceinline__ float tensor_scale(const float* t, int stride, int e) {
  return t == nullptr ? 1.f : t[stride * e];
}

// A lane's 16 values (8 words) as codes and its scale byte (MX: the pair's)
template <bool NV>
__device__ __forceinline__ uint2 quant16(const uint32_t (&p)[8], float t, uint32_t& byte) {
  uint32_t m = bf16_amax16(p);
  if constexpr (!NV) m = max(m, __shfl_xor_sync(kAll, m, 1));
  float inv;
  byte = fp4_scale<NV>(m << 16, t, inv);
  return fp4_codes16(p, inv, NV && fp4_power_of_two(t));
}

// 64 values' scale bytes of four neighbouring lanes, joined in the first of
// them (NV: 4 bytes; MX: 2, the lanes in pairs hold the same)
template <bool NV>
__device__ __forceinline__ uint32_t join_bytes(uint32_t byte) {
  const int lane = threadIdx.x & 31;
  uint32_t w;
  if constexpr (NV) w = byte << (8 * (lane & 3));
  else w = byte << (4 * (lane & 2));
  if constexpr (NV) w |= __shfl_xor_sync(kAll, w, 1);
  w |= __shfl_xor_sync(kAll, w, 2);
  return w;
}

// the codes and scales of values [k0, k0 + 16) of row `row`, by this lane
template <bool NV>
__device__ __forceinline__ void store16(const Fp4QuantArgs& a, const Fp4Place& pl, long long row,
                                        int k0, bool on, uint2 codes, uint32_t scales) {
  if (!on) return;
  *reinterpret_cast<uint2*>(a.q + row * (a.K / 2) + k0 / 2) = codes;
  if ((threadIdx.x & 3) == 0) {
    uint8_t* at = a.s + fp4_scale_at(pl.tile0, row - pl.off, k0 / (NV ? 16 : 32),
                                     fp4_chunks(NV, a.K));
    if constexpr (NV) *reinterpret_cast<uint32_t*>(at) = scales;
    else *reinterpret_cast<uint16_t*>(at) = static_cast<uint16_t>(scales);
  }
}

__device__ __forceinline__ void load16(const uint16_t* p, bool on, uint32_t (&w)[8]) {
  if (on) {
    const uint4 u = __ldcs(reinterpret_cast<const uint4*>(p));
    const uint4 v = __ldcs(reinterpret_cast<const uint4*>(p) + 1);
    w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
    w[4] = v.x; w[5] = v.y; w[6] = v.z; w[7] = v.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 0u;
  }
}

// Rows in their own order; with pair_of_row, row r is token pair_of_row[r] / k
// (pad rows inside an expert: zeros).  Rows outside every expert are left.
template <bool NV>
__global__ void __launch_bounds__(kThreads) rows_kernel(const Fp4QuantArgs a) {
  extern __shared__ int s_off[];
  load_offsets(a.r, s_off, a.err);
  const int lane = threadIdx.x & 31;
  const int segs = (a.K + 511) / 512;
  const long long items = a.r.rows * segs;
  const long long step = static_cast<long long>(gridDim.x) * kWarps;
  for (long long it = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5); it < items;
       it += step) {
    const long long row = it / segs;
    const int k0 = static_cast<int>(it - row * segs) * 512 + lane * 16;
    Fp4Place pl;
    if (!place_of(a.r, s_off, row, pl)) continue;
    const bool on = k0 < a.K;
    long long from = row;
    if (a.pair_of_row != nullptr) {
      const int p = a.pair_of_row[row];
      from = (p >= 0 && p < a.T * a.k) ? p / a.k : -1;
    }
    uint32_t w[8], byte;
    load16(a.src + from * a.K + k0, on && from >= 0, w);
    const uint2 codes = quant16<NV>(w, tensor_scale(a.t, a.t_stride, pl.e), byte);
    store16<NV>(a, pl, row, k0, on, codes, join_bytes<NV>(byte));
  }
}

// A permute in token order: each token's values are read and quantised once.
// The items behind the tokens' look at 32 rows each for pad rows.
template <bool NV>
__global__ void __launch_bounds__(kThreads) tokens_kernel(const Fp4QuantArgs a) {
  extern __shared__ int s_off[];
  load_offsets(a.r, s_off, a.err);
  const int lane = threadIdx.x & 31;
  const int segs = (a.K + 511) / 512;
  const long long tokens = static_cast<long long>(a.T) * segs;
  const long long items = tokens + (a.r.rows + 31) / 32;
  const long long step = static_cast<long long>(gridDim.x) * kWarps;
  const int pairs = a.T * a.k;
  for (long long it = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5); it < items;
       it += step) {
    if (it < tokens) {
      const int t = static_cast<int>(it / segs);
      const int k0 = static_cast<int>(it - static_cast<long long>(t) * segs) * 512 + lane * 16;
      const bool on = k0 < a.K;
      uint32_t w[8], byte;
      load16(a.src + static_cast<long long>(t) * a.K + k0, on, w);
      uint2 codes = make_uint2(0u, 0u);
      uint32_t scales = 0u;
      bool done = false;
      for (int j0 = 0; j0 < a.k; j0 += 32) {
        // lane j finds the place of the token's pair j0 + j
        Fp4Place mine{0, 0, -1};
        int row = -1;
        if (j0 + lane < a.k) {
          const int p = t * a.k + j0 + lane;
          row = a.row_of_pair[p];
          if (row < 0 || row >= a.r.rows || a.pair_of_row[row] != p ||
              !place_of(a.r, s_off, row, mine))
            row = -1;
        }
        if (!done) {      // (a ragged tensor has one scale)
          codes = quant16<NV>(w, tensor_scale(a.t, 0, 0), byte);
          scales = join_bytes<NV>(byte);
          done = true;
        }
        const int n = min(32, a.k - j0);
        for (int j = 0; j < n; ++j) {
          const int to = __shfl_sync(kAll, row, j);
          Fp4Place pl;
          pl.off = __shfl_sync(kAll, mine.off, j);
          pl.tile0 = __shfl_sync(kAll, mine.tile0, j);
          if (to >= 0) store16<NV>(a, pl, to, k0, on, codes, scales);
        }
      }
    } else {
      const long long row0 = (it - tokens) * 32;
      const long long row = row0 + lane;
      bool pad = false;
      if (row < a.r.rows) {
        const int p = a.pair_of_row[row];
        pad = p < 0 || p >= pairs;
      }
      for (unsigned m = __ballot_sync(kAll, pad); m != 0; m &= m - 1) {
        const long long r = row0 + __ffs(m) - 1;
        Fp4Place pl;
        if (!place_of(a.r, s_off, r, pl)) continue;
        for (int k0 = lane * 16; k0 < a.K; k0 += 512)
          store16<NV>(a, pl, r, k0, true, make_uint2(0u, 0u), 0u);
      }
    }
  }
}

template <bool NV>
__global__ void __launch_bounds__(kThreads)
    columns_kernel(const uint16_t* __restrict__ W, int E, int R, int C, const float* __restrict__ t,
                   uint8_t* __restrict__ q, uint8_t* __restrict__ s) {
  const int lane = threadIdx.x & 31;
  const int rb = R / 64, cb = C / 64;
  const long long items = static_cast<long long>(E) * rb * cb;
  const long long step = static_cast<long long>(gridDim.x) * kWarps;
  const int chunks = fp4_chunks(NV, R);
  for (long long it = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5); it < items;
       it += step) {
    // neighbouring warps take neighbouring columns: whole rows of W together
    const int c64 = static_cast<int>(it % cb);
    const long long er = it / cb;
    const int r64 = static_cast<int>(er % rb), e = static_cast<int>(er / rb);
    const float ts = t == nullptr ? 1.f : t[e];
    const bool snap = NV && fp4_power_of_two(ts);
    const uint32_t* src = reinterpret_cast<const uint32_t*>(
        W + (static_cast<long long>(e) * R + r64 * 64) * C + c64 * 64) + lane;
    uint32_t w[64];
#pragma unroll
    for (int i = 0; i < 64; ++i) w[i] = __ldcs(src + static_cast<long long>(i) * (C / 2));
    const long long tile0 = fp4_tile0(static_cast<long long>(e) * C, e);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = c64 * 64 + 2 * lane + h;
      // column h of the lane as 32 words of pairs
      uint32_t p[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) p[i] = __byte_perm(w[2 * i], w[2 * i + 1], h ? 0x7632 : 0x5410);
      uint32_t codes[8], scales = 0;
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        uint32_t m = bf16_amax16(p + 8 * b);
        if constexpr (!NV) m = max(m, bf16_amax16(p + 8 * (b ^ 1)));
        float inv;
        const uint32_t byte = fp4_scale<NV>(m << 16, ts, inv);
        const uint2 u = fp4_codes16(p + 8 * b, inv, snap);
        codes[2 * b] = u.x;
        codes[2 * b + 1] = u.y;
        if constexpr (NV) scales |= byte << (8 * b);
        else if (b % 2 == 0) scales |= byte << (4 * b);
      }
      uint4* dst = reinterpret_cast<uint4*>(q + (static_cast<long long>(e) * C + c) * (R / 2) + r64 * 32);
      dst[0] = make_uint4(codes[0], codes[1], codes[2], codes[3]);
      dst[1] = make_uint4(codes[4], codes[5], codes[6], codes[7]);
      uint8_t* at = s + fp4_scale_at(tile0, c, r64 * (NV ? 4 : 2), chunks);
      if constexpr (NV) *reinterpret_cast<uint32_t*>(at) = scales;
      else *reinterpret_cast<uint16_t*>(at) = static_cast<uint16_t>(scales);
    }
  }
}

template <bool NV, bool F32>
__global__ void __launch_bounds__(kThreads)
    values_kernel(const uint8_t* __restrict__ q, const uint8_t* __restrict__ s, const Fp4Rows r,
                  int K, const float* __restrict__ t, int t_stride, void* __restrict__ out,
                  int32_t* err) {
  extern __shared__ int s_off[];
  load_offsets(r, s_off, err);
  const int lane = threadIdx.x & 31;
  const int segs = (K + 511) / 512;
  const int chunks = fp4_chunks(NV, K);
  const long long items = r.rows * segs;
  const long long step = static_cast<long long>(gridDim.x) * kWarps;
  for (long long it = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5); it < items;
       it += step) {
    const long long row = it / segs;
    const int k0 = static_cast<int>(it - row * segs) * 512 + lane * 16;
    Fp4Place pl;
    if (k0 >= K || !place_of(r, s_off, row, pl)) continue;
    const uint2 w = __ldcs(reinterpret_cast<const uint2*>(q + row * (K / 2) + k0 / 2));
    const uint32_t byte = s[fp4_scale_at(pl.tile0, row - pl.off, k0 / (NV ? 16 : 32), chunks)];
    // (code times block scale is exact, in bf16 too; a t that is no power of
    // two rounds the product once)
    float d;
    if constexpr (NV) d = e4m3_value(byte);
    else d = byte == 0xffu ? __uint_as_float(0x7fc00000u) : mx_scale(byte);
    const float ts = tensor_scale(t, t_stride, pl.e);
    float v[16];
    e2m1_values8(w.x, v);
    e2m1_values8(w.y, v + 8);
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = v[i] * d * ts;
    if constexpr (F32) {
      float4* o = reinterpret_cast<float4*>(static_cast<float*>(out) + row * K + k0);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        __stcs(o + i, make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]));
    } else {
      uint4* o = reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + row * K + k0);
#pragma unroll
      for (int i = 0; i < 2; ++i)
        __stcs(o + i, make_uint4(pack_bf16x2(v[8 * i], v[8 * i + 1]), pack_bf16x2(v[8 * i + 2], v[8 * i + 3]),
                                 pack_bf16x2(v[8 * i + 4], v[8 * i + 5]), pack_bf16x2(v[8 * i + 6], v[8 * i + 7])));
    }
  }
}

// largest finite magnitudes, as bits, by an integer maximum (whatever the
// order, the same result)
__global__ void __launch_bounds__(kThreads)
    amax_kernel(const uint4* __restrict__ src, long long n8, uint32_t* __restrict__ top) {
  const int e = blockIdx.y;
  const uint4* p = src + static_cast<long long>(e) * n8;
  uint32_t m = 0;
  const long long step = static_cast<long long>(gridDim.x) * kThreads;
  for (long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x; i < n8; i += step) {
    const uint4 u = p[i];
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t b = w[j] & 0x7fff7fffu;
      m = __vmaxu2(m, b & __vcmpltu2(b, 0x7f807f80u));
    }
  }
  m = __reduce_max_sync(kAll, max(m & 0xffffu, m >> 16));
  if ((threadIdx.x & 31) == 0 && m != 0) atomicMax(top + e, m << 16);
}

__global__ void power_kernel(float* t, int E) {
  const int e = blockIdx.x * blockDim.x + threadIdx.x;
  if (e >= E) return;
  const float top = t[e];
  float v = 1.f;
  if (top > 0.f) {
    // the power of two at or above top / 2688
    const uint32_t b = __float_as_uint(__fdiv_rn(top, 2688.f));
    uint32_t ex = (b >> 23) + ((b & 0x7fffffu) ? 1u : 0u);
    ex = min(max(ex, 1u), 254u);
    v = __uint_as_float(ex << 23);
  }
  t[e] = v;
}

int blocks_of(long long items, int num_sms) {
  const long long want = (items + kWarps - 1) / kWarps;
  const long long most = 8LL * num_sms;
  return static_cast<int>(want < most ? (want > 0 ? want : 1) : most);
}
size_t off_bytes(const Fp4Rows& r) { return r.offsets ? static_cast<size_t>(r.E + 1) * 4 : 0; }

}  // namespace

cudaError_t launch_fp4_quantize(const Fp4QuantArgs& a, int num_sms, cudaStream_t s) {
  const int segs = (a.K + 511) / 512;
  const size_t smem = off_bytes(a.r);
  if (a.row_of_pair != nullptr) {
    const long long items = static_cast<long long>(a.T) * segs + (a.r.rows + 31) / 32;
    const int b = blocks_of(items, num_sms);
    if (a.nv) tokens_kernel<true><<<b, kThreads, smem, s>>>(a);
    else tokens_kernel<false><<<b, kThreads, smem, s>>>(a);
  } else {
    const int b = blocks_of(a.r.rows * segs, num_sms);
    if (a.nv) rows_kernel<true><<<b, kThreads, smem, s>>>(a);
    else rows_kernel<false><<<b, kThreads, smem, s>>>(a);
  }
  return cudaGetLastError();
}

cudaError_t launch_fp4_quantize_t(const uint16_t* W, int E, int R, int C, bool nv, const float* t,
                                  uint8_t* q, uint8_t* s, int num_sms, cudaStream_t st) {
  const int b = blocks_of(static_cast<long long>(E) * (R / 64) * (C / 64), num_sms);
  if (nv) columns_kernel<true><<<b, kThreads, 0, st>>>(W, E, R, C, t, q, s);
  else columns_kernel<false><<<b, kThreads, 0, st>>>(W, E, R, C, t, q, s);
  return cudaGetLastError();
}

cudaError_t launch_fp4_dequantize(const uint8_t* q, const uint8_t* s, const Fp4Rows& r, int K,
                                  bool nv, const float* t, int t_stride, void* out, bool f32,
                                  int32_t* err, int num_sms, cudaStream_t st) {
  const int b = blocks_of(r.rows * ((K + 511) / 512), num_sms);
  const size_t smem = off_bytes(r);
  if (nv) {
    if (f32) values_kernel<true, true><<<b, kThreads, smem, st>>>(q, s, r, K, t, t_stride, out, err);
    else values_kernel<true, false><<<b, kThreads, smem, st>>>(q, s, r, K, t, t_stride, out, err);
  } else {
    if (f32) values_kernel<false, true><<<b, kThreads, smem, st>>>(q, s, r, K, t, t_stride, out, err);
    else values_kernel<false, false><<<b, kThreads, smem, st>>>(q, s, r, K, t, t_stride, out, err);
  }
  return cudaGetLastError();
}

cudaError_t launch_fp4_tensor_scale(const uint16_t* src, int E, long long n, float* t, int num_sms,
                                    cudaStream_t st, int* launches) {
  *launches = 0;
  cudaError_t e = cudaMemsetAsync(t, 0, static_cast<size_t>(E) * sizeof(float), st);
  if (e != cudaSuccess) return e;
  if (n > 0) {
    const long long want = (n / 8 + 4 * kThreads - 1) / (4 * kThreads);
    const long long most = (8LL * num_sms + E - 1) / E;
    const dim3 grid(static_cast<unsigned>(want < most ? want : most), E);
    amax_kernel<<<grid, kThreads, 0, st>>>(reinterpret_cast<const uint4*>(src), n / 8,
                                           reinterpret_cast<uint32_t*>(t));
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    ++*launches;
  }
  power_kernel<<<(E + 127) / 128, 128, 0, st>>>(t, E);
  ++*launches;
  return cudaGetLastError();
}

}  // namespace moe
