// fp4_quant.cu - quantisation to 4 bits and back (formats and scale layout in
// fp4.cuh).
//
// Rows are read once (2 bytes a value) and written once (0.5 bytes and the scale);
// rows, weights and the values read back are bound by HBM, the gather in token order
// by latency (35% of DRAM, 45% of the warps).  A thread takes 16 consecutive values (two 16-byte
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
constexpr int kTokenBlocks = 4;     // of tokens_kernel an SM, all resident
constexpr unsigned kAll = 0xffffffffu;

// The offsets made safe (clamped to [0, rows], by their running maximum) in
// shared memory, by the whole block; bad ones are reported by block 0.
__device__ __forceinline__ void load_offsets(const Fp4Rows& r, int* s_off, int32_t* err) {
  if (r.offsets == nullptr) return;
  for (int i = threadIdx.x; i <= r.E; i += kThreads) s_off[i] = r.offsets[i];
  __syncthreads();
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    bool bad = false;
    int top = 0;
    for (int base = 0; base <= r.E; base += 32) {
      const int i = base + lane;
      const int raw = i <= r.E ? s_off[i] : 0;
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
    if (r.E == 1) p.e = 0;
    else if (r.rows < (1LL << 31)) p.e = static_cast<int>(static_cast<uint32_t>(row) / static_cast<uint32_t>(r.rows_per_e));
    else p.e = static_cast<int>(row / r.rows_per_e);
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

// where a row's codes and its scales of block 0 begin
struct RowAt {
  long long q, s;
};
template <bool NV>
__device__ __forceinline__ RowAt row_at(const Fp4Place& pl, long long row, int K) {
  return RowAt{row * (K / 2), fp4_scale_at(pl.tile0, row - pl.off, 0, fp4_chunks(NV, K))};
}
// ... of the block that holds value k0 (a multiple of 64)
template <bool NV>
__device__ __forceinline__ long long scales_at(const RowAt& r, int k0) {
  if constexpr (NV) return r.s + static_cast<long long>(k0 / 64) * kFp4ChunkBytes;
  else return r.s + static_cast<long long>(k0 / 128) * kFp4ChunkBytes + (k0 / 32 & 3);
}

// A lane's 16 values (8 words) as codes and its scale byte (MX: the pair's)
template <bool NV>
__device__ __forceinline__ uint2 quant16(uint32_t (&p)[8], const Fp4Tensor& t, uint32_t& byte) {
  if constexpr (NV) fp4_shift(p, t);
  uint32_t m = bf16_amax16(p);
  if constexpr (!NV) m = max(m, __shfl_xor_sync(kAll, m, 1));
  float inv;
  byte = fp4_scale_bf16<NV>(m << 16, t, inv);
  return fp4_codes16<NV>(p, inv, t.exact);
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

// the codes and scales of values [k0, k0 + 16) of a row, by this lane
template <bool NV>
__device__ __forceinline__ void store16(const Fp4QuantArgs& a, const RowAt& r, int k0, bool on,
                                        uint2 codes, uint32_t scales) {
  if (!on) return;
  *reinterpret_cast<uint2*>(a.q + r.q + k0 / 2) = codes;
  if ((threadIdx.x & 3) == 0) {
    uint8_t* at = a.s + scales_at<NV>(r, k0);
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

constexpr int kSegs = 2;          // 512-value segments of a row that a warp takes, all loads first

// Rows in their own order; with pair_of_row, row r is token pair_of_row[r] / k
// (pad rows inside an expert: zeros).  Rows outside every expert are left.  A
// block's y is kSegs segments of K, its warps walk the rows.  (Six blocks an SM hold 40
// registers a thread: 32,768 x 7,168, NV, 124 us with the 48 it would take, 119 so.)
template <bool NV>
__global__ void __launch_bounds__(kThreads, 6) rows_kernel(const Fp4QuantArgs a) {
  extern __shared__ int s_off[];
  load_offsets(a.r, s_off, a.err);
  const int kb = blockIdx.y * (512 * kSegs) + (threadIdx.x & 31) * 16;
  const long long step = static_cast<long long>(gridDim.x) * kWarps;
  const int pairs = a.T * a.k;
  for (long long row = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
       row < a.r.rows; row += step) {
    Fp4Place pl;
    if (!place_of(a.r, s_off, row, pl)) continue;
    long long from = row;
    if (a.pair_of_row != nullptr) {
      const int p = a.pair_of_row[row];
      from = (p >= 0 && p < pairs) ? p / a.k : -1;
    }
    uint32_t w[kSegs][8];
#pragma unroll
    for (int g = 0; g < kSegs; ++g)
      load16(a.src + from * a.K + kb + 512 * g, kb + 512 * g < a.K && from >= 0, w[g]);
    const Fp4Tensor t = fp4_tensor(tensor_scale(a.t, a.t_stride, pl.e));
    const RowAt at = row_at<NV>(pl, row, a.K);
#pragma unroll
    for (int g = 0; g < kSegs; ++g) {
      uint32_t byte;
      const uint2 codes = quant16<NV>(w[g], t, byte);
      store16<NV>(a, at, kb + 512 * g, kb + 512 * g < a.K, codes, join_bytes<NV>(byte));
    }
  }
}

// A permute in token order: each token's values are read and quantised once.  The
// grid is what the device holds at once: every block reads the offsets first, and
// a warp looks up its next token's places while this one's values come (4096 x
// 7168, top-8: 68 us with four waves of blocks, 45.5 so; MX 49.6, 38.7).
template <bool NV>
__global__ void __launch_bounds__(kThreads, kTokenBlocks) tokens_kernel(const Fp4QuantArgs a) {
  extern __shared__ int s_off[];
  load_offsets(a.r, s_off, a.err);
  const int lane = threadIdx.x & 31;
  const long long step = static_cast<long long>(gridDim.x) * kWarps;
  const long long first = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int pairs = a.T * a.k;
  const int kb = blockIdx.y * (512 * kSegs) + lane * 16;
  const Fp4Tensor ts = fp4_tensor(tensor_scale(a.t, 0, 0));     // (a ragged tensor has one scale)
  // the place of pair j0 + lane of token t
  auto place = [&](long long t, int j0) {
    RowAt at{-1, 0};
    if (t < a.T && j0 + lane < a.k) {
      const int p = static_cast<int>(t) * a.k + j0 + lane;
      const int row = a.row_of_pair[p];
      Fp4Place pl;
      if (row >= 0 && row < a.r.rows && a.pair_of_row[row] == p && place_of(a.r, s_off, row, pl))
        at = row_at<NV>(pl, row, a.K);
    }
    return at;
  };
  RowAt next = place(first, 0);
  for (long long t = first; t < a.T; t += step) {
    uint32_t w[kSegs][8];
#pragma unroll
    for (int g = 0; g < kSegs; ++g)
      load16(a.src + t * a.K + kb + 512 * g, kb + 512 * g < a.K, w[g]);
    RowAt mine = next;
    next = place(t + step, 0);        // (its lookups run beside these loads)
    uint2 codes[kSegs];
    uint32_t scales[kSegs];
#pragma unroll
    for (int g = 0; g < kSegs; ++g) {
      uint32_t byte;
      codes[g] = quant16<NV>(w[g], ts, byte);
      scales[g] = join_bytes<NV>(byte);
    }
    for (int j0 = 0; j0 < a.k; j0 += 32) {
      if (j0 > 0) mine = place(t, j0);
      const int n = min(32, a.k - j0);
      for (int j = 0; j < n; ++j) {
        RowAt to;
        to.q = __shfl_sync(kAll, mine.q, j);
        to.s = __shfl_sync(kAll, mine.s, j);
        if (to.q < 0) continue;
#pragma unroll
        for (int g = 0; g < kSegs; ++g)
          store16<NV>(a, to, kb + 512 * g, kb + 512 * g < a.K, codes[g], scales[g]);
      }
    }
  }
  // pad rows: zeros, each by one of the grid's warps
  const long long all = step * gridDim.y;
  for (long long row0 = (blockIdx.y * step + first) * 32; row0 < a.r.rows; row0 += all * 32) {
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
      const RowAt at = row_at<NV>(pl, r, a.K);
      for (int k0 = lane * 16; k0 < a.K; k0 += 512)
        store16<NV>(a, at, k0, true, make_uint2(0u, 0u), 0u);
    }
  }
}

template <bool NV>
__global__ void __launch_bounds__(kThreads)
    columns_kernel(const uint16_t* __restrict__ W, int R, int C, const float* __restrict__ t,
                   uint8_t* __restrict__ q, uint8_t* __restrict__ s) {
  const int lane = threadIdx.x & 31;
  // neighbouring warps take neighbouring columns: whole rows of W together
  const int groups = (C / 64 + kWarps - 1) / kWarps;
  const int r64 = blockIdx.x / groups, e = blockIdx.y;
  const int c64 = (blockIdx.x - r64 * groups) * kWarps + (threadIdx.x >> 5);
  const int chunks = fp4_chunks(NV, R);
  if (c64 * 64 < C) {
    const Fp4Tensor ts = fp4_tensor(t == nullptr ? 1.f : t[e]);
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
      if constexpr (NV) fp4_shift(p, ts);
      uint32_t codes[8], scales = 0;
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        uint32_t m = bf16_amax16(p + 8 * b);
        if constexpr (!NV) m = max(m, bf16_amax16(p + 8 * (b ^ 1)));
        float inv;
        const uint32_t byte = fp4_scale_bf16<NV>(m << 16, ts, inv);
        const uint2 u = fp4_codes16<NV>(p + 8 * b, inv, ts.exact);
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

// The values read back.  A lane takes 8 values of every 256, so that a store of
// the warp is one run of 512 bytes (16 values a lane, 32 bytes in two stores of
// half sectors each: 32,768 x 8,192 148 us,
// now 116, 5.9 TB/s).
constexpr int kRuns = 4;          // 256-value runs of a row that a warp takes, all loads first
template <bool NV, bool F32>
__global__ void __launch_bounds__(kThreads)
    values_kernel(const uint8_t* __restrict__ q, const uint8_t* __restrict__ s, const Fp4Rows r,
                  int K, const float* __restrict__ t, int t_stride, void* __restrict__ out,
                  int32_t* err) {
  extern __shared__ int s_off[];
  load_offsets(r, s_off, err);
  const int kb = blockIdx.y * (256 * kRuns) + (threadIdx.x & 31) * 8;
  const long long step = static_cast<long long>(gridDim.x) * kWarps;
  for (long long row = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
       row < r.rows; row += step) {
    Fp4Place pl;
    if (!place_of(r, s_off, row, pl)) continue;
    const RowAt at = row_at<NV>(pl, row, K);
    const float ts = tensor_scale(t, t_stride, pl.e);
    uint32_t w[kRuns], byte[kRuns];
#pragma unroll
    for (int g = 0; g < kRuns; ++g) {
      const int k0 = kb + 256 * g;
      w[g] = byte[g] = 0u;
      if (k0 < K) {
        w[g] = __ldcs(reinterpret_cast<const uint32_t*>(q + at.q + k0 / 2));
        byte[g] = s[scales_at<NV>(at, k0 & ~63) + (NV ? (k0 / 16 & 3) : (k0 / 32 & 1))];
      }
    }
#pragma unroll
    for (int g = 0; g < kRuns; ++g) {
      const int k0 = kb + 256 * g;
      if (k0 >= K) continue;
      // (code times block scale is exact, in bf16 too; a t that is no power of
      // two rounds the product once)
      float d;
      if constexpr (NV) d = e4m3_value(byte[g]);
      else d = byte[g] == 0xffu ? __uint_as_float(0x7fc00000u) : mx_scale(byte[g]);
      float v[8];
      e2m1_values8(w[g], v);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = v[i] * d * ts;
      if constexpr (F32) {
        float4* o = reinterpret_cast<float4*>(static_cast<float*>(out) + row * K + k0);
        __stcs(o, make_float4(v[0], v[1], v[2], v[3]));
        __stcs(o + 1, make_float4(v[4], v[5], v[6], v[7]));
      } else {
        __stcs(reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + row * K + k0),
               make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                          pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])));
      }
    }
  }
}

// Largest finite magnitudes, as bits, by an integer maximum (whatever the order,
// the same result): of src[e], n8 times 8 values each, or with offsets of the
// experts' rows of row8 times 8 values alone (what lies behind them is not the
// call's).  One atomic a block: one a warp queued up at the word (67 MB that lay in
// L2 18.5 us).
__global__ void __launch_bounds__(kThreads)
    amax_kernel(const uint4* __restrict__ src, long long n8, const Fp4Rows r, int row8,
                uint32_t* __restrict__ top, int32_t* err) {
  const int e = blockIdx.y;
  const uint4* p = src + static_cast<long long>(e) * n8;
  __shared__ uint32_t s_top[kWarps];
  if (r.offsets != nullptr) {
    extern __shared__ int s_off[];
    load_offsets(r, s_off, err);
    p = src + static_cast<long long>(s_off[0]) * row8;
    n8 = static_cast<long long>(s_off[r.E] - s_off[0]) * row8;
  }
  uint32_t m = 0;
  const long long step = static_cast<long long>(gridDim.x) * kThreads;
  auto take = [&](const uint4& u) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t b = w[j] & 0x7fff7fffu;
      m = __vmaxu2(m, b & __vcmpltu2(b, 0x7f807f80u));
    }
  };
  long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
  for (; i + 3 * step < n8; i += 4 * step) {      // four loads in flight
    const uint4 u0 = p[i], u1 = p[i + step], u2 = p[i + 2 * step], u3 = p[i + 3 * step];
    take(u0);
    take(u1);
    take(u2);
    take(u3);
  }
  for (; i < n8; i += step) take(p[i]);
  m = __reduce_max_sync(kAll, max(m & 0xffffu, m >> 16));
  if ((threadIdx.x & 31) == 0) s_top[threadIdx.x >> 5] = m;
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int i = 1; i < kWarps; ++i) m = max(m, s_top[i]);
    if (m != 0) atomicMax(top + e, m << 16);
  }
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

// rows x the segments of K: blocks for every SM, each walking its rows (32 an SM and
// not 16: 32,768 x 7,168 over 256 experts 108 -> 101 us back, 126 -> 125 there)
dim3 grid_of(long long rows, int K, int num_sms) {
  const unsigned y = (K + 512 * kSegs - 1) / (512 * kSegs);
  const long long want = (rows + kWarps - 1) / kWarps;
  const long long most = (32LL * num_sms + y - 1) / y;
  return dim3(static_cast<unsigned>(want < 1 ? 1 : want < most ? want : most), y);
}
size_t off_bytes(const Fp4Rows& r) { return r.offsets ? static_cast<size_t>(r.E + 1) * 4 : 0; }

}  // namespace

cudaError_t launch_fp4_quantize(const Fp4QuantArgs& a, int num_sms, cudaStream_t s) {
  const size_t smem = off_bytes(a.r);
  if (a.row_of_pair != nullptr) {
    dim3 grid = grid_of(a.T, a.K, num_sms);
    const unsigned most = kTokenBlocks * num_sms / grid.y;
    if (grid.x > most) grid.x = most > 0 ? most : 1;
    if (a.nv) tokens_kernel<true><<<grid, kThreads, smem, s>>>(a);
    else tokens_kernel<false><<<grid, kThreads, smem, s>>>(a);
  } else {
    const dim3 grid = grid_of(a.r.rows, a.K, num_sms);
    if (a.nv) rows_kernel<true><<<grid, kThreads, smem, s>>>(a);
    else rows_kernel<false><<<grid, kThreads, smem, s>>>(a);
  }
  return cudaGetLastError();
}

cudaError_t launch_fp4_quantize_t(const uint16_t* W, int E, int R, int C, bool nv, const float* t,
                                  uint8_t* q, uint8_t* s, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>(R / 64) * ((C / 64 + kWarps - 1) / kWarps), E);
  if (nv) columns_kernel<true><<<grid, kThreads, 0, st>>>(W, R, C, t, q, s);
  else columns_kernel<false><<<grid, kThreads, 0, st>>>(W, R, C, t, q, s);
  return cudaGetLastError();
}

cudaError_t launch_fp4_dequantize(const uint8_t* q, const uint8_t* s, const Fp4Rows& r, int K,
                                  bool nv, const float* t, int t_stride, void* out, bool f32,
                                  int32_t* err, int num_sms, cudaStream_t st) {
  const dim3 b = grid_of(r.rows, K, num_sms);    // (256 * kRuns = 512 * kSegs)
  const size_t smem = off_bytes(r);
  static_assert(256 * kRuns == 512 * kSegs, "a block's part of a row");
  if (nv) {
    if (f32) values_kernel<true, true><<<b, kThreads, smem, st>>>(q, s, r, K, t, t_stride, out, err);
    else values_kernel<true, false><<<b, kThreads, smem, st>>>(q, s, r, K, t, t_stride, out, err);
  } else {
    if (f32) values_kernel<false, true><<<b, kThreads, smem, st>>>(q, s, r, K, t, t_stride, out, err);
    else values_kernel<false, false><<<b, kThreads, smem, st>>>(q, s, r, K, t, t_stride, out, err);
  }
  return cudaGetLastError();
}

cudaError_t launch_fp4_tensor_scale(const uint16_t* src, int E, long long n, const Fp4Rows& r,
                                    int K, float* t, int32_t* err, int num_sms, cudaStream_t st,
                                    int* launches) {
  *launches = 0;
  cudaError_t e = cudaMemsetAsync(t, 0, static_cast<size_t>(E) * sizeof(float), st);
  if (e != cudaSuccess) return e;
  if (n > 0) {
    const long long want = (n / 8 + 4 * kThreads - 1) / (4 * kThreads);
    const long long most = (8LL * num_sms + E - 1) / E;
    const dim3 grid(static_cast<unsigned>(want < most ? want : most), E);
    amax_kernel<<<grid, kThreads, off_bytes(r), st>>>(reinterpret_cast<const uint4*>(src), n / 8, r,
                                                      K / 8, reinterpret_cast<uint32_t*>(t), err);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    ++*launches;
  }
  ++*launches;
  return launch_fp4_power(t, E, st);
}

cudaError_t launch_fp4_power(float* t, int E, cudaStream_t st) {
  power_kernel<<<(E + 127) / 128, 128, 0, st>>>(t, E);
  return cudaGetLastError();
}

}  // namespace moe
