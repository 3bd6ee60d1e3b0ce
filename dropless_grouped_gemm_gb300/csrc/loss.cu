// loss.cu - the router's auxiliary losses and its gradient.
//
// With P_te = softmax over all E logits of token t, lse_t its log-sum-exp,
// c_se the pairs of segment s routed to expert e, N_s its valid tokens and
// N = sum N_s:
//   balance = E / (k N) sum_s (1 / N_s) sum_e c_se sum_{t in s} P_te
//   z       = 1 / N sum_t lse_t^2
// (1.0 and the mean squared log-partition; a balanced router gives 1).
// Gradient, with g = dloss and w_se = g0 E c_se / (k N N_s):
//   dz_te = P_te (w_se - sum_e' P_te' w_se' + 2 g1 lse_t / N)
//           + sum_{j: idx_tj = e} p_tj (dp_tj - sum_i p_ti dp_ti)
// the last line being the softmax over the k selected logits that
// moe_router_topk writes.
//
// Forward, two kernels.  loss_rows: a block takes one unit, up to `chunk`
// consecutive tokens of one segment, a warp per token; each lane keeps the
// sums of P of its experts in registers over the warp's tokens, the block
// adds its warps' sums in warp order and writes one partial row per unit, so
// that no order depends on timing.  loss_finish: adds the units of each
// segment in order (32 experts x 32 unit lanes per block); the block that
// finishes last adds the blocks' terms in order.  Backward: one kernel, a
// warp per token, which reads each logit once and writes its gradient.
// All three are bound by HBM on long batches and by launch latency on short
// ones.
#include <cuda_bf16.h>

#include "loss.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kFinishThreads = 1024;

struct Ws {
  float* psum;     // [units, E] sums of P
  int32_t* pcnt;   // [units, E] pairs
  float* pz;       // [units] sums of lse^2
  int32_t* pn;     // [units] valid tokens
  float* term;     // [S, slices] sum_e c S / N_s of a slice of experts
  int32_t* ticket;
};

// Tokens per unit: whole rounds of the block's warps, about two units for
// each of a GB300's 152 SMs (a constant, so that the workspace size and the
// order of the sums do not depend on the device queried).
constexpr int kUnits = 304;
int chunk_of(int T) {
  const int per = (T + kUnits - 1) / kUnits;
  const int c = (per + kWarps - 1) / kWarps * kWarps;
  return c < kWarps ? kWarps : c;
}
int units_cap(int T, int S) {
  const int c = chunk_of(T);
  return (T + c - 1) / c + S + 1;
}
int slices_of(int E) { return (E + 31) / 32; }

size_t up16(size_t b) { return (b + 15) & ~static_cast<size_t>(15); }

Ws carve(void* base, int T, int E, int S, size_t* bytes) {
  const size_t U = static_cast<size_t>(units_cap(T, S));
  uint8_t* p = static_cast<uint8_t*>(base);
  size_t at = 0;
  auto take = [&](size_t b) {
    uint8_t* q = p ? p + at : nullptr;
    at += up16(b);
    return q;
  };
  Ws w;
  w.psum = reinterpret_cast<float*>(take(U * E * 4));
  w.pcnt = reinterpret_cast<int32_t*>(take(U * E * 4));
  w.pz = reinterpret_cast<float*>(take(U * 4));
  w.pn = reinterpret_cast<int32_t*>(take(U * 4));
  w.term = reinterpret_cast<float*>(take(static_cast<size_t>(S) * slices_of(E) * 4));
  w.ticket = reinterpret_cast<int32_t*>(take(4));
  *bytes = at;
  return w;
}

// One segment's place: its tokens [lo, hi) and its first unit.  Segment S
// stands for the tokens after the last segment (never valid).
struct Span {
  int s, lo, hi, unit0;
};

// Walks the segments 32 at a time (one warp): start offsets clamped to
// [0, T] and made non-decreasing, units counted; calls at(lane's span) for
// every segment until one lane returns true, and hands that span to all
// lanes.  bad is set where the offsets had to be corrected.
template <class Pred>
__device__ __forceinline__ bool walk_segments(const int32_t* __restrict__ seg, int S, int T,
                                              int chunk, bool& bad, Span& out, Pred pred) {
  const int lane = threadIdx.x & 31;
  int start_carry = 0, unit_carry = 0;
  for (int base = 0; base <= S; base += 32) {
    const int s = base + lane;
    // segment s begins at seg[s] (segment 0 at 0; S: the tail) and ends
    // where segment s + 1 begins
    int v = 0;
    if (s <= S && seg != nullptr) {
      v = seg[s];
      if (v < 0 || v > T || (s == 0 && v != 0)) bad = true;
      v = (s == 0) ? 0 : min(max(v, 0), T);
    } else if (seg == nullptr && s == 1) {
      v = T;
    }
    int m = max(v, start_carry);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, m, o);
      if (lane >= o) m = max(m, y);
    }
    if (s <= S && m != v) bad = true;
    // the next segment's start: the next lane's, or the first of the next 32
    int nv = __shfl_down_sync(0xffffffffu, m, 1);
    if (lane == 31) {
      const int s1 = s + 1;
      nv = m;
      if (s1 <= S && seg != nullptr) nv = max(m, min(max(seg[s1], 0), T));
    }
    if (s == S) nv = T;
    const int u = (s <= S) ? (nv - m + chunk - 1) / chunk : 0;
    int incl = u;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    Span sp{s, m, nv, unit_carry + incl - u};
    const bool hit = s <= S && pred(sp, u);
    const unsigned b = __ballot_sync(0xffffffffu, hit);
    if (b != 0) {
      const int l = __ffs(b) - 1;
      out.s = __shfl_sync(0xffffffffu, sp.s, l);
      out.lo = __shfl_sync(0xffffffffu, sp.lo, l);
      out.hi = __shfl_sync(0xffffffffu, sp.hi, l);
      out.unit0 = __shfl_sync(0xffffffffu, sp.unit0, l);
      return true;
    }
    start_carry = __shfl_sync(0xffffffffu, m, 31);
    unit_carry += __shfl_sync(0xffffffffu, incl, 31);
  }
  return false;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// A lane's logits of one row: NV values in groups of VEC consecutive ones;
// value i is expert (lane + 32 (i / VEC)) * VEC + i % VEC.  Missing ones are
// -inf.
template <int VEC>
__device__ __forceinline__ int expert_of(int lane, int i) {
  return (lane + 32 * (i / VEC)) * VEC + i % VEC;
}
template <class T, int VEC, int NV>
__device__ __forceinline__ void load_row(const T* __restrict__ row, int E, int lane,
                                         float (&v)[NV]) {
#pragma unroll
  for (int g = 0; g < NV / VEC; ++g) {
    const int e0 = (lane + 32 * g) * VEC;
    if constexpr (VEC == 1) {
      v[g] = -INFINITY;
      if (e0 < E) {
        if constexpr (sizeof(T) == 4) v[g] = row[e0];
        else v[g] = __uint_as_float(static_cast<uint32_t>(row[e0]) << 16);
      }
    } else if (e0 < E) {   // E is a multiple of VEC here
      const uint4 w = *reinterpret_cast<const uint4*>(row + e0);
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
      if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[g * VEC + j] = __uint_as_float(u[j]);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[g * VEC + 2 * j] = bf16_lo(u[j]);
          v[g * VEC + 2 * j + 1] = bf16_hi(u[j]);
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[g * VEC + j] = -INFINITY;
    }
  }
}

// the lowest finite value of the logits' type
template <class T>
__device__ __forceinline__ float lowest() {
  return __uint_as_float(sizeof(T) == 4 ? 0xFF7FFFFFu : 0xFF7F0000u);
}

template <class T, int VEC, int NV>
__global__ void __launch_bounds__(kThreads) loss_rows(const RouterLossArgs a, const Ws w,
                                                      int chunk) {
  extern __shared__ float sm[];             // [kWarps][E] sums, then [E] counts
  int32_t* hist = reinterpret_cast<int32_t*>(sm + kWarps * a.E);
  __shared__ Span s_span;
  __shared__ int s_have;
  __shared__ float s_z[kWarps];
  __shared__ int s_n[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (blockIdx.x == 0 && threadIdx.x == 0) *w.ticket = 0;
  for (int e = threadIdx.x; e < a.E; e += kThreads) hist[e] = 0;
  if (warp == 0) {
    Span sp{0, 0, 0, 0};
    bool bad = false;
    const int u = blockIdx.x;
    const bool have = walk_segments(a.seg, a.S, a.T, chunk, bad, sp, [&](const Span& x, int n) {
      return u >= x.unit0 && u < x.unit0 + n;
    });
    if (lane == 0) {
      s_span = sp;
      s_have = have;
    }
    // the last block of the grid is past every unit, so it walks them all
    if (bad && blockIdx.x == gridDim.x - 1) set_err(a.err, MOE_DEV_BAD_OFFSETS);
  }
  __syncthreads();
  if (!s_have) return;
  const Span sp = s_span;
  const bool seg_ok = sp.s < a.S;
  const int t0 = sp.lo + (blockIdx.x - sp.unit0) * chunk;
  const int t1 = min(t0 + chunk, sp.hi);
  float acc[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) acc[i] = 0.f;
  float zsum = 0.f;
  int nval = 0;
  bool bad_id = false;
  const T* logits = static_cast<const T*>(a.logits);
  for (int t = t0 + warp; t < t1; t += kWarps) {
    float v[NV];
    load_row<T, VEC, NV>(logits + static_cast<long long>(t) * a.E, a.E, lane, v);
    float m = v[0];
#pragma unroll
    for (int i = 1; i < NV; ++i) m = fmaxf(m, v[i]);
    m = warp_max(m);
    float tot = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      v[i] = (v[i] == -INFINITY) ? 0.f : expf(v[i] - m);
      tot += v[i];
    }
    tot = warp_sum(tot);
    // a row that a mask of -inf or of the type's lowest value has emptied
    // has no weight at all (its lse^2 would overflow); NaN goes through
    const float lse = (m <= lowest<T>() && tot == tot) ? -INFINITY : m + logf(tot);
    if (lane == 0) a.lse[t] = lse;
    const bool valid = seg_ok && (a.mask == nullptr || a.mask[t] != 0) && !(lse == -INFINITY);
    if (valid) {
      const float inv = 1.0f / tot;
#pragma unroll
      for (int i = 0; i < NV; ++i) acc[i] += v[i] * inv;
      zsum += lse * lse;
      ++nval;
      for (int j = lane; j < a.k; j += 32) {
        const int e = a.idx[static_cast<long long>(t) * a.k + j];
        if (e >= 0 && e < a.E) atomicAdd(&hist[e], 1);
        else if (e != -1) bad_id = true;
      }
    }
  }
  if (__any_sync(0xffffffffu, bad_id) && lane == 0) set_err(a.err, MOE_DEV_BAD_EXPERT);
  if (!seg_ok) return;    // the tail's tokens count nowhere
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = expert_of<VEC>(lane, i);
    if (e < a.E) sm[warp * a.E + e] = acc[i];
  }
  if (lane == 0) {
    s_z[warp] = zsum;
    s_n[warp] = nval;
  }
  __syncthreads();
  const long long row = static_cast<long long>(blockIdx.x) * a.E;
  for (int e = threadIdx.x; e < a.E; e += kThreads) {
    float x = sm[e];
#pragma unroll
    for (int q = 1; q < kWarps; ++q) x += sm[q * a.E + e];
    w.psum[row + e] = x;
    w.pcnt[row + e] = hist[e];
  }
  if (threadIdx.x == 0) {
    float z = 0.f;
    int n = 0;
    for (int q = 0; q < kWarps; ++q) {
      z += s_z[q];
      n += s_n[q];
    }
    w.pz[blockIdx.x] = z;
    w.pn[blockIdx.x] = n;
  }
}

// block (slice, segment): 32 experts x 32 unit lanes
__global__ void __launch_bounds__(kFinishThreads) loss_finish(const RouterLossArgs a, const Ws w,
                                                              int chunk) {
  __shared__ Span s_span;
  __shared__ float s_sum[32][33];
  __shared__ int s_cnt[32][33];
  __shared__ int s_last, s_nseg;
  const int lane = threadIdx.x & 31, grp = threadIdx.x >> 5;
  const int s = blockIdx.y;
  const int e = blockIdx.x * 32 + lane;
  if (grp == 0) {
    Span sp{0, 0, 0, 0};
    bool bad = false;
    walk_segments(a.seg, a.S, a.T, chunk, bad, sp, [&](const Span& x, int) { return x.s == s; });
    const int n_units = (sp.hi - sp.lo + chunk - 1) / chunk;
    int n = 0;
    for (int u = lane; u < n_units; u += 32) n += w.pn[sp.unit0 + u];
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0) {
      s_span = sp;
      s_nseg = n;
      if (blockIdx.x == 0) a.n_valid[s] = n;
    }
  }
  __syncthreads();
  const Span sp = s_span;
  const int n_units = (sp.hi - sp.lo + chunk - 1) / chunk;
  float x = 0.f;
  int c = 0;
  if (e < a.E) {
    for (int u = grp; u < n_units; u += 32) {
      const long long at = static_cast<long long>(sp.unit0 + u) * a.E + e;
      x += w.psum[at];
      c += w.pcnt[at];
    }
  }
  s_sum[grp][lane] = x;
  s_cnt[grp][lane] = c;
  __syncthreads();
  if (grp == 0) {
    float y = 0.f;
    int d = 0;
#pragma unroll
    for (int q = 0; q < 32; ++q) {
      y += s_sum[q][lane];
      d += s_cnt[q][lane];
    }
    if (e < a.E) a.counts[static_cast<long long>(s) * a.E + e] = d;
    float t = (e < a.E && s_nseg > 0) ? static_cast<float>(d) * (y / static_cast<float>(s_nseg)) : 0.f;
    t = warp_sum(t);
    if (lane == 0) {
      w.term[static_cast<long long>(s) * gridDim.x + blockIdx.x] = t;
      __threadfence();
      s_last = atomicAdd(w.ticket, 1) == static_cast<int>(gridDim.x * gridDim.y) - 1;
    }
  }
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  // the last block: every thread adds a strided part, then a tree
  const int terms = gridDim.x * gridDim.y;
  // units of the segments come first; the tail's, after them, count nowhere
  if (grp == 0) {
    Span tail{0, 0, 0, 0};
    bool bad = false;
    walk_segments(a.seg, a.S, a.T, chunk, bad, tail, [&](const Span& q, int) { return q.s == a.S; });
    if (lane == 0) s_span = tail;
  }
  __syncthreads();
  const int units = s_span.unit0;
  float b = 0.f, z = 0.f;
  int n = 0;
  const volatile float* term = w.term;
  for (int i = threadIdx.x; i < terms; i += kFinishThreads) b += term[i];
  for (int i = threadIdx.x; i < units; i += kFinishThreads) {
    z += w.pz[i];
    n += w.pn[i];
  }
  b = warp_sum(b);
  z = warp_sum(z);
  n = __reduce_add_sync(0xffffffffu, n);
  if (lane == 0) {
    s_sum[0][grp] = b;
    s_sum[1][grp] = z;
    s_cnt[0][grp] = n;
  }
  __syncthreads();
  if (grp == 0) {
    b = warp_sum(s_sum[0][lane]);
    z = warp_sum(s_sum[1][lane]);
    n = __reduce_add_sync(0xffffffffu, s_cnt[0][lane]);
    if (lane == 0) {
      const float N = static_cast<float>(n);
      a.loss[0] = n > 0 ? b * (static_cast<float>(a.E) / (static_cast<float>(a.k) * N)) : 0.f;
      a.loss[1] = n > 0 ? z / N : 0.f;
    }
  }
}

// largest s in [0, S] with start(s) <= t; seg may hold any values, so the
// search is bounded by its index range alone
__device__ __forceinline__ int segment_of(const int32_t* __restrict__ seg, int S, int t) {
  if (seg == nullptr) return 0;
  int lo = 0, hi = S;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (seg[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

template <class T, int VEC, int NV>
__global__ void __launch_bounds__(kThreads) loss_bwd(const RouterLossArgs a, int per_warp) {
  __shared__ int s_part[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int n = 0;
  for (int s = threadIdx.x; s < a.S; s += kThreads) n += a.n_valid[s];
  n = __reduce_add_sync(0xffffffffu, n);
  if (lane == 0) s_part[warp] = n;
  __syncthreads();
  n = 0;
#pragma unroll
  for (int q = 0; q < kWarps; ++q) n += s_part[q];
  const float inv_n = n > 0 ? 1.0f / static_cast<float>(n) : 0.f;
  const float gz = 2.f * a.dloss[1] * inv_n;
  const float gb = a.dloss[0] * static_cast<float>(a.E) / static_cast<float>(a.k) * inv_n;
  const long long first = (static_cast<long long>(blockIdx.x) * kWarps + warp) * per_warp;
  const int t1 = static_cast<int>(min(first + per_warp, static_cast<long long>(a.T)));
  const T* logits = static_cast<const T*>(a.logits);
  float wv[NV];
  int cur = -1;
  for (int t = static_cast<int>(min(first, static_cast<long long>(a.T))); t < t1; ++t) {
    const int s = segment_of(a.seg, a.S, t);
    if (s != cur) {
      cur = s;
      const int ns = s < a.S ? a.n_valid[s] : 0;
      const float f = ns > 0 ? gb / static_cast<float>(ns) : 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int e = expert_of<VEC>(lane, i);
        wv[i] = (s < a.S && e < a.E)
                    ? f * static_cast<float>(a.counts[static_cast<long long>(s) * a.E + e]) : 0.f;
      }
    }
    const long long row = static_cast<long long>(t) * a.E;
    float v[NV];
    load_row<T, VEC, NV>(logits + row, a.E, lane, v);
    const float lse = a.lse[t];
    const bool valid = s < a.S && (a.mask == nullptr || a.mask[t] != 0) && !(lse == -INFINITY);
    if (valid) {
      float dot = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        v[i] = (v[i] == -INFINITY) ? 0.f : expf(v[i] - lse);
        dot += v[i] * wv[i];
      }
      dot = warp_sum(dot) - gz * lse;
#pragma unroll
      for (int i = 0; i < NV; ++i) v[i] *= wv[i] - dot;
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) v[i] = 0.f;
    }
    if (a.probs != nullptr) {
      const long long p0 = static_cast<long long>(t) * a.k;
      float pd = 0.f;
      for (int j = lane; j < a.k; j += 32) {
        const int e = a.idx[p0 + j];
        if (e >= 0 && e < a.E) pd += a.probs[p0 + j] * a.dprobs[p0 + j];
      }
      pd = warp_sum(pd);
      for (int j0 = 0; j0 < a.k; j0 += 32) {
        int e = -1;
        float r = 0.f;
        if (j0 + lane < a.k) {
          e = a.idx[p0 + j0 + lane];
          r = a.probs[p0 + j0 + lane] * (a.dprobs[p0 + j0 + lane] - pd);
        }
        const int jn = min(32, a.k - j0);
        for (int j = 0; j < jn; ++j) {
          const int ej = __shfl_sync(0xffffffffu, e, j);
          const float rj = __shfl_sync(0xffffffffu, r, j);
#pragma unroll
          for (int i = 0; i < NV; ++i)
            if (expert_of<VEC>(lane, i) == ej) v[i] += rj;
        }
      }
    }
#pragma unroll
    for (int g = 0; g < NV / VEC; ++g) {
      const int e0 = (lane + 32 * g) * VEC;
      if (e0 >= a.E) continue;
      if (a.dlogits_bf16) {
        uint16_t* o = static_cast<uint16_t*>(a.dlogits) + row + e0;
        if constexpr (VEC == 8) {
          *reinterpret_cast<uint4*>(o) =
              make_uint4(pack_bf16x2(v[g * 8], v[g * 8 + 1]), pack_bf16x2(v[g * 8 + 2], v[g * 8 + 3]),
                         pack_bf16x2(v[g * 8 + 4], v[g * 8 + 5]), pack_bf16x2(v[g * 8 + 6], v[g * 8 + 7]));
        } else if constexpr (VEC == 4) {
          *reinterpret_cast<uint2*>(o) =
              make_uint2(pack_bf16x2(v[g * 4], v[g * 4 + 1]), pack_bf16x2(v[g * 4 + 2], v[g * 4 + 3]));
        } else {
          *o = static_cast<uint16_t>(pack_bf16x2(v[g], 0.f) & 0xffffu);
        }
      } else {
        float* o = static_cast<float*>(a.dlogits) + row + e0;
        if constexpr (VEC == 1) {
          *o = v[g];
        } else {
#pragma unroll
          for (int q = 0; q < VEC / 4; ++q)
            *reinterpret_cast<float4*>(o + 4 * q) =
                make_float4(v[g * VEC + 4 * q], v[g * VEC + 4 * q + 1], v[g * VEC + 4 * q + 2],
                            v[g * VEC + 4 * q + 3]);
        }
      }
    }
  }
}

template <class T, int VEC, int NV>
cudaError_t go(const RouterLossArgs& a, int num_sms, cudaStream_t s, bool bwd, int chunk,
               const Ws& w) {
  if (bwd) {
    // consecutive tokens of a warp share their segment's weights: eight at
    // most, fewer while the SMs are not full
    int per = (a.T + num_sms * 4 * kWarps - 1) / (num_sms * 4 * kWarps);
    per = per < 1 ? 1 : (per > 8 ? 8 : per);
    const long long blocks = (static_cast<long long>(a.T) + per * kWarps - 1) / (per * kWarps);
    loss_bwd<T, VEC, NV><<<static_cast<int>(blocks), kThreads, 0, s>>>(a, per);
  } else {
    const size_t smem = static_cast<size_t>(kWarps + 1) * a.E * 4;   // at most 36 KB
    loss_rows<T, VEC, NV><<<units_cap(a.T, a.S), kThreads, smem, s>>>(a, w, chunk);
  }
  return cudaGetLastError();
}

// values per lane: the smallest instance that covers E
template <class T, int VEC>
cudaError_t pick(const RouterLossArgs& a, int num_sms, cudaStream_t s, bool bwd, int chunk,
                 const Ws& w) {
  const int groups = (a.E + 32 * VEC - 1) / (32 * VEC);
  if constexpr (VEC == 1) {
    if (groups <= 1) return go<T, VEC, 1>(a, num_sms, s, bwd, chunk, w);
    if (groups <= 2) return go<T, VEC, 2>(a, num_sms, s, bwd, chunk, w);
    if (groups <= 4) return go<T, VEC, 4>(a, num_sms, s, bwd, chunk, w);
    if (groups <= 8) return go<T, VEC, 8>(a, num_sms, s, bwd, chunk, w);
    if (groups <= 16) return go<T, VEC, 16>(a, num_sms, s, bwd, chunk, w);
    return go<T, VEC, 32>(a, num_sms, s, bwd, chunk, w);
  } else {
    if (groups * VEC <= 4) return go<T, VEC, VEC>(a, num_sms, s, bwd, chunk, w);
    if (groups * VEC <= 8) return go<T, VEC, 8>(a, num_sms, s, bwd, chunk, w);
    if (groups * VEC <= 16) return go<T, VEC, 16>(a, num_sms, s, bwd, chunk, w);
    return go<T, VEC, 32>(a, num_sms, s, bwd, chunk, w);
  }
}

cudaError_t dispatch(const RouterLossArgs& a, int num_sms, cudaStream_t s, bool bwd, int chunk,
                     const Ws& w) {
  // 16-byte loads need whole 16-byte groups in every row
  if (a.logits_bf16)
    return a.E % 8 == 0 ? pick<uint16_t, 8>(a, num_sms, s, bwd, chunk, w)
                        : pick<uint16_t, 1>(a, num_sms, s, bwd, chunk, w);
  return a.E % 4 == 0 ? pick<float, 4>(a, num_sms, s, bwd, chunk, w)
                      : pick<float, 1>(a, num_sms, s, bwd, chunk, w);
}

}  // namespace

size_t router_loss_workspace_bytes(int T, int E, int S) {
  size_t b = 0;
  carve(nullptr, T, E, S, &b);
  return b;
}

cudaError_t launch_router_loss(const RouterLossArgs& a, int num_sms, cudaStream_t s,
                               int* launches) {
  size_t bytes = 0;
  const Ws w = carve(a.ws, a.T, a.E, a.S, &bytes);
  const int chunk = chunk_of(a.T);
  *launches = 0;
  const cudaError_t e = dispatch(a, num_sms, s, false, chunk, w);
  if (e != cudaSuccess) return e;
  loss_finish<<<dim3(slices_of(a.E), a.S), kFinishThreads, 0, s>>>(a, w, chunk);
  *launches = 2;
  return cudaGetLastError();
}

cudaError_t launch_router_loss_bwd(const RouterLossArgs& a, int num_sms, cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
  return dispatch(a, num_sms, s, true, 0, Ws{});
}

}  // namespace moe
