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
// consecutive tokens of one segment.  A group of L lanes (4 to 32, so that
// each holds 8 to 32 logits) takes a token and keeps the sums of P of its
// experts in registers over its tokens; the block adds its groups' sums in a
// fixed order and writes one partial row per unit, so that no order depends
// on timing.  loss_finish, launched programmatically behind it: adds the
// units of each segment in order (a block per segment and slice of experts);
// the block that finishes last adds the blocks' terms in order.  Backward:
// one kernel, a group of lanes per token, which reads each logit once and
// writes its gradient.
// All are bound by HBM on long batches and by launch latency on short ones.
#include <cuda_bf16.h>

#include "loss.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kBwdThreads = 256;

struct Ws {
  float* psum;     // [units, E] sums of P
  int32_t* pcnt;   // [units, E] pairs
  float* pz;       // [units] sums of lse^2
  int32_t* pn;     // [units] valid tokens
  float* term;     // [S, slices] sum_e c S / N_s of a slice of experts
  float* zseg;     // [S] sums of lse^2
  int32_t* ticket;
};

// Tokens per unit: about one unit (a block of 16 warps) for each of the 304
// places that 152 SMs have at two blocks each, a few left for segments that
// end inside a unit (a constant, so that the workspace size and the order of
// the sums do not depend on the device queried).  65,536 tokens x 256 experts
// in 16 sequences, forward as a whole: 22.0 us, against 25.9 with 440 units,
// whose second wave is short.
constexpr int kUnits = 300;
int chunk_of(int T) {
  const int per = (T + kUnits - 1) / kUnits;
  const int c = (per + 15) / 16 * 16;
  return c < 16 ? 16 : c;
}
int units_cap(int T, int S) {
  const int c = chunk_of(T);
  return (T + c - 1) / c + S + 1;
}
// experts per block of loss_finish
int finish_experts(int S) { return S < 4 ? 8 : 32; }
int slices_of(int E, int S) { return (E + finish_experts(S) - 1) / finish_experts(S); }

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
  w.term = reinterpret_cast<float*>(take(static_cast<size_t>(S) * slices_of(E, S) * 4));
  w.zseg = reinterpret_cast<float*>(take(static_cast<size_t>(S) * 4));
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
// sums and maxima over the L lanes of a group
template <int L>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
template <int L>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// A lane's logits of one row: NV values in groups of VEC consecutive ones;
// value i of lane l of its group is expert (l + L (i / VEC)) * VEC + i % VEC.
// Missing ones are -inf.
template <int VEC, int L>
__device__ __forceinline__ int expert_of(int l, int i) {
  return (l + L * (i / VEC)) * VEC + i % VEC;
}
template <class T, int VEC, int NV, int L>
__device__ __forceinline__ void load_row(const T* __restrict__ row, int E, int l, bool ok,
                                         float (&v)[NV]) {
#pragma unroll
  for (int g = 0; g < NV / VEC; ++g) {
    const int e0 = (l + L * g) * VEC;
    if constexpr (VEC == 1) {
      v[g] = -INFINITY;
      if (ok && e0 < E) {
        if constexpr (sizeof(T) == 4) v[g] = __ldcs(row + e0);
        else v[g] = __uint_as_float(static_cast<uint32_t>(__ldcs(row + e0)) << 16);
      }
    } else if (ok && e0 < E) {   // E is a multiple of VEC here
      const uint4 w = __ldcs(reinterpret_cast<const uint4*>(row + e0));
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

// The softmax in base 2: e^(z - m) = 2^((z - m) log2 e), the subtraction
// first: it is exact where z and m are close, so that a row's offset, however
// large, costs nothing (m log2 e, rounded, is off by 64 at m = 1e9 and past
// float32 at 3e38).  lse = m + ln sum, rounded once.
constexpr float kLog2E = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
__device__ __forceinline__ float exp2_(float x) {
  float y;
  asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Nothing at or below bf16's lowest finite value counts as a logit (float32's
// lowest is below it): masks use either, on rows of either type.
constexpr float kLowest = -3.3895313892515355e38f;

template <class T, int VEC, int NV, int L, int W>
__global__ void __launch_bounds__(32 * W, NV <= 16 ? 2 : 1) loss_rows(const RouterLossArgs a, const Ws w, int chunk) {
  constexpr int G = 32 / L;                 // tokens of a warp at a time
  extern __shared__ float sm[];             // [W][E] sums, then [E] counts
  int32_t* hist = reinterpret_cast<int32_t*>(sm + W * a.E);
  __shared__ Span s_span;
  __shared__ int s_have;
  __shared__ float s_z[W];
  __shared__ int s_n[W];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int l = lane % L, grp = lane / L;
  if (blockIdx.x == 0 && threadIdx.x == 0) *w.ticket = 0;
  for (int e = threadIdx.x; e < a.E; e += 32 * W) hist[e] = 0;
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
  // a round is G tokens of each warp.  Loads are not staged ahead: with 32
  // warps an SM, one warp's wait is covered by the others' arithmetic
  for (int tw = t0 + warp * G; tw < t1; tw += W * G) {
    const int t = tw + grp;
    const bool have = t < t1;
    float v[NV];
    load_row<T, VEC, NV, L>(logits + static_cast<long long>(t) * a.E, a.E, l, have, v);
    const long long p0 = static_cast<long long>(t) * a.k;
    int e0 = -1;
    if (have && l < a.k) e0 = a.idx[p0 + l];
    bool on = have && seg_ok;
    if (on && a.mask != nullptr) on = a.mask[t] != 0;
    float m = v[0];
#pragma unroll
    for (int i = 1; i < NV; ++i) m = fmaxf(m, v[i]);
    m = group_max<L>(m);
    // a row that a mask of -inf or of a type's lowest value has emptied
    // has no weight at all (its lse^2 would overflow): with m = 0 every term
    // is 0 and lse = log 0; NaN goes through
    if (m <= kLowest) m = 0.f;
    float tot = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      v[i] = exp2_((v[i] - m) * kLog2E);
      tot += v[i];
    }
    tot = group_sum<L>(tot);
    const float lse = fmaf(log2f(tot), kLn2, m);
    if (have && l == 0) a.lse[t] = lse;
    if (on && !(lse == -INFINITY)) {
      const float inv = __fdividef(1.0f, tot);
#pragma unroll
      for (int i = 0; i < NV; ++i) acc[i] = fmaf(v[i], inv, acc[i]);
      if (l == 0) {
        zsum = fmaf(lse, lse, zsum);
        ++nval;
      }
      if (e0 >= 0 && e0 < a.E) atomicAdd(&hist[e0], 1);
      else if (e0 != -1) bad_id = true;
      for (int j = l + L; j < a.k; j += L) {
        const int e = a.idx[p0 + j];
        if (e >= 0 && e < a.E) atomicAdd(&hist[e], 1);
        else if (e != -1) bad_id = true;
      }
    }
  }
  // loss_finish may come in once every block is here (it waits for this grid
  // to end; earlier its blocks would take the place of this grid's)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (__any_sync(0xffffffffu, bad_id) && lane == 0) set_err(a.err, MOE_DEV_BAD_EXPERT);
  if (!seg_ok) return;    // the tail's tokens count nowhere
  // the warp's groups, by a tree
#pragma unroll
  for (int o = L; o < 32; o <<= 1) {
#pragma unroll
    for (int i = 0; i < NV; ++i) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
    zsum += __shfl_xor_sync(0xffffffffu, zsum, o);
    nval += __shfl_xor_sync(0xffffffffu, nval, o);
  }
  if (grp == 0) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = expert_of<VEC, L>(l, i);
      if (e < a.E) sm[warp * a.E + e] = acc[i];
    }
    if (l == 0) {
      s_z[warp] = zsum;
      s_n[warp] = nval;
    }
  }
  __syncthreads();
  const long long row = static_cast<long long>(blockIdx.x) * a.E;
  for (int e = threadIdx.x; e < a.E; e += 32 * W) {
    float x = sm[e];
#pragma unroll
    for (int q = 1; q < W; ++q) x += sm[q * a.E + e];
    w.psum[row + e] = x;
    w.pcnt[row + e] = hist[e];
  }
  if (threadIdx.x == 0) {
    float z = 0.f;
    int n = 0;
#pragma unroll
    for (int q = 0; q < W; ++q) {
      z += s_z[q];
      n += s_n[q];
    }
    w.pz[blockIdx.x] = z;
    w.pn[blockIdx.x] = n;
  }
}

// block (slice of EB experts, segment), blockDim / EB unit lanes: EB = 8 with
// 1024 threads where a segment has many units, 32 with 256 threads where
// there are many segments (a 1024-thread block for each of 16 segments took
// 21 us, as long as loss_rows)
template <int EB, int TH>
__global__ void __launch_bounds__(TH) loss_finish(const RouterLossArgs a, const Ws w, int chunk) {
  constexpr int LANES = TH / EB;      // unit lanes
  constexpr int NW = TH / 32;
  __shared__ Span s_span;
  __shared__ float s_sum[NW][EB];
  __shared__ int s_cnt[NW][EB];
  __shared__ float s_red[2][NW];
  __shared__ int s_num[NW];
  __shared__ int s_last;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int xe = threadIdx.x % EB, ul = threadIdx.x / EB;
  const int s = blockIdx.y;
  const int e = blockIdx.x * EB + xe;
  if (warp == 0) {     // the segment's place, from the caller's offsets alone
    Span sp{0, 0, 0, 0};
    bool bad = false;
    walk_segments(a.seg, a.S, a.T, chunk, bad, sp, [&](const Span& x, int) { return x.s == s; });
    if (lane == 0) s_span = sp;
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");   // loss_rows has ended
  __syncthreads();
  const Span sp = s_span;
  const int n_units = (sp.hi - sp.lo + chunk - 1) / chunk;
  int n = 0;
  float z = 0.f;
  for (int u = threadIdx.x; u < n_units; u += TH) {
    n += w.pn[sp.unit0 + u];
    z += w.pz[sp.unit0 + u];
  }
  float x = 0.f;
  int c = 0;
  if (e < a.E) {
    const float* ps = w.psum + static_cast<long long>(sp.unit0) * a.E + e;
    const int32_t* pc = w.pcnt + static_cast<long long>(sp.unit0) * a.E + e;
#pragma unroll 4
    for (int u = ul; u < n_units; u += LANES) {
      x += ps[static_cast<long long>(u) * a.E];
      c += pc[static_cast<long long>(u) * a.E];
    }
  }
  // the warp's unit lanes by a tree, then the warps in order
#pragma unroll
  for (int o = EB; o < 32; o <<= 1) {
    x += __shfl_xor_sync(0xffffffffu, x, o);
    c += __shfl_xor_sync(0xffffffffu, c, o);
  }
  n = __reduce_add_sync(0xffffffffu, n);
  z = warp_sum(z);
  if (lane < EB) {
    s_sum[warp][xe] = x;
    s_cnt[warp][xe] = c;
  }
  if (lane == 0) {
    s_num[warp] = n;
    s_red[0][warp] = z;
  }
  __syncthreads();
  if (warp == 0) {
    const int nseg = __reduce_add_sync(0xffffffffu, lane < NW ? s_num[lane] : 0);
    z = warp_sum(lane < NW ? s_red[0][lane] : 0.f);
    float y = 0.f;
    int d = 0;
#pragma unroll
    for (int q = lane / EB; q < NW; q += 32 / EB) {
      y += s_sum[q][xe];
      d += s_cnt[q][xe];
    }
#pragma unroll
    for (int o = EB; o < 32; o <<= 1) {
      y += __shfl_xor_sync(0xffffffffu, y, o);
      d += __shfl_xor_sync(0xffffffffu, d, o);
    }
    const bool mine = lane < EB && e < a.E;
    if (mine) a.counts[static_cast<long long>(s) * a.E + e] = d;
    float t = (mine && nseg > 0) ? static_cast<float>(d) * (y / static_cast<float>(nseg)) : 0.f;
    t = warp_sum(t);
    if (lane == 0) {
      if (blockIdx.x == 0) {
        a.n_valid[s] = nseg;
        w.zseg[s] = z;
      }
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
  float b = 0.f;
  n = 0;
  z = 0.f;
  const volatile float* term = w.term;
  const volatile float* zseg = w.zseg;
  const volatile int32_t* nv = a.n_valid;
#pragma unroll 4
  for (int i = threadIdx.x; i < terms; i += TH) b += term[i];
  for (int i = threadIdx.x; i < a.S; i += TH) {
    z += zseg[i];
    n += nv[i];
  }
  b = warp_sum(b);
  z = warp_sum(z);
  n = __reduce_add_sync(0xffffffffu, n);
  if (lane == 0) {
    s_red[0][warp] = b;
    s_red[1][warp] = z;
    s_num[warp] = n;
  }
  __syncthreads();
  if (warp == 0) {
    b = warp_sum(lane < NW ? s_red[0][lane] : 0.f);
    z = warp_sum(lane < NW ? s_red[1][lane] : 0.f);
    n = __reduce_add_sync(0xffffffffu, lane < NW ? s_num[lane] : 0);
    if (lane == 0) {
      const float N = static_cast<float>(n);
      a.loss[0] = n > 0 ? b * (static_cast<float>(a.E) / (static_cast<float>(a.k) * N)) : 0.f;
      a.loss[1] = n > 0 ? z / N : 0.f;
    }
  }
}

// The sequence of token t, as walk_segments lays them out: segment 0 begins
// at 0, the others at the running maximum of the offsets.  Of non-decreasing
// offsets (ordered) the last one at or below t, by bisection; else the one
// before the first offset above t, one by one.
__device__ __forceinline__ int segment_of(const int32_t* __restrict__ seg, int S, int t,
                                          bool ordered) {
  if (seg == nullptr) return 0;
  int lo = 0, hi = S;
  if (!ordered) {
    while (lo < S && seg[lo + 1] <= t) ++lo;
    return lo;
  }
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (seg[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

template <class T, int VEC, int NV, int L, bool ROUTER>
__global__ void __launch_bounds__(kBwdThreads) loss_bwd(const RouterLossArgs a, int per_warp) {
  constexpr int G = 32 / L;
  constexpr int W = kBwdThreads / 32;
  extern __shared__ float s_add[];    // ROUTER: a row of E zeros for each group of lanes
  __shared__ int s_part[W];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int l = lane % L, grp = lane / L;
  if constexpr (ROUTER)
    for (int i = threadIdx.x; i < W * G * a.E; i += kBwdThreads) s_add[i] = 0.f;
  // this warp's tokens: G at a time, per_warp rounds
  const long long first = (static_cast<long long>(blockIdx.x) * W + warp) * per_warp * G;
  const T* logits = static_cast<const T*>(a.logits);
  int n = 0;
  bool unordered = false;
  for (int s = threadIdx.x; s < a.S; s += kBwdThreads) {
    n += a.n_valid[s];
    if (a.seg != nullptr && s > 0 && a.seg[s] > a.seg[s + 1]) unordered = true;
  }
  n = __reduce_add_sync(0xffffffffu, n);
  if (lane == 0) s_part[warp] = n;
  const bool ordered = !__syncthreads_or(unordered);
  n = 0;
#pragma unroll
  for (int q = 0; q < W; ++q) n += s_part[q];
  const float inv_n = n > 0 ? 1.0f / static_cast<float>(n) : 0.f;
  const float gz = 2.f * a.dloss[1] * inv_n;
  const float gb = a.dloss[0] * static_cast<float>(a.E) / static_cast<float>(a.k) * inv_n;
  float wv[NV];
  int cur = -1;
  for (int r = 0; r < per_warp; ++r) {
    const long long tl = first + static_cast<long long>(r) * G;
    if (tl >= a.T) break;                       // the same for the whole warp
    const bool have = tl + grp < a.T;
    const int t = static_cast<int>(have ? tl + grp : a.T - 1);
    float v[NV];
    load_row<T, VEC, NV, L>(logits + static_cast<long long>(t) * a.E, a.E, l, have, v);
    const float lse = a.lse[t];
    // the router's own part: lane j of the group has the token's pair j
    const long long p0 = static_cast<long long>(t) * a.k;
    int e0 = -1;
    float pr = 0.f, dp = 0.f;
    if (ROUTER && l < a.k) {
      e0 = a.idx[p0 + l];
      pr = a.probs[p0 + l];
      dp = a.dprobs[p0 + l];
    }
    bool valid = !(lse == -INFINITY) && (a.mask == nullptr || a.mask[t] != 0);
    const int s = segment_of(a.seg, a.S, t, ordered);
    if (s != cur) {
      cur = s;
      const int ns = s < a.S ? a.n_valid[s] : 0;
      const float f = ns > 0 ? gb / static_cast<float>(ns) : 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int e = expert_of<VEC, L>(l, i);
        wv[i] = (s < a.S && e < a.E)
                    ? f * static_cast<float>(a.counts[static_cast<long long>(s) * a.E + e]) : 0.f;
      }
    }
    valid = valid && s < a.S;
    // P is normalised by the row's own sum, so that what the exponents are
    // shifted by cancels: 2^((z - lse) log2 e) alone would carry the rounding
    // of the stored lse, |lse| 2^-24 relative, and not sum to 1.  lse serves as
    // the shift while its rounding is far inside the exponent's range, and the
    // row's maximum past that (always the maximum: 34.7 us for 65,536 x 256,
    // 32.9 with lse).  An empty or masked token's values are dropped below.
    float shift = lse;
    const bool far = !(fabsf(lse) < 1048576.f);
    if (__any_sync(0xffffffffu, far)) {
      float m = v[0];
#pragma unroll
      for (int i = 1; i < NV; ++i) m = fmaxf(m, v[i]);
      m = group_max<L>(m);
      if (far) shift = m;     // this row's alone: no row's bits depend on its neighbours
    }
    float tot = 0.f, dot = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      v[i] = exp2_((v[i] - shift) * kLog2E);
      tot += v[i];
      dot += v[i] * wv[i];
    }
    const float inv = __fdividef(1.0f, group_sum<L>(tot));
    dot = group_sum<L>(dot) * inv - gz * lse;
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = valid ? v[i] * inv * (wv[i] - dot) : 0.f;
    if constexpr (ROUTER) {
      const bool ok0 = e0 >= 0 && e0 < a.E;
      float pd = ok0 ? pr * dp : 0.f;
      for (int j = l + L; j < a.k; j += L) {
        const int e = a.idx[p0 + j];
        if (e >= 0 && e < a.E) pd += a.probs[p0 + j] * a.dprobs[p0 + j];
      }
      pd = group_sum<L>(pd);
      // The pairs' terms reach the lanes that hold their experts through
      // the group's row in shared memory: each pair leaves its number at its
      // expert and reads it back, so that an expert chosen twice shows; such
      // tokens (no router makes them) take their pairs one after another.
      // (__match_any_sync in place of the numbers: 34.2 us against 31.7, both
      // before the row's sum was taken.)
      float* add = s_add + (warp * G + grp) * a.E;
      int* tag = reinterpret_cast<int*>(add);
      for (int j0 = 0; j0 < a.k; j0 += L) {
        int e = e0;
        float rr = pr * (dp - pd);
        if (j0 > 0) {
          e = -1;
          if (j0 + l < a.k) {
            e = a.idx[p0 + j0 + l];
            rr = a.probs[p0 + j0 + l] * (a.dprobs[p0 + j0 + l] - pd);
          }
        }
        const bool in = e >= 0 && e < a.E;
        if (in) tag[e] = l;
        __syncwarp();
        const bool twice = in && tag[e] != l;
        const bool any_twice = __any_sync(0xffffffffu, twice);
        __syncwarp();
        if (!any_twice) {
          if (in) add[e] = rr;
        } else {
          if (in) add[e] = 0.f;
          __syncwarp();
          for (int j = 0; j < L; ++j) {
            if (in && l == j) add[e] += rr;
            __syncwarp();
          }
        }
        __syncwarp();
        // every lane takes its experts' terms (zero where there is none) ...
#pragma unroll
        for (int g = 0; g < NV / VEC; ++g) {
          const int c0 = (l + L * g) * VEC;
          if (c0 < a.E) {
#pragma unroll
            for (int q = 0; q < VEC; ++q) v[g * VEC + q] += add[c0 + q];
          }
        }
        __syncwarp();
        if (in) add[e] = 0.f;    // ... and the row is zero again
        __syncwarp();
      }
    }
    if (!have) continue;
    const long long row = static_cast<long long>(t) * a.E;
#pragma unroll
    for (int g = 0; g < NV / VEC; ++g) {
      const int c0 = (l + L * g) * VEC;
      if (c0 >= a.E) continue;
      if (a.dlogits_bf16) {
        uint16_t* o = static_cast<uint16_t*>(a.dlogits) + row + c0;
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
        float* o = static_cast<float*>(a.dlogits) + row + c0;
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

template <class T, int VEC, int NV, int L>
cudaError_t go_bwd(const RouterLossArgs& a, int num_sms, cudaStream_t s) {
  // rounds of a warp: one while the SMs' 2048 threads are not full, then
  // up to eight, whose tokens mostly share their segment's weights
  constexpr int G = 32 / L, W = kBwdThreads / 32;
  const long long waves = static_cast<long long>(num_sms) * 64 * G;
  long long per = (a.T + waves - 1) / waves;
  per = per < 1 ? 1 : (per > 8 ? 8 : per);
  const long long blocks = (a.T + per * G * W - 1) / (per * G * W);
  const int grid = static_cast<int>(blocks), rounds = static_cast<int>(per);
  if (a.probs != nullptr)   // with a row of E terms for each group: at most 32 KB
    loss_bwd<T, VEC, NV, L, true>
        <<<grid, kBwdThreads, static_cast<size_t>(W) * G * a.E * 4, s>>>(a, rounds);
  else
    loss_bwd<T, VEC, NV, L, false><<<grid, kBwdThreads, 0, s>>>(a, rounds);
  return cudaGetLastError();
}
template <class T, int VEC, int NV, int L>
cudaError_t go_fwd(const RouterLossArgs& a, cudaStream_t s, int chunk, const Ws& w) {
  constexpr int W = NV <= 16 ? 16 : 8;    // [W][E] sums: at most 37 KB
  const size_t smem = static_cast<size_t>(W + 1) * a.E * 4;
  loss_rows<T, VEC, NV, L, W><<<units_cap(a.T, a.S), 32 * W, smem, s>>>(a, w, chunk);
  return cudaGetLastError();
}
template <class T, int VEC, int NV, int L>
cudaError_t go(const RouterLossArgs& a, int num_sms, cudaStream_t s, bool bwd, int chunk,
               const Ws& w) {
  return bwd ? go_bwd<T, VEC, NV, L>(a, num_sms, s) : go_fwd<T, VEC, NV, L>(a, s, chunk, w);
}

// Lanes and values per lane: the smallest instance that covers E.  The
// forward, bound by its instructions, takes 16 values a lane and half the
// lanes, which halves the shuffles and the per-token work (65,536 x 256: 26.4
// -> 22.0 us); the backward, which also holds the counts, 8 (31.7 us, 33.9
// with 16, both before the row's sum was taken; 33 with it).
template <class T, int VEC>
cudaError_t pick(const RouterLossArgs& a, int num_sms, cudaStream_t s, bool bwd, int chunk,
                 const Ws& w) {
  if (a.E <= 32) return go<T, VEC, 8, 4>(a, num_sms, s, bwd, chunk, w);
  if (bwd) {
    if (a.E <= 64) return go_bwd<T, VEC, 8, 8>(a, num_sms, s);
    if (a.E <= 128) return go_bwd<T, VEC, 8, 16>(a, num_sms, s);
    if (a.E <= 256) return go_bwd<T, VEC, 8, 32>(a, num_sms, s);
  } else {
    if (a.E <= 64) return go_fwd<T, VEC, 16, 4>(a, s, chunk, w);
    if (a.E <= 128) return go_fwd<T, VEC, 16, 8>(a, s, chunk, w);
    if (a.E <= 256) return go_fwd<T, VEC, 16, 16>(a, s, chunk, w);
  }
  if (a.E <= 512) return go<T, VEC, 16, 32>(a, num_sms, s, bwd, chunk, w);
  return go<T, VEC, 32, 32>(a, num_sms, s, bwd, chunk, w);
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
  // programmatic launch: loss_finish's blocks come in behind loss_rows and
  // wait on the device for it to end
  cudaLaunchConfig_t cfg = {};
  const bool few = finish_experts(a.S) == 8;
  cfg.gridDim = dim3(slices_of(a.E, a.S), a.S);
  cfg.blockDim = dim3(few ? 1024 : 256);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  *launches = 2;
  return few ? cudaLaunchKernelEx(&cfg, loss_finish<8, 1024>, a, w, chunk)
             : cudaLaunchKernelEx(&cfg, loss_finish<32, 256>, a, w, chunk);
}

cudaError_t launch_router_loss_bwd(const RouterLossArgs& a, int num_sms, cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
  return dispatch(a, num_sms, s, true, 0, Ws{});
}

}  // namespace moe
