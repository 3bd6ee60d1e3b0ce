// select.cu - the router's choice of experts by scores, and its gradient.
//
//   s_te = softmax_e(z_t) or sigmoid(z_te);  c_te = s_te + bias_e
//   group g's score = the sum of its `best` (1 or 2) largest c; the top_groups
//   best groups stay; the k largest c inside them are chosen, in decreasing
//   order (ties: the lower index, of groups and of experts)
//   w_tj = scale s_tj / sum_i s_ti (renorm), or scale s_tj
// An expert whose logit is NaN or at most bf16's lowest finite value (a mask)
// takes no part; picks that no expert is left for are -1 with weight 0.
//
// The choice is that of the real numbers, not of float32's: without a bias the
// experts' order is that of z, which is exact; with one (or for groups' sums), c is computed in
// float32 and a row in which two neighbours of the order (or the last kept and
// the first dropped group) lie nearer than c's error is done again in 64 bits
// (some 0.4% of rows of 256 experts).  Equal logits with equal biases are equal
// and need no second look.
//
// Forward: a warp per token, lane l holding the E / 32 experts from l E / 32
// on, so that the lowest lane of equals has the lowest index; k rounds of a
// maximum over the lane's keys and over the warp.  Bound by the rounds'
// instructions on long batches, by launch latency on short ones.  Backward: a
// warp per token, the k gradients scattered into a row in shared memory that
// leaves in 16-byte stores; bound by those writes.
#include <cuda_bf16.h>

#include <type_traits>

#include "ptx.cuh"
#include "select.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = kThreads / 32;      // tokens of a block, one a warp
constexpr unsigned kAll = 0xffffffffu;
// bf16's lowest finite value: a mask's logit is there, at float32's lowest, or -inf
constexpr float kMasked = -3.3895313892515355e38f;

__device__ __forceinline__ bool takes_part(float z) { return z > kMasked; }   // (false for NaN)

// unsigned keys in the order of the floats (-0 as +0); 0: none
__device__ __forceinline__ uint32_t key_of(float f) {
  uint32_t b = __float_as_uint(f + 0.f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
  return v;
}
template <class F>
__device__ __forceinline__ F warp_add(F v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

template <class T>
__device__ __forceinline__ float logit(const T* p) {
  if constexpr (sizeof(T) == 4) return *p;
  else return __uint_as_float(static_cast<uint32_t>(*p) << 16);
}

// e^(z - m) of a logit that takes part, m the largest (equal: 1, at +inf too)
__device__ __forceinline__ float exp_below(float z, float m) { return z == m ? 1.f : expf(z - m); }
__device__ __forceinline__ double exp_below(double z, double m) { return z == m ? 1.0 : exp(z - m); }

// the largest and second largest of two such pairs
template <class F>
__device__ __forceinline__ void top2(F& a1, F& a2, F b1, F b2) {
  const F lo = a1 < b1 ? a1 : b1;
  a1 = a1 < b1 ? b1 : a1;
  a2 = a2 < b2 ? b2 : a2;
  a2 = a2 < lo ? lo : a2;
}
// a group's score from its two largest c (what is missing adds nothing)
template <class F>
__device__ __forceinline__ F group_score(F t1, F t2, int best) {
  return (best == 2 && t2 > static_cast<F>(-INFINITY)) ? t1 + t2 : t1;
}

// One row's choice in 64 bits: lane j returns pick j (-1: none).  Rarely
// called, so it keeps its values in local memory.
template <class T>
__device__ __noinline__ int select_exact(const SelectArgs& a, long long t, int nv) {
  const int lane = threadIdx.x & 31;
  const T* row = static_cast<const T*>(a.logits) + t * a.E;
  double c[32];
  float mf = -INFINITY;
  for (int i = 0; i < nv; ++i) {
    const int e = lane * nv + i;
    if (e < a.E) {
      const float z = logit(row + e);
      if (takes_part(z)) mf = fmaxf(mf, z);
    }
  }
  const double m = warp_max(mf);
  double sum = 0;
  for (int i = 0; i < nv; ++i) {
    const int e = lane * nv + i;
    const float z = e < a.E ? logit(row + e) : -INFINITY;
    c[i] = -INFINITY;
    if (!takes_part(z)) continue;
    c[i] = a.score == MOE_SCORE_SIGMOID ? 1.0 / (1.0 + exp(-static_cast<double>(z)))
                                        : exp_below(static_cast<double>(z), m);
    sum += c[i];
  }
  if (a.score == MOE_SCORE_SOFTMAX) {
    sum = warp_add(sum);
    for (int i = 0; i < nv; ++i) c[i] = c[i] / sum;      // (-inf stays)
  }
  if (a.bias != nullptr)
    for (int i = 0; i < nv; ++i) {
      const int e = lane * nv + i;
      if (e < a.E) c[i] += a.bias[e];
      if (!(c[i] > -INFINITY)) c[i] = -INFINITY;
    }
  if (a.top_groups < a.groups) {
    const int n = a.E / a.groups;
    double mine = -INFINITY;             // lane g: group g's score
    for (int g = 0; g < a.groups; ++g) {
      double t1 = -INFINITY, t2 = -INFINITY;
      for (int i = 0; i < nv; ++i) {
        const int e = lane * nv + i;
        if (e >= g * n && e < (g + 1) * n) top2(t1, t2, c[i], static_cast<double>(-INFINITY));
      }
      for (int o = 16; o > 0; o >>= 1) {
        const double b1 = __shfl_xor_sync(kAll, t1, o), b2 = __shfl_xor_sync(kAll, t2, o);
        top2(t1, t2, b1, b2);
      }
      if (lane == g) mine = group_score(t1, t2, a.best);
    }
    int before = 0;
    for (int g = 0; g < a.groups; ++g) {
      const double other = __shfl_sync(kAll, mine, g);
      if (other > mine || (other == mine && g < lane)) ++before;
    }
    const unsigned keep = __ballot_sync(kAll, lane < a.groups && before < a.top_groups);
    for (int i = 0; i < nv; ++i) {
      const int e = lane * nv + i;
      if (e >= a.E) continue;
      if (!((keep >> (e / n)) & 1u)) c[i] = -INFINITY;
      else if (a.bias == nullptr && c[i] > -INFINITY) c[i] = logit(row + e);
    }
  }
  int pick = -1;
  for (int j = 0; j < a.k; ++j) {
    double bv = -INFINITY;
    int be = 0x7fffffff;
    for (int i = 0; i < nv; ++i)
      if (c[i] > bv) { bv = c[i]; be = lane * nv + i; }
    for (int o = 16; o > 0; o >>= 1) {
      const double ov = __shfl_xor_sync(kAll, bv, o);
      const int oe = __shfl_xor_sync(kAll, be, o);
      if (ov > bv || (ov == bv && oe < be)) { bv = ov; be = oe; }
    }
    if (be == 0x7fffffff) break;         // (the same on every lane)
    if (be / nv == lane) c[be - lane * nv] = -INFINITY;
    if (lane == j) pick = be;
  }
  return pick;
}

// Float32's c is at most 2^-20 (1 + |c|) off.  Sigmoid: the exponential is
// 2 + 1.16 |z| units off, which s (1 - s) scales to under 1.2 of s <= 1, and the
// division 2; softmax: expf 2 units, z - m 2^-24 |z - m| of an s that is as much
// smaller, the sum's chains of 8 + 2 + 5 additions 15 halves; then half a unit
// of |c|.  Two such are in doubt within twice that, sums of two within four times.
__device__ __forceinline__ bool in_doubt(float hi, float lo, float times) {
  return !(hi - lo > times * 1.9073486328125e-6f * (1.f + fmaxf(fabsf(hi), fabsf(lo))));
}

// NV: experts a lane (32 NV >= E).  SCORED: the order is that of c (a bias, or
// groups by the sum of two scores), else that of z.
template <class T, int NV, bool SCORED, bool VEC>
__global__ void __launch_bounds__(kThreads) select_kernel(const SelectArgs a) {
  const int lane = threadIdx.x & 31;
  const int e0 = lane * NV;
  const int n = a.E / a.groups;                       // experts of a group
  const bool limited = a.top_groups < a.groups;
  // whole lanes to a group, a power of two of them: each lane has one group
  const int lanes = (n % NV == 0 && ((n / NV) & (n / NV - 1)) == 0) ? n / NV : 0;
  float b[SCORED ? NV : 1];
  if constexpr (SCORED) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      b[i] = (a.bias != nullptr && e0 + i < a.E) ? a.bias[e0 + i] : 0.f;
  }
  const int step = gridDim.x * kRows;
  for (int t = blockIdx.x * kRows + (threadIdx.x >> 5); t < a.T; t += step) {
    const T* row = static_cast<const T*>(a.logits) + static_cast<long long>(t) * a.E;
    float z[NV];
    if constexpr (VEC) {                              // E is a multiple of NV: all or nothing
      if (e0 < a.E) {
        uint32_t w[NV * sizeof(T) / 4];
        if constexpr (NV * sizeof(T) >= 16) {
#pragma unroll
          for (int i = 0; i < static_cast<int>(NV * sizeof(T) / 16); ++i) {
            const uint4 u = __ldcs(reinterpret_cast<const uint4*>(row + e0) + i);
            w[4 * i] = u.x; w[4 * i + 1] = u.y; w[4 * i + 2] = u.z; w[4 * i + 3] = u.w;
          }
        } else {
          const uint2 u = __ldcs(reinterpret_cast<const uint2*>(row + e0));
          w[0] = u.x;
          w[1] = u.y;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          if constexpr (sizeof(T) == 4) z[i] = __uint_as_float(w[i]);
          else z[i] = (i & 1) ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) z[i] = -INFINITY;
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) z[i] = e0 + i < a.E ? logit(row + e0 + i) : -INFINITY;
    }
    float m = -INFINITY, sum = 0.f;                   // of a softmax over all experts
    if (a.score == MOE_SCORE_SOFTMAX && (SCORED || !a.renorm)) {
#pragma unroll
      for (int i = 0; i < NV; ++i) m = fmaxf(m, takes_part(z[i]) ? z[i] : -INFINITY);
      m = warp_max(m);
      float part[4] = {0.f, 0.f, 0.f, 0.f};           // (short chains: the doubt's bound counts them)
#pragma unroll
      for (int i = 0; i < NV; ++i) part[i & 3] += takes_part(z[i]) ? exp_below(z[i], m) : 0.f;
      sum = warp_add((part[0] + part[1]) + (part[2] + part[3]));
    }
    uint32_t key[NV];
    if constexpr (SCORED) {
      const float inv = 1.f / sum;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const float s = a.score == MOE_SCORE_SIGMOID ? __fdividef(1.f, 1.f + __expf(-z[i]))
                                                     : exp_below(z[i], m) * inv;
        const float c = s + b[i];
        key[i] = takes_part(z[i]) && c > -INFINITY ? key_of(c) : 0u;
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) key[i] = takes_part(z[i]) ? key_of(z[i]) : 0u;
    }
    bool doubt = false;
    if (limited) {
      if (lanes > 0) {
        float t1 = -INFINITY, t2 = -INFINITY;
#pragma unroll
        for (int i = 0; i < NV; ++i)
          top2(t1, t2, key[i] ? value_of(key[i]) : -INFINITY, -INFINITY);
        for (int o = lanes / 2; o > 0; o >>= 1) {
          const float b1 = __shfl_xor_sync(kAll, t1, o), b2 = __shfl_xor_sync(kAll, t2, o);
          top2(t1, t2, b1, b2);
        }
        const float score = group_score(t1, t2, a.best);
        const int mine = lane / lanes;
        int before = 0;
        for (int g = 0; g < a.groups; ++g) {
          const float other = __shfl_sync(kAll, score, g * lanes);
          before += other > score || (other == score && g < mine);
        }
        const bool in = mine < a.groups, keep = in && before < a.top_groups;
        if constexpr (SCORED) {
          const uint32_t lo = __reduce_min_sync(kAll, keep ? key_of(score) : kAll);
          const uint32_t hi = __reduce_max_sync(kAll, in && !keep ? key_of(score) : 0u);
          doubt |= in_doubt(value_of(lo), value_of(hi), 2.f) && value_of(hi) > -INFINITY;
        }
        if (!keep) {
#pragma unroll
          for (int i = 0; i < NV; ++i) key[i] = 0u;
        }
      } else {
        float score = -INFINITY;                      // lane g: group g's
        for (int g = 0; g < a.groups; ++g) {
          float t1 = -INFINITY, t2 = -INFINITY;
#pragma unroll
          for (int i = 0; i < NV; ++i)
            if (key[i] && e0 + i >= g * n && e0 + i < (g + 1) * n)
              top2(t1, t2, value_of(key[i]), -INFINITY);
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) {
            const float b1 = __shfl_xor_sync(kAll, t1, o), b2 = __shfl_xor_sync(kAll, t2, o);
            top2(t1, t2, b1, b2);
          }
          if (lane == g) score = group_score(t1, t2, a.best);
        }
        int before = 0;
        for (int g = 0; g < a.groups; ++g) {
          const float other = __shfl_sync(kAll, score, g);
          before += other > score || (other == score && g < lane);
        }
        const bool in = lane < a.groups, keep = in && before < a.top_groups;
        if constexpr (SCORED) {
          const uint32_t lo = __reduce_min_sync(kAll, keep ? key_of(score) : kAll);
          const uint32_t hi = __reduce_max_sync(kAll, in && !keep ? key_of(score) : 0u);
          doubt |= in_doubt(value_of(lo), value_of(hi), 2.f) && value_of(hi) > -INFINITY;
        }
        const unsigned kept = __ballot_sync(kAll, keep);
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (!((kept >> min((e0 + i) / n, 31)) & 1u)) key[i] = 0u;
      }
    }
    const bool biased = SCORED && a.bias != nullptr;
    if constexpr (SCORED) {
      if (!biased) {                                  // (the groups' scores were all that c was for)
#pragma unroll
        for (int i = 0; i < NV; ++i) key[i] = key[i] ? key_of(z[i]) : 0u;
      }
    }
    // the rounds; a biased choice looks at one more, for the last pick's doubt
    int pick = -1;                                    // lane j: pick j
    uint32_t last = 0u;
    int last_e = -1;
    const int rounds = a.k + (biased ? 1 : 0);
    for (int j = 0; j < rounds; ++j) {
      uint32_t top = key[0];
#pragma unroll
      for (int i = 1; i < NV; ++i) top = max(top, key[i]);
      const uint32_t best = __reduce_max_sync(kAll, top);
      if (best == 0u) break;
      const int owner = __ffs(__ballot_sync(kAll, top == best)) - 1;
      int at = 0;
#pragma unroll
      for (int i = NV - 1; i >= 0; --i)
        if (key[i] == best) at = i;
      const int e = __shfl_sync(kAll, e0 + at, owner);
      if (lane == owner) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (i == at) key[i] = 0u;
      }
      if (lane == j && j < a.k) pick = e;
      if constexpr (SCORED) {
        if (biased && last_e >= 0 && in_doubt(value_of(last), value_of(best), 1.f))
          doubt |= logit(row + e) != logit(row + last_e) || a.bias[e] != a.bias[last_e];
        last = best;
        last_e = e;
      }
    }
    if constexpr (SCORED) {
      if (doubt) pick = select_exact<T>(a, t, NV);
    }
    // the weights, lane j's of pick j
    const bool on = pick >= 0;
    const float zj = on ? logit(row + pick) : -INFINITY;
    float w = 0.f;
    if (a.score == MOE_SCORE_SIGMOID) {
      if (on) w = 1.f / (1.f + expf(-zj));
      if (a.renorm) {
        const float tot = warp_add(w);
        w = tot > 0.f ? w / tot : 0.f;
      }
    } else if (a.renorm) {
      const float mx = warp_max(zj);
      if (on) w = exp_below(zj, mx);
      const float tot = warp_add(w);
      w = tot > 0.f ? w / tot : 0.f;
    } else if (on) {
      w = exp_below(zj, m) / sum;
    }
    if (lane < a.k) {
      const long long o = static_cast<long long>(t) * a.k + lane;
      a.idx[o] = pick;
      a.probs[o] = a.scale * w;
    }
  }
}

// Backward.  With g_j = w_j (dw_j - sum_i w_i dw_i / scale) (renorm) or
// w_j dw_j, the gradient of the weights through their normalisation:
//   sigmoid:           dz_j = g_j (1 - s_j)
//   softmax, renorm:   dz_j = g_j          (the softmax's own sum cancels)
//   softmax:           dz_e = [e chosen] g_e - s_e sum_j g_j   (every e)
// A pair with an id outside [0, E) takes no part; an expert chosen twice by a
// token gets both terms, in the order of the pairs.
template <class T, class TO, int VEC, bool DENSE>
__global__ void __launch_bounds__(kThreads) select_bwd_kernel(const SelectArgs a) {
  extern __shared__ __align__(16) float rows[];       // [kRows][E padded to 4]
  const int lane = threadIdx.x & 31;
  float* acc = rows + (threadIdx.x >> 5) * ((a.E + 3) & ~3);
  for (int e = lane; e < a.E; e += 32) acc[e] = 0.f;
  __syncwarp();
  const int step = gridDim.x * kRows;
  for (int t = blockIdx.x * kRows + (threadIdx.x >> 5); t < a.T; t += step) {
    const T* row = static_cast<const T*>(a.logits) + static_cast<long long>(t) * a.E;
    TO* out = static_cast<TO*>(a.dlogits) + static_cast<long long>(t) * a.E;
    int e = -1;
    float w = 0.f, g = 0.f;
    if (lane < a.k) {
      const long long o = static_cast<long long>(t) * a.k + lane;
      e = a.idx[o];
      if (e < 0 || e >= a.E) e = -1;
      if (e >= 0) {
        w = a.probs[o];
        g = a.dprobs[o];
      }
    }
    const float dot = warp_add(w * g);
    g = a.renorm ? w * (g - dot / a.scale) : w * g;
    if (a.score == MOE_SCORE_SIGMOID && e >= 0) g *= 1.f / (1.f + expf(logit(row + e)));
    const unsigned twins = __match_any_sync(kAll, e);
    if (e >= 0) {
      const bool first = lane == __ffs(twins) - 1;
      if (twins & (twins - 1)) {                      // chosen more than once
        float s = 0.f;
        for (unsigned r = twins; r != 0; r &= r - 1) s += __shfl_sync(twins, g, __ffs(r) - 1);
        if (first) acc[e] = s;
      } else {
        acc[e] = g;
      }
    }
    float m = -INFINITY, share = 0.f;
    if constexpr (DENSE) {
      const float total = warp_add(e >= 0 ? g : 0.f);
      float sum = 0.f;
      for (int i = lane; i < a.E; i += 32) {
        const float z = logit(row + i);
        if (takes_part(z)) m = fmaxf(m, z);
      }
      m = warp_max(m);
      for (int i = lane; i < a.E; i += 32) {
        const float z = logit(row + i);
        if (takes_part(z)) sum += exp_below(z, m);
      }
      sum = warp_add(sum);
      share = sum > 0.f ? total / sum : 0.f;
    }
    __syncwarp();
    for (int i = lane * VEC; i < a.E; i += 32 * VEC) {
      float v[VEC];
      if constexpr (VEC == 4) {
        const float4 f = *reinterpret_cast<const float4*>(acc + i);
        v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
      } else {
        v[0] = acc[i];
      }
      if constexpr (DENSE) {
#pragma unroll
        for (int x = 0; x < VEC; ++x) {
          const float z = logit(row + i + x);
          if (takes_part(z)) v[x] -= exp_below(z, m) * share;
        }
      }
      if (a.accumulate) {
#pragma unroll
        for (int x = 0; x < VEC; ++x) v[x] += logit(out + i + x);
      }
      if constexpr (VEC == 4 && sizeof(TO) == 4) {
        *reinterpret_cast<float4*>(out + i) = make_float4(v[0], v[1], v[2], v[3]);
      } else if constexpr (VEC == 4) {
        *reinterpret_cast<uint2*>(out + i) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
      } else if constexpr (sizeof(TO) == 4) {
        out[i] = v[0];
      } else {
        out[i] = static_cast<TO>(pack_bf16x2(v[0], 0.f) & 0xffffu);
      }
    }
    __syncwarp();
    if (e >= 0) acc[e] = 0.f;
    __syncwarp();
  }
}

// experts a lane: the smallest power of two that holds E
template <class F>
cudaError_t with_lane(int E, F&& f) {
  if (E <= 32) return f(std::integral_constant<int, 1>{});
  if (E <= 64) return f(std::integral_constant<int, 2>{});
  if (E <= 128) return f(std::integral_constant<int, 4>{});
  if (E <= 256) return f(std::integral_constant<int, 8>{});
  if (E <= 512) return f(std::integral_constant<int, 16>{});
  return f(std::integral_constant<int, 32>{});
}

int blocks_of(int T, int num_sms) {
  const long long want = (static_cast<long long>(T) + kRows - 1) / kRows;
  return static_cast<int>(want < 8LL * num_sms ? want : 8LL * num_sms);
}

template <class T, int NV, bool SCORED>
cudaError_t select_t(const SelectArgs& a, int num_sms, cudaStream_t s) {
  const int blocks = blocks_of(a.T, num_sms);
  // lanes' experts in 8- and 16-byte loads: whole lanes, and rows that keep the alignment
  constexpr int bytes = NV * static_cast<int>(sizeof(T));
  constexpr int align = bytes < 16 ? bytes : 16;
  if constexpr (bytes >= 8) {
    if (a.E % NV == 0 && (a.E * sizeof(T)) % align == 0 &&
        reinterpret_cast<uintptr_t>(a.logits) % align == 0) {
      select_kernel<T, NV, SCORED, true><<<blocks, kThreads, 0, s>>>(a);
      return cudaGetLastError();
    }
  }
  select_kernel<T, NV, SCORED, false><<<blocks, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

template <class T, class TO>
cudaError_t bwd_t(const SelectArgs& a, int num_sms, cudaStream_t s) {
  const int blocks = blocks_of(a.T, num_sms);
  const size_t smem = static_cast<size_t>(kRows) * ((a.E + 3) & ~3) * sizeof(float);
  const bool dense = a.score == MOE_SCORE_SOFTMAX && !a.renorm;
  const bool vec = a.E % 4 == 0 && reinterpret_cast<uintptr_t>(a.dlogits) % (4 * sizeof(TO)) == 0;
  if (vec)
    dense ? select_bwd_kernel<T, TO, 4, true><<<blocks, kThreads, smem, s>>>(a)
          : select_bwd_kernel<T, TO, 4, false><<<blocks, kThreads, smem, s>>>(a);
  else
    dense ? select_bwd_kernel<T, TO, 1, true><<<blocks, kThreads, smem, s>>>(a)
          : select_bwd_kernel<T, TO, 1, false><<<blocks, kThreads, smem, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_router_select(const SelectArgs& a, int num_sms, cudaStream_t s) {
  if (a.T <= 0) return cudaSuccess;
  const bool scored = a.bias != nullptr || (a.top_groups < a.groups && a.best == 2);
  return with_lane(a.E, [&](auto nv) {
    constexpr int NV = decltype(nv)::value;
    if (a.logits_bf16)
      return scored ? select_t<uint16_t, NV, true>(a, num_sms, s)
                    : select_t<uint16_t, NV, false>(a, num_sms, s);
    return scored ? select_t<float, NV, true>(a, num_sms, s)
                  : select_t<float, NV, false>(a, num_sms, s);
  });
}

cudaError_t launch_router_select_bwd(const SelectArgs& a, int num_sms, cudaStream_t s) {
  if (a.T <= 0) return cudaSuccess;
  if (a.logits_bf16)
    return a.dlogits_bf16 ? bwd_t<uint16_t, uint16_t>(a, num_sms, s)
                          : bwd_t<uint16_t, float>(a, num_sms, s);
  return a.dlogits_bf16 ? bwd_t<float, uint16_t>(a, num_sms, s)
                        : bwd_t<float, float>(a, num_sms, s);
}

}  // namespace moe
