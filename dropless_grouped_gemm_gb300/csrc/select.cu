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
// experts' order is that of z, which is exact; with one (or for groups' sums), c
// is computed in float32 and a row in which two neighbours of the order (or the
// last kept and the first dropped group) lie nearer than c's error is done again
// in 64 bits (some 0.2% of rows of 256 experts).  Equal logits with equal biases
// are equal and need no second look, nor do groups that are equal place by place
// (65,536 rows of 256 zeros, zero bias, 8 groups: 154 us, in 64 bits 3,040; rows of
// random logits 98 us without this look at their groups, 101 with it).
//
// Forward: a warp per token, lane l holding the E / 32 experts from l E / 32 on.
// A lane's values become 32-bit keys in the order of the floats, their last bits
// replaced by the expert's place in the lane (so that one number says which, and
// equals go to the lower index; what those bits hid counts as doubt), sorted once
// by a network of minima and maxima.  Each of the k rounds then is one maximum
// over the warp, one ballot, and a shift of the owner's keys: 18 instructions.
// Bound by instructions on long batches (65,536 x 256, sigmoid, bias, 8 groups:
// 144 us with a search of the lane's values in every round, 91 with the sort; by a batch's
// rows in doubt 90 to 112 now), by launch latency on short ones.  Backward: a warp per token, the k gradients scattered into a row
// in shared memory that leaves in 16-byte stores, the next token's pairs read
// meanwhile; a softmax's exponentials are taken once and wait in that row (taken
// again for the output: 48 us for 65,536 x 256, now 39).  Bound by latency and by
// the writes (by sigmoid 25.7 us, 2.6 TB/s of them; 34 with more blocks than are resident).
#include <cuda_bf16.h>

#include <type_traits>

#include "ptx.cuh"
#include "select.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = kThreads / 32;      // tokens of a block, one a warp
constexpr int kBwdBlocks = 5;             // of the gradient's an SM, all resident
constexpr unsigned kAll = 0xffffffffu;
// bf16's lowest finite value: a mask's logit is there, at float32's lowest, or -inf
constexpr float kMasked = -3.3895313892515355e38f;

// below this a float32 sigmoid is subnormal (and from -88.8 on 0); from the second
// one on a 64-bit one is 0, and counts as 0 here
constexpr float kLowSigmoid = -87.f;
constexpr float kNoSigmoid = -709.7827f;

__device__ __forceinline__ bool takes_part(float z) { return z > kMasked; }   // (false for NaN)

// signed keys in the order of the floats (-0 as +0); kNone: none
constexpr int kNone = static_cast<int>(0x80000000u);
__device__ __forceinline__ int key_of(float f) {
  const int b = __float_as_int(f + 0.f);
  return b ^ ((b >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float value_of(int k) {
  return __int_as_float(k ^ ((k >> 31) & 0x7fffffff));
}

// descending order by compare-exchanges (Batcher's odd-even merge sort)
template <int N>
__device__ __forceinline__ void sort_keys(int (&k)[N]) {
#pragma unroll
  for (int p = 1; p < N; p *= 2) {
#pragma unroll
    for (int q = p; q >= 1; q /= 2) {
#pragma unroll
      for (int j = q % p; j <= N - 1 - q; j += 2 * q) {
#pragma unroll
        for (int i = 0; i < q; ++i) {
          if (i + j + q < N && (i + j) / (2 * p) == (i + j + q) / (2 * p)) {
            const int hi = max(k[i + j], k[i + j + q]);
            k[i + j + q] = min(k[i + j], k[i + j + q]);
            k[i + j] = hi;
          }
        }
      }
    }
  }
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

// What a block needs to do a row again in 64 bits
struct Exact {
  double c[MOE_MAX_EXPERTS];
  double part[kRows];
  float top[kRows];
  int8_t doubt[kRows];
};

// c of row t in 64 bits (the logits where there is no bias and no group's sum to
// take), by the whole block: with a warp's lanes doing eight experts each, one
// after the other, a row took 20 us, and there is hardly a batch without one.
template <class T>
__device__ __noinline__ void exact_scores(const SelectArgs& a, long long t, Exact& x) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const T* row = static_cast<const T*>(a.logits) + t * a.E;
  const bool plain = a.bias == nullptr && !(a.top_groups < a.groups && a.best == 2);
  double m = 0, sum = 1;
  if (a.score == MOE_SCORE_SOFTMAX && !plain) {
    float mf = -INFINITY;
    for (int e = threadIdx.x; e < a.E; e += kThreads) {
      const float z = logit(row + e);
      if (takes_part(z)) mf = fmaxf(mf, z);
    }
    mf = warp_max(mf);
    if (lane == 0) x.top[warp] = mf;
    __syncthreads();
    for (int w = 0; w < kRows; ++w) mf = fmaxf(mf, x.top[w]);
    m = mf;
    double s = 0;
    for (int e = threadIdx.x; e < a.E; e += kThreads) {
      const float z = logit(row + e);
      if (takes_part(z)) s += exp_below(static_cast<double>(z), m);
    }
    s = warp_add(s);
    if (lane == 0) x.part[warp] = s;
    __syncthreads();
    sum = 0;
    for (int w = 0; w < kRows; ++w) sum += x.part[w];
  }
  for (int e = threadIdx.x; e < a.E; e += kThreads) {
    const float z = logit(row + e);
    double c = -INFINITY;
    if (takes_part(z)) {
      if (plain) c = z;
      else
        c = a.score == MOE_SCORE_SIGMOID ? 1.0 / (1.0 + exp(-static_cast<double>(z)))
                                         : exp_below(static_cast<double>(z), m) / sum;
      if (a.bias != nullptr) c += a.bias[e];
      if (!(c > -INFINITY)) c = -INFINITY;
    }
    x.c[e] = c;
  }
  __syncthreads();
}

// That row's choice, by one warp: lane j returns pick j (-1: none)
template <class T>
__device__ __noinline__ int exact_choice(const SelectArgs& a, long long t, Exact& x) {
  const int lane = threadIdx.x & 31;
  const T* row = static_cast<const T*>(a.logits) + t * a.E;
  if (a.top_groups < a.groups) {
    const int n = a.E / a.groups;
    double mine = -INFINITY;             // lane g: group g's score
    for (int g = 0; g < a.groups; ++g) {
      double t1 = -INFINITY, t2 = -INFINITY;
      for (int e = g * n + lane; e < (g + 1) * n; e += 32)
        top2(t1, t2, x.c[e], static_cast<double>(-INFINITY));
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
    for (int e = lane; e < a.E; e += 32) {
      if (!((keep >> (e / n)) & 1u)) x.c[e] = -INFINITY;
      else if (a.bias == nullptr && x.c[e] > -INFINITY) x.c[e] = logit(row + e);
    }
    __syncwarp();
  }
  int pick = -1;
  for (int j = 0; j < a.k; ++j) {
    double bv = -INFINITY;
    int be = 0x7fffffff;
    for (int e = lane; e < a.E; e += 32)
      if (x.c[e] > bv) { bv = x.c[e]; be = e; }
    for (int o = 16; o > 0; o >>= 1) {
      const double ov = __shfl_xor_sync(kAll, bv, o);
      const int oe = __shfl_xor_sync(kAll, be, o);
      if (ov > bv || (ov == bv && oe < be)) { bv = ov; be = oe; }
    }
    if (be == 0x7fffffff) break;         // (the same on every lane)
    if (lane == (be & 31)) x.c[be] = -INFINITY;
    __syncwarp();
    if (lane == j) pick = be;
  }
  return pick;
}

// How near two float32 c's have to be for their order to be in doubt, in units u
// = 2^-24.  A sigmoid is at most 6 u off (the exponential 2 + 1.16 |z| units in
// the last place, which s (1 - s) scales to 0.65; 1 + e^-z half a unit, the
// division two, of s <= 1), a softmax's s 22 u (expf two units, z - m u |z - m|
// of an s that is as much smaller, the sum's chains of 8 + 2 + 5 additions, the
// reciprocal and the product); c's addition rounds by u |c|, and a key's last bits
// hide up to NV - 1 units of 2 u |c|.
template <int NV>
__device__ __forceinline__ bool in_doubt(int score, float hi, float lo) {
  const float own = score == MOE_SCORE_SIGMOID ? 12.f : 44.f;
  const float tol = 5.9604644775390625e-8f * (own + 2.f * NV * fmaxf(fabsf(hi), fabsf(lo)));
  return !(hi - lo > tol);
}

// How far a float32 group score may be off: its terms' errors (own: half of
// in_doubt's for each of two), and by the terms' sizes, which its own may be far
// below, the keys' hidden bits, both additions and what is done with it here.
template <int NV>
__device__ __forceinline__ float group_slack(int score, float t1, float t2, int best) {
  const float own = score == MOE_SCORE_SIGMOID ? 12.f : 44.f;
  const float size = fabsf(t1) + ((best == 2 && t2 > -INFINITY) ? fabsf(t2) : 0.f);
  return size < INFINITY ? 5.9604644775390625e-8f * (own + (2.f * NV + 2.f) * size) : 0.f;
}

// Whether an expert other than pick `at` (the last one chosen), and not equal to
// it, lies within the doubt around it: the first one that was not chosen did, and
// what comes behind it was not looked at.  Rarely called.
template <class T>
__device__ __noinline__ bool doubt_around(const SelectArgs& a, long long t, int at, float m, float sum) {
  const int lane = threadIdx.x & 31;
  const T* row = static_cast<const T*>(a.logits) + t * a.E;
  auto value = [&](int e) {
    const float z = logit(row + e);
    if (a.bias == nullptr) return z;
    return (a.score == MOE_SCORE_SIGMOID ? 1.f / (1.f + expf(-z)) : exp_below(z, m) / sum) + a.bias[e];
  };
  const float v0 = value(at), z0 = logit(row + at), b0 = a.bias ? a.bias[at] : 0.f;
  bool other = false;
#pragma unroll 1
  for (int e = lane; e < a.E; e += 32) {
    const float z = logit(row + e);
    if (!takes_part(z) || (z == z0 && (a.bias == nullptr || a.bias[e] == b0))) continue;
    const float v = value(e);
    // (twice what a key of 32 hides and c's own error)
    other |= !(fabsf(v - v0) > 7.62939453125e-6f * (a.bias ? 1.f + fabsf(v0) : fabsf(v0)));
  }
  return __any_sync(kAll, other);
}

// Whether any of the groups in `which` (a bit for lane g * step: group g) has
// other logits or biases than the first of them, place by place.  Without such a
// difference their scores are equal, in float32 as in truth, and the lower index
// has been taken.
template <class T>
__device__ __noinline__ bool groups_differ(const SelectArgs& a, long long t, unsigned which, int step) {
  const int n = a.E / a.groups, lane = threadIdx.x & 31;
  const T* row = static_cast<const T*>(a.logits) + t * a.E;
  const int ref = (__ffs(which) - 1) / step * n;
#pragma unroll 1
  for (int at = 0; at < a.E; at += 32) {
    const int e = min(at + lane, a.E - 1);
    const int g = e / n, r = ref + e - g * n;
    const float z = logit(row + e), zr = logit(row + r);
    const bool same = (z == zr && (a.bias == nullptr || a.bias[e] == a.bias[r])) ||
                      (!takes_part(z) && !takes_part(zr));
    if (__any_sync(kAll, ((which >> (g * step)) & 1u) && !same)) return true;
  }
  return false;
}

// NV: experts a lane (32 NV >= E).  SCORED: c is needed (a bias, or groups by the
// sum of two scores), else the order is that of z.
template <class T, int NV, bool SCORED, bool VEC>
__global__ void __launch_bounds__(kThreads, NV == 8 && SCORED ? 4 : 0)    // (one instance took 75 registers)
    select_kernel(const SelectArgs a) {
  constexpr int kLow = NV - 1;                        // the bits that say which of the lane's
  const int lane = threadIdx.x & 31;
  const int e0 = lane * NV;
  const int n = a.E / a.groups;                       // experts of a group
  const bool limited = a.top_groups < a.groups;
  const bool biased = SCORED && a.bias != nullptr;
  // whole lanes to a group, a power of two of them: each lane has one group
  const int lanes = (n % NV == 0 && ((n / NV) & (n / NV - 1)) == 0) ? n / NV : 0;
  float b[SCORED ? NV : 1];
  if constexpr (SCORED) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      b[i] = (a.bias != nullptr && e0 + i < a.E) ? a.bias[e0 + i] : 0.f;
  }
  __shared__ Exact exact;
  const int step = gridDim.x * kRows;
  for (int t0 = blockIdx.x * kRows; t0 < a.T; t0 += step) {
    const bool here = t0 + (threadIdx.x >> 5) < a.T;      // (the block stays together)
    const int t = here ? t0 + (threadIdx.x >> 5) : a.T - 1;
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
    int key[NV];
    if constexpr (SCORED) {
      const float inv = 1.f / sum;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const float s = a.score == MOE_SCORE_SIGMOID ? __fdividef(1.f, 1.f + __expf(-z[i]))
                                                     : exp_below(z[i], m) * inv;
        const float c = s + b[i];
        key[i] = takes_part(z[i]) && c > -INFINITY ? (key_of(c) & ~kLow) | (kLow - i) : kNone;
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) key[i] = takes_part(z[i]) ? (key_of(z[i]) & ~kLow) | (kLow - i) : kNone;
    }
    sort_keys(key);
    bool doubt = false, keep = true;
    unsigned kept = kAll;                             // groups, a bit each
    unsigned near_groups = 0;                         // lanes of the ones in doubt
    if (limited) {
      float score = -INFINITY, slack = 0.f;           // lane's group's, or lane g: group g's
      int mine = lane;
      if (lanes > 0) {
        // (values without the keys' last bits)
        float t1 = key[0] != kNone ? value_of(key[0] & ~kLow) : -INFINITY;
        float t2 = -INFINITY;
        if constexpr (NV > 1) t2 = key[1] != kNone ? value_of(key[1] & ~kLow) : -INFINITY;
        for (int o = lanes / 2; o > 0; o >>= 1) {
          const float b1 = __shfl_xor_sync(kAll, t1, o), b2 = __shfl_xor_sync(kAll, t2, o);
          top2(t1, t2, b1, b2);
        }
        score = group_score(t1, t2, a.best);
        if constexpr (SCORED) slack = group_slack<NV>(a.score, t1, t2, a.best);
        mine = lane / lanes;
      } else {
        for (int g = 0; g < a.groups; ++g) {
          float t1 = -INFINITY, t2 = -INFINITY;
#pragma unroll
          for (int i = 0; i < NV; ++i) {
            const int e = e0 + kLow - (key[i] & kLow);
            if (key[i] != kNone && e >= g * n && e < (g + 1) * n)
              top2(t1, t2, value_of(key[i] & ~kLow), -INFINITY);
          }
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) {
            const float b1 = __shfl_xor_sync(kAll, t1, o), b2 = __shfl_xor_sync(kAll, t2, o);
            top2(t1, t2, b1, b2);
          }
          if (lane == g) {
            score = group_score(t1, t2, a.best);
            if constexpr (SCORED) slack = group_slack<NV>(a.score, t1, t2, a.best);
          }
        }
      }
      int before = 0;
      const int first = lanes > 0 ? lanes : 1;
      for (int g = 0; g < a.groups; ++g) {
        const float other = __shfl_sync(kAll, score, g * first);
        before += other > score || (other == score && g < mine);
      }
      const bool in = mine < a.groups;
      keep = in && before < a.top_groups;
      // the least that a kept group's score may be, the most that a dropped one's
      const float lo = value_of(__reduce_min_sync(kAll, keep ? key_of(score - slack) : 0x7fffffff));
      const int hk = __reduce_max_sync(kAll, in && !keep ? key_of(score + slack) : kNone);
      const float hi = value_of(hk);
      // (scores without a bias, each group's largest: the largest logits, of which
      // the keys hide the last bits of float32)
      if (hk != kNone && hi > -INFINITY && (SCORED || sizeof(T) == 4) && !(lo > hi)) {
        const bool near = keep ? !(score - slack > hi) : in && !(score + slack < lo);
        // (equal groups' float32 scores are equal)
        doubt = __reduce_min_sync(kAll, near ? key_of(score) : 0x7fffffff) !=
                __reduce_max_sync(kAll, near ? key_of(score) : kNone);
        near_groups = __ballot_sync(kAll, near);
      }
      if (lanes == 0) kept = __ballot_sync(kAll, keep);
      if (!SCORED || biased) {                        // (keys at a group's end become none, not in order)
        bool gap = false;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const bool out = lanes > 0 ? !keep
                                     : !((kept >> min((e0 + kLow - (key[i] & kLow)) / n, 31)) & 1u);
          if (out && key[i] != kNone) {
            key[i] = kNone;
            gap = true;
          }
        }
        if (lanes == 0 && __any_sync(kAll, gap)) sort_keys(key);
      }
    }
    if constexpr (SCORED) {
      if (!biased) {                                  // (the groups' scores were all that c was for)
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const bool in = lanes > 0 ? keep : (kept >> min((e0 + i) / n, 31)) & 1u;
          key[i] = in && takes_part(z[i]) ? (key_of(z[i]) & ~kLow) | (kLow - i) : kNone;
        }
        sort_keys(key);
      }
    }
    // the rounds, one more for what the last pick was chosen from (lane k holds
    // it), and a look at what comes then
    int pick = -1, mykey = kNone, next = kNone, after = kNone;       // lane j: pick j
    for (int j = 0; j <= a.k + 1; ++j) {
      const int head = key[0] & ~kLow;                // (of equals the lowest lane, then place)
      const int best = __reduce_max_sync(kAll, head);
      if (best == kNone) break;
      if (j == a.k + 1) {
        after = best;
        break;
      }
      const int owner = __ffs(__ballot_sync(kAll, head == best)) - 1;
      const int low = __shfl_sync(kAll, key[0], owner) & kLow;
      if (lane == j) {
        pick = owner * NV + kLow - low;
        mykey = best;
      }
      if (j == a.k) next = best;
      if (lane == owner) {
#pragma unroll
        for (int i = 0; i + 1 < NV; ++i) key[i] = key[i + 1];
        key[NV - 1] = kNone;
      }
    }
    float zj = pick >= 0 ? logit(row + pick) : -INFINITY;
    // neighbours in doubt: of a biased order by c's error, of the logits' by the
    // bits that the keys hide (bf16 logits have none there)
    if (biased || sizeof(T) == 4) {
      auto near = [&](int hi, int lo) {
        return biased ? in_doubt<NV>(a.score, value_of(hi), value_of(lo)) : hi == lo;
      };
      int nk = __shfl_down_sync(kAll, mykey, 1);
      const int ne = __shfl_down_sync(kAll, pick, 1);
      const float nz = __shfl_down_sync(kAll, zj, 1);
      const bool last = lane == a.k - 1;
      if (last) nk = next;
      const bool close = lane < a.k && nk != kNone && near(mykey, nk);
      bool pair = false;
      if (close && (!last || a.k < 32)) pair = zj != nz || (biased && a.bias[pick] != a.bias[ne]);
      bool some = __any_sync(kAll, pair);
      // more than one beyond the last pick: whether any of them differs from it
      const int edge = __shfl_sync(kAll, mykey, a.k - 1);
      const bool open = __any_sync(kAll, close && last) && after != kNone && near(edge, after);
      if (!doubt && (open || (a.k == 32 && __any_sync(kAll, close && last))))
        doubt = doubt_around<T>(a, t, __shfl_sync(kAll, pick, a.k - 1), m, sum);
      if (a.k == 32 || (biased && a.score == MOE_SCORE_SOFTMAX)) doubt |= some;
      else if (some && !doubt) {
        // the order of the picks and the one behind them alone: each lane its own
        // in 64 bits, then its rank among them
        double c = -INFINITY;
        if (pick >= 0)
          c = biased ? 1.0 / (1.0 + exp(-static_cast<double>(zj))) + a.bias[pick] : static_cast<double>(zj);
        int rank = 0;
        for (int i = 0; i <= a.k; ++i) {
          const double oc = __shfl_sync(kAll, c, i);
          const int oe = __shfl_sync(kAll, pick, i);
          rank += oc > c || (oc == c && oe < pick);
        }
        const int was = pick;
        for (int i = 0; i <= a.k; ++i) {
          const int r = __shfl_sync(kAll, rank, i), e = __shfl_sync(kAll, was, i);
          if (r == lane && e >= 0) pick = e;
        }
        zj = pick >= 0 ? logit(row + pick) : -INFINITY;
      }
    }
    if (lane >= a.k) {                                // (lane k's was not chosen)
      pick = -1;
      zj = -INFINITY;
    }
    float zs = zj;
    if (SCORED || sizeof(T) == 4) {
      // (asked here, where few registers are live)
      if (near_groups != 0 && !doubt) doubt = groups_differ<T>(a, t, near_groups, lanes > 0 ? lanes : 1);
      if (__syncthreads_or(doubt && here)) {
        if (lane == 0) exact.doubt[threadIdx.x >> 5] = doubt && here;
        __syncthreads();
        for (int w = 0; w < kRows; ++w) {
          if (!exact.doubt[w]) continue;
          exact_scores<T>(a, t0 + w, exact);
          if (static_cast<int>(threadIdx.x >> 5) == w) {
            pick = exact_choice<T>(a, t, exact);
            zs = pick >= 0 ? logit(row + pick) : -INFINITY;
          }
          __syncthreads();
        }
      }
    }
    // the weights, lane j's of pick j
    const bool on = pick >= 0;
    float w = 0.f;
    if (a.score == MOE_SCORE_SIGMOID) {
      if (on) w = 1.f / (1.f + expf(-zs));
      if (a.renorm) {
        if (__any_sync(kAll, on && zs < kLowSigmoid)) {
          // all below 0: numerator and sum times e^-m, m the largest logit
          const float m0 = warp_max(on ? zs : -INFINITY);
          if (m0 < 0.f) w = on && zs > kNoSigmoid ? expf(zs - m0) / (1.f + expf(zs)) : 0.f;
        }
        const float tot = warp_add(w);
        w = tot > 0.f ? w / tot : 0.f;
      }
    } else if (a.renorm) {
      const float mx = warp_max(zs);
      if (on) w = exp_below(zs, mx);
      const float tot = warp_add(w);
      w = tot > 0.f ? w / tot : 0.f;
    } else if (on) {
      w = exp_below(zs, m) / sum;
    }
    if (here && lane < a.k) {
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
__global__ void __launch_bounds__(kThreads, kBwdBlocks) select_bwd_kernel(const SelectArgs a) {
  extern __shared__ __align__(16) float rows[];       // [kRows][E padded to 4]
  const int lane = threadIdx.x & 31;
  float* acc = rows + (threadIdx.x >> 5) * ((a.E + 3) & ~3);
  for (int e = lane; e < a.E; e += 32) acc[e] = 0.f;
  __syncwarp();
  const int step = gridDim.x * kRows;
  // lane j: pair j of a token, read while the token before is worked on
  struct Pair {
    int e;
    float w, g;
  };
  auto pair_of = [&](int t) {
    Pair p{-1, 0.f, 0.f};
    if (lane < a.k && t < a.T) {
      const long long o = static_cast<long long>(t) * a.k + lane;
      p = Pair{a.idx[o], a.probs[o], a.dprobs[o]};
    }
    return p;
  };
  const int t0 = blockIdx.x * kRows + (threadIdx.x >> 5);
  Pair ahead = pair_of(t0);
  for (int t = t0; t < a.T; t += step) {
    const T* row = static_cast<const T*>(a.logits) + static_cast<long long>(t) * a.E;
    TO* out = static_cast<TO*>(a.dlogits) + static_cast<long long>(t) * a.E;
    const Pair pair = ahead;
    ahead = pair_of(t + step);
    const int e = pair.e >= 0 && pair.e < a.E ? pair.e : -1;
    const float w = e >= 0 ? pair.w : 0.f;
    float g = e >= 0 ? pair.g : 0.f;
    const float dot = warp_add(w * g);
    g = a.renorm ? w * (g - dot / a.scale) : w * g;
    if (a.score == MOE_SCORE_SIGMOID && e >= 0) g *= 1.f / (1.f + expf(logit(row + e)));
    const unsigned twins = __match_any_sync(kAll, e);
    const bool first = e >= 0 && lane == __ffs(twins) - 1;
    float mine = g;
    if (e >= 0 && (twins & (twins - 1))) {            // chosen more than once
      mine = 0.f;
      for (unsigned r = twins; r != 0; r &= r - 1) mine += __shfl_sync(twins, g, __ffs(r) - 1);
    }
    if constexpr (!DENSE) {
      if (first) acc[e] = mine;
    } else {
      const float total = warp_add(e >= 0 ? g : 0.f);
      float m = -INFINITY, sum = 0.f;
      for (int i = lane; i < a.E; i += 32) {
        const float z = logit(row + i);
        if (takes_part(z)) m = fmaxf(m, z);
      }
      m = warp_max(m);
      // the exponentials in the row, -1 for a mask; then the gradients in their place
      for (int i = lane; i < a.E; i += 32) {
        const float z = logit(row + i);
        const float x = takes_part(z) ? exp_below(z, m) : -1.f;
        if (x >= 0.f) sum += x;
        acc[i] = x;
      }
      sum = warp_add(sum);
      const float share = sum > 0.f ? total / sum : 0.f;
      __syncwarp();
      if (first && acc[e] >= 0.f) mine -= acc[e] * share;
      __syncwarp();
      for (int i = lane; i < a.E; i += 32) acc[i] = acc[i] >= 0.f ? -acc[i] * share : 0.f;
      __syncwarp();
      if (first) acc[e] = mine;
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
    if (!DENSE && e >= 0) acc[e] = 0.f;
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

int blocks_of(int T, int most) {
  const int want = static_cast<int>((static_cast<long long>(T) + kRows - 1) / kRows);
  return want < most ? want : most;
}

template <class T, int NV, bool SCORED>
cudaError_t select_t(const SelectArgs& a, int num_sms, cudaStream_t s) {
  const int blocks = blocks_of(a.T, 8 * num_sms);
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
  const int blocks = blocks_of(a.T, kBwdBlocks * num_sms);
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
