// act.cuh - gate nonlinearities of the gated expert MLP and their
// derivatives, shared by the bf16 and MXFP8 epilogues.
//   SwiGLU: phi(g) = g * sigmoid(g) (Swish on the gate side, times the up
//           projection) - [CuTe] "핵심 아이디어 / 구조 / 동작 방식".
//   GeGLU:  phi(g) = 0.5 g (1 + tanh(sqrt(2/pi) (g + 0.044715 g^3))), the
//           tanh approximation of GELU (Hendrycks & Gimpel), evaluated as
//           g sigmoid(2 sqrt(2/pi) (g + 0.044715 g^3)), the same function.
#pragma once

#include "ptx.cuh"

namespace moe {

__device__ __forceinline__ float sigmoidf_(float g) { return 1.0f / (1.0f + __expf(-g)); }
constexpr float kGeluC = 0.7978845608028654f;  // sqrt(2/pi)
constexpr float kGeluA = 0.044715f;

template <int ACT>
__device__ __forceinline__ float gate_phi(float g) {
  if constexpr (ACT == MOE_ACT_SWIGLU) {
    return g * sigmoidf_(g);
  } else {
    // 1 + tanh(z) = 2 sigmoid(2z): no tanh, and no cancellation for
    // negative gates, where 1 + tanh(z) is small
    const float z = kGeluC * (g + kGeluA * g * g * g);
    return g * sigmoidf_(2.0f * z);
  }
}
// phi and phi' together
template <int ACT>
__device__ __forceinline__ void gate_phi_dphi(float g, float& ph, float& dph) {
  if constexpr (ACT == MOE_ACT_SWIGLU) {
    const float s = sigmoidf_(g);
    ph = g * s;
    dph = s * (1.0f + g * (1.0f - s));
  } else {
    // with s = sigmoid(2z): 1 + tanh z = 2s and 1 - tanh^2 z = 4 s (1 - s), so
    // phi = g s and phi' = s + 2 g s (1 - s) z'(g), z' = c (1 + 3 a g^2)
    const float z = kGeluC * (g + kGeluA * g * g * g);
    const float s = sigmoidf_(2.0f * z);
    ph = g * s;
    dph = s + 2.0f * g * s * (1.0f - s) * kGeluC * (1.0f + 3.0f * kGeluA * g * g);
  }
}

// ------------------------------------------------ the linear operator's set
// relu, silu, gelu (tanh form) and srelu as above; NaN goes through (the
// comparison is false for it).
__device__ __forceinline__ float relu_(float x) { return x < 0.f ? 0.f : x; }
// The sigmoid with the approximate division (2 ulp, against an IEEE division
// that is a call of its own): where a few threads finish a tile, four gated
// outputs took 0.5 us with the latter.
__device__ __forceinline__ float sigmoid_(float x) { return __fdividef(1.0f, 1.0f + __expf(-x)); }
__device__ __forceinline__ float silu_(float x) { return x * sigmoid_(x); }
__device__ __forceinline__ float gelu_(float x) {
  return x * sigmoid_(2.0f * kGeluC * (x + kGeluA * x * x * x));
}
// phi and phi' (phi silu or gelu)
template <bool GELU>
__device__ __forceinline__ void linear_phi(float x, float& p, float& d) {
  if constexpr (!GELU) {
    const float s = sigmoid_(x);
    p = x * s;
    d = s * (1.0f + x * (1.0f - s));
  } else {
    const float s = sigmoid_(2.0f * kGeluC * (x + kGeluA * x * x * x));
    p = x * s;
    // (x bounded: s (1 - s) is 0 long before, and 0 times an overflow is not)
    const float y = fminf(fmaxf(x, -1e15f), 1e15f);
    d = s + 2.0f * kGeluC * y * s * (1.0f - s) * (1.0f + 3.0f * kGeluA * y * y);
  }
}

template <int N, class F>
__device__ __forceinline__ void each(float (&v)[N], F f) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = f(v[i]);
}
// act is the same for the whole grid, so the switch does not diverge
template <int N>
__device__ __forceinline__ void linear_act(int act, float (&v)[N]) {
  switch (act) {
    case MOE_ACT_RELU: each(v, [](float x) { return relu_(x); }); break;
    case MOE_ACT_SILU: each(v, [](float x) { return silu_(x); }); break;
    case MOE_ACT_GELU: each(v, [](float x) { return gelu_(x); }); break;
    case MOE_ACT_SRELU: each(v, [](float x) { const float r = relu_(x); return r * r; }); break;
    default: break;
  }
}
// N / 2 (gate, up) pairs -> N / 2 outputs
template <int N>
__device__ __forceinline__ void linear_glu(int act, const float (&v)[N], float (&u)[N / 2]) {
  if (act == MOE_ACT_SWIGLU) {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) u[i] = silu_(v[2 * i]) * v[2 * i + 1];
  } else {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) u[i] = gelu_(v[2 * i]) * v[2 * i + 1];
  }
}
// the derivative at x times the gradient g
template <int ACT>
__device__ __forceinline__ float linear_dact(float x, float g) {
  if constexpr (ACT == MOE_ACT_RELU) {
    return x > 0.f ? g : (x == x ? 0.f : x);
  } else if constexpr (ACT == MOE_ACT_SRELU) {
    return 2.f * relu_(x) * g;
  } else if constexpr (ACT == MOE_ACT_SILU || ACT == MOE_ACT_GELU) {
    float p, d;
    linear_phi<ACT == MOE_ACT_GELU>(x, p, d);
    return g * d;
  } else {
    return g;
  }
}
// v += N bf16 values at p (16-byte aligned)
template <int N>
__device__ __forceinline__ void add_bf16(const uint16_t* p, float* v) {
#pragma unroll
  for (int i = 0; i < N / 8; ++i) {
    const uint4 w = reinterpret_cast<const uint4*>(p)[i];
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[8 * i + 2 * j] += bf16_lo(u[j]);
      v[8 * i + 2 * j + 1] += bf16_hi(u[j]);
    }
  }
}

}  // namespace moe
