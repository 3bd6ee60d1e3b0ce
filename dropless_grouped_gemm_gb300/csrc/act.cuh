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

template <class F>
__device__ __forceinline__ void each32(float (&v)[32], F f) {
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = f(v[i]);
}
// act is the same for the whole grid, so the switch does not diverge
__device__ __forceinline__ void linear_act32(int act, float (&v)[32]) {
  switch (act) {
    case MOE_ACT_RELU: each32(v, [](float x) { return relu_(x); }); break;
    case MOE_ACT_SILU: each32(v, [](float x) { return gate_phi<MOE_ACT_SWIGLU>(x); }); break;
    case MOE_ACT_GELU: each32(v, [](float x) { return gate_phi<MOE_ACT_GEGLU>(x); }); break;
    case MOE_ACT_SRELU: each32(v, [](float x) { const float r = relu_(x); return r * r; }); break;
    default: break;
  }
}
// 16 (gate, up) pairs -> 16 outputs
__device__ __forceinline__ void glu16(int act, const float (&v)[32], float (&u)[16]) {
  if (act == MOE_ACT_SWIGLU) {
#pragma unroll
    for (int i = 0; i < 16; ++i) u[i] = gate_phi<MOE_ACT_SWIGLU>(v[2 * i]) * v[2 * i + 1];
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) u[i] = gate_phi<MOE_ACT_GEGLU>(v[2 * i]) * v[2 * i + 1];
  }
}
// one value (not gated), and its derivative times the gradient
__device__ __forceinline__ float linear_act1(int act, float x) {
  switch (act) {
    case MOE_ACT_RELU: return relu_(x);
    case MOE_ACT_SILU: return gate_phi<MOE_ACT_SWIGLU>(x);
    case MOE_ACT_GELU: return gate_phi<MOE_ACT_GEGLU>(x);
    case MOE_ACT_SRELU: { const float r = relu_(x); return r * r; }
    default: return x;
  }
}
template <int ACT>
__device__ __forceinline__ float linear_dact(float x, float g) {
  if constexpr (ACT == MOE_ACT_RELU) {
    return x > 0.f ? g : (x == x ? 0.f : x);
  } else if constexpr (ACT == MOE_ACT_SRELU) {
    return 2.f * relu_(x) * g;
  } else if constexpr (ACT == MOE_ACT_SILU || ACT == MOE_ACT_GELU) {
    float p, d;
    gate_phi_dphi<ACT == MOE_ACT_SILU ? MOE_ACT_SWIGLU : MOE_ACT_GEGLU>(x, p, d);
    return g * d;
  } else {
    return g;
  }
}
// v += 32 (16) bf16 values at p (16-byte aligned)
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
__device__ __forceinline__ void add_bf16x32(const uint16_t* p, float (&v)[32]) { add_bf16<32>(p, v); }
__device__ __forceinline__ void add_bf16x16(const uint16_t* p, float (&v)[16]) { add_bf16<16>(p, v); }

}  // namespace moe
