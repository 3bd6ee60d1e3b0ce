// select.cuh - host-side interface of the router's choice by scores (select.cu).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace moe {

constexpr int kSelectMaxK = 32;        // a lane holds each pick
constexpr int kSelectMaxGroups = 32;   // a lane holds each group's score

struct SelectArgs {
  const void* logits;      // [T, E] float32, or bf16 with logits_bf16
  int logits_bf16;
  int T, E, k;
  int score;               // MOE_SCORE_*
  const float* bias;       // [E] or NULL
  int groups, top_groups, best;
  int renorm;
  float scale;
  int32_t* idx;            // [T, k]
  float* probs;            // [T, k]
  // backward (idx and probs are read)
  const float* dprobs;     // [T, k]
  int accumulate;
  void* dlogits;           // [T, E]
  int dlogits_bf16;
};

cudaError_t launch_router_select(const SelectArgs& a, int num_sms, cudaStream_t s);
cudaError_t launch_router_select_bwd(const SelectArgs& a, int num_sms, cudaStream_t s);

}  // namespace moe
