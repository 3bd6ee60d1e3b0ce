// loss.cuh - host-side interface of the router's losses (loss.cu).
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace moe {

constexpr int kMaxSegments = 4096;

struct RouterLossArgs {
  const void* logits;          // [T, E] float32, or bf16 with logits_bf16
  int logits_bf16;
  const int32_t* idx;          // [T, k]
  int T, E, k;
  const int32_t* seg;          // [S+1] or NULL (one segment of all T tokens)
  int S;
  const uint8_t* mask;         // [T] or NULL
  int32_t* err;
  // forward
  float* loss;                 // [2]: balance, z
  int32_t* counts;             // [S, E]
  float* lse;                  // [T]
  int32_t* n_valid;            // [S]
  void* ws;
  // backward (counts, lse and n_valid are read)
  const float* dloss;          // [2]
  const float* probs;          // [T, k] or NULL
  const float* dprobs;         // [T, k]
  void* dlogits;               // [T, E]
  int dlogits_bf16;
};

size_t router_loss_workspace_bytes(int T, int E, int S);
cudaError_t launch_router_loss(const RouterLossArgs& a, int num_sms, cudaStream_t s,
                               int* launches);
cudaError_t launch_router_loss_bwd(const RouterLossArgs& a, int num_sms, cudaStream_t s);

}  // namespace moe
