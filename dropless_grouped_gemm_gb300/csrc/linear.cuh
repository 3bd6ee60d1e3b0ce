// linear.cuh - host-side interface of the linear operator's own kernels
// (linear.cu): the product for few rows, and the elementwise part of its
// backward.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace moe {

struct FewArgs {
  const int32_t* offsets;    // [E+1] device; NULL (E = 1): all M_cap rows
  int E, M_cap, K, N;
  const uint16_t* bias;      // [E, N] or NULL
  int act;                   // MOE_ACT_*
  const uint16_t* residual;  // [M_cap, ldo] or NULL
  uint16_t* z;               // [M_cap, N] or NULL
  uint16_t* out;             // [M_cap, ldo] bf16, or
  float* out_f32;            // float32
  long long ldo;
  int32_t* err;
};

// How the few-row kernel serves a product of this size: tokens per tile (0:
// it does not, the 128 x 256-tile kernel does; bf16 outputs only), how many
// parts of K the CTAs of a cluster take, whether two CTAs form a pair over
// 256 columns, and the rows of a's box that a CTA loads.
struct FewPlan {
  int tn = 0;
  int split = 1;
  bool pair = false;
  int x_rows = 0;
};
FewPlan few_plan(int E, int M_cap, int K, int N, bool ragged, bool f32, int num_sms);

// tw: the weights [E, K, N] (kn) or [E, N, K] (nk) with boxes of 64 columns x
// 64 rows; tx: a [M_cap, K] with 64 x plan.x_rows
cudaError_t launch_few(const CUtensorMap& tw, const CUtensorMap& tx, bool kn, const FewArgs& g,
                       const FewPlan& plan, int num_sms, cudaStream_t s);

// dz = act'(z) dout (bf16; NULL with act none: dz is dout) and the bias
// gradient's column sums of each expert, from the float32 dz
struct LinearDzArgs {
  const uint16_t* dout;      // [M_cap, N or N/2]
  const uint16_t* z;         // [M_cap, N] or NULL (act none)
  const int32_t* offsets;    // as FewArgs
  int E, M_cap, N, act;
  uint16_t* dz;              // [M_cap, N] or NULL
  float* dbias;              // [E, N] or NULL
  int accumulate;            // dbias += the sums
  float* part;               // workspace
  uint32_t* top;             // dz's largest finite magnitude, as bits: raised to it; or NULL
  int blocks;                // row blocks of the grid (set by the launcher)
  int32_t* err;
};
size_t linear_dz_workspace_bytes(int E, int M_cap, int N);
cudaError_t launch_linear_dz(const LinearDzArgs& g, cudaStream_t s, int* launches);

}  // namespace moe
