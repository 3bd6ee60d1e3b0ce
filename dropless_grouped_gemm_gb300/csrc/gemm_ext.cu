// gemm_ext.cu - further instances of the grouped GEMM kernel: the linear
// operator (bias, activation and residual in the epilogue) and the expert
// MLP's FC1 and FC2-dgrad with H kept in 8 bits.  A translation unit of its
// own, so that it compiles beside gemm.cu.
#include "gemm_kernel.cuh"

namespace moe {

cudaError_t launch_gemm_ext(GemmKind kind, int act, const CUtensorMap& ta, const CUtensorMap& tb,
                            const CUtensorMap& tc, const CUtensorMap& td, const GemmArgs& g,
                            int num_sms, cudaStream_t s, bool pair) {
#define MOE_GO(KIND, ACT, Q8)                                                                     \
  (pair ? launch_t<KIND, ACT, false, false, false, true, Q8>(ta, tb, tc, td, g, num_sms, s)       \
        : launch_t<KIND, ACT, false, false, false, false, Q8>(ta, tb, tc, td, g, num_sms, s))
  // the linear epilogue is built gated or not; the activation itself is an
  // argument (a uniform switch per 32 columns, against 128 reduction blocks
  // of MMAs per tile on the benchmark shape)
  const bool gated = act == MOE_ACT_SWIGLU || act == MOE_ACT_GEGLU;
  switch (kind) {
    case GemmKind::kLinearKN:
      return gated ? MOE_GO(GemmKind::kLinearKN, MOE_ACT_SWIGLU, false)
                   : MOE_GO(GemmKind::kLinearKN, MOE_ACT_NONE, false);
    case GemmKind::kLinearNK:
      return gated ? MOE_GO(GemmKind::kLinearNK, MOE_ACT_SWIGLU, false)
                   : MOE_GO(GemmKind::kLinearNK, MOE_ACT_NONE, false);
    case GemmKind::kFc1Act:
      switch (act) {
        case MOE_ACT_SWIGLU: return MOE_GO(GemmKind::kFc1Act, MOE_ACT_SWIGLU, true);
        case MOE_ACT_GEGLU: return MOE_GO(GemmKind::kFc1Act, MOE_ACT_GEGLU, true);
        case MOE_ACT_SRELU: return MOE_GO(GemmKind::kFc1Act, MOE_ACT_SRELU, true);
        default: return cudaErrorInvalidValue;
      }
    case GemmKind::kDgradAct:
      switch (act) {
        case MOE_ACT_SWIGLU: return MOE_GO(GemmKind::kDgradAct, MOE_ACT_SWIGLU, true);
        case MOE_ACT_GEGLU: return MOE_GO(GemmKind::kDgradAct, MOE_ACT_GEGLU, true);
        case MOE_ACT_SRELU: return MOE_GO(GemmKind::kDgradAct, MOE_ACT_SRELU, true);
        default: return cudaErrorInvalidValue;
      }
    default: return cudaErrorInvalidValue;
  }
#undef MOE_GO
}

}  // namespace moe
