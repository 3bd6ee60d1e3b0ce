// gemm.cu - host side of the grouped GEMMs of the expert MLP: pair mode, unit
// order, the launch split of skinny layers (the kernel: gemm_kernel.cuh).
#include <cuda_runtime.h>

#include <atomic>

#include "gemm_kernel.cuh"

namespace moe {
namespace {

// ragged-row kind in pair mode or not, per activation
template <GemmKind KIND, bool MX, bool PAIR>
cudaError_t launch_act(int act, const CUtensorMap& ta, const CUtensorMap& tb,
                       const CUtensorMap& tc, const CUtensorMap& td, const GemmArgs& g,
                       int num_sms, cudaStream_t s) {
  switch (act) {
    case MOE_ACT_SWIGLU: return launch_t<KIND, MOE_ACT_SWIGLU, MX, false, false, PAIR>(ta, tb, tc, td, g, num_sms, s);
    case MOE_ACT_GEGLU: return launch_t<KIND, MOE_ACT_GEGLU, MX, false, false, PAIR>(ta, tb, tc, td, g, num_sms, s);
    case MOE_ACT_SRELU: return launch_t<KIND, MOE_ACT_SRELU, MX, false, false, PAIR>(ta, tb, tc, td, g, num_sms, s);
    default: return cudaErrorInvalidValue;
  }
}

std::atomic<int> g_pair_mode{kPairAuto};

}  // namespace

int pair_mode() { return g_pair_mode.load(); }

int set_pair_mode(int mode) {
  if (mode < kPairNever || mode > kPairAlways) return -1;
  return g_pair_mode.exchange(mode);
}

bool use_pair(GemmKind kind, const GemmArgs& g) {
  if (g.gather_pair != nullptr) return false;
  const int m = g_pair_mode.load();
  if (m == kPairNever) return false;
  if (m == kPairAlways) return true;
  // experts of 256 rows or more on average: a 256-row unit rarely idles a
  // CTA, and the halved stages let six of them cover the load latency
  return static_cast<long long>(g.M_cap) >= static_cast<long long>(kPairRows) * g.E;
}

bool wgrad_skinny(const GemmArgs& g) {
  return static_cast<long long>(g.M_cap) < static_cast<long long>(kSkinnyRows) * g.E;
}

namespace {
// one launch in the given configuration (pair: 2-SM MMAs; skinny: the
// weight gradient's skinny-expert configuration, whose output box tc has)
cudaError_t launch_cfg(GemmKind kind, int act, const CUtensorMap& ta, const CUtensorMap& tb,
                       const CUtensorMap& tc, const CUtensorMap& td, const GemmArgs& g_in,
                       int num_sms, cudaStream_t s, bool mx, bool pair, bool skinny) {
  // Unit order: when an expert has no more row-pair units than column
  // tiles, sweep column tiles outermost, so that a wave of clusters reuses
  // each B column tile across the expert's row pairs while the A block stays
  // in L2; otherwise row pairs outermost.  Measured on the balanced layer
  // (E=8 x 4096 rows, d=8192, n=2048), column order against row order:
  // FC1-dgrad -4.7%, FC2-wgrad -1.4%, FC1 -1.2%, FC2 +2.0%; FC1-wgrad (32
  // row pairs, 16 column tiles) +1.6%, so it keeps row order.
  GemmArgs g = g_in;
  {
    const long long rows = (kind == GemmKind::kWgrad)
                               ? g.R
                               : (static_cast<long long>(g.M_cap) + g.E - 1) / (g.E > 0 ? g.E : 1);
    const long long units_m = ((rows + BM - 1) / BM + kCluster - 1) / kCluster;
    const long long nt = (g.N + BN - 1) / BN;
    g.col_major = units_m <= nt ? 1 : 0;
    // FC1 reads x over K = d (64 MB per expert on the balanced layer), more
    // than an L2 half keeps between two column sweeps: sweeping kRowGroup
    // row pairs at a time re-reads less of it (ncu, two balanced experts:
    // DRAM reads 678 -> 580 MB per launch; groups of 4 read 704 MB), at the
    // same speed
    const bool linear = kind == GemmKind::kLinearKN || kind == GemmKind::kLinearNK;
    if ((kind == GemmKind::kFc1Act || linear) && units_m > kRowGroup) g.col_major = 2;
    if (linear || g.h_q != nullptr) {
      if (mx || g.gather_pair != nullptr) return cudaErrorInvalidValue;
      return launch_gemm_ext(kind, act, ta, tb, tc, td, g, num_sms, s, pair);
    }
  }
  if (g.gather_pair != nullptr) {
    // the gathering producer is its own instantiation, so that the other
    // kernels keep their code and registers
    if (mx) return cudaErrorInvalidValue;
    if (kind == GemmKind::kWgrad)
      return skinny ? launch_t<GemmKind::kWgrad, 0, false, true, true>(ta, tb, tc, td, g, num_sms, s)
                             : launch_t<GemmKind::kWgrad, 0, false, false, true>(ta, tb, tc, td, g, num_sms, s);
#define MOE_GATHER_SWITCH(KIND)                                                                  \
  switch (act) {                                                                                 \
    case MOE_ACT_SWIGLU: return launch_t<KIND, MOE_ACT_SWIGLU, false, false, true>(ta, tb, tc, td, g, num_sms, s); \
    case MOE_ACT_GEGLU: return launch_t<KIND, MOE_ACT_GEGLU, false, false, true>(ta, tb, tc, td, g, num_sms, s);   \
    case MOE_ACT_SRELU: return launch_t<KIND, MOE_ACT_SRELU, false, false, true>(ta, tb, tc, td, g, num_sms, s);   \
    default: return cudaErrorInvalidValue;                                                       \
  }
    if (kind == GemmKind::kFc1Act) MOE_GATHER_SWITCH(GemmKind::kFc1Act)
    if (kind == GemmKind::kDgradAct) MOE_GATHER_SWITCH(GemmKind::kDgradAct)
#undef MOE_GATHER_SWITCH
    return cudaErrorInvalidValue;
  }
  if (mx) {
    if (kind != GemmKind::kFc1Act) return cudaErrorInvalidValue;
    return pair ? launch_act<GemmKind::kFc1Act, true, true>(act, ta, tb, tc, td, g, num_sms, s)
                             : launch_act<GemmKind::kFc1Act, true, false>(act, ta, tb, tc, td, g, num_sms, s);
  }
  if (pair) {
    switch (kind) {
      case GemmKind::kFc1Act: return launch_act<GemmKind::kFc1Act, false, true>(act, ta, tb, tc, td, g, num_sms, s);
      case GemmKind::kDgradAct: return launch_act<GemmKind::kDgradAct, false, true>(act, ta, tb, tc, td, g, num_sms, s);
      case GemmKind::kFc2: return launch_t<GemmKind::kFc2, 0, false, false, false, true>(ta, tb, tc, td, g, num_sms, s);
      case GemmKind::kDgrad: return launch_t<GemmKind::kDgrad, 0, false, false, false, true>(ta, tb, tc, td, g, num_sms, s);
      default: break;   // kWgrad: below
    }
  }
#define MOE_ACT_SWITCH(KIND)                                                         \
  switch (act) {                                                                     \
    case MOE_ACT_SWIGLU: return launch_t<KIND, MOE_ACT_SWIGLU>(ta, tb, tc, td, g, num_sms, s); \
    case MOE_ACT_GEGLU: return launch_t<KIND, MOE_ACT_GEGLU>(ta, tb, tc, td, g, num_sms, s);   \
    case MOE_ACT_SRELU: return launch_t<KIND, MOE_ACT_SRELU>(ta, tb, tc, td, g, num_sms, s);   \
    default: return cudaErrorInvalidValue;                                           \
  }
  switch (kind) {
    case GemmKind::kFc1Act: MOE_ACT_SWITCH(GemmKind::kFc1Act)
    case GemmKind::kDgradAct: MOE_ACT_SWITCH(GemmKind::kDgradAct)
    case GemmKind::kFc2: return launch_t<GemmKind::kFc2, 0>(ta, tb, tc, td, g, num_sms, s);
    case GemmKind::kDgrad: return launch_t<GemmKind::kDgrad, 0>(ta, tb, tc, td, g, num_sms, s);
    case GemmKind::kWgrad:
      if (pair)
        return skinny
                   ? launch_t<GemmKind::kWgrad, 0, false, true, false, true>(ta, tb, tc, td, g, num_sms, s)
                   : launch_t<GemmKind::kWgrad, 0, false, false, false, true>(ta, tb, tc, td, g, num_sms, s);
      return skinny ? launch_t<GemmKind::kWgrad, 0, false, true>(ta, tb, tc, td, g, num_sms, s)
                             : launch_t<GemmKind::kWgrad, 0, false, false>(ta, tb, tc, td, g, num_sms, s);
  }
#undef MOE_ACT_SWITCH
  return cudaErrorInvalidValue;
}
}  // namespace

cudaError_t launch_grouped_gemm(GemmKind kind, int act, const CUtensorMap& ta,
                                const CUtensorMap& tb, const CUtensorMap& tc, const GemmArgs& g,
                                int num_sms, cudaStream_t s, bool mx, const CUtensorMap* td_in,
                                int* launched) {
  const CUtensorMap& td = td_in ? *td_in : tc;
  if (launched) *launched = 1;
  if (g.gather_pair == nullptr && g.row_min == 0 && g.row_max == 0 && g.E > 1 &&
      g_pair_mode.load() == kPairAuto && !use_pair(kind, g)) {
    // A skinny layer's experts of kPairRows rows or more (hot experts of a
    // fine-grained layer) run first with the pair configuration, the rest
    // after them with the single-CTA one.  The two launches write disjoint
    // experts; experts with no rows belong to the second.
    GemmArgs gh = g;
    gh.row_min = kPairRows;
    GemmArgs gl = g;
    gl.row_max = kPairRows;
    const bool wl = (kind == GemmKind::kWgrad);
    cudaError_t e = launch_cfg(kind, act, ta, tb, (wl && td_in) ? *td_in : tc, td, gh, num_sms, s,
                               mx, true, wl && !td_in && wgrad_skinny(g));
    if (e != cudaSuccess) return e;
    if (launched) *launched = 2;
    return launch_cfg(kind, act, ta, tb, tc, td, gl, num_sms, s, mx, false, wgrad_skinny(g));
  }
  return launch_cfg(kind, act, ta, tb, tc, td, g, num_sms, s, mx, use_pair(kind, g),
                    wgrad_skinny(g));
}

}  // namespace moe
