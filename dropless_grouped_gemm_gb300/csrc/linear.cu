// linear.cu - the linear operator where it has few rows, and the elementwise
// part of its backward.
//
// out_e = act(a_e B_e + bias_e) + residual.  With few rows per expert (a
// token or a small batch in decoding, a router's gate) the product reads
// every weight once for little arithmetic: it is bound by the weights' bytes
// and by how many SMs stream them.  Tiles of 128 rows x 256 columns would
// leave most SMs idle (a dense K x 4096 layer has 16) and load 128 rows of
// `a` for one.  So the tile is turned: the weights are the MMA's M operand
// (128 output columns x 64 of K, 16 KB) and TN = 16..128 tokens its N
// operand, D[column, token] in TMEM; and `split` CTAs of a cluster share one
// tile's reduction, each streaming its part of K into its own TMEM.  They
// join through distributed shared memory: each CTA leaves its float32
// partials in its own buffer, and token t's sum is formed by one of the CTAs
// in the order of the ranks, so reruns are bitwise identical and no
// workspace, atomic or second launch is needed.
//
// A dense product with more tokens than 64 (a gate over a batch, a large
// decode batch) has arithmetic to do.  There two CTAs form a pair (2-SM MMAs,
// tcgen05.mma.cta_group::2): 256 columns x 128 tokens, each CTA with its 128
// columns of the weights and 64 of the tokens, 24 KB a stage instead of 32
// (8192 x 4096 x 4096 float32: 221 us against 293 without pairs).
//
// The tensor cores add into their float32 accumulator with less than a
// float32 addition's rounding, an error that grows with the number of
// additions (K = 7168 in one chain: 3.7e-6 of the result, against 8.4e-7 for
// a float32 product).  A float32 output therefore ends its chains after 64
// additions an accumulator and adds them in shared memory: 8.5e-7.  A stage's
// MMAs take two accumulators in turn, which the epilogue adds: half as many
// drains of these chains (221 us against 287 with one accumulator; bf16, 512
// x 4096 x 4096, 23.4 against 24.4).
//
// Roles (192 threads, one CTA an SM, so that the stages can hold 130 to 200
// KB of loads in flight): warp 0 TMA producer, warp 1 TMEM owner and MMA
// issuer, warps 2-5 epilogue.  (Eight epilogue warps shorten a single tile's
// output pass, and slowed the streaming of many tiles by 4 to 6%.)
#include <cuda_runtime.h>

#include "act.cuh"
#include "drain.cuh"
#include "linear.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int FT = 192;               // threads
constexpr int FE = 4;                 // epilogue warps, one for each TMEM lane quadrant
constexpr int FM = 128;               // output columns per tile
constexpr int FK = 64;                // reduction elements per stage
constexpr int W_BYTES = FM * FK * 2;  // 16 KB
constexpr int W_BOX = 64 * FK * 2;    // a 64 (columns) x 64 (K) box
constexpr int MAX_SPLIT = 8;
constexpr int PAIR_TN = 128;          // tokens of a pair's tile
constexpr int NACC = 2;               // accumulators that a stage's MMAs take in turn
constexpr int CHAIN = 64;             // MMAs per accumulation chain, float32 output

template <int TN, bool PAIR>
struct FC {
  static constexpr int x_rows = PAIR ? TN / 2 : TN;
  static constexpr int x_bytes = x_rows * FK * 2;
  static constexpr int stage_bytes = W_BYTES + x_bytes;
  static constexpr int stages = PAIR ? 6 : TN == 16 ? 11 : TN == 32 ? 9 : TN == 64 ? 7 : 4;
  static constexpr int red_bytes = TN * FM * 4;   // the tile's float32 sums
  static constexpr int tmem_cols = 2 * NACC * TN;   // two buffers: 64 to 512, a power of two
  static constexpr size_t smem(int E) {
    return 1024 + static_cast<size_t>(stages) * stage_bytes + red_bytes + (2 * stages + 7) * 8 +
           16 + 2 * (E + 1) * 4;
  }
};

struct FTile {
  int e, row0, rows, n0;
};

// unit u -> tile: an expert's units run over its token tiles first, so that
// consecutive units share their weights through L2.  Dense (no offsets): by
// arithmetic alone.  Pair: 256 columns, of which CTA sh has 128.
template <int TN, bool PAIR>
__device__ __forceinline__ FTile few_tile(const FewArgs& g, const int* s_off, const int* s_ts,
                                          int u, int sh) {
  int lo = 0, first = 0, rows = g.M_cap, at = 0;
  if (g.offsets != nullptr) {
    int hi = g.E - 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (s_ts[mid + 1] <= u) lo = mid + 1;
      else hi = mid;
    }
    rows = s_off[lo + 1] - s_off[lo];
    first = s_off[lo];
    at = s_ts[lo];
  }
  const int tt = (rows + TN - 1) / TN;
  const int local = u - at;
  const int ni = local / tt;
  const int ti = local - ni * tt;
  FTile t;
  t.e = lo;
  t.row0 = first + ti * TN;
  t.rows = min(TN, rows - ti * TN);
  t.n0 = PAIR ? (2 * ni + sh) * FM : ni * FM;
  return t;
}

// 8 float32 values from the same place in each CTA of a split (ranks first,
// first + stride, ...), loaded, then added in the order of the ranks
template <int S>
__device__ __forceinline__ void load8(const float* p, int first, int stride, float (&w)[S][8]) {
  const uint32_t at = smem_u32(p);
#pragma unroll
  for (int r = 0; r < S; ++r) {
    if constexpr (S == 1) {
      const float4 a = *reinterpret_cast<const float4*>(p);
      const float4 b = *reinterpret_cast<const float4*>(p + 4);
      w[0][0] = a.x; w[0][1] = a.y; w[0][2] = a.z; w[0][3] = a.w;
      w[0][4] = b.x; w[0][5] = b.y; w[0][6] = b.z; w[0][7] = b.w;
    } else {
      const uint32_t pa = mapa_shared(at, first + r * stride);
      ld_cluster_v4(pa, w[r][0], w[r][1], w[r][2], w[r][3]);
      ld_cluster_v4(pa + 16, w[r][4], w[r][5], w[r][6], w[r][7]);
    }
  }
}
template <int S>
__device__ __forceinline__ void add8(const float (&w)[S][8], float (&z)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    z[i] = w[0][i];
#pragma unroll
    for (int r = 1; r < S; ++r) z[i] += w[r][i];
  }
}

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                    pack_bf16x2(v[6], v[7]));
}

// 8 neighbouring columns from c (a multiple of 8 below N) of row `row`: bias,
// pre-activation, activation, residual, output
template <bool GATED>
__device__ __forceinline__ void few_out(const FewArgs& g, long long row, int c, const uint4& bias,
                                        float (&z)[8]) {
  const uint32_t b[4] = {bias.x, bias.y, bias.z, bias.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    z[2 * i] += bf16_lo(b[i]);
    z[2 * i + 1] += bf16_hi(b[i]);
  }
  if (g.z != nullptr) *reinterpret_cast<uint4*>(g.z + row * g.N + c) = pack8(z);
  if constexpr (!GATED) {
    linear_act(g.act, z);
    const long long at = row * g.ldo + c;
    if (g.residual != nullptr) add_bf16<8>(g.residual + at, z);
    if (g.out_f32 != nullptr) {
      float4* o = reinterpret_cast<float4*>(g.out_f32 + at);
      o[0] = make_float4(z[0], z[1], z[2], z[3]);
      o[1] = make_float4(z[4], z[5], z[6], z[7]);
    } else {
      *reinterpret_cast<uint4*>(g.out + at) = pack8(z);
    }
  } else {
    float v[4];
    linear_glu(g.act, z, v);
    const long long at = row * g.ldo + c / 2;
    if (g.residual != nullptr) {
      const uint2 r = *reinterpret_cast<const uint2*>(g.residual + at);
      v[0] += bf16_lo(r.x); v[1] += bf16_hi(r.x); v[2] += bf16_lo(r.y); v[3] += bf16_hi(r.y);
    }
    if (g.out_f32 != nullptr)
      *reinterpret_cast<float4*>(g.out_f32 + at) = make_float4(v[0], v[1], v[2], v[3]);
    else
      *reinterpret_cast<uint2*>(g.out + at) =
          make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
  }
}

// the accumulators' columns of the tile's tokens of this thread's lane into its
// column of the tile's sums (put, or added to what earlier chains left)
template <int TN>
__device__ __forceinline__ void take_chain(uint32_t tb, int tokens, bool first, float* col) {
#pragma unroll 1
  for (int t = 0; t < tokens; t += 16) {
    uint32_t r[NACC][16];
#pragma unroll
    for (int a = 0; a < NACC; ++a) tmem_ld16(tb + a * TN + t, r[a]);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float v = first ? 0.f : col[(t + i) * FM];
#pragma unroll
      for (int a = 0; a < NACC; ++a) v += __uint_as_float(r[a][i]);
      col[(t + i) * FM] = v;
    }
  }
}

// the output pass of one tile for a split over S CTAs: a thread takes 8
// neighbouring columns from c of a token, 16 threads a token, tokens rank,
// rank + S, ...; as many tokens' loads in flight as 64 registers hold
template <bool GATED, int S>
__device__ __forceinline__ void few_store(const FewArgs& g, const FTile& t, const float* src,
                                          int k0, int c, const uint4& bias, int first, int stride) {
  constexpr int U = S <= 2 ? 4 : S == 4 ? 2 : 1;
  constexpr int STEP = 2 * FE * S;
#pragma unroll 1
  for (int k = k0; k < t.rows; k += U * STEP) {
    float w[U][S][8];
#pragma unroll
    for (int b = 0; b < U; ++b)
      if (k + b * STEP < t.rows) load8<S>(src + (k + b * STEP) * FM, first, stride, w[b]);
#pragma unroll
    for (int b = 0; b < U; ++b)
      if (k + b * STEP < t.rows) {
        float z[8];
        add8<S>(w[b], z);
        few_out<GATED>(g, static_cast<long long>(t.row0) + k + b * STEP, c, bias, z);
      }
  }
}

template <bool KN, int TN, bool GATED, bool PAIR>
__global__ void __launch_bounds__(FT, 1)
    few_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
               const FewArgs g) {
  using C = FC<TN, PAIR>;
  constexpr int NST = C::stages;
  constexpr int SH = PAIR ? 2 : 1;
  constexpr uint32_t IDESC = idesc_bf16(SH * FM, TN, KN, false);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  float* red = reinterpret_cast<float*>(smem + NST * C::stage_bytes);   // [TN][FM]
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(red) + C::red_bytes);
  uint64_t* empty_bar = full_bar + NST;
  uint64_t* tfull_bar = empty_bar + NST;
  uint64_t* tempty_bar = tfull_bar + 2;
  uint64_t* rfull_bar = tempty_bar + 2;    // every CTA's partials are in its buffer
  uint64_t* rempty_bar = rfull_bar + 1;    // every CTA has read this CTA's partials
  uint64_t* drain_bar = rempty_bar + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain_bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint32_t* loads = tmem_slot + 2;    // stages loaded: by this CTA, by the pair's second
  int* s_off = reinterpret_cast<int*>(tmem_slot + 4);
  int* s_ts = s_off + (g.E + 1);

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);   // (uniform to the compiler too)
  const int lane = threadIdx.x & 31;
  // the cluster: split parts of K, each a CTA or a pair
  const int csize = static_cast<int>(cluster_nctarank());
  const int crank = static_cast<int>(cluster_ctarank());
  const int split = csize / SH;
  const int sh = crank % SH;
  const int rank = crank / SH;
  const uint16_t pair = static_cast<uint16_t>(3u << (crank - sh));   // both CTAs of the pair
  const int unit0 = blockIdx.x / csize;
  const int unit_step = gridDim.x / csize;
  const int nt = (g.N + SH * FM - 1) / (SH * FM);
  const int kblocks = g.K / FK;
  const int kb0 = static_cast<int>(static_cast<long long>(kblocks) * rank / split);
  const int kb1 = static_cast<int>(static_cast<long long>(kblocks) * (rank + 1) / split);
  const int chain = g.out_f32 != nullptr ? CHAIN * NACC / (FK / 16) : kblocks;   // in stages

  // a pair's bytes all count on its first CTA's barrier
  const uint32_t full0 = PAIR ? mapa_shared(smem_u32(full_bar), crank - sh) : 0u;
  auto load = [&](const FTile& t, int kb, int stage) {
    uint8_t* sw = smem + stage * C::stage_bytes;
    uint64_t* fb = &full_bar[stage];
    const uint32_t fbc = full0 + stage * 8;
    if (!PAIR || sh == 0) mbar_arrive_expect_tx(fb, SH * C::stage_bytes);
    // the weights' 16 KB in one load (KN: two groups of 64 columns)
    if constexpr (KN) {
      if constexpr (PAIR) tma_load_4d_pair(sw, &tmW, fbc, 0, kb * FK, t.n0 / 64, t.e);
      else tma_load_4d(sw, &tmW, fb, 0, kb * FK, t.n0 / 64, t.e);
    } else {
      if constexpr (PAIR) tma_load_3d_pair(sw, &tmW, fbc, kb * FK, t.n0, t.e);
      else tma_load_3d(sw, &tmW, fb, kb * FK, t.n0, t.e);
    }
    if constexpr (PAIR) tma_load_2d_pair(sw + W_BYTES, &tmX, fbc, kb * FK, t.row0 + C::x_rows * sh);
    else tma_load_2d(sw + W_BYTES, &tmX, fb, kb * FK, t.row0);
  };
  // a role that gives up takes the pair's other CTA with it
  auto gave_up = [&](bool ok) {
    if (PAIR && !ok && elect_one())
      st_cluster_u32(mapa_shared(smem_u32(const_cast<int*>(abort_flag)), crank ^ 1), 1u);
  };
  int ahead = 0;      // stages of the first unit that are already loading

  if (warp == 0) {
    if (lane == 0) {
      for (int i = 0; i < NST; ++i) {
        mbar_init(&full_bar[i], 1);
        mbar_init(&empty_bar[i], 1);
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(&tfull_bar[i], 1);
        mbar_init(&tempty_bar[i], SH * FE);   // a pair's first CTA issues for both
      }
      mbar_init(rfull_bar, FE * split);
      mbar_init(rempty_bar, FE * split);
      mbar_init(drain_bar, 1);
      *abort_flag = 0;
      fence_mbar_init();
    }
    __syncwarp();
    // dense: the first unit is known, so its loads start before anything else
    if (!PAIR && g.offsets == nullptr && unit0 < nt * ((g.M_cap + TN - 1) / TN)) {
      const FTile t = few_tile<TN, PAIR>(g, nullptr, nullptr, unit0, sh);
      ahead = min(NST, kb1 - kb0);
      if (elect_one())
        for (int i = 0; i < ahead; ++i) load(t, kb0 + i, i);
      __syncwarp();
    }
  }
  if (warp == 1) {
    if constexpr (PAIR) tmem_alloc_pair(tmem_slot, C::tmem_cols);
    else tmem_alloc(tmem_slot, C::tmem_cols);
  }
  if (warp == 2 && g.offsets != nullptr) {
    // offsets made safe (within [0, M_cap], non-decreasing by their running
    // maximum, as in the grouped GEMM) and the experts' first units, 32
    // experts at a time
    bool bad = false;
    int top = 0, carry = 0;
    for (int base = 0; base <= g.E; base += 32) {
      const int i = base + lane;
      const int raw = i <= g.E ? g.offsets[i] : 0;
      int m = max(min(max(raw, 0), g.M_cap), top);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, m, o);
        if (lane >= o) m = max(m, y);
      }
      if (i <= g.E) {
        if (m != raw || (i == 0 && m != 0)) bad = true;
        s_off[i] = m;
      }
      // expert i - 1 ends at m
      int prev = __shfl_up_sync(0xffffffffu, m, 1);
      if (lane == 0) prev = top;
      int c = (i >= 1 && i <= g.E) ? (m - prev + TN - 1) / TN * nt : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, c, o);
        if (lane >= o) c += y;
      }
      if (i <= g.E) s_ts[i] = carry + c;
      top = __shfl_sync(0xffffffffu, m, 31);
      carry += __shfl_sync(0xffffffffu, c, 31);
    }
    if (__any_sync(0xffffffffu, bad) && lane == 0 && blockIdx.x == 0) set_err(g.err, MOE_DEV_BAD_OFFSETS);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // the peers' barriers are initialised before the epilogue arrives on them
  // (it waits then; everything before runs ahead), and before a pair's loads
  // and commits
  cluster_arrive();
  if constexpr (PAIR) cluster_wait();

  const uint32_t tmem_base = *tmem_slot;
  const int units =
      g.offsets != nullptr ? s_ts[g.E] : nt * ((g.M_cap + TN - 1) / TN);

  if (warp == 0) {
    // the whole warp walks the stages, one elected lane issues (as the MMA
    // warp does, and for the same reason)
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true, ready = false;
    uint32_t issued = ahead;          // stages loaded so far
    for (int u = unit0; u < units && ok; u += unit_step) {
      const FTile t = few_tile<TN, PAIR>(g, s_off, s_ts, u, sh);
      for (int kb = kb0; kb < kb1; ++kb) {
        const int ns = stage + 1 == NST ? 0 : stage + 1;
        if (ahead > 0) {
          --ahead;
        } else {
          if (!ready) {
            ok = __all_sync(0xffffffffu, mbar_wait(&empty_bar[stage], phase ^ 1, abort_flag));
            if (!ok) break;
          }
          const bool next = mbar_test(&empty_bar[ns], ns == 0 ? phase : phase ^ 1);
          if (elect_one()) load(t, kb, stage);
          ready = __all_sync(0xffffffffu, next);
          ++issued;
        }
        stage = ns;
        if (ns == 0) phase ^= 1;
      }
    }
    if (elect_one()) {
      if (PAIR && sh != 0) st_cluster_u32(mapa_shared(smem_u32(loads + 1), crank - 1), issued);
      else loads[0] = issued;
    }
    gave_up(ok);
    __syncwarp();
    if constexpr (!PAIR) cluster_wait();
  } else if (warp == 1) {
    // The whole warp walks the stages, one elected lane issues: with stage,
    // addresses and descriptors warp-uniform the four MMAs of a stage cost
    // few cycles to issue.  (Issued from a branch on the lane they took 330
    // cycles, more than the MMAs themselves and, with the wait, than the
    // stage's loads: 0.27 us a stage whatever the tile.)
    if (sh == 0) {      // a pair's first CTA issues for both
      int stage = 0;
      uint32_t phase = 0;
      int local = 0;                    // chains so far
      bool ok = true;
      bool ready = false;               // the stage was seen full ahead of its turn
      const uint32_t w_lo0 = sdesc_lo(smem_u32(smem), KN ? W_BOX : 16);
      const uint32_t x_lo0 = sdesc_lo(smem_u32(smem) + W_BYTES, 16);
      for (int u = unit0; u < units && ok; u += unit_step) {
        for (int c0 = kb0; c0 < kb1 && ok; c0 += chain, ++local) {
          const int buf = local & 1;
          const uint32_t tph = ((local >> 1) & 1) ^ 1;
          ok = __all_sync(0xffffffffu, PAIR ? mbar_wait_cluster(&tempty_bar[buf], tph, abort_flag)
                                            : mbar_wait(&tempty_bar[buf], tph, abort_flag));
          if (!ok) break;
          tc_fence_after();
          const uint32_t d0 = tmem_base + buf * (NACC * TN);
          const int c1 = min(c0 + chain, kb1);
          for (int kb = c0; kb < c1; ++kb) {
            if (!ready) {
              ok = __all_sync(0xffffffffu, mbar_wait(&full_bar[stage], phase, abort_flag));
              if (!ok) break;
            }
            tc_fence_after();
            // look at the next stage while this one's MMAs are issued
            const int ns = stage + 1 == NST ? 0 : stage + 1;
            const bool next = mbar_test(&full_bar[ns], ns == 0 ? phase ^ 1 : phase);
            const uint32_t w_lo = w_lo0 + stage * (C::stage_bytes >> 4);
            const uint32_t x_lo = x_lo0 + stage * (C::stage_bytes >> 4);
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < FK / 16; ++kk) {
                const uint64_t wd = sdesc_of(w_lo + kk * (KN ? 2048 >> 4 : 32 >> 4));
                const uint64_t xd = sdesc_of(x_lo + kk * (32 >> 4));
                const uint32_t d = d0 + (kk % NACC) * TN;
                const uint32_t add = (kb > c0 || kk >= NACC) ? 1u : 0u;
                if constexpr (PAIR) umma_bf16_pair(d, wd, xd, IDESC, add);
                else umma_bf16(d, wd, xd, IDESC, add);
              }
              if constexpr (PAIR) umma_commit_pair_mask(&empty_bar[stage], pair);
              else umma_commit(&empty_bar[stage]);
            }
            ready = __all_sync(0xffffffffu, next);
            stage = ns;
            if (ns == 0) phase ^= 1;
          }
          if (ok && elect_one()) {
            if constexpr (PAIR) umma_commit_pair_mask(&tfull_bar[buf], pair);
            else umma_commit(&tfull_bar[buf]);
          }
          __syncwarp();
        }
      }
      gave_up(ok);
    }
    __syncwarp();
    if constexpr (!PAIR) cluster_wait();
  } else {
    const int q = warp & 3;                 // TMEM lane quadrant
    const int tid = q * 32 + lane;          // its column of the tile, then its place in the output pass
    int local = 0, mine = 0;                // chains and units so far
    bool ok = true, joined = PAIR;
    const uint32_t tempty0 = PAIR ? mapa_shared(smem_u32(tempty_bar), crank - sh) : 0u;
    for (int u = unit0; u < units && ok; u += unit_step, ++mine) {
      const FTile t = few_tile<TN, PAIR>(g, s_off, s_ts, u, sh);
      // the output's part of the tile: a thread takes 8 neighbouring columns
      // of a token, 16 threads a token, tokens rank, rank + split, ...  What
      // it reads there is on its way while the tile is computed.
      const int c = t.n0 + (tid & 15) * 8;
      uint4 bias = make_uint4(0, 0, 0, 0);
      if (c < g.N) {
        if (g.bias != nullptr)
          bias = __ldg(reinterpret_cast<const uint4*>(g.bias + static_cast<long long>(t.e) * g.N + c));
        const int k = rank + (tid >> 4) * split;
        if (g.residual != nullptr && k < t.rows)
          prefetch_l2(g.residual + (static_cast<long long>(t.row0) + k) * g.ldo + (GATED ? c / 2 : c));
      }
      for (int c0 = kb0; c0 < kb1 && ok; c0 += chain, ++local) {
        const int buf = local & 1;
        if (lane == 0) {
          ok = mbar_wait(&tfull_bar[buf], (local >> 1) & 1, abort_flag);
          // the previous unit's sums have been read
          if (ok && c0 == kb0)
            ok = mbar_wait_cluster(rempty_bar, (mine & 1) ^ 1, abort_flag);
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        __syncwarp();     // what lane 0 acquired orders every lane's writes
        tc_fence_after();
        take_chain<TN>(
            tmem_base + (static_cast<uint32_t>(q * 32) << 16) + buf * (NACC * TN), t.rows,
            c0 == kb0, red + tid);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (PAIR && sh != 0) mbar_arrive_cluster(tempty0 + buf * 8);
          else mbar_arrive(&tempty_bar[buf]);
        }
      }
      if (!joined) {      // every CTA of the cluster has its barriers
        cluster_wait();
        joined = true;
      }
      // The tile's sums are in shared memory, a CTA's part in each; tell
      // every CTA of the cluster (split 1: this CTA's other warps), and wait
      // for all.
      __syncwarp();
      if (ok) {
        if (lane < split) mbar_arrive_cluster(mapa_shared(smem_u32(rfull_bar), lane * SH + sh));
        if (lane == 0) ok = mbar_wait_cluster(rfull_bar, mine & 1, abort_flag);
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      // every lane reads what other warps wrote, so every lane acquires (the
      // phase is complete and the next one needs this warp: no waiting)
      while (!mbar_try_wait_cluster(smem_u32(rfull_bar), mine & 1) && !*abort_flag) {}
      if (c < g.N) {
        const float* src = red + (tid & 15) * 8;
        const int k0 = rank + (tid >> 4) * split;
        switch (split) {
          case 1: few_store<GATED, 1>(g, t, src, k0, c, bias, sh, SH); break;
          case 2: few_store<GATED, 2>(g, t, src, k0, c, bias, sh, SH); break;
          case 4: few_store<GATED, 4>(g, t, src, k0, c, bias, sh, SH); break;
          default:
            if constexpr (!PAIR) few_store<GATED, 8>(g, t, src, k0, c, bias, sh, SH);
        }
      }
      // this warp has read its peers' sums: the arrival releases the reads of
      // all its lanes, after which the peers overwrite what was read
      __syncwarp();
      if (lane < split) mbar_arrive_cluster(mapa_shared(smem_u32(rempty_bar), lane * SH + sh));
    }
    if (!joined) cluster_wait();
    gave_up(ok);
  }

  tc_fence_before();
  __syncwarp();
  // no CTA leaves while a peer may still read its sums or arrive on it: the
  // arrival releases this thread's reads of and arrivals on its peers
  cluster_sync();
  if (*abort_flag && threadIdx.x == 0) set_err(g.err, MOE_DEV_TIMEOUT);
  if (warp == 1) {
    // Given up (both CTAs of a pair, or neither): what is in flight ends
    // (waits bounded) before TMEM is freed and shared memory left: the MMAs
    // already issued, then the copies, a pair's on its first CTA's barriers;
    // the second waits for the first's word.
    if (*abort_flag && elect_one()) {
      const uint64_t t0 = globaltimer_ns();
      auto ends = [&](uint64_t* bar, uint32_t parity, uint64_t limit_ns) {
        const uint32_t a = smem_u32(bar);
        for (;;)
          if (mbar_try_wait(a, parity) || globaltimer_ns() - t0 > limit_ns) break;
      };
      if (sh == 0) {
        if constexpr (PAIR) umma_commit_pair(drain_bar);
        else umma_commit(drain_bar);
        ends(drain_bar, 0, kWaitLimitNs);
        for (uint32_t i = 0; i < NST; ++i) {
          const StageDrain d = stage_drain(loads[0], PAIR ? loads[1] : loads[0], NST, i);
          if (d.make_up) mbar_complete_tx(&full_bar[i], C::stage_bytes);
          if (d.arrive) mbar_arrive_expect_tx(&full_bar[i], C::stage_bytes);
          if (d.wait) ends(&full_bar[i], d.parity, 2 * kWaitLimitNs);
        }
        if constexpr (PAIR) mbar_arrive_cluster(mapa_shared(smem_u32(drain_bar), crank + 1));
      } else {
        ends(drain_bar, 0, 3 * kWaitLimitNs);
      }
    }
    __syncwarp();
    tc_fence_after();
    if constexpr (PAIR) tmem_dealloc_pair(tmem_base, C::tmem_cols);
    else tmem_dealloc(tmem_base, C::tmem_cols);
  }
}

constexpr int kMaxDevices = 64;

int split_index(int split) { return split == 1 ? 0 : split == 2 ? 1 : split == 4 ? 2 : 3; }

void few_config(cudaLaunchConfig_t& cfg, cudaLaunchAttribute& at, int split) {
  cfg.blockDim = dim3(FT);
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = split;
  at.val.clusterDim.y = 1;
  at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
}

// Clusters of `split` CTAs (any kernel's), one an SM, that the device holds at
// once (a GPC's SMs are not a multiple of 8: 152, 76, 36 and 15 for 1, 2, 4 and
// 8), found once per device.  It sizes grids only; no cluster waits for another.
int few_clusters(int split, int num_sms) {
  static int known[kMaxDevices][4] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return num_sms / split;
  int& k = known[dev][split_index(split)];
  if (k == 0) {
    auto kern = few_kernel<true, 16, false, false>;
    const int smem = static_cast<int>(FC<16, false>::smem(1));
    int n = 0;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at;
    few_config(cfg, at, split);
    cfg.gridDim = dim3(num_sms / split * split);
    cfg.dynamicSmemBytes = smem;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(FC<16, false>::smem(MOE_MAX_EXPERTS))) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n < 1)
      n = num_sms / split;
    k = n < 1 ? 1 : n;
  }
  return k;
}

long long few_units(int E, int M_cap, int N, int tn, bool pair, bool ragged) {
  const long long nt = (N + (pair ? 2 : 1) * FM - 1) / ((pair ? 2 : 1) * FM);
  // ragged: an upper bound over all ways the rows can lie
  const long long tiles = ragged ? static_cast<long long>(M_cap) / tn + (E < M_cap ? E : M_cap)
                                 : (static_cast<long long>(M_cap) + tn - 1) / tn;
  return nt * tiles;
}

template <bool KN, int TN, bool GATED, bool PAIR>
cudaError_t few_t(const CUtensorMap& tw, const CUtensorMap& tx, const FewArgs& g, int split,
                  int num_sms, cudaStream_t s) {
  using C = FC<TN, PAIR>;
  auto kern = few_kernel<KN, TN, GATED, PAIR>;
  static_assert(C::smem(MOE_MAX_EXPERTS) <= 227 * 1024, "shared memory of a CTA");
  static bool set[kMaxDevices] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  if (!set[dev]) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(C::smem(MOE_MAX_EXPERTS)));
    if (e != cudaSuccess) return e;
    set[dev] = true;
  }
  constexpr int SH = PAIR ? 2 : 1;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at;
  few_config(cfg, at, SH * split);
  cfg.stream = s;
  const long long units = few_units(g.E, g.M_cap, g.N, TN, PAIR, g.offsets != nullptr);
  const long long fit = few_clusters(SH * split, num_sms);
  cfg.gridDim = dim3(static_cast<unsigned>((units < fit ? units : fit) * SH * split));
  cfg.dynamicSmemBytes = C::smem(g.E);
  return cudaLaunchKernelEx(&cfg, kern, tw, tx, g);
}

template <bool KN, bool GATED>
cudaError_t few_tn(const CUtensorMap& tw, const CUtensorMap& tx, const FewArgs& g,
                   const FewPlan& p, int num_sms, cudaStream_t s) {
  switch (p.tn) {
    case 16: return few_t<KN, 16, GATED, false>(tw, tx, g, p.split, num_sms, s);
    case 32: return few_t<KN, 32, GATED, false>(tw, tx, g, p.split, num_sms, s);
    case 64: return few_t<KN, 64, GATED, false>(tw, tx, g, p.split, num_sms, s);
    case 128:
      return p.pair ? few_t<KN, PAIR_TN, GATED, true>(tw, tx, g, p.split, num_sms, s)
                    : few_t<KN, 128, GATED, false>(tw, tx, g, p.split, num_sms, s);
    default: return cudaErrorInvalidValue;
  }
}

// ------------------------------------------------------------- backward
// dz = act'(z) dout and the bias gradient, bound by HBM: z and dout are read
// once (evict-first, so that dz, which the two products read next, stays in
// L2) and dz written.  A block takes kDzRows rows of one expert and 256
// columns of dz; a thread 8 columns (one 16-byte load of z) of every eighth
// row, four rows' loads in flight, its column sums in registers; the block
// adds its eight row lanes in order and writes one partial row per (block of
// rows, columns), which dbias_sum, launched programmatically behind it, adds
// in order.  dz is rounded to bf16, as the operand of both products (their
// error against 64 bits is 1.4 times that of one rounding: 0.0023 of the
// magnitude in place of 0.0017); the sums take it before.  16384 x 8192, silu:
// 133 us with the sums, 6.05 TB/s (one row in
// flight: 48 us for 8191 x 4096 swiglu, now 38; two rows 45, eight 43).
constexpr int kDzRows = 128;
constexpr int kDzThreads = 256;
constexpr int kDzUnroll = 4;

__device__ __forceinline__ int safe_off(const LinearDzArgs& g, int e) {
  if (g.offsets == nullptr) return e == 0 ? 0 : g.M_cap;
  return min(max(g.offsets[e], 0), g.M_cap);
}

// The rows [lo, hi) of expert x = 32 i + lane, for a warp that walks the
// experts in order: the offsets clamped and by their running maximum, which
// are the rows that the products take.  top: where the 32 before ended (the
// first offset to begin with).
__device__ __forceinline__ void expert_rows(const LinearDzArgs& g, int x, int& top, int& lo,
                                            int& hi) {
  const int lane = threadIdx.x & 31;
  hi = max(x < g.E ? safe_off(g, x + 1) : 0, top);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, hi, o);
    if (lane >= o) hi = max(hi, y);
  }
  lo = __shfl_up_sync(0xffffffffu, hi, 1);
  if (lane == 0) lo = top;
  top = __shfl_sync(0xffffffffu, hi, 31);
}

// the row block `b` of the ragged rows: expert e and rows [r0, r1); experts
// are walked by one warp, 32 at a time
__device__ __forceinline__ bool dz_block(const LinearDzArgs& g, int b, int& e, int& r0, int& r1) {
  const int lane = threadIdx.x & 31;
  int carry = 0, top = safe_off(g, 0);
  for (int base = 0; base < g.E; base += 32) {
    const int x = base + lane;
    int lo, hi;
    expert_rows(g, x, top, lo, hi);
    // the grid's last block is past every row block, so it sees all experts
    if (b == g.blocks - 1 && g.offsets != nullptr && x < g.E &&
        (g.offsets[x + 1] != hi || (x == 0 && g.offsets[0] != 0)))
      set_err(g.err, MOE_DEV_BAD_OFFSETS);
    const int c = (hi - lo + kDzRows - 1) / kDzRows;
    int incl = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const int first = carry + incl - c;
    const bool hit = b >= first && b < first + c;
    const unsigned m = __ballot_sync(0xffffffffu, hit);
    if (m != 0) {
      const int l = __ffs(m) - 1;
      e = base + l;
      r0 = __shfl_sync(0xffffffffu, lo + (b - first) * kDzRows, l);
      r1 = min(r0 + kDzRows, __shfl_sync(0xffffffffu, hi, l));
      return true;
    }
    carry += __shfl_sync(0xffffffffu, incl, 31);
  }
  return false;
}

// 8 dz values from 8 of z and 8 (gated: 4) of dout
template <int ACT>
__device__ __forceinline__ void dz8(const uint4& z, const uint32_t* d, float (&o)[8]) {
  const uint32_t zw[4] = {z.x, z.y, z.z, z.w};
  if constexpr (ACT == MOE_ACT_SWIGLU || ACT == MOE_ACT_GEGLU) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float gr = (i & 1) ? bf16_hi(d[i >> 1]) : bf16_lo(d[i >> 1]);
      float p, dp;
      linear_phi<ACT == MOE_ACT_GEGLU>(bf16_lo(zw[i]), p, dp);
      o[2 * i] = gr * bf16_hi(zw[i]) * dp;
      o[2 * i + 1] = gr * p;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o[2 * i] = linear_dact<ACT>(bf16_lo(zw[i]), bf16_lo(d[i]));
      o[2 * i + 1] = linear_dact<ACT>(bf16_hi(zw[i]), bf16_hi(d[i]));
    }
  }
}

template <int ACT>
__global__ void __launch_bounds__(kDzThreads, 4) dz_kernel(const LinearDzArgs g) {
  constexpr bool GATED = (ACT == MOE_ACT_SWIGLU || ACT == MOE_ACT_GEGLU);
  __shared__ int s_e, s_r0, s_r1, s_have;
  __shared__ float s_sum[8][256];
  if (threadIdx.x < 32) {
    int e = 0, r0 = 0, r1 = 0;
    const bool have = dz_block(g, blockIdx.x, e, r0, r1);
    if (threadIdx.x == 0) { s_e = e; s_r0 = r0; s_r1 = r1; s_have = have; }
  }
  __syncthreads();
  if (!s_have) return;
  const int c8 = threadIdx.x & 31, rl = threadIdx.x >> 5;
  const int col = blockIdx.y * 256 + c8 * 8;
  float sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (col < g.N) {
    const int ldd = GATED ? g.N / 2 : g.N;
    const uint16_t* zp = g.z + col;
    const uint16_t* dp = g.dout + (GATED ? col / 2 : col);
    for (int r0 = s_r0 + rl; r0 < s_r1; r0 += 8 * kDzUnroll) {
      uint4 zv[kDzUnroll], dv[kDzUnroll];
#pragma unroll
      for (int u = 0; u < kDzUnroll; ++u) {
        const long long row = r0 + 8 * u;
        if (row < s_r1) {
          if constexpr (GATED) {
            const uint2 d = __ldcs(reinterpret_cast<const uint2*>(dp + row * ldd));
            dv[u] = make_uint4(d.x, d.y, 0, 0);
          } else {
            dv[u] = __ldcs(reinterpret_cast<const uint4*>(dp + row * ldd));
          }
          if constexpr (ACT != MOE_ACT_NONE) zv[u] = __ldcs(reinterpret_cast<const uint4*>(zp + row * g.N));
          else zv[u] = dv[u];
        }
      }
#pragma unroll
      for (int u = 0; u < kDzUnroll; ++u) {
        const long long row = r0 + 8 * u;
        if (row < s_r1) {
          const uint32_t dw[4] = {dv[u].x, dv[u].y, dv[u].z, dv[u].w};
          float o[8];
          dz8<ACT>(zv[u], dw, o);
          if (ACT != MOE_ACT_NONE)
            *reinterpret_cast<uint4*>(g.dz + row * g.N + col) = pack8(o);
#pragma unroll
          for (int i = 0; i < 8; ++i) sum[i] += o[i];
        }
      }
    }
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (g.dbias == nullptr) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) s_sum[rl][c8 * 8 + i] = sum[i];
  __syncthreads();
  const int c = blockIdx.y * 256 + threadIdx.x;
  if (c < g.N) {
    float t = s_sum[0][threadIdx.x];
#pragma unroll
    for (int i = 1; i < 8; ++i) t += s_sum[i][threadIdx.x];
    g.part[static_cast<long long>(blockIdx.x) * g.N + c] = t;
  }
}

// dbias[e][c] (+)= the sum of e's row blocks, in order: 32 columns x 8 lanes
// of blocks
__global__ void __launch_bounds__(kDzThreads) dbias_sum(const LinearDzArgs g) {
  __shared__ float s_sum[8][33];
  __shared__ int s_b0, s_b1;
  const int lane = threadIdx.x & 31, q = threadIdx.x >> 5;
  const int e = blockIdx.y, c = blockIdx.x * 32 + lane;
  if (q == 0) {
    int n = 0, mine = 0, top = safe_off(g, 0);
    for (int base = 0; base <= e; base += 32) {
      const int x = base + lane;
      int lo, hi;
      expert_rows(g, x, top, lo, hi);
      const int k = (hi - lo + kDzRows - 1) / kDzRows;
      if (x < e) n += k;
      else if (x == e) mine = k;
    }
    n = __reduce_add_sync(0xffffffffu, n);
    mine = __reduce_add_sync(0xffffffffu, mine);
    if (lane == 0) { s_b0 = n; s_b1 = n + mine; }
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");   // dz_kernel has ended
  __syncthreads();
  float t = 0.f;
  if (c < g.N)
#pragma unroll 4
    for (int b = s_b0 + q; b < s_b1; b += 8) t += g.part[static_cast<long long>(b) * g.N + c];
  s_sum[q][lane] = t;
  __syncthreads();
  if (q == 0 && c < g.N) {
    t = s_sum[0][lane];
#pragma unroll
    for (int i = 1; i < 8; ++i) t += s_sum[i][lane];
    float* o = g.dbias + static_cast<long long>(e) * g.N + c;
    *o = g.accumulate ? *o + t : t;
  }
}

int dz_blocks_cap(int E, int M_cap) {
  return M_cap / kDzRows + (E < M_cap ? E : M_cap) + 1;
}

}  // namespace

// The choice, by an estimate of the time in nanoseconds, with these measured
// rates: a stage (64 of K) takes 220 ns, a TN = 128 tile's 260, a pair's 240,
// and its 16 KB of weights' share of 6.6 TB/s where no other tile reads them;
// joining a split 2.5 us (TN = 128: 5 us), ending a tile 1 us; a 128 x 256 tile
// of the grouped GEMM (256 rows or more: a 256 x 256 one on two SMs) 290 ns a
// stage, its 32 KB of weights' share of 5.6 TB/s, and 4 us of start and end.
// Measured, us, this kernel / the grouped GEMM: dense 64 x 4096 x 4096
// 14.4 / 37.4, 512 x 4096 x 4096 24.1 / 30.0, 1024 x 4096 x 4096 38.1 / 30.7,
// 1024 x 7168 x 2048 33.9 / 45.7; 8 experts, 4096 x 4096: 64 rows 47.3 / 54.5,
// 2048 rows 90.6 / 59.4.  float32 outputs stay here for their accuracy.
FewPlan few_plan(int E, int M_cap, int K, int N, bool ragged, bool f32, int num_sms) {
  const long long active = ragged ? (E < M_cap ? E : M_cap) : 1;
  const long long avg = (M_cap + active - 1) / active;
  const long long kb = K / FK;
  FewPlan p;
  const long long r = ragged ? 2 * avg : avg;
  p.tn = r <= 16 ? 16 : r <= 32 ? 32 : r <= 64 ? 64 : 128;
  p.pair = !ragged && p.tn == PAIR_TN && N > FM;
  const int sh = p.pair ? 2 : 1;
  p.x_rows = p.tn / sh;
  const long long units = (avg + p.tn - 1) / p.tn * active * ((N + sh * FM - 1) / (sh * FM));
  long long best = -1;
  for (int split = 1; split * sh <= MAX_SPLIT; split *= 2) {
    if (split > 1 && kb < 4 * split) break;
    const long long fit = few_clusters(split * sh, num_sms);
    const long long ctas = (units < fit ? units : fit) * split * sh;
    long long stage = p.pair ? 240 : 260;
    if (p.tn <= 64) stage = 220;
    if (avg <= p.tn && ctas * 16384 / 6600 > stage) stage = ctas * 16384 / 6600;
    const long long join = split == 1 ? 1000 : p.tn == 128 ? 5000 : 2500;
    const long long cost = (units + fit - 1) / fit * ((kb + split - 1) / split * stage + join);
    if (best < 0 || cost < best) {
      best = cost;
      p.split = split;
    }
  }
  if (f32) return p;
  const bool two = avg >= 256;
  const long long tiles = (avg + (two ? 255 : 127)) / (two ? 256 : 128) * active * ((N + 255) / 256);
  const long long places = two ? num_sms / 2 : num_sms;
  long long stage = 290;
  if (avg <= 128 && (tiles < places ? tiles : places) * 32768 / 5600 > stage)
    stage = (tiles < places ? tiles : places) * 32768 / 5600;
  const long long big = (tiles + places - 1) / places * kb * stage + 4000;
  return big < best ? FewPlan{} : p;
}

cudaError_t launch_few(const CUtensorMap& tw, const CUtensorMap& tx, bool kn, const FewArgs& g,
                       const FewPlan& plan, int num_sms, cudaStream_t s) {
  const bool gated = g.act == MOE_ACT_SWIGLU || g.act == MOE_ACT_GEGLU;
  if (kn)
    return gated ? few_tn<true, true>(tw, tx, g, plan, num_sms, s)
                 : few_tn<true, false>(tw, tx, g, plan, num_sms, s);
  return gated ? few_tn<false, true>(tw, tx, g, plan, num_sms, s)
               : few_tn<false, false>(tw, tx, g, plan, num_sms, s);
}

size_t linear_dz_workspace_bytes(int E, int M_cap, int N) {
  return static_cast<size_t>(dz_blocks_cap(E, M_cap)) * N * sizeof(float);
}

cudaError_t launch_linear_dz(const LinearDzArgs& in, cudaStream_t s, int* launches) {
  *launches = 0;
  LinearDzArgs g = in;
  g.blocks = dz_blocks_cap(g.E, g.M_cap);
  const dim3 grid(g.blocks, (g.N + 255) / 256);
  if (g.M_cap > 0) {
    switch (g.act) {
      case MOE_ACT_SWIGLU: dz_kernel<MOE_ACT_SWIGLU><<<grid, kDzThreads, 0, s>>>(g); break;
      case MOE_ACT_GEGLU: dz_kernel<MOE_ACT_GEGLU><<<grid, kDzThreads, 0, s>>>(g); break;
      case MOE_ACT_SRELU: dz_kernel<MOE_ACT_SRELU><<<grid, kDzThreads, 0, s>>>(g); break;
      case MOE_ACT_NONE: dz_kernel<MOE_ACT_NONE><<<grid, kDzThreads, 0, s>>>(g); break;
      case MOE_ACT_RELU: dz_kernel<MOE_ACT_RELU><<<grid, kDzThreads, 0, s>>>(g); break;
      case MOE_ACT_SILU: dz_kernel<MOE_ACT_SILU><<<grid, kDzThreads, 0, s>>>(g); break;
      case MOE_ACT_GELU: dz_kernel<MOE_ACT_GELU><<<grid, kDzThreads, 0, s>>>(g); break;
      default: return cudaErrorInvalidValue;
    }
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    ++*launches;
  }
  if (g.dbias != nullptr) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((g.N + 31) / 32, g.E);
    cfg.blockDim = dim3(kDzThreads);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, dbias_sum, g);
    if (e != cudaSuccess) return e;
    ++*launches;
  }
  return cudaGetLastError();
}

}  // namespace moe
