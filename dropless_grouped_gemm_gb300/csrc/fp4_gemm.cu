// fp4_gemm.cu - block-scaled 4-bit grouped product
// (tcgen05.mma.kind::mxf4nvf4.block_scale) with bias, activation, residual and
// a 4-bit output in its epilogue, for many rows.
//
//   z = t_a t_e sum_blocks s_a s_w (sum of a block's code products) + bias
//   out = act(z) + residual
// Persistent and warp-specialised in CTA pairs, as the MXFP8 grouped GEMM: 256
// rows x 256 columns a tile, each CTA with 128 rows of a and 128 columns of w in
// shared memory (2-SM MMAs, M = 256, N = 256, K = 64).  A stage is one 128-byte
// swizzle row of K (256 values): 32 KB of codes and, NV, 6 KB of scales (MX 3)
// for 33.5 MFLOP.  TMEM: a 256-column accumulator and each stage's scale columns;
// the epilogue moves the accumulator to registers and releases it at once, so
// the next tile's MMAs overlap bias, activation, quantisation and stores.
//
// Measured: a stage's four MMAs take 0.280 us (MX: 9.1 PFLOP/s while they run) and
// 0.288 us (NV, with twelve copies of scales into TMEM a stage where MX has six),
// and 2.2 to 2.7 us pass between two tiles' MMAs (commit, TMEM to registers,
// release in both CTAs).  Some 0.6 of that is the second CTA's release of the
// accumulator: its arrival is on a barrier of the first CTA, so it releases at
// cluster scope, and that waits for the output stores that the SM has under way.
// Bound by the MMAs where K is long (32,768 x 8,192 x 4,096 over 8 experts, bf16
// out: 330 us NV, 311 MX, 6.7 and 7.1 PFLOP/s, at the power cap), by those gaps where it is
// short (8,192 x 1,024 x 4,864 32 us NV, 31 MX).
//   Tried, and compared when that arrival still released at CTA scope, which does
// not reach the thread that waits (320 us, 301; 27, 27):
//   Tiles of 192 columns leave TMEM for two accumulators and hide the gaps, but
// an MMA of N = 192 takes 123 cycles (142 NV), nearly what one of N = 256 takes (130):
// 8,192 rows x 4,864, NV, K = 1,024 26.2 us against 27.4, 2,048 41.8 against 39.7, 8,192
// 116 against 96.  Not worth a second tile.  Pairs that share a's rows by multicast changed
// nothing.  Eight epilogue warps that hold 128 columns each, with room for 32 KB
// more of boxes and four stages in place of five: 8,192 x 1,024 x 4,864 26 us plain but 58
// gated (37 with 16 warps), and K = 8,192 104 in place of 96.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "drain.cuh"
#include "fp4_mma.cuh"

namespace moe {
namespace {

constexpr int GEPI = 16;                         // epilogue warps
constexpr int GT = 64 + 32 * GEPI;               // threads
constexpr int GCOLS = 64;                        // columns of a tile that an epilogue warp takes
constexpr int GM = 128;                          // rows, and columns of w, that a CTA holds
constexpr int GN = 256;                          // columns of a tile
constexpr int OP_BYTES = GM * 128;               // 16 KB: 128 rows x 256 codes
constexpr int BOX_BYTES = 32 * 64;               // an epilogue warp's, for its stores
constexpr int STAGES = 5;
constexpr int SF_TMEM = GN;                      // scale columns after the accumulator

template <bool NV>
struct GC {
  static constexpr int sf_bytes = 3 * Fp4Sf<NV>::bytes;        // a's, and both halves of w's
  static constexpr int stage_bytes = 2 * OP_BYTES;
  static constexpr int stage_tx = stage_bytes + sf_bytes;      // a CTA's bytes
  static constexpr int sf_cols = 3 * Fp4Sf<NV>::cols;
  static_assert(SF_TMEM + STAGES * sf_cols <= 512, "TMEM columns");
  // the tables of many experts leave NV no room for the epilogue's boxes
  static constexpr int box_experts = NV ? 448 : MOE_MAX_EXPERTS;
  static __host__ __device__ constexpr bool boxes(int E) { return E <= box_experts; }
  static constexpr size_t smem(int E) {
    return 1024 + static_cast<size_t>(STAGES) * stage_tx + (boxes(E) ? GEPI * BOX_BYTES : 0) +
           (2 * STAGES + 4) * 8 + 32 + 2 * (E + 1) * 4;
  }
  static constexpr size_t most =
      smem(MOE_MAX_EXPERTS) > smem(box_experts) ? smem(MOE_MAX_EXPERTS) : smem(box_experts);
};

struct GTile {
  int e, row0, rows, n0;    // first row of this CTA's block, its valid rows, first column
  long long tile;           // its scale tile
};

// unit u: 256 rows x 256 columns, of which CTA `rank` of the pair has 128 rows
__device__ __forceinline__ GTile gemm_tile(const Fp4GemmArgs& g, const int* s_off, const int* s_ts,
                                           int u, int rank) {
  const int e = fp4_expert_of(s_ts, g.E, u);
  const int nt = (g.N + GN - 1) / GN;
  const int local = u - s_ts[e];
  const int pm = local / nt;
  const int mi = 2 * pm + rank;
  GTile t;
  t.e = e;
  t.row0 = s_off[e] + mi * GM;
  t.rows = max(0, min(GM, s_off[e + 1] - t.row0));
  t.n0 = (local - pm * nt) * GN;
  t.tile = fp4_tile0(s_off[e], e) + mi;
  return t;
}

// What a kernel's epilogue can do: the plain one adds a bias alone (a second
// product of an MLP, a data gradient), without the tests and the registers of
// the others.
enum class Epi { kPlain, kFull, kGated };

// A warp's 32 rows of a tile, from the warp's first column on
struct GRows {
  bool biased;
  uint32_t bias;            // columns 2 lane and 2 lane + 1: one register, where each thread's own
                            // loads of all 64 took 32 (and spilled others)
  const uint16_t* residual; // this thread's row
  uint8_t* box;             // the warp's 2 KB of shared memory; NULL: none
  int rows;                 // valid ones
  bool on;                  // this thread's is
};

// 64 bytes of each row (w: this thread's) to `dst` (the first row's), rows
// `pitch` bytes apart: row y and column x of `map`.  Through the box and a TMA
// store, which runs on while the warp goes on: stores from registers hold a warp
// until L2 has taken them, some 2500 cycles where all SMs end a tile at once.
// 16-byte piece j of row r lies at place j ^ (r / 2 % 4): the 64-byte swizzle.  A
// block that ends early goes row by row.
__device__ __forceinline__ void store_rows(const GRows& p, const CUtensorMap* map, int x, int y,
                                           uint8_t* dst, uint32_t pitch, const uint32_t (&w)[16]) {
  const uint32_t lane = threadIdx.x & 31;
  if (p.box == nullptr) {
    if (p.on) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *reinterpret_cast<uint4*>(dst + static_cast<uint64_t>(lane) * pitch + 16 * j) =
            make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
    }
    return;
  }
  if (lane == 0) bulk_wait_read_0();      // the box's store before has read it
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 4; ++j)
    *reinterpret_cast<uint4*>(p.box + lane * 64 + ((j ^ ((lane >> 1) & 3)) * 16)) =
        make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
  fence_proxy_async_smem();
  __syncwarp();
  if (p.rows == 32) {
    if (lane == 0) {
      tma_store_2d(map, p.box, x, y);
      bulk_commit();
    }
    return;
  }
  const uint32_t j = lane & 3;
#pragma unroll 1
  for (uint32_t r = lane >> 2; static_cast<int>(r) < p.rows; r += 8)
    *reinterpret_cast<uint4*>(dst + static_cast<uint64_t>(r) * pitch + 16 * j) =
        *reinterpret_cast<const uint4*>(p.box + r * 64 + ((j ^ ((r >> 1) & 3)) * 16));
}

// 8 pre-activations, the i-th of the warp's columns on
__device__ __forceinline__ void gemm_z8(const GRows& p, float alpha, int i, const uint32_t* acc,
                                        float (&z)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) z[j] = __uint_as_float(acc[j]) * alpha;
  if (p.biased) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t b = __shfl_sync(0xffffffffu, p.bias, i / 2 + j);
      z[2 * j] += bf16_lo(b);
      z[2 * j + 1] += bf16_hi(b);
    }
  }
}
// 32 of them in bf16
__device__ __forceinline__ void gemm_z32(const GRows& p, float alpha, int i, const uint32_t* acc,
                                         uint32_t (&w)[16]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float z[8];
    gemm_z8(p, alpha, i + 8 * j, acc + 8 * j, z);
#pragma unroll
    for (int m = 0; m < 4; ++m) w[4 * j + m] = pack_bf16x2(z[2 * m], z[2 * m + 1]);
  }
}
// the outputs of 8 accumulator columns: 8, or 4 when gated; and, where wanted,
// the pre-activations in bf16
template <bool GATED>
__device__ __forceinline__ void gemm_out8(const GRows& p, int act, float alpha, int i,
                                          const uint32_t* acc, float* v, bool keep, uint32_t* zw) {
  float z[8];
  gemm_z8(p, alpha, i, acc, z);
  if (keep) {
#pragma unroll
    for (int j = 0; j < 4; ++j) zw[j] = pack_bf16x2(z[2 * j], z[2 * j + 1]);
  }
  if constexpr (GATED) {
    float u[4];
    linear_glu(act, z, u);
    if (p.residual && p.on) {
      const uint2 r = *reinterpret_cast<const uint2*>(p.residual + i / 2);
      u[0] += bf16_lo(r.x); u[1] += bf16_hi(r.x); u[2] += bf16_lo(r.y); u[3] += bf16_hi(r.y);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = u[j];
  } else {
    linear_act(act, z);
    if (p.residual && p.on) {
      const uint4 r = *reinterpret_cast<const uint4*>(p.residual + i);
      const uint32_t rw[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) { z[2 * j] += bf16_lo(rw[j]); z[2 * j + 1] += bf16_hi(rw[j]); }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = z[j];
  }
}

__device__ __forceinline__ uint32_t amax_bits(const float* v, int n) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < n; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
  return m;
}

template <bool NV, Epi EPI>
__global__ void __launch_bounds__(GT, 1)
    fp4_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmW,
                    const __grid_constant__ CUtensorMap tmSA,
                    const __grid_constant__ CUtensorMap tmSW,
                    const __grid_constant__ CUtensorMap tmO, const __grid_constant__ CUtensorMap tmZ,
                    const Fp4GemmArgs g) {
  using C = GC<NV>;
  using SF = Fp4Sf<NV>;
  constexpr bool GATED = EPI == Epi::kGated;
  constexpr uint32_t IDESC = fp4_idesc<NV>(2 * GM, GN);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sf_region = smem + STAGES * C::stage_bytes;
  uint8_t* boxes = sf_region + STAGES * C::sf_bytes;
  uint64_t* full_bar =
      reinterpret_cast<uint64_t*>(boxes + (C::boxes(g.E) ? GEPI * BOX_BYTES : 0));
  uint64_t* empty_bar = full_bar + STAGES;
  uint64_t* tfull_bar = empty_bar + STAGES;
  uint64_t* tempty_bar = tfull_bar + 1;
  uint64_t* drain_bar = tempty_bar + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain_bar + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint32_t* loads = tmem_slot + 2;    // stages loaded: by the first CTA, by the second
  int* s_off = reinterpret_cast<int*>(tmem_slot + 4);
  int* s_ts = s_off + (g.E + 1);

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
  const int lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const int unit0 = blockIdx.x / 2, unit_step = gridDim.x / 2;
  const int nt = (g.N + GN - 1) / GN;
  const int kblocks = (g.K + kFp4StageK - 1) / kFp4StageK;
  const int chunks = fp4_chunks(NV, g.K);

  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(&full_bar[i], 1);
      mbar_init(&empty_bar[i], 1);
    }
    mbar_init(tfull_bar, 1);
    mbar_init(tempty_bar, 2 * GEPI);    // the first CTA's MMAs wait for both CTAs' epilogues
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&tmA);
    prefetch_tmap(&tmW);
    prefetch_tmap(&tmSA);
    prefetch_tmap(&tmSW);
  }
  if (warp == 1) tmem_alloc_pair(tmem_slot, 512);
  if (warp == 2)
    fp4_schedule(g.offsets, g.E, g.M_cap, s_off, s_ts, g.err,
                 [&](int rows) { return (rows + 2 * GM - 1) / (2 * GM) * nt; });
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int units = s_ts[g.E];
  // a role that gives up takes the other CTA with it
  auto tell_other = [&]() {
    st_cluster_u32(mapa_shared(smem_u32(const_cast<int*>(abort_flag)), rank ^ 1), 1u);
  };
  auto gave_up = [&](bool ok) {
    if (!ok && elect_one()) tell_other();
  };

  if (warp == 0) {
    // producer: this CTA's rows of a, its columns of w and three runs of scale
    // chunks; every byte counts on the first CTA's barrier.  Chunks and rows
    // past a buffer read as zeros, those of a neighbour belong to columns and
    // rows that are not stored.
    const uint32_t full0 = mapa_shared(smem_u32(full_bar), 0);
    int stage = 0;
    uint32_t phase = 0, issued = 0;
    bool ok = true;
    for (int u = unit0; u < units && ok; u += unit_step) {
      const GTile t = gemm_tile(g, s_off, s_ts, u, rank);
      const long long ca = t.tile * chunks;
      const long long cw =
          (fp4_tile0(static_cast<long long>(t.e) * g.N, t.e) + t.n0 / GM) * chunks;
      for (int kb = 0; kb < kblocks; ++kb) {
        ok = __all_sync(0xffffffffu, mbar_wait(&empty_bar[stage], phase ^ 1, abort_flag));
        if (!ok) break;
        if (elect_one()) {
          uint8_t* sa = smem + stage * C::stage_bytes;
          uint8_t* ss = sf_region + stage * C::sf_bytes;
          const uint32_t fb = full0 + stage * 8;
          if (rank == 0) mbar_arrive_expect_tx(&full_bar[stage], 2 * C::stage_tx);
          tma_load_2d_pair(sa, &tmA, fb, kb * 128, t.row0);
          tma_load_3d_pair(sa + OP_BYTES, &tmW, fb, kb * 128, t.n0 + rank * GM, t.e);
          const long long c = kb * SF::chunks;
          tma_load_2d_pair(ss, &tmSA, fb, 0, static_cast<int>(2 * (ca + c)));
          tma_load_2d_pair(ss + SF::bytes, &tmSW, fb, 0, static_cast<int>(2 * (cw + c)));
          tma_load_2d_pair(ss + 2 * SF::bytes, &tmSW, fb, 0, static_cast<int>(2 * (cw + chunks + c)));
        }
        ++issued;
        if (++stage == STAGES) { stage = 0; phase ^= 1; }
      }
    }
    if (elect_one()) {
      if (rank != 0) st_cluster_u32(mapa_shared(smem_u32(loads + 1), 0), issued);
      else loads[0] = issued;
    }
    gave_up(ok);
  } else if (warp == 1) {
    // MMA issuer: one thread of the first CTA, for both (no other thread of the
    // warp to agree with between the stages)
    if (rank == 0 && elect_one()) {
      int stage = 0, local = 0;
      uint32_t phase = 0;
      bool ok = true;
      const uint32_t a_lo0 = sdesc_lo(smem_u32(smem), 16);
      const uint32_t w_lo0 = sdesc_lo(smem_u32(smem) + OP_BYTES, 16);
      const uint32_t sf0 = smem_u32(sf_region);
      for (int u = unit0; u < units && ok; u += unit_step, ++local) {
        ok = mbar_wait_cluster(tempty_bar, (local & 1) ^ 1, abort_flag);
        if (!ok) break;
        tc_fence_after();
        for (int kb = 0; kb < kblocks; ++kb) {
          ok = mbar_wait(&full_bar[stage], phase, abort_flag);
          if (!ok) break;
          tc_fence_after();
          const uint32_t ss = sf0 + stage * C::sf_bytes;
          const uint32_t ta = tmem_base + SF_TMEM + stage * C::sf_cols;
          const uint32_t tw = ta + SF::cols;
#pragma unroll
          for (int c = 0; c < SF::chunks; ++c) {
            tmem_cp_sf_pair(ta + 4 * c, fp4_sf_desc(ss + c * kFp4ChunkBytes));
            tmem_cp_sf_pair(tw + 8 * c, fp4_sf_desc(ss + SF::bytes + c * kFp4ChunkBytes));
            tmem_cp_sf_pair(tw + 8 * c + 4, fp4_sf_desc(ss + 2 * SF::bytes + c * kFp4ChunkBytes));
          }
          const uint32_t a_lo = a_lo0 + stage * (C::stage_bytes >> 4);
          const uint32_t w_lo = w_lo0 + stage * (C::stage_bytes >> 4);
          auto mma = [&](int kk) {
            umma_fp4<NV, true>(tmem_base, sdesc_of(a_lo + kk * 2), sdesc_of(w_lo + kk * 2),
                               IDESC | fp4_select<NV>(kk), ta + 4 * fp4_step_chunk<NV>(kk),
                               tw + 8 * fp4_step_chunk<NV>(kk), (kb > 0 || kk > 0) ? 1u : 0u);
          };
          const int steps = min(4, (g.K - kb * kFp4StageK) / kFp4StepK);
          if (steps == 4) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) mma(kk);
          } else {          // the end of a K that is no multiple of 256
#pragma unroll
            for (int kk = 0; kk < 3; ++kk)
              if (kk < steps) mma(kk);
          }
          umma_commit_pair_mc(&empty_bar[stage]);
          if (++stage == STAGES) { stage = 0; phase ^= 1; }
        }
        if (ok) umma_commit_pair_mc(tfull_bar);
      }
      if (!ok) tell_other();
    }
    __syncwarp();
  } else {
    // epilogue: warpgroup wg takes 64 of the tile's columns, warp q of it 32
    // rows, a thread one row
    const int q = warp & 3, wg = (warp - 2) >> 2;
    const int r = q * 32 + lane;
    const uint32_t tempty0 = mapa_shared(smem_u32(tempty_bar), 0);
    const int out_chunks = g.out_q ? fp4_chunks(NV, g.ldo) : 0;
    const float out_t = (g.out_q && g.out_t) ? *g.out_t : 1.f;
    int local = 0;
    bool ok = true;
    for (int u = unit0; u < units && ok; u += unit_step, ++local) {
      const GTile t = gemm_tile(g, s_off, s_ts, u, rank);
      const float alpha = fp4_alpha(g, t.e);
      const int col0 = t.n0 + wg * GCOLS;
      const bool mine = col0 < g.N && q * 32 < t.rows;
      const int ocol = GATED ? col0 / 2 : col0;
      GRows p;
      p.biased = g.bias != nullptr;
      p.bias = 0u;
      if (p.biased && mine)
        p.bias = *reinterpret_cast<const uint32_t*>(g.bias + static_cast<long long>(t.e) * g.N + col0 + 2 * lane);
      if (lane == 0) ok = mbar_wait(tfull_bar, local & 1, abort_flag);
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      tc_fence_after();
      const uint32_t tb = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + wg * GCOLS;
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (rank != 0) mbar_arrive_cluster(tempty0);    // (the waiter is in the other CTA)
          else mbar_arrive(tempty_bar);
        }
      };
      if (!mine) {
        release();
        continue;
      }
      p.box = C::boxes(g.E) ? boxes + (warp - 2) * BOX_BYTES : nullptr;
      p.rows = min(32, t.rows - q * 32);
      p.on = r < t.rows;
      const int y = t.row0 + q * 32;                  // the warp's first row
      const long long row0 = y;
      if constexpr (EPI == Epi::kPlain) {
        if (g.out) {      // packed at once: half the registers, and none spilled
          uint32_t w[2][16];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t v[32];
            tmem_ld32(tb + 32 * c, v);
            tmem_wait_ld();
            gemm_z32(p, alpha, 32 * c, v, w[c]);
          }
          release();
          uint8_t* out = reinterpret_cast<uint8_t*>(g.out + row0 * g.ldo + ocol);
#pragma unroll
          for (int c = 0; c < 2; ++c) store_rows(p, &tmO, ocol + 32 * c, y, out + 64 * c, 2 * g.ldo, w[c]);
          continue;
        }
      }
      const long long row = row0 + lane;
      const bool on = p.on;
      const long long at = row0 * g.ldo + ocol;
      p.residual = g.residual ? g.residual + at + static_cast<long long>(lane) * g.ldo : nullptr;
      uint8_t* out = g.out ? reinterpret_cast<uint8_t*>(g.out + at) : reinterpret_cast<uint8_t*>(g.out_f32 + at);
      const uint32_t pitch = g.ldo * (g.out ? 2 : 4);
      uint8_t* zp = g.z ? reinterpret_cast<uint8_t*>(g.z + row0 * g.N + col0) : nullptr;
      if constexpr (EPI == Epi::kPlain) {     // float32
#pragma unroll 1
        for (int c = 0; c < 2; ++c) {
          uint32_t v[32];
          tmem_ld32(tb + 32 * c, v);
          tmem_wait_ld();
          if (c == 1) release();
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t w[16];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              float z[8];
              gemm_z8(p, alpha, 32 * c + 16 * h + 8 * j, v + 16 * h + 8 * j, z);
#pragma unroll
              for (int i = 0; i < 8; ++i) w[8 * j + i] = __float_as_uint(z[i]);
            }
            store_rows(p, &tmO, ocol + 32 * c + 16 * h, y, out + 128 * c + 64 * h, pitch, w);
          }
        }
        continue;
      }
      const long long tile0 = fp4_tile0(s_off[t.e], t.e);
      const long long in_e = row - s_off[t.e];
      uint32_t bytes = 0;
      float held[GATED && !NV ? 16 : 1];
      uint32_t half[GATED ? 8 : 1];
      // 32 columns at a time from TMEM, which is released with the second load:
      // both at once spill registers (8192 x 1024 x 4864, geglu with z and stores from
      // registers: 68 us, 52 so; where K is long it costs 3%)
#pragma unroll 1
      for (int c = 0; c < 2; ++c) {
        const int col = col0 + 32 * c;
        uint32_t v[32];
        tmem_ld32(tb + 32 * c, v);
        tmem_wait_ld();
        if (c == 1) release();
        uint32_t zw[16];
        if constexpr (GATED) {
          float o[16];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            gemm_out8<true>(p, g.act, alpha, 32 * c + 8 * j, v + 8 * j, o + 4 * j, zp != nullptr, zw + 4 * j);
          if (zp) store_rows(p, &tmZ, col, y, zp + 64 * c, 2 * g.N, zw);
          if (g.out) {
            if (c == 0) {
#pragma unroll
              for (int i = 0; i < 8; ++i) half[i] = pack_bf16x2(o[2 * i], o[2 * i + 1]);
            } else {
              uint32_t w[16];
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                w[i] = half[i];
                w[8 + i] = pack_bf16x2(o[2 * i], o[2 * i + 1]);
              }
              store_rows(p, &tmO, ocol, y, out, pitch, w);
            }
          } else if (g.out_f32) {
            uint32_t w[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(o[i]);
            store_rows(p, &tmO, ocol + 16 * c, y, out + 64 * c, pitch, w);
          } else {                      // 16 outputs from oc on
            const int oc = col / 2;
            uint8_t* q8 = g.out_q + row * (g.ldo / 2) + oc / 2;
            if constexpr (NV) {
              float inv;
              bytes |= fp4_scale<true>(amax_bits(o, 16), out_t, inv) << (8 * c);
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] *= inv;
              if (on) {
                *reinterpret_cast<uint2*>(q8) = make_uint2(e2m1x8(o), e2m1x8(o + 8));
                if (c == 1)
                  *reinterpret_cast<uint16_t*>(g.out_s + fp4_scale_at(tile0, in_e, col0 / 32, out_chunks)) =
                      static_cast<uint16_t>(bytes);
              }
            } else if (c == 0) {
#pragma unroll
              for (int i = 0; i < 16; ++i) held[i] = o[i];
            } else {
              float inv;
              const uint32_t s = fp4_scale<false>(max(amax_bits(held, 16), amax_bits(o, 16)), 1.f, inv);
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                held[i] *= inv;
                o[i] *= inv;
              }
              if (on) {
                *reinterpret_cast<uint4*>(q8 - 8) =
                    make_uint4(e2m1x8(held), e2m1x8(held + 8), e2m1x8(o), e2m1x8(o + 8));
                g.out_s[fp4_scale_at(tile0, in_e, col0 / 64, out_chunks)] = static_cast<uint8_t>(s);
              }
            }
          }
        } else {
          float o[32];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            gemm_out8<false>(p, g.act, alpha, 32 * c + 8 * j, v + 8 * j, o + 8 * j, zp != nullptr, zw + 4 * j);
          if (zp) store_rows(p, &tmZ, col, y, zp + 64 * c, 2 * g.N, zw);
          if (g.out) {
            uint32_t w[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) w[i] = pack_bf16x2(o[2 * i], o[2 * i + 1]);
            store_rows(p, &tmO, ocol + 32 * c, y, out + 64 * c, pitch, w);
          } else if (g.out_f32) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t w[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(o[16 * h + i]);
              store_rows(p, &tmO, ocol + 32 * c + 16 * h, y, out + 128 * c + 64 * h, pitch, w);
            }
          } else {                      // 32 outputs from col on
            float inv;
            if constexpr (NV) {
#pragma unroll
              for (int b = 0; b < 2; ++b) {
                bytes |= fp4_scale<true>(amax_bits(o + 16 * b, 16), out_t, inv) << (8 * (2 * c + b));
#pragma unroll
                for (int i = 0; i < 16; ++i) o[16 * b + i] *= inv;
              }
            } else {
              bytes |= fp4_scale<false>(amax_bits(o, 32), 1.f, inv) << (8 * c);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] *= inv;
            }
            if (on) {
              *reinterpret_cast<uint4*>(g.out_q + row * (g.ldo / 2) + col / 2) =
                  make_uint4(e2m1x8(o), e2m1x8(o + 8), e2m1x8(o + 16), e2m1x8(o + 24));
              if (c == 1) {
                uint8_t* s8 = g.out_s + fp4_scale_at(tile0, in_e, col0 / (NV ? 16 : 32), out_chunks);
                if constexpr (NV) *reinterpret_cast<uint32_t*>(s8) = bytes;
                else *reinterpret_cast<uint16_t*>(s8) = static_cast<uint16_t>(bytes);
              }
            }
          }
        }
      }
    }
    if (lane == 0) bulk_wait_all();       // (shared memory is left behind them)
    __syncwarp();
    gave_up(ok);
  }
  tc_fence_before();
  __syncwarp();
  cluster_sync();
  if (*abort_flag && threadIdx.x == 0) set_err(g.err, MOE_DEV_TIMEOUT);
  if (warp == 1) {
    // Given up (both CTAs): what is in flight ends (waits bounded) before TMEM
    // is freed and shared memory left
    if (*abort_flag && elect_one()) {
      const uint64_t t0 = globaltimer_ns();
      auto ends = [&](uint64_t* bar, uint32_t parity, uint64_t limit_ns) {
        const uint32_t a = smem_u32(bar);
        for (;;)
          if (mbar_try_wait(a, parity) || globaltimer_ns() - t0 > limit_ns) break;
      };
      if (rank == 0) {
        umma_commit_pair(drain_bar);
        ends(drain_bar, 0, kWaitLimitNs);
        for (uint32_t i = 0; i < STAGES; ++i) {
          const StageDrain d = stage_drain(loads[0], loads[1], STAGES, i);
          if (d.make_up) mbar_complete_tx(&full_bar[i], C::stage_tx);
          if (d.arrive) mbar_arrive_expect_tx(&full_bar[i], C::stage_tx);
          if (d.wait) ends(&full_bar[i], d.parity, 2 * kWaitLimitNs);
        }
        mbar_arrive_cluster(mapa_shared(smem_u32(drain_bar), 1));
      } else {
        ends(drain_bar, 0, 3 * kWaitLimitNs);
      }
    }
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 512);
  }
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}
// a scale buffer as rows of 256 bytes; a box holds `chunks` whole chunks
bool map_scales(CUtensorMap* m, const uint8_t* base, long long total, int chunks) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t gdim[2] = {256, static_cast<cuuint64_t>(2 * total)};
  cuuint64_t gstride[1] = {256};
  cuuint32_t bdim[2] = {256, static_cast<cuuint32_t>(2 * chunks)}, estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(base), gdim, gstride, bdim,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [rows, cols] outputs, bf16 or float32, written 32 rows x 64 bytes at a time
bool map_rows(CUtensorMap* m, const void* base, int rows, int cols, bool f32) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t gdim[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t gstride[1] = {static_cast<cuuint64_t>(cols) * (f32 ? 4 : 2)};
  const cuuint32_t bdim[2] = {f32 ? 16u : 32u, 32u}, estr[2] = {1, 1};
  return fn(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
            const_cast<void*>(base), gdim, gstride, bdim, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool NV, Epi EPI>
cudaError_t gemm_t(const CUtensorMap& ta, const CUtensorMap& tw, const Fp4GemmArgs& g, int num_sms,
                   cudaStream_t s) {
  using C = GC<NV>;
  static_assert(C::most <= 227 * 1024, "shared memory of a CTA");
  auto kern = fp4_pair_kernel<NV, EPI>;
  CUtensorMap tsa, tsw;
  const int chunks = fp4_chunks(NV, g.K);
  if (!map_scales(&tsa, g.a_s, g.a_tiles * chunks, Fp4Sf<NV>::chunks) ||
      !map_scales(&tsw, g.w_s, g.w_tiles * chunks, Fp4Sf<NV>::chunks))
    return cudaErrorInvalidValue;
  CUtensorMap to = tsa, tz = tsa;       // (not used where there is no such output)
  if ((!g.out_q && !map_rows(&to, g.out ? static_cast<const void*>(g.out) : g.out_f32, g.M_cap, g.ldo, !g.out)) ||
      (g.z && !map_rows(&tz, g.z, g.M_cap, g.N, false)))
    return cudaErrorInvalidValue;
  // the pairs that the device holds at once and the shared-memory attribute, set
  // up once per device and instantiation
  static int pairs_of[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 2;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(num_sms / 2 * 2);
  cfg.blockDim = dim3(GT);
  cfg.dynamicSmemBytes = C::most;
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  int& pairs = pairs_of[dev];
  if (pairs == 0) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(C::most));
    if (e != cudaSuccess) return e;
    int n = 0;
    e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg);
    if (e != cudaSuccess) return e;
    pairs = n > 0 && n < num_sms / 2 ? n : num_sms / 2;
  }
  // at most so many units, however the rows lie
  const long long units = (static_cast<long long>(g.M_cap) / (2 * GM) + (g.E < g.M_cap ? g.E : g.M_cap)) *
                          ((g.N + GN - 1) / GN);
  cfg.gridDim = dim3(2 * static_cast<unsigned>(units < pairs ? units : pairs));
  cfg.dynamicSmemBytes = C::smem(g.E);
  return cudaLaunchKernelEx(&cfg, kern, ta, tw, tsa, tsw, to, tz, g);
}

}  // namespace

cudaError_t launch_fp4_gemm(const CUtensorMap& ta, const CUtensorMap& tw, const Fp4GemmArgs& g,
                            int num_sms, cudaStream_t s) {
  auto run = [&](auto nv) {
    constexpr bool NV = decltype(nv)::value;
    if (g.act == MOE_ACT_SWIGLU || g.act == MOE_ACT_GEGLU)
      return gemm_t<NV, Epi::kGated>(ta, tw, g, num_sms, s);
    if (g.act == MOE_ACT_NONE && !g.residual && !g.z && !g.out_q)
      return gemm_t<NV, Epi::kPlain>(ta, tw, g, num_sms, s);
    return gemm_t<NV, Epi::kFull>(ta, tw, g, num_sms, s);
  };
  return g.nv ? run(BoolC<true>{}) : run(BoolC<false>{});
}

}  // namespace moe
