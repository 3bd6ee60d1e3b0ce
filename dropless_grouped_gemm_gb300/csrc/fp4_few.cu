// fp4_few.cu - the 4-bit product for few rows (decoding: a token, or a few
// per expert; small dense batches).
//
// As the bf16 few-row kernel (linear.cu) it turns the tile: the weights are the
// MMA's M operand (128 output columns x 256 of K a stage: 16 KB of codes, NV 2
// KB of scales), up to 64 tokens its N operand, D[column, token] in TMEM, and
// the CTAs of a cluster share one tile's reduction and join through distributed
// shared memory in the order of their ranks: one launch, no workspace, no
// atomics, the same bits in every run.  The MMA's N and the boxes loaded follow
// the tile's tokens (16 at a time), so one token costs 2 KB a stage.  Bound by
// the weights' bytes and, for one small layer, by launch, prologue and join.
//
// A tile begins at a multiple of 64 rows of its expert: 64 rows of a scale
// chunk are two of its four TMEM columns, so an odd tile's scales begin two
// columns in.
//
// Roles (192 threads, one CTA an SM): warp 0 TMA producer, warp 1 TMEM owner
// and MMA issuer, warps 2-5 epilogue.
#include <cuda.h>
#include <cuda_runtime.h>

#include "drain.cuh"
#include "fp4_mma.cuh"

namespace moe {
namespace {

constexpr int FT = 192;
constexpr int FE = 4;                   // epilogue warps, one for each TMEM lane quadrant
constexpr int FM = 128;                 // output columns per tile
constexpr int TN = 64;                  // tokens per tile
constexpr int W_BYTES = FM * 128;
constexpr int X_BYTES = TN * 128;
constexpr int BOX_BYTES = kFp4FewBox * 128;
constexpr int RED_BYTES = TN * FM * 4;  // the tile's float32 sums
constexpr int MAX_SPLIT = 8;
constexpr int SF_TMEM = 2 * TN;         // scale columns after the two accumulators

template <bool NV>
struct FC {
  static constexpr int stages = 6;
  static constexpr int stage_bytes = W_BYTES + X_BYTES;
  static constexpr int sf_bytes = 2 * Fp4Sf<NV>::bytes;   // w's, a's
  static constexpr int sf_cols = 2 * Fp4Sf<NV>::cols;
  static_assert(SF_TMEM + stages * sf_cols <= 512, "TMEM columns");
  static constexpr size_t smem(int E) {
    return 1024 + static_cast<size_t>(stages) * (stage_bytes + sf_bytes) + RED_BYTES +
           (2 * stages + 7) * 8 + 24 + 2 * (E + 1) * 4;
  }
};

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

struct FTile {
  int e, row0, rows, n0;
  int off;              // the expert's first row
  int ti;               // the tile's number in the expert
};

// unit u -> tile: an expert's units run over its token tiles first, so that
// consecutive units share their weights through L2
__device__ __forceinline__ FTile few_tile(const Fp4GemmArgs& g, const int* s_off, const int* s_ts,
                                          int u) {
  int e = 0, first = 0, rows = g.M_cap, at = 0;
  if (g.offsets != nullptr) {
    e = fp4_expert_of(s_ts, g.E, u);
    first = s_off[e];
    rows = s_off[e + 1] - first;
    at = s_ts[e];
  }
  const int tt = (rows + TN - 1) / TN;
  const int local = u - at;
  const int ni = local / tt;
  FTile t;
  t.e = e;
  t.off = first;
  t.ti = local - ni * tt;
  t.row0 = first + t.ti * TN;
  t.rows = min(TN, rows - t.ti * TN);
  t.n0 = ni * FM;
  return t;
}

// 8 float32 sums from the same place in each CTA of a split, in the order of the ranks
template <int S>
__device__ __forceinline__ void sum8(const float* p, float (&z)[8]) {
  if constexpr (S == 1) {
    const float4 a = *reinterpret_cast<const float4*>(p);
    const float4 b = *reinterpret_cast<const float4*>(p + 4);
    z[0] = a.x; z[1] = a.y; z[2] = a.z; z[3] = a.w;
    z[4] = b.x; z[5] = b.y; z[6] = b.z; z[7] = b.w;
  } else {
    const uint32_t at = smem_u32(p);
    float w[S][8];
#pragma unroll
    for (int r = 0; r < S; ++r) {
      const uint32_t pa = mapa_shared(at, r);
      ld_cluster_v4(pa, w[r][0], w[r][1], w[r][2], w[r][3]);
      ld_cluster_v4(pa + 16, w[r][4], w[r][5], w[r][6], w[r][7]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      z[i] = w[0][i];
#pragma unroll
      for (int r = 1; r < S; ++r) z[i] += w[r][i];
    }
  }
}

// `n` outputs of a thread (4 when gated, else 8) as 4 bits: the threads of a
// block are neighbouring lanes of `mask`
template <bool NV, int N>
__device__ __forceinline__ void few_quant(const Fp4GemmArgs& g, const FTile& t, long long row,
                                          int oc, float (&v)[8], float out_t, unsigned mask) {
  constexpr int threads = (NV ? 16 : 32) / N;
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
#pragma unroll
  for (int o = threads / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(mask, m, o));
  float inv;
  const uint32_t byte = fp4_scale<NV>(m, out_t, inv);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = i < N ? v[i] * inv : 0.f;
  const uint32_t codes = e2m1x8(v);
  uint8_t* q = g.out_q + row * (g.ldo / 2) + oc / 2;
  if constexpr (N == 4) *reinterpret_cast<uint16_t*>(q) = static_cast<uint16_t>(codes);
  else *reinterpret_cast<uint32_t*>(q) = codes;
  if (oc % (NV ? 16 : 32) == 0)
    g.out_s[fp4_scale_at(fp4_tile0(t.off, t.e), row - t.off, oc / (NV ? 16 : 32),
                         fp4_chunks(NV, g.ldo))] = static_cast<uint8_t>(byte);
}

// 8 neighbouring columns from c of row `row`: bias, pre-activation, activation,
// residual, output
template <bool NV, bool GATED>
__device__ __forceinline__ void few_out(const Fp4GemmArgs& g, const FTile& t, long long row, int c,
                                        const uint4& bias, float alpha, float out_t, unsigned mask,
                                        float (&z)[8]) {
  const uint32_t b[4] = {bias.x, bias.y, bias.z, bias.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    z[2 * i] = fmaf(z[2 * i], alpha, bf16_lo(b[i]));
    z[2 * i + 1] = fmaf(z[2 * i + 1], alpha, bf16_hi(b[i]));
  }
  if (g.z != nullptr)
    *reinterpret_cast<uint4*>(g.z + row * g.N + c) =
        make_uint4(pack_bf16x2(z[0], z[1]), pack_bf16x2(z[2], z[3]), pack_bf16x2(z[4], z[5]),
                   pack_bf16x2(z[6], z[7]));
  float v[8];
  constexpr int N = GATED ? 4 : 8;
  const int oc = GATED ? c / 2 : c;
  const long long at = row * g.ldo + oc;
  if constexpr (GATED) {
    float u[4];
    linear_glu(g.act, z, u);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = u[i];
    if (g.residual != nullptr) {
      const uint2 r = *reinterpret_cast<const uint2*>(g.residual + at);
      v[0] += bf16_lo(r.x); v[1] += bf16_hi(r.x); v[2] += bf16_lo(r.y); v[3] += bf16_hi(r.y);
    }
  } else {
    linear_act(g.act, z);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = z[i];
    if (g.residual != nullptr) {
      const uint4 r = *reinterpret_cast<const uint4*>(g.residual + at);
      const uint32_t rw[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) { v[2 * i] += bf16_lo(rw[i]); v[2 * i + 1] += bf16_hi(rw[i]); }
    }
  }
  if (g.out_q != nullptr) {
    few_quant<NV, N>(g, t, row, oc, v, out_t, mask);
  } else if (g.out_f32 != nullptr) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i)
      *reinterpret_cast<float4*>(g.out_f32 + at + 4 * i) =
          make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
  } else if constexpr (GATED) {
    *reinterpret_cast<uint2*>(g.out + at) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
  } else {
    *reinterpret_cast<uint4*>(g.out + at) =
        make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                   pack_bf16x2(v[6], v[7]));
  }
}

template <bool NV, bool GATED, int S>
__device__ __forceinline__ void few_store(const Fp4GemmArgs& g, const FTile& t, const float* src,
                                          int k0, int c, const uint4& bias, float alpha, float out_t,
                                          unsigned mask) {
#pragma unroll 1
  for (int k = k0; k < t.rows; k += 2 * FE * S) {
    float z[8];
    sum8<S>(src + k * FM, z);
    few_out<NV, GATED>(g, t, static_cast<long long>(t.row0) + k, c, bias, alpha, out_t, mask, z);
  }
}

template <bool NV, bool GATED>
__global__ void __launch_bounds__(FT, 1)
    fp4_few_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                   const Fp4GemmArgs g) {
  using C = FC<NV>;
  using SF = Fp4Sf<NV>;
  constexpr int NST = C::stages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sf_region = smem + NST * C::stage_bytes;
  float* red = reinterpret_cast<float*>(sf_region + NST * C::sf_bytes);   // [TN][FM]
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(red) + RED_BYTES);
  uint64_t* empty_bar = full_bar + NST;
  uint64_t* tfull_bar = empty_bar + NST;
  uint64_t* tempty_bar = tfull_bar + 2;
  uint64_t* rfull_bar = tempty_bar + 2;    // every CTA's partials are in its buffer
  uint64_t* rempty_bar = rfull_bar + 1;    // every CTA has read this CTA's partials
  uint64_t* drain_bar = rempty_bar + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain_bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint32_t* loads = tmem_slot + 2;
  int* s_off = reinterpret_cast<int*>(tmem_slot + 4);
  int* s_ts = s_off + (g.E + 1);

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
  const int lane = threadIdx.x & 31;
  const int split = static_cast<int>(cluster_nctarank());
  const int rank = static_cast<int>(cluster_ctarank());
  const int unit0 = blockIdx.x / split;
  const int unit_step = gridDim.x / split;
  const int nt = (g.N + FM - 1) / FM;
  const int kblocks = (g.K + kFp4StageK - 1) / kFp4StageK;
  const int chunks = fp4_chunks(NV, g.K);
  const int kb0 = static_cast<int>(static_cast<long long>(kblocks) * rank / split);
  const int kb1 = static_cast<int>(static_cast<long long>(kblocks) * (rank + 1) / split);

  auto load = [&](const FTile& t, int kb, int stage) {
    uint8_t* sw = smem + stage * C::stage_bytes;
    uint8_t* ss = sf_region + stage * C::sf_bytes;
    uint64_t* fb = &full_bar[stage];
    const int boxes = (t.rows + kFp4FewBox - 1) / kFp4FewBox;
    const uint32_t sfb =
        static_cast<uint32_t>(min(SF::chunks, chunks - kb * SF::chunks)) * kFp4ChunkBytes;
    mbar_arrive_expect_tx(fb, W_BYTES + boxes * BOX_BYTES + 2 * sfb);
    tma_load_3d(sw, &tmW, fb, kb * 128, t.n0, t.e);
    const long long cw =
        (fp4_tile0(static_cast<long long>(t.e) * g.N, t.e) + t.n0 / FM) * chunks + kb * SF::chunks;
    bulk_load(ss, g.w_s + cw * kFp4ChunkBytes, sfb, fb);
    for (int b = 0; b < boxes; ++b)
      tma_load_2d(sw + W_BYTES + b * BOX_BYTES, &tmX, fb, kb * 128, t.row0 + b * kFp4FewBox);
    const long long ca = (fp4_tile0(t.off, t.e) + t.ti / 2) * chunks + kb * SF::chunks;
    bulk_load(ss + SF::bytes, g.a_s + ca * kFp4ChunkBytes, sfb, fb);
  };

  if (warp == 0 && lane == 0) {
    for (int i = 0; i < NST; ++i) {
      mbar_init(&full_bar[i], 1);
      mbar_init(&empty_bar[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull_bar[i], 1);
      mbar_init(&tempty_bar[i], FE);
    }
    mbar_init(rfull_bar, FE * split);
    mbar_init(rempty_bar, FE * split);
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&tmW);
    prefetch_tmap(&tmX);
  }
  if (warp == 1) tmem_alloc(tmem_slot, 512);
  if (warp == 2 && g.offsets != nullptr)
    fp4_schedule(g.offsets, g.E, g.M_cap, s_off, s_ts, g.err,
                 [&](int rows) { return (rows + TN - 1) / TN * nt; });
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // the peers' barriers are initialised before the epilogue arrives on them
  // (it waits then; everything before runs ahead)
  cluster_arrive();

  const uint32_t tmem_base = *tmem_slot;
  const int units = g.offsets != nullptr ? s_ts[g.E] : nt * ((g.M_cap + TN - 1) / TN);

  if (warp == 0) {
    if (elect_one()) {          // (one thread throughout: none to agree with between stages)
      int stage = 0;
      uint32_t phase = 0, issued = 0;
      bool ok = true;
      for (int u = unit0; u < units && ok; u += unit_step) {
        const FTile t = few_tile(g, s_off, s_ts, u);
        for (int kb = kb0; kb < kb1; ++kb) {
          ok = mbar_wait(&empty_bar[stage], phase ^ 1, abort_flag);
          if (!ok) break;
          load(t, kb, stage);
          ++issued;
          if (++stage == NST) { stage = 0; phase ^= 1; }
        }
      }
      loads[0] = issued;
    }
    __syncwarp();
    cluster_wait();
  } else if (warp == 1) {
    if (elect_one()) {
      int stage = 0, local = 0;
      uint32_t phase = 0;
      bool ok = true;
      const uint32_t w_lo0 = sdesc_lo(smem_u32(smem), 16);
      const uint32_t x_lo0 = sdesc_lo(smem_u32(smem) + W_BYTES, 16);
      const uint32_t sf0 = smem_u32(sf_region);
      for (int u = unit0; u < units && ok; u += unit_step, ++local) {
        const FTile t = few_tile(g, s_off, s_ts, u);
        const int buf = local & 1;
        ok = mbar_wait(&tempty_bar[buf], ((local >> 1) & 1) ^ 1, abort_flag);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tmem_base + buf * TN;
        const uint32_t idesc =
            fp4_idesc<NV>(FM, (t.rows + kFp4FewBox - 1) / kFp4FewBox * kFp4FewBox);
        const uint32_t half = 2 * (t.ti & 1);
        for (int kb = kb0; kb < kb1; ++kb) {
          ok = mbar_wait(&full_bar[stage], phase, abort_flag);
          if (!ok) break;
          tc_fence_after();
          const uint32_t ss = sf0 + stage * C::sf_bytes;
          const uint32_t tw = tmem_base + SF_TMEM + stage * C::sf_cols;
          const uint32_t tx = tw + SF::cols;
          const int steps = min(4, (g.K - kb * kFp4StageK) / kFp4StepK);
#pragma unroll
          for (int c = 0; c < SF::chunks; ++c)
            if (c * (4 / SF::chunks) < steps) {
              fp4_sf_copy(tw + 4 * c, fp4_sf_desc(ss + c * kFp4ChunkBytes));
              fp4_sf_copy(tx + 4 * c, fp4_sf_desc(ss + SF::bytes + c * kFp4ChunkBytes));
            }
          const uint32_t w_lo = w_lo0 + stage * (C::stage_bytes >> 4);
          const uint32_t x_lo = x_lo0 + stage * (C::stage_bytes >> 4);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            if (kk < steps)
              umma_fp4<NV, false>(d, sdesc_of(w_lo + kk * 2), sdesc_of(x_lo + kk * 2),
                                  idesc | fp4_select<NV>(kk), tw + 4 * fp4_step_chunk<NV>(kk),
                                  tx + 4 * fp4_step_chunk<NV>(kk) + half,
                                  (kb > kb0 || kk > 0) ? 1u : 0u);
          umma_commit(&empty_bar[stage]);
          if (++stage == NST) { stage = 0; phase ^= 1; }
        }
        if (ok) umma_commit(&tfull_bar[buf]);
      }
    }
    __syncwarp();
    cluster_wait();
  } else {
    const int q = warp & 3;                 // TMEM lane quadrant
    const int tid = q * 32 + lane;          // its column of the tile, then its place in the output pass
    const float out_t = (g.out_q && g.out_t) ? *g.out_t : 1.f;
    int local = 0;
    bool ok = true, joined = false;
    for (int u = unit0; u < units && ok; u += unit_step, ++local) {
      const FTile t = few_tile(g, s_off, s_ts, u);
      const int c = t.n0 + (tid & 15) * 8;
      const float alpha = fp4_alpha(g, t.e);
      uint4 bias = make_uint4(0, 0, 0, 0);
      if (c < g.N && g.bias != nullptr)
        bias = __ldg(reinterpret_cast<const uint4*>(g.bias + static_cast<long long>(t.e) * g.N + c));
      const int buf = local & 1;
      if (lane == 0) {
        ok = mbar_wait(&tfull_bar[buf], (local >> 1) & 1, abort_flag);
        // the previous unit's sums have been read
        if (ok)
          ok = split == 1 ? mbar_wait(rempty_bar, (local & 1) ^ 1, abort_flag)
                          : mbar_wait_cluster(rempty_bar, (local & 1) ^ 1, abort_flag);
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      __syncwarp();     // what lane 0 acquired orders every lane's writes
      tc_fence_after();
      const uint32_t tb = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + buf * TN;
#pragma unroll 1
      for (int k = 0; k < t.rows; k += 16) {
        uint32_t r[16];
        tmem_ld16(tb + k, r);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) red[(k + i) * FM + tid] = __uint_as_float(r[i]);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tempty_bar[buf]);
      if (!joined) {      // every CTA of the cluster has its barriers
        cluster_wait();
        joined = true;
      }
      // The tile's sums are in shared memory, a CTA's part in each: tell every
      // CTA of the cluster, and wait for all.  Every lane reads what other warps
      // wrote, so every lane acquires (after lane 0 has waited the phase is
      // complete, and the next one needs this warp: no waiting).  A CTA on its
      // own stays with its own barriers, at CTA scope: a unit of 8 stages took
      // 4.1 us at cluster scope, most of it here.
      __syncwarp();
      if (split == 1) {
        if (lane == 0) {
          mbar_arrive(rfull_bar);
          ok = mbar_wait(rfull_bar, local & 1, abort_flag);
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        while (!mbar_try_wait(smem_u32(rfull_bar), local & 1) && !*abort_flag) {}
      } else {
        if (lane < split) mbar_arrive_cluster(mapa_shared(smem_u32(rfull_bar), lane));
        if (lane == 0) ok = mbar_wait_cluster(rfull_bar, local & 1, abort_flag);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        while (!mbar_try_wait_cluster(smem_u32(rfull_bar), local & 1) && !*abort_flag) {}
      }
      if (c < g.N) {
        const float* src = red + (tid & 15) * 8;
        const int k0 = rank + (tid >> 4) * split;
        // the lanes of this token that hold columns (N is a multiple of 64)
        const unsigned mask = (g.N - t.n0 >= FM ? 0xffffu : 0xffu) << (lane & 16);
        switch (split) {
          case 1: few_store<NV, GATED, 1>(g, t, src, k0, c, bias, alpha, out_t, mask); break;
          case 2: few_store<NV, GATED, 2>(g, t, src, k0, c, bias, alpha, out_t, mask); break;
          case 4: few_store<NV, GATED, 4>(g, t, src, k0, c, bias, alpha, out_t, mask); break;
          default: few_store<NV, GATED, 8>(g, t, src, k0, c, bias, alpha, out_t, mask);
        }
      }
      // this warp has read its peers' sums: the arrival releases the reads of
      // all its lanes, after which the peers overwrite what was read
      __syncwarp();
      if (split == 1) {
        if (lane == 0) mbar_arrive(rempty_bar);
      } else if (lane < split) {
        mbar_arrive_cluster(mapa_shared(smem_u32(rempty_bar), lane));
      }
    }
    if (!joined) cluster_wait();
  }

  tc_fence_before();
  __syncwarp();
  // no CTA leaves while a peer may still read its sums or arrive on it
  cluster_sync();
  if (*abort_flag && threadIdx.x == 0) set_err(g.err, MOE_DEV_TIMEOUT);
  if (warp == 1) {
    // Given up: what is in flight ends (waits bounded) before TMEM is freed and
    // shared memory left: the MMAs already issued, then the copies
    if (*abort_flag && elect_one()) {
      const uint64_t t0 = globaltimer_ns();
      auto ends = [&](uint64_t* bar, uint32_t parity, uint64_t limit_ns) {
        const uint32_t a = smem_u32(bar);
        for (;;)
          if (mbar_try_wait(a, parity) || globaltimer_ns() - t0 > limit_ns) break;
      };
      umma_commit(drain_bar);
      ends(drain_bar, 0, kWaitLimitNs);
      for (uint32_t i = 0; i < NST; ++i) {
        const StageDrain d = stage_drain(loads[0], loads[0], NST, i);
        if (d.wait) ends(&full_bar[i], d.parity, 2 * kWaitLimitNs);
      }
    }
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
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

// Clusters of `split` CTAs, one an SM, that the device holds at once, found
// once per device.  It sizes grids only; no cluster waits for another.
int few_clusters(int split, int num_sms) {
  static int known[kMaxDevices][4] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return num_sms / split;
  int& k = known[dev][split_index(split)];
  if (k == 0) {
    auto kern = fp4_few_kernel<true, false>;
    const int smem = static_cast<int>(FC<true>::smem(MOE_MAX_EXPERTS));
    int n = 0;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at;
    few_config(cfg, at, split);
    cfg.gridDim = dim3(num_sms / split * split);
    cfg.dynamicSmemBytes = smem;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n < 1)
      n = num_sms / split;
    k = n < 1 ? 1 : n;
  }
  return k;
}

long long few_units(int E, int M_cap, int N, bool ragged) {
  const long long nt = (N + FM - 1) / FM;
  // ragged: an upper bound over all ways the rows can lie
  const long long tiles = ragged ? static_cast<long long>(M_cap) / TN + (E < M_cap ? E : M_cap)
                                 : (static_cast<long long>(M_cap) + TN - 1) / TN;
  return nt * tiles;
}

template <bool NV, bool GATED>
cudaError_t few_t(const CUtensorMap& tw, const CUtensorMap& tx, const Fp4GemmArgs& g, int split,
                  int num_sms, cudaStream_t s) {
  using C = FC<NV>;
  auto kern = fp4_few_kernel<NV, GATED>;
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
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at;
  few_config(cfg, at, split);
  cfg.stream = s;
  const long long units = few_units(g.E, g.M_cap, g.N, g.offsets != nullptr);
  const long long fit = few_clusters(split, num_sms);
  cfg.gridDim = dim3(static_cast<unsigned>((units < fit ? units : fit) * split));
  cfg.dynamicSmemBytes = C::smem(g.E);
  return cudaLaunchKernelEx(&cfg, kern, tw, tx, g);
}

}  // namespace

// The choice, by an estimate of the time in nanoseconds with these measured
// rates.  This kernel: 3.5 us of launch, prologue and end; a stage (256 of K)
// 260 ns, 350 with more than 16 tokens; ending a tile 1.5 us, joining a split 2.5;
// where no other tile reads a tile's weights, their share of 6.6 TB/s at least.
// The pairs' kernel: 4 us, a stage 300 ns, a tile's end 1.9 us, and the same
// share.  (Fitted before the release of the pairs' accumulator took 0.6 us more, from a
// pair's second tile on.)  Measured, us, this kernel / the pairs': dense 64 x 4096 x 4096 8.7 /
// 10.1, 128 rows 9.6 / 10.7, 256 rows 11.5 / 10.7, 512 rows 16.7 / 10.8, 1024 rows
// 28.7 / 12.3, 256 x 7168 x 2048 11.5 / 13.9; 57 experts with 128 rows, 2048 x 7168
// 77.2 / 90.3, 7168 x 4096 142 / 153, with 2000 rows, 2048 x 7168 83.7 / 96.4; 8
// experts, 4096 x 4096, 512 rows 24.4 / 21.7, 1000 rows 30.9 / 23.6.
Fp4Plan fp4_plan(int E, int M_cap, int K, int N, bool ragged, int num_sms) {
  const long long active = ragged ? (E < M_cap ? E : M_cap) : 1;
  const long long avg = (M_cap + active - 1) / active;
  const long long kb = (K + kFp4StageK - 1) / kFp4StageK;
  Fp4Plan p;
  p.tn = TN;
  const long long units = (avg + TN - 1) / TN * active * ((N + FM - 1) / FM);
  long long best = -1;
  for (int split = 1; split <= MAX_SPLIT; split *= 2) {
    if (split > 1 && kb < 2 * split) break;
    const long long fit = few_clusters(split, num_sms);
    const long long ctas = (units < fit ? units : fit) * split;
    const long long stages = (kb + split - 1) / split;
    long long tile = stages * (avg <= kFp4FewBox ? 260 : 350) + (split == 1 ? 1500 : 2500);
    const long long read = stages * (ctas * 18432 / 6600);
    if (avg <= TN && read > tile) tile = read;
    const long long cost = 3500 + (units + fit - 1) / fit * tile;
    if (best < 0 || cost < best) {
      best = cost;
      p.split = split;
    }
  }
  const long long tiles = (avg + 255) / 256 * active * ((N + 255) / 256);
  const long long places = num_sms / 2;
  long long tile = kb * 300 + 1900;
  const long long read = kb * ((tiles < places ? tiles : places) * 36864 / 6600);
  if (avg <= 256 && read > tile) tile = read;
  const long long big = 4000 + (tiles + places - 1) / places * tile;
  return big < best ? Fp4Plan{} : p;
}

cudaError_t launch_fp4_few(const CUtensorMap& ta, const CUtensorMap& tw, const Fp4GemmArgs& g,
                           const Fp4Plan& plan, int num_sms, cudaStream_t s) {
  const bool gated = g.act == MOE_ACT_SWIGLU || g.act == MOE_ACT_GEGLU;
  const int split = plan.split;
  if (g.nv) return gated ? few_t<true, true>(tw, ta, g, split, num_sms, s) : few_t<true, false>(tw, ta, g, split, num_sms, s);
  return gated ? few_t<false, true>(tw, ta, g, split, num_sms, s) : few_t<false, false>(tw, ta, g, split, num_sms, s);
}

}  // namespace moe
