// fp4.cuh - 4-bit floating point: the two block formats, their scale layout,
// and the host-side interface of the quantisers (fp4_quant.cu) and of the
// products (fp4_gemm.cu, fp4_few.cu).
//
// A value is an E2M1 code (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives; two
// codes a byte, the first in the low half) times its block's scale:
//   NV  blocks of 16, E4M3 scale, and one float32 scale t for the tensor:
//       s = E4M3(amax / (6 t)), code = E2M1(v / (s t))
//   MX  blocks of 32, E8M0 scale (OCP MX v1.0):
//       s = 2^(floor(log2 amax) - 2), code = E2M1(v / s)
// each rounded to nearest, ties to even, saturating.  A block that holds a NaN
// or an infinity has a NaN scale: all of it reads back as NaN.
//
// Scales lie in 512-byte chunks of 128 rows x 4 consecutive blocks (NV: 64
// values, MX: 128), the order in which tcgen05.cp moves them into TMEM: row r
// of the tile, block b at byte (r % 32) * 16 + (r / 32) * 4 + b.  Tile i of
// expert e (rows off_e + 128 i ...) is number off_e / 128 + e + i, a place that
// needs no prefix over the experts: an expert of n rows from off_e on has at
// most (off_e + n) / 128 - off_e / 128 + 1 tiles.  Chunk (tile, c) is at byte
// (tile * chunks + c) * 512.  Weights are experts of N rows each.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace moe {

constexpr int kFp4ChunkBytes = 512;

// chunks of a row of K values
inline __host__ __device__ int fp4_chunks(bool nv, int K) { return nv ? K / 64 : (K + 127) / 128; }
// chunks hold these many values of K
inline __host__ __device__ int fp4_chunk_values(bool nv) { return nv ? 64 : 128; }
// 128-row tiles of E experts with `rows` rows in all
inline __host__ __device__ long long fp4_tiles(long long rows, int E) { return rows / 128 + E; }
inline __host__ __device__ long long fp4_tile0(long long off, int e) { return off / 128 + e; }

// Where rows and their scales lie: ragged (offsets), or E experts of
// rows_per_e rows each.
struct Fp4Rows {
  const int32_t* offsets;    // [E+1] or NULL
  int E;
  long long rows;            // rows of the buffer (M_cap, or E * rows_per_e)
  long long rows_per_e;      // without offsets
};

struct Fp4QuantArgs {
  const uint16_t* src;       // [rows, K] bf16, or with pair_of_row [T, K]
  Fp4Rows r;
  int K;
  bool nv;
  const float* t;            // tensor scale: one value (t_stride 0) or one per expert (1); NULL: 1
  int t_stride;
  const int32_t* pair_of_row;    // [rows] or NULL
  const int32_t* row_of_pair;    // [T*k] or NULL: walk the tokens instead
  int T, k;
  uint8_t* q;                // [rows, K/2]
  uint8_t* s;
  int32_t* err;              // (ragged)
};
cudaError_t launch_fp4_quantize(const Fp4QuantArgs& a, int num_sms, cudaStream_t s);

// W [E, R, C] with blocks along R: q [E, C, R/2]
cudaError_t launch_fp4_quantize_t(const uint16_t* W, int E, int R, int C, bool nv, const float* t,
                                  uint8_t* q, uint8_t* s, cudaStream_t st);

// the values [rows, K], bf16 or float32
cudaError_t launch_fp4_dequantize(const uint8_t* q, const uint8_t* s, const Fp4Rows& r, int K,
                                  bool nv, const float* t, int t_stride, void* out, bool f32,
                                  int32_t* err, int num_sms, cudaStream_t st);

// t[e] = the smallest power of two with max|v| <= 6 * 448 t over the finite
// values of src[e] (n of each, a multiple of 8); 1 where they are all zero.  With
// r.offsets (E 1, n = r.rows K) of the experts' rows alone (bad offsets: err)
cudaError_t launch_fp4_tensor_scale(const uint16_t* src, int E, long long n, const Fp4Rows& r,
                                    int K, float* t, int32_t* err, int num_sms, cudaStream_t st,
                                    int* launches);
// ... t [E] holding the largest magnitudes
cudaError_t launch_fp4_power(float* t, int E, cudaStream_t st);

// ------------------------------------------------------------- products
// out_e = act(t_a t_e a4_e w4_e^T + bias_e) + residual, w4 [E, N, K]
struct Fp4GemmArgs {
  const int32_t* offsets;    // [E+1]; NULL (E = 1): all M_cap rows
  int E, M_cap, K, N;
  bool nv;
  const uint8_t* a_s;        // scales of a and of w
  const uint8_t* w_s;
  long long a_tiles, w_tiles;
  const float* a_t;          // [1] or NULL
  const float* w_t;          // [E] or NULL
  const uint16_t* bias;      // [E, N] or NULL
  int act;
  const uint16_t* residual;  // [M_cap, ldo] or NULL
  uint16_t* z;               // [M_cap, N] or NULL
  uint16_t* out;             // [M_cap, ldo] bf16, or
  float* out_f32;            // float32, or
  uint8_t* out_q;            // 4 bits: codes [M_cap, ldo / 2]
  uint8_t* out_s;            //   and scales
  const float* out_t;        // their tensor scale ([1] or NULL)
  int ldo;
  int32_t* err;
};

// How a product of this size runs: tokens of a tile of the few-row kernel (0:
// the 256 x 256 tiles of the pairs' kernel) and the parts of its reduction.
struct Fp4Plan {
  int tn = 0;
  int split = 1;
};
Fp4Plan fp4_plan(int E, int M_cap, int K, int N, bool ragged, int num_sms);

// ta: a's codes [M_cap, K/2] with boxes of 128 bytes x 128 rows; tw: w's [E, N,
// K/2] with 128 x 128
cudaError_t launch_fp4_gemm(const CUtensorMap& ta, const CUtensorMap& tw, const Fp4GemmArgs& g,
                            int num_sms, cudaStream_t s);
// ta: with boxes of 128 bytes x kFp4FewBox rows
constexpr int kFp4FewBox = 16;
cudaError_t launch_fp4_few(const CUtensorMap& ta, const CUtensorMap& tw, const Fp4GemmArgs& g,
                           const Fp4Plan& plan, int num_sms, cudaStream_t s);

}  // namespace moe
