// Launches of the operators with which a layer is put together from calls:
// the norm with the residual's addition, rotary rows into the caches, products
// with 4-bit weights.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "q8d_internal.cuh"

namespace q8d {

// ---- q8d_rmsnorm_rows (q8d_norm.cu) ---------------------------------------
constexpr int kNormMaxN = 16384;  // 1024 threads of 16 elements
struct NormParams {
  const void *x, *r;  // rows of row_dtype; r or nullptr
  void* sum;          // or nullptr
  int row_dtype;
  long long ldx, ldr, lds;
  const float* w;
  float eps;
  void* y;
  int y_dtype;  // Q8D_KV_F32, Q8D_KV_F16 or Q8D_KV_Q8_0 (ldy in elements)
  long long ldy;
  int rows, n;
};
int norm_launch(const NormParams& P, cudaStream_t stream);

// ---- q8d_rope_table, q8d_rope_append_rows (q8d_rope.cu) --------------------
int rope_table_launch(float* table, int max_pos, int rot_dim, double theta, int scaling, double factor,
                      double orig_ctx, double beta_fast, double beta_slow, double mscale,
                      cudaStream_t stream);
struct RopeRowsParams {
  q8d_rope_desc d;
  const void *q, *k, *v;
  void* q_out;
  uint8_t *kc, *vc;
  long long seq_bytes;
  int batch, rows;
  const int *d_pos, *d_rope_pos, *d_counts;
  int* d_err;
};
int rope_rows_launch(const RopeRowsParams& P, cudaStream_t stream);

// ---- 4-bit matrices (q8d_q4_pack.cu, q8d_q4.cu) ----------------------------
// A matrix [p][n] is cut into tiles of 16 rows by 128 columns, the last ones
// filled up with zeros; the tiles of one strip of 16 rows lie one behind the
// other, strip after strip.  A tile is 1024 bytes of quants, then its scales.
//
// The order of a tile is the order in which the lanes of a warp feed them to
// mma.sync m16n8k16 as its 16 x 16 operand, so that a product loads them
// straight into registers, 16 bytes a lane and no byte twice: lane 4 g + t of
// half h (rows g + 8 h) has the 16 bytes from 512 h + 16 (4 g + t), word b of
// them the columns 32 b + 8 t + (0..7) of its row.  Half-byte i < 4 of a word is
// column 2 i of those, half-byte i + 4 column 2 i + 1: a mask then leaves two
// neighbours in the two halves of a register.
// The scales of rows g and g + 8 lie together, 128 / group each, g after g.
constexpr int kQ4Rows = 16, kQ4Cols = 128, kQ4QuantBytes = 1024;
__host__ __device__ constexpr int q4_scales(int group) { return kQ4Cols / group; }  // a row and tile
__host__ __device__ constexpr int q4_tile_bytes(int group) {
  return kQ4QuantBytes + kQ4Rows * q4_scales(group) * 2;
}
inline long long q4_strips(int p) { return ((long long)p + kQ4Rows - 1) / kQ4Rows; }
inline int q4_tiles(int n) { return (n + kQ4Cols - 1) / kQ4Cols; }
inline bool q4_group_known(int group) { return group == 32 || group == 64 || group == 128; }

struct Q4CopyParams {
  void* rows;  // f32, f16 or (packing only) Q8_0 rows, ld elements apart
  int dtype;
  long long ld;
  uint8_t* w;
  int p, n, group;
};
int q4_pack_launch(const Q4CopyParams& P, cudaStream_t stream);
int q4_unpack_launch(const Q4CopyParams& P, cudaStream_t stream);

constexpr int kQ4MaxRows = 16;      // activation rows of a call
constexpr int kQ4MaxN = 32768;      // columns
struct Q4Params {
  const uint8_t* w[2];  // one matrix, or gate and up
  int nmat, group;
  const void* X;
  int x_dtype;
  long long ldx;  // elements
  const float* bias;
  const float* residual;
  long long ldr;
  float* Y;
  long long ldy;
  int m, n, p;
};
int q4_launch(const Q4Params& P, cudaStream_t stream);
void q4_set_wait_limit(uint32_t polls);  // of launches from now on; 0: the default

}  // namespace q8d
