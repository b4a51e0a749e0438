// Storing and reading back rows of the KV caches, and the 4-bit cache's
// layout and quantizer.
#pragma once
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "q8d_internal.cuh"

namespace q8d {

// n / d for any 32-bit n by a multiplication (d fixed by the host; Granlund and
// Montgomery's division by an invariant integer): q = (((n - t) >> 1) + t) >> s
// with t = n * m >> 32.
struct FastDiv {
  uint32_t d, m, s;
  __device__ __forceinline__ uint32_t div(uint32_t n) const {
    const uint32_t t = __umulhi(n, m);
    return d == 1 ? n : ((n - t) / 2 + t) >> s;
  }
};
inline FastDiv fast_div(uint32_t d) {
  uint32_t l = 0;  // ceil(log2 d)
  while (l < 32 && (1ull << l) < d) ++l;
  FastDiv f;
  f.d = d;
  f.m = (uint32_t)(((1ull << 32) * ((1ull << l) - d)) / d + 1);
  f.s = l ? l - 1 : 0;
  return f;
}

struct KvRowsParams {
  void* k;  // rows outside the cache: row i of sequence s at element (s * rows + i) * ld
  void* v;
  int row_dtype;  // Q8D_KV_F32 or Q8D_KV_F16
  int ld;
  uint8_t* kc;  // caches: sequence s at seq_bytes * s
  uint8_t* vc;
  int kv_dtype;
  long long seq_bytes;
  int batch, rows, width, cap;
  const int* d_pos;
  const int* d_counts;  // or nullptr: `rows` rows of every sequence
  int* d_err;
  FastDiv groups;  // items a row (set by the launch)
};

int kv_append_rows_launch(const KvRowsParams& P, cudaStream_t stream);
int kv_read_rows_launch(const KvRowsParams& P, cudaStream_t stream);

// ---- 4-bit cache (Q8D_KV_Q4) ----------------------------------------------
// One sequence's cache is two planes: the quants of its cap rows (width / 2
// bytes a row, 16 bytes a block of 32), then their f16 scales (width / 16
// bytes a row).  Split like this a KV head's quants (32 or 64 bytes a row)
// and both planes start on 16-byte boundaries, so the attention copies and
// ldmatrix-reads them as whole 16-byte blocks; blocks with their scale
// inside (18 bytes) would start on any even byte.
__host__ __device__ inline long long q4_scale_plane(int cap, int width) {
  return (long long)cap * (width / 2);
}

// Scale and inverse of a block from its element m of largest magnitude (the
// first of them): d = m / -8 is exact, so m itself becomes nibble 0 and
// every element lies in [-8 d, 8 d].
__device__ __forceinline__ void q4_scale(float m, float& d, float& id) {
  d = m * -0.125f;
  id = __frcp_rn(d);
  if (!isfinite(id)) id = 0.f;  // (an all-zero block, or 1 / d beyond f32: all nibbles 8)
}
// n = min(floor(x / d + 8.5), 15) in single correctly rounded f32 steps (the
// sum is never below 0.49).  The floor is the sum with 2^23 rounded down (its
// low bits): the rounding and conversion instructions run at a quarter of the
// rate and would bound the store.
__device__ __forceinline__ uint32_t q4_bits(float x, float id) {  // n in the low byte
  const float t = __fadd_rn(__fmul_rn(x, id), 8.5f);
  return __float_as_uint(__fadd_rd(fminf(t, 15.5f), 8388608.f));
}
// Keeps of (m, o) the larger magnitude, on a tie the one of lower index.
__device__ __forceinline__ float q4_larger(float m, float o, bool o_first) {
  const float am = fabsf(m), ao = fabsf(o);
  return (ao > am || (ao == am && o_first)) ? o : m;
}

// Stores one 32-element block held by a warp (lane j: element j): byte i is
// element i in its low half and element i + 16 in its high half.
__device__ __forceinline__ void quantize_q4_warp(float x, uint8_t* quants, uint8_t* scale, int lane) {
  // (distances upwards: at each step a lane stands for `o` neighbouring
  // elements, all before or all behind those of the lane it asks)
  float m = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1)
    m = q4_larger(m, __shfl_xor_sync(0xffffffffu, m, o), (lane & o) != 0);
  float d, id;
  q4_scale(m, d, id);
  const uint32_t n = q4_bits(x, id) & 15u;
  const uint32_t hi = __shfl_down_sync(0xffffffffu, n, 16);
  if (lane < 16) quants[lane] = (uint8_t)(n | hi << 4);
  if (lane == 0) *reinterpret_cast<unsigned short*>(scale) = __half_as_ushort(__float2half_rn(d));
}

}  // namespace q8d
