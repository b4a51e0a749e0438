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

// ---- blocks shared by neighbouring lanes ------------------------------------
// amax / 127 rounded to nearest, without a division: a quotient from the rounded
// reciprocal, corrected by its exact remainder, is the rounded one (Markstein,
// "Computation of elementary functions on the IBM RISC System/6000 processor",
// 1990), as long as nothing leaves the normal range.
__device__ __forceinline__ float q8_0_step(float amax) {
  constexpr float kInv = 1.0f / 127.0f;
  const float q = __fmul_rn(amax, kInv);
  const float d = __fmaf_rn(__fmaf_rn(-127.0f, q, amax), kInv, q);
  return amax > 0x1p-100f && amax < 0x1p100f ? d : __fdiv_rn(amax, 127.0f);
}
// (int)roundf(v), halves away from zero: half a step added towards zero cannot
// reach the next whole number unless the exact sum does.
__device__ __forceinline__ uint32_t q8_0_round(float v) {
  return (uint32_t)__float2int_rz(__fadd_rz(v, copysignf(0.5f, v)));
}

// The 32 / kE lanes of a Q8_0 block (lane `part` holds its elements kE * part
// and on) quantize it with the operations of quantize_q8_0_warp, so the bytes
// are the same.  Every lane of the warp calls; lanes that are not live store
// nothing.
template <int kE>
__device__ __forceinline__ void put_q8_0(uint8_t* blk, int part, const float (&f)[kE], bool live) {
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < kE; ++i) amax = max_nan(amax, fabsf(f[i]));
#pragma unroll
  for (int o = 1; o < 32 / kE; o <<= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if (!live) return;
  const float d = q8_0_step(amax);
  const float id = d != 0.f ? __frcp_rn(d) : 0.f;
  unsigned short* q = reinterpret_cast<unsigned short*>(blk + 2 + kE * part);
#pragma unroll
  for (int i = 0; i < kE / 2; ++i)
    q[i] = (unsigned short)__byte_perm(q8_0_round(__fmul_rn(f[2 * i], id)), q8_0_round(__fmul_rn(f[2 * i + 1], id)), 0x0040);
  if (part == 0) *reinterpret_cast<unsigned short*>(blk) = __half_as_ushort(__float2half_rn(d));
}

// The element of largest magnitude (the first of them) among the values of
// `lanes` neighbouring lanes, lane after lane.
template <int kE>
__device__ __forceinline__ float first_largest(const float (&f)[kE], int lanes) {
  // the largest magnitude among the positive and among the negative elements;
  // only where they tie (a block of zeros, say) does the order decide
  float hi = f[0], lo = f[0];
#pragma unroll
  for (int i = 1; i < kE; ++i) {
    hi = fmaxf(hi, f[i]);
    lo = fminf(lo, f[i]);
  }
#pragma unroll
  for (int o = 1; o < lanes; o <<= 1) {
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
  }
  float m = hi > -lo ? hi : lo;
  if (__any_sync(0xffffffffu, hi == -lo)) {
    m = f[0];
#pragma unroll
    for (int i = 1; i < kE; ++i) m = q4_larger(m, f[i], false);
#pragma unroll
    for (int o = 1; o < lanes; o <<= 1)
      m = q4_larger(m, __shfl_xor_sync(0xffffffffu, m, o), (threadIdx.x & o) != 0);
  }
  return m;
}

// The 32 / kE lanes of a 4-bit block (kE 4 or 8).  The lower half of them holds
// elements 0-15 (low halves of the 16 bytes), the upper half elements 16-31
// (high halves): a lane and its opposite exchange the nibbles of one word and
// write a word each (kE 8), or the lower one writes (kE 4).
template <int kE>
__device__ __forceinline__ void put_q4(uint8_t* quants, uint8_t* scale, int part, const float (&f)[kE],
                                       bool live) {
  const float m = first_largest<kE>(f, 32 / kE);
  float d, id;
  q4_scale(m, d, id);
  uint32_t w[kE / 4];  // a byte an element
#pragma unroll
  for (int i = 0; i < kE / 4; ++i)
    w[i] = __byte_perm(__byte_perm(q4_bits(f[4 * i], id), q4_bits(f[4 * i + 1], id), 0x0040),
                       __byte_perm(q4_bits(f[4 * i + 2], id), q4_bits(f[4 * i + 3], id), 0x0040), 0x5410);
  constexpr int kHalf = 16 / kE;
  const bool high = part >= kHalf;
  if constexpr (kE == 8) {
    const uint32_t got = __shfl_xor_sync(0xffffffffu, high ? w[0] : w[1], kHalf);
    if (!live) return;
    const uint32_t word = high ? (got | w[1] << 4) : (w[0] | got << 4);
    reinterpret_cast<uint32_t*>(quants)[2 * (part & 1) + (high ? 1 : 0)] = word;
  } else {
    static_assert(kE == 4, "");
    const uint32_t got = __shfl_xor_sync(0xffffffffu, w[0], kHalf);
    if (!live) return;
    if (!high) reinterpret_cast<uint32_t*>(quants)[part] = w[0] | got << 4;
  }
  if (part == 0) *reinterpret_cast<unsigned short*>(scale) = __half_as_ushort(__float2half_rn(d));
}

}  // namespace q8d
