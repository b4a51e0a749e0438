// 4-bit matrices: rows of f32, f16 or Q8_0 weights into the tiles of
// q8d_layer.cuh, and back into rows.
//
// The quantizer is the 4-bit cache's over groups of 32, 64 or 128: the element
// of largest magnitude (the first of them) / -8 is the scale.  A block of 256
// threads takes a tile: sixteen neighbouring lanes a row of it, eight columns
// (one word) a lane.  Run once for a model, and not made fast: 18944 x 3584 in groups
// of 32 from f32 takes 63 us (46 at the copy rate), from f16 63 (26), from Q8_0 70
// (16), back into f32 61, into f16 129, whose elements are moved one by one.
#include "q8d_kv_rows.cuh"
#include "q8d_layer.cuh"

namespace q8d {
namespace {

struct Place {
  long long tile;
  int row, col;  // in the matrix; eight columns from col on
  int word, scale;  // bytes in the tile
  bool leader;      // the group's first lane
};

__device__ __forceinline__ Place place(const Q4CopyParams& P, int tiles) {
  Place a;
  a.tile = blockIdx.x;
  const int r = threadIdx.x / 16, w = threadIdx.x & 15, h = r / 8, g = r & 7;
  a.row = (int)(a.tile / tiles) * kQ4Rows + r;
  a.col = (int)(a.tile % tiles) * kQ4Cols + 8 * w;
  a.word = 512 * h + 16 * (4 * g + (w & 3)) + 4 * (w >> 2);
  const int ns = q4_scales(P.group), lanes = P.group / 8;
  a.scale = kQ4QuantBytes + 2 * (ns * (2 * g + h) + w / lanes);
  a.leader = w % lanes == 0;
  return a;
}

// (the row's elements are read one by one where it starts off 16 bytes)
__device__ __forceinline__ void source8(const Q4CopyParams& P, const Place& a, float (&f)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = 0.f;
  if (a.row >= P.p || a.col >= P.n) return;  // (n is a multiple of 32)
  if (P.dtype == Q8D_KV_Q8_0) {
    const uint8_t* blk = static_cast<const uint8_t*>(P.rows) +
                         (a.row * (P.ld / kQBlock) + a.col / kQBlock) * kQBlockBytes;
    const float d = f16_bits_to_f32(*reinterpret_cast<const unsigned short*>(blk));
    const unsigned short* q = reinterpret_cast<const unsigned short*>(blk + 2 + (a.col & 31));
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t v = q[e];
      f[2 * e] = d * (float)(int8_t)(v & 0xff);
      f[2 * e + 1] = d * (float)(int8_t)(v >> 8);
    }
  } else if (P.dtype == Q8D_KV_F16) {
    const __half* p = static_cast<const __half*>(P.rows) + a.row * P.ld + a.col;
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = __half2float(p[e]);
  } else {
    const float* p = static_cast<const float*>(P.rows) + a.row * P.ld + a.col;
    if (reinterpret_cast<uintptr_t>(p) % 16 == 0) {
      const float4 x = reinterpret_cast<const float4*>(p)[0], y = reinterpret_cast<const float4*>(p)[1];
      f[0] = x.x, f[1] = x.y, f[2] = x.z, f[3] = x.w, f[4] = y.x, f[5] = y.y, f[6] = y.z, f[7] = y.w;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = p[e];
    }
  }
}

__global__ void __launch_bounds__(256) q4_pack_kernel(const Q4CopyParams P, int tiles) {
  griddep_launch_dependents();
  griddep_wait();
  const Place a = place(P, tiles);
  float f[8];
  source8(P, a, f);
  const float m = first_largest<8>(f, P.group / 8);
  float d, id;
  q4_scale(m, d, id);
  uint32_t word = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) word |= (q4_bits(f[e], id) & 15u) << (4 * (e / 2 + 4 * (e & 1)));
  uint8_t* tile = P.w + a.tile * q4_tile_bytes(P.group);
  *reinterpret_cast<uint32_t*>(tile + a.word) = word;
  if (a.leader) *reinterpret_cast<unsigned short*>(tile + a.scale) = __half_as_ushort(__float2half_rn(d));
}

__global__ void __launch_bounds__(256) q4_unpack_kernel(const Q4CopyParams P, int tiles) {
  griddep_launch_dependents();
  griddep_wait();
  const Place a = place(P, tiles);
  if (a.row >= P.p || a.col >= P.n) return;
  const uint8_t* tile = P.w + a.tile * q4_tile_bytes(P.group);
  const uint32_t word = *reinterpret_cast<const uint32_t*>(tile + a.word);
  const float d = f16_bits_to_f32(*reinterpret_cast<const unsigned short*>(tile + a.scale));
  float f[8];
#pragma unroll
  for (int e = 0; e < 8; ++e)
    f[e] = d * ((float)(word >> (4 * (e / 2 + 4 * (e & 1))) & 15u) - 8.f);
  if (P.dtype == Q8D_KV_F16) {
    __half* p = static_cast<__half*>(P.rows) + a.row * P.ld + a.col;
#pragma unroll
    for (int e = 0; e < 8; ++e) p[e] = __float2half_rn(f[e]);
  } else {
    float* p = static_cast<float*>(P.rows) + a.row * P.ld + a.col;
    if (reinterpret_cast<uintptr_t>(p) % 16 == 0) {
      reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
      reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) p[e] = f[e];
    }
  }
}

int launch_copy(void (*kernel)(Q4CopyParams, int), const Q4CopyParams& P, cudaStream_t stream) {
  const int tiles = q4_tiles(P.n);
  const long long all = q4_strips(P.p) * tiles;
  if (all > 0x7fffffffLL) return Q8D_EUNSUPPORTED;
  return launch_ex(kernel, dim3((unsigned)all), dim3(256), 0, stream, true, P, tiles);
}

}  // namespace

int q4_pack_launch(const Q4CopyParams& P, cudaStream_t stream) { return launch_copy(q4_pack_kernel, P, stream); }
int q4_unpack_launch(const Q4CopyParams& P, cudaStream_t stream) {
  return launch_copy(q4_unpack_kernel, P, stream);
}

}  // namespace q8d
