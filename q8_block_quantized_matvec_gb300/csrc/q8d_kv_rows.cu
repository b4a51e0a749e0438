// Rows of the KV caches: storing a batch of rows (a prompt, or one row of
// every sequence) and reading rows back, for f32, f16, packed Q8_0 and 4-bit
// caches.  The rows outside the cache are f32 or f16.
//
// Both directions move every byte once and do a handful of operations on
// it, so HBM bounds them (and the launch does for a few rows).  A thread
// takes eight consecutive elements: one or two 16-byte accesses outside the
// cache, and four neighbouring threads make a packed block of 32, whose
// largest element they find with two shuffles.  grid.y runs over the
// sequences and grid.z over k and v, so a ragged batch's unused threads are
// whole CTAs that leave at once.
#include <algorithm>

#include "q8d_attn.cuh"
#include "q8d_kv_rows.cuh"

namespace q8d {
namespace {

constexpr int kRowThreads = 256;
constexpr int kGroupE = 8;  // elements a thread

// The rows of sequence s: their count, and their first cache row.  A bad
// count or position sets its bit (one thread) and leaves count 0.
__device__ __forceinline__ bool seq_rows(const KvRowsParams& P, int s, bool report, int& pos,
                                         int& count) {
  pos = P.d_pos[s];
  count = P.d_counts ? P.d_counts[s] : P.rows;
  int bad = 0;
  if (count < 0 || count > P.rows)
    bad = Q8D_DERR_LEN_RANGE;
  else if (count > 0 && (pos < 0 || pos > P.cap - count))
    bad = Q8D_DERR_POS_RANGE;
  if (bad) {
    if (report && P.d_err) atomicOr(P.d_err, bad);
    count = 0;
  }
  return !bad;
}

// Eight elements of a row outside the cache (n of them exist).
template <typename T, bool kVec>
__device__ __forceinline__ void load8(const T* p, int n, float (&f)[kGroupE]) {
  if constexpr (kVec && sizeof(T) == 4) {
    const float4 a = *reinterpret_cast<const float4*>(p);
    const float4 b = reinterpret_cast<const float4*>(p)[1];
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
    f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  } else if constexpr (kVec) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      f[2 * i] = t.x;
      f[2 * i + 1] = t.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kGroupE; ++i) f[i] = i < n ? (float)p[i] : 0.f;
  }
}

template <typename T, bool kVec>
__device__ __forceinline__ void store8(T* p, int n, const float (&f)[kGroupE]) {
  if constexpr (kVec && sizeof(T) == 4) {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
  } else if constexpr (kVec) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
#pragma unroll
    for (int i = 0; i < kGroupE; ++i)
      if (i < n) p[i] = (T)f[i];
  }
}

// Element i of the group in the cache: types F32 / F16 as T.
template <int KV>
struct CacheT {
  using T = float;
};
template <>
struct CacheT<Q8D_KV_F16> {
  using T = __half;
};

// The four lanes of a Q8_0 block quantize its 32 elements (the operations
// of quantize_q8_0_warp: the bytes are the same).
__device__ __forceinline__ void put_q8_0(uint8_t* blk, int part, const float (&f)[kGroupE], bool live) {
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < kGroupE; ++i) amax = fmaxf(amax, fabsf(f[i]));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  if (!live) return;
  const float d = __fdiv_rn(amax, 127.0f);
  const float id = d != 0.f ? __fdiv_rn(1.0f, d) : 0.f;
  unsigned short* q = reinterpret_cast<unsigned short*>(blk + 2 + 8 * part);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int a = (int)roundf(__fmul_rn(f[2 * i], id)), b = (int)roundf(__fmul_rn(f[2 * i + 1], id));
    q[i] = (unsigned short)((a & 0xff) | (b & 0xff) << 8);
  }
  if (part == 0) *reinterpret_cast<unsigned short*>(blk) = __half_as_ushort(__float2half_rn(d));
}

// The four lanes of a 4-bit block.  Lanes 0, 1 hold elements 0-15 (low
// halves of the 16 bytes), lanes 2, 3 elements 16-31 (high halves): lane p
// and lane p ^ 2 exchange four nibbles each and write one word each.
__device__ __forceinline__ void put_q4(uint8_t* quants, uint8_t* scale, int part,
                                       const float (&f)[kGroupE], bool live) {
  float m = f[0];
#pragma unroll
  for (int i = 1; i < kGroupE; ++i) m = q4_larger(m, f[i], false);
  m = q4_larger(m, __shfl_xor_sync(0xffffffffu, m, 1), (part & 1) != 0);
  m = q4_larger(m, __shfl_xor_sync(0xffffffffu, m, 2), (part & 2) != 0);
  float d, id;
  q4_scale(m, d, id);
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < kGroupE; ++i) w[i >> 2] |= q4_nibble(f[i], id) << (8 * (i & 3));
  const bool high = part >= 2;
  const uint32_t got = __shfl_xor_sync(0xffffffffu, high ? w[0] : w[1], 2);
  if (!live) return;
  const uint32_t word = high ? (got | w[1] << 4) : (w[0] | got << 4);
  reinterpret_cast<uint32_t*>(quants)[2 * (part & 1) + (high ? 1 : 0)] = word;
  if (part == 0) *reinterpret_cast<unsigned short*>(scale) = __half_as_ushort(__float2half_rn(d));
}

template <typename T, int KV, bool kVec>
__global__ void __launch_bounds__(kRowThreads) kv_append_rows_kernel(const KvRowsParams P) {
  griddep_launch_dependents();
  griddep_wait();  // (a programmatic dependent: the previous work is complete)
  const T* src = static_cast<const T*>(blockIdx.z ? P.v : P.k);
  uint8_t* cache = blockIdx.z ? P.vc : P.kc;
  const int groups = (P.width + kGroupE - 1) / kGroupE;
  const long long item = (long long)blockIdx.x * kRowThreads + threadIdx.x;
  for (int s = blockIdx.y; s < P.batch; s += gridDim.y) {
    int pos, count;
    seq_rows(P, s, blockIdx.x == 0 && blockIdx.z == 0 && threadIdx.x == 0, pos, count);
    const long long items = (long long)count * groups;
    if ((long long)blockIdx.x * kRowThreads >= items) continue;  // (the whole CTA)
    const bool live = item < items;
    const int i = live ? (int)(item / groups) : 0, g = live ? (int)(item - (long long)i * groups) : 0;
    const int n = min(kGroupE, P.width - g * kGroupE);
    float f[kGroupE];
    load8<T, kVec>(src + ((long long)s * P.rows + i) * P.ld + g * kGroupE, n, f);
    uint8_t* seq = cache + P.seq_bytes * s;
    const long long row = pos + i;
    if constexpr (KV == Q8D_KV_Q4) {
      const int blk = g >> 2;
      put_q4(seq + row * (P.width / 2) + blk * 16,
             seq + q4_scale_plane(P.cap, P.width) + row * (P.width / 16) + blk * 2, g & 3, f, live);
    } else if constexpr (KV == Q8D_KV_Q8_0) {
      put_q8_0(seq + (row * (P.width / kQBlock) + (g >> 2)) * kQBlockBytes, g & 3, f, live);
    } else {
      using C = typename CacheT<KV>::T;
      C* dst = reinterpret_cast<C*>(seq) + row * P.width + g * kGroupE;
      if (live) {
        if (P.width % kGroupE == 0)
          store8<C, true>(dst, n, f);
        else
          store8<C, false>(dst, n, f);
      }
    }
  }
}

// Reading: for a packed 4-bit row a thread takes half a block (8 bytes:
// elements 8h .. 8h+7 and 16+8h .. 16+8h+7), so every access outside is 16
// bytes or more; otherwise eight consecutive elements.
template <typename T, int KV, bool kVec>
__global__ void __launch_bounds__(kRowThreads) kv_read_rows_kernel(const KvRowsParams P) {
  griddep_launch_dependents();
  griddep_wait();
  constexpr int kItemE = KV == Q8D_KV_Q4 ? 16 : kGroupE;
  T* dst = static_cast<T*>(blockIdx.z ? P.v : P.k);
  const uint8_t* cache = blockIdx.z ? P.vc : P.kc;
  const int groups = (P.width + kItemE - 1) / kItemE;
  const long long item = (long long)blockIdx.x * kRowThreads + threadIdx.x;
  for (int s = blockIdx.y; s < P.batch; s += gridDim.y) {
    int pos, count;
    const bool ok =
        seq_rows(P, s, blockIdx.x == 0 && blockIdx.z == 0 && threadIdx.x == 0, pos, count);
    // (the rows of a refused sequence become NaN)
    if (item >= (long long)(ok ? count : P.rows) * groups) continue;
    const int i = (int)(item / groups), g = (int)(item - (long long)i * groups);
    T* out = dst + ((long long)s * P.rows + i) * P.ld;
    const uint8_t* seq = cache + P.seq_bytes * s;
    const long long row = pos + i;
    float f[kGroupE];
    if constexpr (KV == Q8D_KV_Q4) {
      const int blk = g >> 1, h = g & 1;
      uint2 w = make_uint2(0u, 0u);
      float d = __int_as_float(0x7fc00000);
      if (ok) {
        w = *reinterpret_cast<const uint2*>(seq + row * (P.width / 2) + blk * 16 + h * 8);
        d = f16_bits_to_f32(*reinterpret_cast<const unsigned short*>(
            seq + q4_scale_plane(P.cap, P.width) + row * (P.width / 16) + blk * 2));
      }
#pragma unroll
      for (int hi = 0; hi < 2; ++hi) {
#pragma unroll
        for (int e = 0; e < kGroupE; ++e) {
          const uint32_t word = e < 4 ? w.x : w.y;
          f[e] = d * ((float)((word >> (8 * (e & 3) + 4 * hi)) & 15u) - 8.f);
        }
        store8<T, kVec>(out + blk * 32 + hi * 16 + h * 8, kGroupE, f);
      }
    } else {
      const int n = min(kGroupE, P.width - g * kGroupE);
      if (!ok) {
#pragma unroll
        for (int e = 0; e < kGroupE; ++e) f[e] = __int_as_float(0x7fc00000);
      } else if constexpr (KV == Q8D_KV_Q8_0) {
        const uint8_t* blk = seq + (row * (P.width / kQBlock) + (g >> 2)) * kQBlockBytes;
        const float d = f16_bits_to_f32(*reinterpret_cast<const unsigned short*>(blk));
        const unsigned short* q = reinterpret_cast<const unsigned short*>(blk + 2 + 8 * (g & 3));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const unsigned short u = q[e];
          f[2 * e] = d * (float)(int8_t)(u & 0xff);
          f[2 * e + 1] = d * (float)(int8_t)(u >> 8);
        }
      } else {
        using C = typename CacheT<KV>::T;
        const C* p = reinterpret_cast<const C*>(seq) + row * P.width + g * kGroupE;
        if (P.width % kGroupE == 0)
          load8<C, true>(p, n, f);
        else
          load8<C, false>(p, n, f);
      }
      store8<T, kVec>(out + g * kGroupE, n, f);
    }
  }
}

template <bool kRead, typename T, int KV>
int launch_rows(const KvRowsParams& P, cudaStream_t stream) {
  const int item_e = kRead && KV == Q8D_KV_Q4 ? 16 : kGroupE;
  const long long items = (long long)P.rows * ((P.width + item_e - 1) / item_e);
  const long long gx = (items + kRowThreads - 1) / kRowThreads;
  if (gx > 0x7fffffffLL) return Q8D_EUNSUPPORTED;
  const dim3 grid((unsigned)gx, (unsigned)std::min(P.batch, 65535), 2);
  // 16-byte accesses outside the cache where every row allows them
  const bool vec = P.width % kGroupE == 0 && (reinterpret_cast<uintptr_t>(P.k) % 16) == 0 &&
                   (reinterpret_cast<uintptr_t>(P.v) % 16) == 0 && (P.ld * sizeof(T)) % 16 == 0;
  if constexpr (kRead)
    return vec ? launch_ex(kv_read_rows_kernel<T, KV, true>, grid, dim3(kRowThreads), 0, stream, true, P)
               : launch_ex(kv_read_rows_kernel<T, KV, false>, grid, dim3(kRowThreads), 0, stream, true, P);
  else
    return vec ? launch_ex(kv_append_rows_kernel<T, KV, true>, grid, dim3(kRowThreads), 0, stream, true, P)
               : launch_ex(kv_append_rows_kernel<T, KV, false>, grid, dim3(kRowThreads), 0, stream, true, P);
}

template <bool kRead, typename T>
int launch_rows_kv(const KvRowsParams& P, cudaStream_t stream) {
  switch (P.kv_dtype) {
    case Q8D_KV_F32: return launch_rows<kRead, T, Q8D_KV_F32>(P, stream);
    case Q8D_KV_F16: return launch_rows<kRead, T, Q8D_KV_F16>(P, stream);
    case Q8D_KV_Q8_0: return launch_rows<kRead, T, Q8D_KV_Q8_0>(P, stream);
    default: return launch_rows<kRead, T, Q8D_KV_Q4>(P, stream);
  }
}

template <bool kRead>
int launch_rows_any(const KvRowsParams& P, cudaStream_t stream) {
  return P.row_dtype == Q8D_KV_F16 ? launch_rows_kv<kRead, __half>(P, stream)
                                   : launch_rows_kv<kRead, float>(P, stream);
}

}  // namespace

int kv_append_rows_launch(const KvRowsParams& P, cudaStream_t stream) {
  return launch_rows_any<false>(P, stream);
}
int kv_read_rows_launch(const KvRowsParams& P, cudaStream_t stream) {
  return launch_rows_any<true>(P, stream);
}

}  // namespace q8d
