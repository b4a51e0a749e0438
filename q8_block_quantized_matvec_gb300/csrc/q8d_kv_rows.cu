// Rows of the KV caches: storing a batch of rows (a prompt, or one row of
// every sequence) and reading rows back, for f32, f16, packed Q8_0 and 4-bit
// caches.  The rows outside the cache are f32 or f16.
//
// Both directions move every byte once and do a handful of operations on
// it, so HBM bounds them (and the launch does for a few rows; storing packed
// blocks, the conversions' instructions).  A thread that stores takes eight
// consecutive elements (four into an f32 cache), one that reads 16 bytes of
// the output; four neighbours make a packed block of 32, whose largest element
// they find with two shuffles.  Large calls give a thread several such groups,
// loaded before any is used, because a CTA that moves 8 KB spends as long
// starting as working: 8 sequences of up to 2047 rows of 1024, f16 and Q8_0,
// took 21.8 us to append and 18.9 to read with one group a thread, 16.4 and
// 13.4 with four; 131071 rows of 512 out of 4 bits into f16 57.6, now 51 (6.7
// TB/s).  Staging the 34-byte blocks through shared memory, for whole 16-byte
// lines on the cache's side, was slower than the 2-byte accesses (21.8 against
// 18.9 us to read): the lines are put together in L1 and L2 anyway.  grid.y
// runs over the sequences and grid.z over k and v, so a ragged batch's unused
// threads are whole CTAs that leave at once.
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

// Four elements, all of which exist where kVec.
template <typename T, bool kVec>
__device__ __forceinline__ void load4(const T* p, int n, float (&f)[4]) {
  if constexpr (kVec && sizeof(T) == 4) {
    const float4 a = *reinterpret_cast<const float4*>(p);
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
  } else if constexpr (kVec) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&u.x));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&u.y));
    f[0] = a.x, f[1] = a.y, f[2] = b.x, f[3] = b.y;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = i < n ? (float)p[i] : 0.f;
  }
}
template <typename T, bool kVec>
__device__ __forceinline__ void store4(T* p, int n, const float (&f)[4]) {
  if constexpr (kVec) {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) p[i] = (T)f[i];
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

template <typename T, bool kVec, int kE>
__device__ __forceinline__ void load_e(const T* p, int n, float (&f)[kE]) {
  if constexpr (kE == 4)
    load4<T, kVec>(p, n, f);
  else
    load8<T, kVec>(p, n, f);
}
template <typename T, bool kVec, int kE>
__device__ __forceinline__ void store_e(T* p, int n, const float (&f)[kE]) {
  if constexpr (kE == 4)
    store4<T, kVec>(p, n, f);
  else
    store8<T, kVec>(p, n, f);
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

// The four lanes of a Q8_0 block quantize its 32 elements (the operations of
// quantize_q8_0_warp, so the bytes are the same).
__device__ __forceinline__ void put_q8_0(uint8_t* blk, int part, const float (&f)[kGroupE], bool live) {
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < kGroupE; ++i) amax = fmaxf(amax, fabsf(f[i]));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  if (!live) return;
  const float d = __fdiv_rn(amax, 127.0f);
  const float id = d != 0.f ? __frcp_rn(d) : 0.f;
  unsigned short* q = reinterpret_cast<unsigned short*>(blk + 2 + 8 * part);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t pair = 0;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int r = (int)roundf(__fmul_rn(f[2 * i + k], id));
      pair |= (uint32_t)(uint8_t)(int8_t)r << (8 * k);
    }
    q[i] = (unsigned short)pair;
  }
  if (part == 0) *reinterpret_cast<unsigned short*>(blk) = __half_as_ushort(__float2half_rn(d));
}

// The four lanes of a 4-bit block.  Lanes 0, 1 hold elements 0-15 (low
// halves of the 16 bytes), lanes 2, 3 elements 16-31 (high halves): lane p
// and lane p ^ 2 exchange four nibbles each and write one word each.
__device__ __forceinline__ void put_q4(uint8_t* quants, uint8_t* scale, int part,
                                       const float (&f)[kGroupE], bool live) {
  // the largest magnitude among the positive and among the negative elements;
  // only where they tie (a block of zeros, say) does the order decide
  float hi = f[0], lo = f[0];
#pragma unroll
  for (int i = 1; i < kGroupE; ++i) {
    hi = fmaxf(hi, f[i]);
    lo = fminf(lo, f[i]);
  }
#pragma unroll
  for (int o = 1; o <= 2; o <<= 1) {
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
  }
  float m = hi > -lo ? hi : lo;
  if (__any_sync(0xffffffffu, hi == -lo)) {
    m = f[0];
#pragma unroll
    for (int i = 1; i < kGroupE; ++i) m = q4_larger(m, f[i], false);
    m = q4_larger(m, __shfl_xor_sync(0xffffffffu, m, 1), (part & 1) != 0);
    m = q4_larger(m, __shfl_xor_sync(0xffffffffu, m, 2), (part & 2) != 0);
  }
  float d, id;
  q4_scale(m, d, id);
  uint32_t w[2];  // a byte an element
#pragma unroll
  for (int i = 0; i < 2; ++i)
    w[i] = __byte_perm(__byte_perm(q4_bits(f[4 * i], id), q4_bits(f[4 * i + 1], id), 0x0040),
                       __byte_perm(q4_bits(f[4 * i + 2], id), q4_bits(f[4 * i + 3], id), 0x0040), 0x5410);
  const bool high = part >= 2;
  const uint32_t got = __shfl_xor_sync(0xffffffffu, high ? w[0] : w[1], 2);
  if (!live) return;
  const uint32_t word = high ? (got | w[1] << 4) : (w[0] | got << 4);
  reinterpret_cast<uint32_t*>(quants)[2 * (part & 1) + (high ? 1 : 0)] = word;
  if (part == 0) *reinterpret_cast<unsigned short*>(scale) = __half_as_ushort(__float2half_rn(d));
}

// Elements an append's thread takes at once: a packed block's quarter, or 16
// bytes of the cache (eight of an f32 cache would be two stores, each of half
// of every 32-byte sector).
template <int KV>
constexpr int append_item() {
  return KV == Q8D_KV_F32 ? 4 : kGroupE;
}

template <typename T, int KV, bool kVec, int kPer>
__global__ void __launch_bounds__(kRowThreads) kv_append_rows_kernel(const KvRowsParams P) {
  constexpr int kE = append_item<KV>();
  griddep_launch_dependents();
  griddep_wait();  // (a programmatic dependent: the previous work is complete)
  const T* src = static_cast<const T*>(blockIdx.z ? P.v : P.k);
  uint8_t* cache = blockIdx.z ? P.vc : P.kc;
  const uint32_t groups = P.groups.d, first = blockIdx.x * (kRowThreads * kPer);
  for (int s = blockIdx.y; s < P.batch; s += gridDim.y) {
    int pos, count;
    seq_rows(P, s, blockIdx.x == 0 && blockIdx.z == 0 && threadIdx.x == 0, pos, count);
    const uint32_t items = (uint32_t)count * groups;
    if (first >= items) continue;  // (the whole CTA)
    const T* rows = src + (long long)s * P.rows * P.ld;
    uint8_t* seq = cache + P.seq_bytes * s;
    float f[kPer][kE];
    int row[kPer], g[kPer];
    bool live[kPer];
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const uint32_t item = first + threadIdx.x + u * kRowThreads;
      live[u] = item < items;
      row[u] = live[u] ? (int)P.groups.div(item) : 0;
      g[u] = live[u] ? (int)(item - (uint32_t)row[u] * groups) : 0;
      load_e<T, kVec, kE>(rows + (long long)row[u] * P.ld + g[u] * kE, min(kE, P.width - g[u] * kE), f[u]);
      row[u] += pos;
    }
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const long long r = row[u];
      if constexpr (KV == Q8D_KV_Q4) {
        const int blk = g[u] >> 2;
        put_q4(seq + r * (P.width / 2) + blk * 16,
               seq + q4_scale_plane(P.cap, P.width) + r * (P.width / 16) + blk * 2, g[u] & 3, f[u], live[u]);
      } else if constexpr (KV == Q8D_KV_Q8_0) {
        put_q8_0(seq + (r * (P.width / kQBlock) + (g[u] >> 2)) * kQBlockBytes, g[u] & 3, f[u], live[u]);
      } else {
        using C = typename CacheT<KV>::T;
        C* dst = reinterpret_cast<C*>(seq) + r * P.width + g[u] * kE;
        if (!live[u]) continue;
        if (P.width % kE == 0)
          store_e<C, true, kE>(dst, kE, f[u]);
        else
          store_e<C, false, kE>(dst, min(kE, P.width - g[u] * kE), f[u]);
      }
    }
  }
}

// Reading: a store outside is 16 bytes, kE elements (with two stores a lane
// of f32 each instruction would fill half of every 32-byte sector: 16384 rows
// of 1024 from f16 37.6 us, now 30.3; 12 x 10127 of 128 from 4 bits, 21.9, now
// 14.5),
// and an item one store; for a 4-bit row two: kE / 2 of a block's bytes, their
// low and their high halves.  kPer items a thread, kRowThreads apart, loaded
// before any is converted.
template <typename T>
constexpr int store_e() {
  return 16 / sizeof(T);
}
template <int KV, typename T>
constexpr int read_item() {
  return (KV == Q8D_KV_Q4 ? 2 : 1) * store_e<T>();
}
template <typename T, int KV, bool kVec, int kPer>
__global__ void __launch_bounds__(kRowThreads) kv_read_rows_kernel(const KvRowsParams P) {
  constexpr int kE = store_e<T>();
  constexpr int kParts = KV == Q8D_KV_Q4 ? 16 / kE : kQBlock / kE;  // items a block
  griddep_launch_dependents();
  griddep_wait();
  T* dst = static_cast<T*>(blockIdx.z ? P.v : P.k);
  const uint8_t* cache = blockIdx.z ? P.vc : P.kc;
  const uint32_t groups = P.groups.d, first = blockIdx.x * (kRowThreads * kPer);
  const float nan = __int_as_float(0x7fc00000);
  for (int s = blockIdx.y; s < P.batch; s += gridDim.y) {
    int pos, count;
    const bool ok =
        seq_rows(P, s, blockIdx.x == 0 && blockIdx.z == 0 && threadIdx.x == 0, pos, count);
    // (the rows of a refused sequence become NaN)
    const uint32_t items = (uint32_t)(ok ? count : P.rows) * groups;
    if (first >= items) continue;  // (the whole CTA)
    const uint8_t* seq = cache + P.seq_bytes * s;
    T* rows = dst + (long long)s * P.rows * P.ld;
    uint32_t w[kPer][kE / 2];  // packed: two quants a word; 4 bits: four bytes a word
    float scale[kPer];
    float f[kPer][kE];
    int row[kPer], g[kPer];
    bool live[kPer];
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const uint32_t item = first + threadIdx.x + u * kRowThreads;
      live[u] = item < items;
      row[u] = live[u] ? (int)P.groups.div(item) : 0;
      g[u] = live[u] ? (int)(item - (uint32_t)row[u] * groups) : 0;
      const long long r = ok ? pos + row[u] : 0;  // (row 0 for a refused sequence: not used)
      if constexpr (KV == Q8D_KV_Q4) {
        const int blk = g[u] / kParts, part = g[u] % kParts;
        const uint8_t* q = seq + r * (P.width / 2) + blk * 16 + part * kE;
        if constexpr (kE == 8) {
          const uint2 v = *reinterpret_cast<const uint2*>(q);
          w[u][0] = v.x;
          w[u][1] = v.y;
        } else {
          w[u][0] = *reinterpret_cast<const uint32_t*>(q);
        }
        scale[u] = f16_bits_to_f32(*reinterpret_cast<const unsigned short*>(
            seq + q4_scale_plane(P.cap, P.width) + r * (P.width / 16) + blk * 2));
      } else if constexpr (KV == Q8D_KV_Q8_0) {
        const uint8_t* blk = seq + (r * (P.width / kQBlock) + g[u] / kParts) * kQBlockBytes;
        scale[u] = f16_bits_to_f32(*reinterpret_cast<const unsigned short*>(blk));
        const unsigned short* q = reinterpret_cast<const unsigned short*>(blk + 2 + kE * (g[u] % kParts));
#pragma unroll
        for (int e = 0; e < kE / 2; ++e) w[u][e] = q[e];
      } else {
        using C = typename CacheT<KV>::T;
        const C* p = reinterpret_cast<const C*>(seq) + r * P.width + g[u] * kE;
        if (P.width % kE == 0)
          load_e<C, true, kE>(p, kE, f[u]);
        else
          load_e<C, false, kE>(p, min(kE, P.width - g[u] * kE), f[u]);
      }
    }
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      if (!live[u]) continue;
      T* out = rows + (long long)row[u] * P.ld;
      if constexpr (KV == Q8D_KV_Q4) {
        const float d = ok ? scale[u] : nan;
#pragma unroll
        for (int hi = 0; hi < 2; ++hi) {
#pragma unroll
          for (int e = 0; e < kE; ++e) {
            // half-byte n under the exponent of 2^23: 2^23 + n, exactly
            const uint32_t n = (w[u][e / 4] >> (8 * (e & 3) + 4 * hi)) & 15u;
            f[u][e] = d * (__uint_as_float(n | 0x4B000000u) - 8388616.f);
          }
          store_e<T, kVec, kE>(out + g[u] / kParts * 32 + g[u] % kParts * kE + hi * 16, kE, f[u]);
        }
      } else {
        if constexpr (KV == Q8D_KV_Q8_0) {
#pragma unroll
          for (int e = 0; e < kE / 2; ++e) {
            const uint32_t q = w[u][e] ^ 0x8080u;
            f[u][2 * e] = scale[u] * (__uint_as_float((q & 0xffu) | kMagicHi) - kMagicBias);
            f[u][2 * e + 1] = scale[u] * (__uint_as_float((q >> 8) | kMagicHi) - kMagicBias);
          }
        }
        if (!ok) {
#pragma unroll
          for (int e = 0; e < kE; ++e) f[u][e] = nan;
        }
        store_e<T, kVec, kE>(out + g[u] * kE, min(kE, P.width - g[u] * kE), f[u]);
      }
    }
  }
}

template <bool kRead, typename T, int KV, bool kVec, int kPer>
int launch_rows_per(const KvRowsParams& P, cudaStream_t stream) {
  const long long items = (long long)P.rows * P.groups.d, cta = kRowThreads * kPer;
  const dim3 grid((unsigned)((items + cta - 1) / cta), (unsigned)std::min(P.batch, 65535), 2);
  if constexpr (kRead)
    return launch_ex(kv_read_rows_kernel<T, KV, kVec, kPer>, grid, dim3(kRowThreads), 0, stream, true, P);
  else
    return launch_ex(kv_append_rows_kernel<T, KV, kVec, kPer>, grid, dim3(kRowThreads), 0, stream, true, P);
}

template <bool kRead, typename T, int KV>
int launch_rows(KvRowsParams P, cudaStream_t stream) {
  const int item_e = kRead ? read_item<KV, T>() : append_item<KV>();
  P.groups = fast_div(((uint32_t)P.width + item_e - 1) / item_e);
  const long long items = (long long)P.rows * P.groups.d;
  if (items > 0xffff0000LL) return Q8D_EUNSUPPORTED;  // (item numbers are 32 bits)
  // 16-byte accesses outside the cache where every row allows them
  const bool vec = P.width % kGroupE == 0 && (reinterpret_cast<uintptr_t>(P.k) % 16) == 0 &&
                   (reinterpret_cast<uintptr_t>(P.v) % 16) == 0 && (P.ld * sizeof(T)) % 16 == 0;
  // Several items a thread once one each would take more than two full
  // machines (from one on: 5.3 against 5.0 us for 4096 rows of 512 f32
  // into 4 bits).  Four or two, whichever measured better, us: Q8_0, 8
  // sequences of up to 2047 rows of 1024 f16, append 15.8 / 16.4 (with a
  // rounding of fewer instructions that was not roundf's for NaN), read 13.4 /
  // 14.0; 4 bits, 32768 rows of 1024 f32, append 67.8 / 59.1 (it holds 32 f32
  // values a thread at four; 51 now), read 27.1 / 27.0; f32 rows in 16-byte items,
  // 16384 of 1024 from f16, read 30.3 / 33.8.
  constexpr int kMany = KV == Q8D_KV_Q8_0 || KV == Q8D_KV_F32 || (kRead && sizeof(T) == 4) ? 4 : 2;
  const bool many = items * P.batch * 2 > 2LL * 2048 * sm_count();
  if (!vec) return launch_rows_per<kRead, T, KV, false, 1>(P, stream);
  return many ? launch_rows_per<kRead, T, KV, true, kMany>(P, stream)
              : launch_rows_per<kRead, T, KV, true, 1>(P, stream);
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
