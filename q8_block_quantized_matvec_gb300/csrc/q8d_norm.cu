// Root-mean-square norm of rows, with the residual's addition before it:
//   h = x + r,  sum = h,  y = h / sqrt(mean(h^2) + eps) * w
// y as f32, f16 or Q8_0 blocks (the caches' quantizer).
//
// Every element is read once, kept in registers between the sum of squares and
// the product, and written once (and the sum once), so HBM bounds it; a few rows
// take a launch and one reduction.  A row belongs to a group of threads, at most
// 32 elements each; f32 is moved in 16 bytes a thread, f16 in 16 where the
// output is no wider.  See q8d_rms.cuh for the sum.
#include <algorithm>
#include <type_traits>

#include "q8d_kv_rows.cuh"
#include "q8d_layer.cuh"
#include "q8d_rms.cuh"

namespace q8d {
namespace {

struct NormArgs {
  NormParams P;
  Pair inv_n;
  int tpr;     // threads a row: a power of two up to 32, or a multiple of 32
  int per;     // rows a block
};

// kV consecutive elements (16 or 8 bytes at once, or one element).  Rows are
// read once: they do not displace the weights in L1.
template <typename T, int kV>
__device__ __forceinline__ void row_load(const T* p, float (&f)[kV]) {
  if constexpr (kV == 1) {
    f[0] = (float)__ldcs(p);
  } else if constexpr (sizeof(T) == 4) {
    static_assert(kV == 4, "");
    const float4 a = __ldcs(reinterpret_cast<const float4*>(p));
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
  } else {
    uint32_t w[kV / 2];
    if constexpr (kV == 8) {
      const uint4 u = __ldcs(reinterpret_cast<const uint4*>(p));
      w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
    } else {
      const uint2 u = __ldcs(reinterpret_cast<const uint2*>(p));
      w[0] = u.x, w[1] = u.y;
    }
#pragma unroll
    for (int i = 0; i < kV / 2; ++i) {
      const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      f[2 * i] = t.x;
      f[2 * i + 1] = t.y;
    }
  }
}
template <typename T, int kV>
__device__ __forceinline__ void row_store(T* p, const float (&f)[kV]) {
  if constexpr (kV == 1) {
    *p = (T)f[0];
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < kV / 4; ++i)
      reinterpret_cast<float4*>(p)[i] = make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
  } else {
    uint32_t w[kV / 2];
#pragma unroll
    for (int i = 0; i < kV / 2; ++i) {
      const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    if constexpr (kV == 8)
      *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else
      *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  }
}

// Barrier of one row's threads (whole warps).
__device__ __forceinline__ void row_barrier(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// T: the rows' type; OUT: the output's type number; kV elements at once, kK
// times a thread.
// (32 elements and as many of the residual need more than 64 registers, so
// groups of at most 512 threads)
constexpr int most_threads(int elements) { return elements > 16 ? 512 : 1024; }

template <typename T, int OUT, int kV, int kK>
__global__ void __launch_bounds__(most_threads(kV * kK)) rmsnorm_kernel(const NormArgs A) {
  __shared__ Pair part[32];
  __shared__ double wide[32];
  griddep_launch_dependents();
  griddep_wait();
  const NormParams& P = A.P;
  const int tpr = A.tpr, group = threadIdx.x / tpr, t = threadIdx.x - group * tpr;
  const long long row = (long long)blockIdx.x * A.per + group;
  const bool live = group < A.per && row < P.rows;  // (the same for a row's whole threads)
  const int lanes = min(tpr, 32), lane = threadIdx.x & 31;
  // (dead threads of a warp go on with it: they hold zeros and store nothing)
  float h[kK][kV];
  {
    const T* x = static_cast<const T*>(P.x) + row * P.ldx;
    const T* r = static_cast<const T*>(P.r) + row * P.ldr;
    float b[kK][kV];
#pragma unroll
    for (int k = 0; k < kK; ++k) {
      const int i = (t + k * tpr) * kV;
#pragma unroll
      for (int e = 0; e < kV; ++e) h[k][e] = b[k][e] = 0.f;
      if (live && i < P.n) {
        row_load<T, kV>(x + i, h[k]);
        if (P.r) row_load<T, kV>(r + i, b[k]);
      }
    }
    if (P.r) {
#pragma unroll
      for (int k = 0; k < kK; ++k)
#pragma unroll
        for (int e = 0; e < kV; ++e) h[k][e] = __fadd_rn(h[k][e], b[k][e]);
    }
  }
  Pair ss{0.f, 0.f};
#pragma unroll
  for (int k = 0; k < kK; ++k)
#pragma unroll
    for (int e = 0; e < kV; ++e) pair_add_square(ss, h[k][e]);
  if (P.sum && live) {
    T* s = static_cast<T*>(P.sum) + row * P.lds;
#pragma unroll
    for (int k = 0; k < kK; ++k) {
      const int i = (t + k * tpr) * kV;
      if (i < P.n) row_store<T, kV>(s + i, h[k]);
    }
  }
  ss = pair_sum(ss, lanes, 0xffffffffu);
  const int warp0 = group * (tpr / 32);  // (tpr > 32: the row's first warp)
  if (tpr > 32) {
    if (lane == 0) part[threadIdx.x / 32] = ss;
    row_barrier(1 + group, tpr);
    ss = lane < tpr / 32 ? part[warp0 + lane] : Pair{0.f, 0.f};
    ss = pair_sum(ss, 32, 0xffffffffu);
  }
  float inv = rms_factor(ss, A.inv_n, P.eps);
  const bool good = !live || rms_in_range(ss);
  // (whole rows enter together; of rows that share a warp each keeps its own
  // factor, whatever the others hold)
  if (!__all_sync(0xffffffffu, good)) {
    double d = 0.0;
#pragma unroll
    for (int k = 0; k < kK; ++k)
#pragma unroll
      for (int e = 0; e < kV; ++e) d += (double)h[k][e] * (double)h[k][e];
    for (int o = 1; o < lanes; o <<= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
    if (tpr > 32) {
      if (lane == 0) wide[threadIdx.x / 32] = d;
      row_barrier(1 + group, tpr);
      d = 0.0;
      for (int i = 0; i < tpr / 32; ++i) d += wide[warp0 + i];
    }
    if (!good) inv = rms_factor_wide(d, P.n, P.eps);
  }
#pragma unroll
  for (int k = 0; k < kK; ++k) {
    const int i = (t + k * tpr) * kV;
    const bool in = live && i < P.n;
    float w[kV], y[kV];
    if constexpr (kV == 1) {
      w[0] = in ? __ldg(P.w + i) : 0.f;
    } else {
#pragma unroll
      for (int e = 0; e < kV; e += 4) {
        const float4 a = in ? __ldg(reinterpret_cast<const float4*>(P.w + i + e)) : make_float4(0, 0, 0, 0);
        w[e] = a.x, w[e + 1] = a.y, w[e + 2] = a.z, w[e + 3] = a.w;
      }
    }
#pragma unroll
    for (int e = 0; e < kV; ++e) y[e] = __fmul_rn(__fmul_rn(h[k][e], inv), w[e]);
    if constexpr (OUT == Q8D_KV_Q8_0) {
      // a block is 32 / kV neighbouring lanes, all of which are in the row or behind it
      uint8_t* blk = static_cast<uint8_t*>(P.y) + (row * (P.ldy / kQBlock) + i / kQBlock) * kQBlockBytes;
      put_q8_0<kV>(blk, t & (kQBlock / kV - 1), y, in);
    } else {
      using O = typename std::conditional<OUT == Q8D_KV_F16, __half, float>::type;
      if (in) row_store<O, kV>(static_cast<O*>(P.y) + row * P.ldy + i, y);
    }
  }
}

template <typename T, int OUT, int kV, int kK>
int launch_k(const NormArgs& A, cudaStream_t stream) {
  const int threads = (A.per * A.tpr + 31) / 32 * 32;
  const dim3 grid((unsigned)((A.P.rows + A.per - 1) / A.per));
  return launch_ex(rmsnorm_kernel<T, OUT, kV, kK>, grid, dim3(threads), 0, stream, true, A);
}

template <typename T, int OUT, int kV>
int launch_v(const NormParams& P, cudaStream_t stream) {
  constexpr int kMost = 32 / kV;  // groups of kV elements a thread
  const int items = (P.n + kV - 1) / kV;
  // threads a row with k groups each: whole warps, or a power of two that
  // holds a Q8_0 block
  const auto threads = [&](int k) {
    const int t = (items + k - 1) / k;
    if (t > 32) return (t + 31) / 32 * 32;
    int q = 32 / kV;
    while (q < t) q <<= 1;
    return q;
  };
  // as many groups a thread as leave the machine full: more loads in flight a
  // thread and fewer partial sums; a few rows take one or two for the latency
  int k = 1;
  while (k < kMost && (threads(k) > most_threads(k * kV) ||
                       (threads(2 * k) <= most_threads(2 * k * kV) &&
                        (long long)P.rows * threads(2 * k) >= 1024LL * sm_count())))
    k *= 2;
  NormArgs A{P, pair_inverse(P.n), threads(k), 1};
  A.per = std::max(1, 256 / A.tpr);
  switch (k) {
    case 1: return launch_k<T, OUT, kV, 1>(A, stream);
    case 2: return launch_k<T, OUT, kV, 2>(A, stream);
    case 4: return launch_k<T, OUT, kV, 4>(A, stream);
    default:
      if constexpr (kMost >= 8) {
        if (k == 8) return launch_k<T, OUT, kV, 8>(A, stream);
        if constexpr (kMost >= 32) {
          if (k == 16) return launch_k<T, OUT, kV, 16>(A, stream);
          return launch_k<T, OUT, kV, 32>(A, stream);
        }
      }
      return Q8D_EUNSUPPORTED;
  }
}

template <typename T, int OUT>
int launch_out(const NormParams& P, cudaStream_t stream) {
  const auto on = [&](const void* p, long long ld, int e, int bytes) {
    return !p || (reinterpret_cast<uintptr_t>(p) % bytes == 0 && (ld * e) % bytes == 0);
  };
  // an f16 row in eights where the output is f16 or 8 bits wide (f32 would be
  // stored in halves of every sector)
  constexpr int kV = sizeof(T) == 2 && OUT != Q8D_KV_F32 ? 8 : 4;
  constexpr int e = sizeof(T), oe = OUT == Q8D_KV_F32 ? 4 : 2;
  const bool vec = P.n % kV == 0 && on(P.x, P.ldx, e, e * kV) && on(P.r, P.ldr, e, e * kV) &&
                   on(P.sum, P.lds, e, e * kV) && on(P.w, 0, 4, 16) &&
                   (OUT == Q8D_KV_Q8_0 || on(P.y, P.ldy, oe, oe * kV > 16 ? 16 : oe * kV));
  return vec ? launch_v<T, OUT, kV>(P, stream) : launch_v<T, OUT, 1>(P, stream);
}

template <typename T>
int launch_t(const NormParams& P, cudaStream_t stream) {
  switch (P.y_dtype) {
    case Q8D_KV_F32: return launch_out<T, Q8D_KV_F32>(P, stream);
    case Q8D_KV_F16: return launch_out<T, Q8D_KV_F16>(P, stream);
    default: return launch_out<T, Q8D_KV_Q8_0>(P, stream);
  }
}

}  // namespace

int norm_launch(const NormParams& P, cudaStream_t stream) {
  return P.row_dtype == Q8D_KV_F16 ? launch_t<__half>(P, stream) : launch_t<float>(P, stream);
}

}  // namespace q8d
