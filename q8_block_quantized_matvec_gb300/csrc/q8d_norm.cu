// Root-mean-square norm of rows, with the residual's addition before it:
//   h = x + r,  sum = h,  y = h / sqrt(mean(h^2) + eps) * w
// y as f32, f16 or Q8_0 blocks (the caches' quantizer).
//
// Every element is read once, kept in registers between the sum of squares and
// the product, and written once (and the sum once), so HBM bounds it; a few rows
// take a launch and one reduction.  A row belongs to a group of threads, 64 bytes
// of each operand a thread at most; f32 is moved in 16 bytes a thread, f16 in 16
// where the output is no wider.  See q8d_rms.cuh for the sum.
//
// us in a graph (and TB/s): 4096 rows of 3584 with the residual in f16 20.8 (5.65),
// in f32 39.1 (6.0), from f16 into Q8_0 26.0 (4.0: a quarter of the instructions
// are the quantizer's); 4000 rows of 2887 f32 35.0 (5.3); one row 2.5.  What is
// left is latency: half the issue slots are used, by 27 warps an SM whose rows are
// loaded, summed and written in turn.  (A block that walks several rows, the next
// one's loads in flight, needed more registers: 41.7 for 39.1.)
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
  int tpr;    // threads a row: a power of two up to 32, or a multiple of 32
  int per;    // rows a block
  int warps;  // of a row, rounded up to a power of two
};

// How a row is moved: kV elements at once from boundary to boundary; the same
// for rows that start off a boundary, all operands alike (a row's groups start
// at the boundary before it, the first and the last one are moved element by
// element); or all of it element by element.
enum Access { kWhole, kShifted, kScalar };

// kV consecutive elements of a row as they lie in memory: 16 or 8 bytes.  Loads
// are kept apart from the conversions, so that all of a thread's are in flight
// before the first is used.  Rows are read once: they do not displace the
// weights in L1.
template <typename T, int kV>
struct Raw {
  uint32_t w[kV * sizeof(T) / 4];
};
// Elements i .. i + kV - 1 of a row of n that are to be had at once (zeros else).
template <typename T, int kV, int ACCESS>
__device__ __forceinline__ void raw_load(const T* row, int i, int n, Raw<T, kV>& f) {
  constexpr int kW = kV * sizeof(T) / 4;
#pragma unroll
  for (int e = 0; e < kW; ++e) f.w[e] = 0;
  if constexpr (ACCESS == kScalar) {
#pragma unroll
    for (int e = 0; e < kV; ++e) {
      if constexpr (sizeof(T) == 4) {
        if (i + e < n) f.w[e] = __ldcs(reinterpret_cast<const uint32_t*>(row) + i + e);
      } else {
        uint32_t v = 0;
        if (i + e < n) v = __ldcs(reinterpret_cast<const unsigned short*>(row) + i + e);
        f.w[e / 2] |= v << (16 * (e & 1));
      }
    }
  } else if (ACCESS == kWhole ? i < n : i >= 0 && i + kV <= n) {
    if constexpr (kW == 4) {
      const uint4 u = __ldcs(reinterpret_cast<const uint4*>(row + i));
      f.w[0] = u.x, f.w[1] = u.y, f.w[2] = u.z, f.w[3] = u.w;
    } else {
      const uint2 u = __ldcs(reinterpret_cast<const uint2*>(row + i));
      f.w[0] = u.x, f.w[1] = u.y;
    }
  }
}
// The elements of a shifted row's first or last group that are inside.
template <typename T, int kV>
__device__ __forceinline__ void raw_ends(const T* row, int i, int n, Raw<T, kV>& f) {
  if (i >= n || (i >= 0 && i + kV <= n)) return;
#pragma unroll
  for (int e = 0; e < kV; ++e) {
    if (i + e < 0 || i + e >= n) continue;
    if constexpr (sizeof(T) == 4)
      f.w[e] = reinterpret_cast<const uint32_t*>(row)[i + e];
    else
      f.w[e / 2] |= (uint32_t) reinterpret_cast<const unsigned short*>(row)[i + e] << (16 * (e & 1));
  }
}
// As packed pairs of f32.
template <typename T, int kV>
__device__ __forceinline__ void expand(const Raw<T, kV>& r, uint64_t (&f)[kV / 2]) {
#pragma unroll
  for (int i = 0; i < kV / 2; ++i) {
    if constexpr (sizeof(T) == 4) {
      f[i] = pack2(__uint_as_float(r.w[2 * i]), __uint_as_float(r.w[2 * i + 1]));
    } else {
      const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&r.w[i]));
      f[i] = pack2(t.x, t.y);
    }
  }
}
template <typename T, int kV>
__device__ __forceinline__ void row_store(T* p, const uint64_t (&f)[kV / 2]) {
  float v[kV];
#pragma unroll
  for (int i = 0; i < kV / 2; ++i) unpack2(f[i], v[2 * i], v[2 * i + 1]);
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < kV / 4; ++i)
      reinterpret_cast<float4*>(p)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
  } else {
    uint32_t w[kV / 2];
#pragma unroll
    for (int i = 0; i < kV / 2; ++i) {
      const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    if constexpr (kV == 8)
      *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else
      *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  }
}
// Elements i .. i + kV - 1 of a row of n, those that are inside.
template <typename T, int kV, int ACCESS>
__device__ __forceinline__ void part_store(T* row, int i, int n, const uint64_t (&f)[kV / 2]) {
  if (ACCESS == kWhole || (ACCESS == kShifted && i >= 0 && i + kV <= n)) {
    row_store<T, kV>(row + i, f);
  } else {
    float v[kV];
#pragma unroll
    for (int e = 0; e < kV / 2; ++e) unpack2(f[e], v[2 * e], v[2 * e + 1]);
#pragma unroll
    for (int e = 0; e < kV; ++e)
      if (i + e >= 0 && i + e < n) row[i + e] = (T)v[e];
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

template <typename T, int OUT, int kV, int kK, int ACCESS>
__global__ void __launch_bounds__(most_threads(kV * kK)) rmsnorm_kernel(const NormArgs A) {
  constexpr int kP = kV / 2;
  __shared__ Pair part[32];
  __shared__ double wide[32];
  griddep_launch_dependents();
  griddep_wait();
  const NormParams& P = A.P;
  const int tpr = blockDim.x, group = threadIdx.y, t = threadIdx.x;  // a row's threads
  const long long row = (long long)blockIdx.x * blockDim.y + group;
  const bool live = row < P.rows;  // (the same for a row's whole threads)
  const int thread = group * tpr + t, lanes = min(tpr, 32), lane = thread & 31;
  const T* x = static_cast<const T*>(P.x) + row * P.ldx;
  // elements from the boundary to the row's start
  const int off = ACCESS == kShifted ? (int)(reinterpret_cast<uintptr_t>(x) / sizeof(T)) & (kV - 1) : 0;
  // (dead threads of a warp go on with it: they hold zeros and store nothing)
  const int n = live ? P.n : -kV;
  uint64_t h[kK][kP];
  {
    const T* r = static_cast<const T*>(P.r) + row * P.ldr;
    const int nr = P.r ? n : -kV;
    Raw<T, kV> a[kK], b[kK];
#pragma unroll
    for (int k = 0; k < kK; ++k) raw_load<T, kV, ACCESS>(x, (t + k * tpr) * kV - off, n, a[k]);
#pragma unroll
    for (int k = 0; k < kK; ++k) raw_load<T, kV, ACCESS>(r, (t + k * tpr) * kV - off, nr, b[k]);
    if constexpr (ACCESS == kShifted) {
#pragma unroll
      for (int k = 0; k < kK; ++k) {
        raw_ends<T, kV>(x, (t + k * tpr) * kV - off, n, a[k]);
        raw_ends<T, kV>(r, (t + k * tpr) * kV - off, nr, b[k]);
      }
    }
#pragma unroll
    for (int k = 0; k < kK; ++k) {
      uint64_t v[kP];
      expand<T, kV>(a[k], h[k]);
      expand<T, kV>(b[k], v);
#pragma unroll
      for (int e = 0; e < kP; ++e) h[k][e] = P.r ? add2(h[k][e], v[e]) : h[k][e];
    }
  }
  Pair2 both{0, 0};
#pragma unroll
  for (int k = 0; k < kK; ++k)
#pragma unroll
    for (int e = 0; e < kP; ++e) pair2_add_square(both, h[k][e]);
  if (P.sum) {
    T* s = static_cast<T*>(P.sum) + row * P.lds;
#pragma unroll
    for (int k = 0; k < kK; ++k) {
      const int i = (t + k * tpr) * kV - off;
      if (i < n) part_store<T, kV, ACCESS>(s, i, n, h[k]);
    }
  }
  Pair ss = pair_sum(pair2_join(both), lanes, 0xffffffffu);
  const int warp0 = group * (tpr / 32);  // (tpr > 32: the row's first warp)
  if (tpr > 32) {
    if (lane == 0) part[thread / 32] = ss;
    row_barrier(1 + group, tpr);
    // (every `warps` neighbouring lanes take all of the row's warps)
    const int w = lane & (A.warps - 1);
    ss = w < tpr / 32 ? part[warp0 + w] : Pair{0.f, 0.f};
    ss = pair_sum(ss, A.warps, 0xffffffffu);
  }
  float inv = rms_factor(ss, A.inv_n, P.eps);
  const bool good = !live || rms_in_range(ss, P.eps);
  // (whole rows enter together; of rows that share a warp each keeps its own
  // factor, whatever the others hold)
  if (!__all_sync(0xffffffffu, good)) {
    double d = 0.0;
#pragma unroll
    for (int k = 0; k < kK; ++k)
#pragma unroll
      for (int e = 0; e < kP; ++e) {
        float a, b;
        unpack2(h[k][e], a, b);
        d += (double)a * (double)a;
        d += (double)b * (double)b;
      }
    for (int o = 1; o < lanes; o <<= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
    if (tpr > 32) {
      if (lane == 0) wide[thread / 32] = d;
      row_barrier(1 + group, tpr);
      d = 0.0;
      for (int i = 0; i < tpr / 32; ++i) d += wide[warp0 + i];
    }
    if (!good) inv = rms_factor_wide(d, P.n, P.eps);
  }
  const uint64_t inv2 = pack2(inv, inv);
#pragma unroll
  for (int k = 0; k < kK; ++k) {
    const int i = (t + k * tpr) * kV - off;
    const bool in = i < n;
    uint64_t y[kP];
    if constexpr (ACCESS != kWhole) {
      float w[kV];
#pragma unroll
      for (int e = 0; e < kV; ++e) w[e] = i + e >= 0 && i + e < n ? __ldg(P.w + i + e) : 0.f;
#pragma unroll
      for (int e = 0; e < kP; ++e) y[e] = pack2(w[2 * e], w[2 * e + 1]);
    } else {
#pragma unroll
      for (int e = 0; e < kV; e += 4) {
        const float4 a = in ? __ldg(reinterpret_cast<const float4*>(P.w + i + e)) : make_float4(0, 0, 0, 0);
        y[e / 2] = pack2(a.x, a.y);
        y[e / 2 + 1] = pack2(a.z, a.w);
      }
    }
#pragma unroll
    for (int e = 0; e < kP; ++e) y[e] = mul2(mul2(h[k][e], inv2), y[e]);
    if constexpr (OUT == Q8D_KV_Q8_0) {
      // a block is 32 / kV neighbouring lanes, all of which are in the row or behind it
      uint8_t* blk = static_cast<uint8_t*>(P.y) + (row * (P.ldy / kQBlock) + i / kQBlock) * kQBlockBytes;
      float v[kV];
#pragma unroll
      for (int e = 0; e < kV; e += 2) unpack2(y[e / 2], v[e], v[e + 1]);
      put_q8_0<kV>(blk, t & (kQBlock / kV - 1), v, in);
    } else {
      using O = typename std::conditional<OUT == Q8D_KV_F16, __half, float>::type;
      if (in) part_store<O, kV, ACCESS>(static_cast<O*>(P.y) + row * P.ldy, i, n, y);
    }
  }
}

template <typename T, int OUT, int kV, int ACCESS, int kK>
int launch_k(const NormArgs& A, cudaStream_t stream) {
  const dim3 grid((unsigned)((A.P.rows + (A.per - 1LL)) / A.per));
  return launch_ex(rmsnorm_kernel<T, OUT, kV, kK, ACCESS>, grid, dim3(A.tpr, A.per), 0, stream, true, A);
}

template <typename T, int OUT, int kV, int ACCESS>
int launch_v(const NormParams& P, cudaStream_t stream) {
  // groups of kV elements a thread: 64 bytes of a row (us for 16 / 32 elements:
  // 4096 x 3584 with the residual 40.5 / 46.8 in f32, 23.5 / 21.5 in f16)
  constexpr int kMost = 64 / (int)sizeof(T) / kV;
  const int items = (P.n + kV - 1) / kV + (ACCESS == kShifted ? 1 : 0);
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
  NormArgs A{P, pair_inverse(P.n), threads(k), 1, 1};
  A.per = std::max(1, 256 / A.tpr);
  while (A.warps * 32 < A.tpr) A.warps *= 2;
  switch (k) {
    case 1: return launch_k<T, OUT, kV, ACCESS, 1>(A, stream);
    case 2: return launch_k<T, OUT, kV, ACCESS, 2>(A, stream);
    case 4: return launch_k<T, OUT, kV, ACCESS, 4>(A, stream);
    default:
      if constexpr (kMost == 8) return launch_k<T, OUT, kV, ACCESS, 8>(A, stream);
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
  if (vec) return launch_v<T, OUT, kV, kWhole>(P, stream);
  if constexpr (OUT != Q8D_KV_Q8_0) {
    // all operands alike off a boundary of four elements, as tensors of odd n are
    const auto place = [&](const void* p, long long ld, int bytes) {  // of row 0, and a row's step
      return reinterpret_cast<uintptr_t>(p) / bytes % 4 + ld % 4 * 4;
    };
    const auto at = place(P.x, P.ldx, e);
    if ((!P.r || place(P.r, P.ldr, e) == at) && (!P.sum || place(P.sum, P.lds, e) == at) &&
        place(P.y, P.ldy, oe) == at && P.n <= kNormMaxN - 8)
      return launch_v<T, OUT, 4, kShifted>(P, stream);
  }
  return launch_v<T, OUT, 4, kScalar>(P, stream);
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
