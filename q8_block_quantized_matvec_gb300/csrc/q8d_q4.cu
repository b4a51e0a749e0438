// Products with 4-bit weights and group scales for 1 to 16 activation rows:
//   Y[i][r] = sum_g s(r, g) sum_{j in g} (n(r, j) - 8) X[i][j]  (+ bias, + residual)
// and the gated pair silu(Wg x) * (Wu x).
//
// The weights' bytes bound it: an SM's share of HBM brings a tile of 16 rows by
// 128 columns (1056 to 1152 bytes) every 49 clocks, so that a tile has about
// 190 issue slots.  On CUDA cores its 2048 products alone take 64 (and their
// unpacking twice that); the tensor cores take them in eight mma.sync m16n8k16.
//  * The weights are the 16 x 16 operand, eight rows of the batch (four f32 ones
//    as f16 hi and lo) its 8 columns.  tcgen05's smallest shape spends 93 clocks
//    on as many weights as mma.sync multiplies in 32 a column group.
//  * Tiles lie in memory in the order in which lanes feed them (q8d_layer.cuh):
//    two 16-byte loads a lane bring a tile into registers, no byte twice, with
//    no shared memory between.  Four tiles a warp are in flight.
//  * A pair of quants costs one LOP3 under the exponent of 1024 (1024 + n, or
//    1024 + 16 n of the half-byte above) and one exact f16 subtraction or fma
//    that leaves n - 8.
//  * An f32 row enters as f16 hi + lo under a power of two for every 128 columns
//    (2^-22 relative, at least 2^-39 of the tile's largest), f16 rows as they
//    are, Q8_0 rows as their whole numbers, their scales applied to the sums.
//    The products of 32 columns are exact in f32 and summed from zero on the
//    tensor cores; the scales are applied outside and all further sums are
//    rounded f32 additions, because the tensor core cuts its own off.
//  * A cluster of CTAs takes whole strips of 16 rows, each of its CTAs a part of
//    their columns; a CTA's tiles, strip after strip, are cut into equal ranges
//    for its warps.  The warps' sums of a strip meet in shared memory, the CTAs'
//    through the cluster's, both in a fixed order.
#include <algorithm>
#include <map>
#include <mutex>
#include <tuple>

#include "q8d_layer.cuh"

namespace q8d {
namespace {

constexpr int kWarps = 16;
constexpr int kThreads = kWarps * 32;
constexpr int kAhead = 4;       // tiles a warp has in flight
// Strips (of either matrix) summed up at once, for mp rows of the batch, and
// how many of them a warp's range of a pass may touch.
__host__ __device__ constexpr int pass_parts(int mp) { return mp <= 8 ? 32 : 16; }
__host__ __device__ constexpr int pass_slots(int mp) { return pass_parts(mp) / kWarps + 2; }
constexpr int kMaxSmem = 232448;

enum Mode { kF32 = 0, kF16 = 1, kQ8 = 2 };

// Rows of the batch a column group of eight takes, and sums a lane keeps of it.
__host__ __device__ constexpr int group_rows(int mode) { return mode == kF32 ? 4 : 8; }

struct Q4Args {
  Q4Params P;
  int kt;        // tiles a strip
  int cs, ncl;   // CTAs a cluster, clusters
  int ncol;      // columns of the operand in use
  int passes;
};

struct Smem {  // offsets
  int scale, part, red, total;
};
__host__ __device__ inline Smem smem_layout(int mode, int ng, int ktl, int ncol, bool cluster) {
  const int mp = ng * group_rows(mode);
  Smem s;
  s.scale = ktl * 4 * ncol * 64;
  // the power of two of every 128 columns, or the scales of every 32
  s.part = s.scale + (mode == kF32 ? ktl * mp * 4 : mode == kQ8 ? ktl * 4 * mp * 4 : 0);
  s.part = (s.part + 15) & ~15;
  s.red = s.part + kWarps * pass_slots(mp) * mp * 16 * 4;
  s.total = s.red + (cluster ? pass_parts(mp) * mp * 16 * 4 : 0);
  return s;
}

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 load_once(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// Eight quants of a word as four pairs of f16 n - 8, columns ascending.
__device__ __forceinline__ void unpack(uint32_t w, uint32_t (&p)[4]) {
  const uint32_t magic = 0x64006400u;  // 1024, twice
  const __half2 off = __half2half2(__ushort_as_half(0x6408));    // 1032
  const __half2 sixteenth = __half2half2(__ushort_as_half(0x2c00));  // 1 / 16
  const __half2 off16 = __half2half2(__ushort_as_half(0xd480));  // -72
  const uint32_t v = w >> 8;
  const uint32_t q[4] = {(w & 0x000f000fu) | magic, (w & 0x00f000f0u) | magic, (v & 0x000f000fu) | magic,
                         (v & 0x00f000f0u) | magic};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = *reinterpret_cast<const __half2*>(&q[i]);
    const __half2 r = (i & 1) ? __hfma2(h, sixteenth, off16) : __hsub2(h, off);
    p[i] = *reinterpret_cast<const uint32_t*>(&r);
  }
}

template <int NS>
struct Tile {
  uint4 a[2];  // rows g and g + 8: a word a block of 32 columns
  uint32_t s[NS];  // their scales: NS / 2 words each (one half word each for NS 1)
};
// NS: scales a row and tile (4, 2, 1): words of the two rows' scales
template <int NS>
__device__ __forceinline__ void load_tile(const uint8_t* tile, int lane, Tile<NS>& t) {
  t.a[0] = load_once(tile + 16 * lane);
  t.a[1] = load_once(tile + 512 + 16 * lane);
  const uint8_t* s = tile + kQ4QuantBytes + (lane >> 2) * (4 * NS);
  if constexpr (NS == 4) {
    const uint4 v = load_once(s);
    t.s[0] = v.x, t.s[1] = v.y, t.s[2] = v.z, t.s[3] = v.w;
  } else if constexpr (NS == 2) {
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(t.s[0]), "=r"(t.s[1]) : "l"(s));
  } else {
    asm volatile("ld.global.nc.L1::no_allocate.u32 %0, [%1];" : "=r"(t.s[0]) : "l"(s));
  }
}
// The scale of row g (h = 0) or g + 8 for block b of 32 columns.
template <int NS>
__device__ __forceinline__ float scale_of(const Tile<NS>& t, int h, int b) {
  const int i = h * NS + b * NS / 4;  // the half word
  return f16_bits_to_f32(i & 1 ? t.s[i / 2] >> 16 : t.s[i / 2] & 0xffffu);
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float cluster_load(const float* p, uint32_t rank) {
  uint32_t a;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}

// The activations' columns [128 k0, 128 (k0 + ktl)) as the MMA's second operand:
// [tile][block of 32][column][32] f16, eight neighbouring values a lane.
template <int MODE>
__device__ __forceinline__ void build_x(const Q4Args& A, int k0, int ktl, int mp, __half* xf, float* scale) {
  const Q4Params& P = A.P;
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const int b = lane / 8, at = (lane & 7) * 4;
  for (int it = warp; it < P.m * ktl; it += kWarps) {
    const int j = it / ktl, k = it - j * ktl;
    const int col = (k0 + k) * kQ4Cols + 4 * lane;
    float f[4] = {0.f, 0.f, 0.f, 0.f};
    __half* dst = xf + ((k * 4 + b) * A.ncol + (MODE == kF32 ? 2 * j : j)) * 32 + at;
    if constexpr (MODE == kF32) {
      if (col < P.n) {
        const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(P.X) + j * P.ldx + col);
        f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
      }
      // (bits of magnitudes are ordered as they are; infinities and NaN, the
      // largest, stay what they are and make the row's sums NaN)
      uint32_t top = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) top = max(top, __float_as_uint(f[e]) & 0x7fffffffu);
      top = __reduce_max_sync(0xffffffffu, top);
      const int up = top ? min(14 - ((int)(top >> 23) - 127), 126) : 0;  // largest into [2^14, 2^15)
      const float by = __uint_as_float((uint32_t)(up + 127) << 23);
      __half hi[4], lo[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float v = f[e] * by;
        hi[e] = __float2half_rn(v);
        lo[e] = __float2half_rn(v - __half2float(hi[e]));
      }
      *reinterpret_cast<uint2*>(dst) = *reinterpret_cast<const uint2*>(hi);
      *reinterpret_cast<uint2*>(dst + 32) = *reinterpret_cast<const uint2*>(lo);
      if (lane == 0) scale[k * mp + j] = __uint_as_float((uint32_t)(127 - up) << 23);
    } else if constexpr (MODE == kF16) {
      uint2 v = make_uint2(0, 0);
      if (col < P.n) v = *reinterpret_cast<const uint2*>(static_cast<const __half*>(P.X) + j * P.ldx + col);
      *reinterpret_cast<uint2*>(dst) = v;
    } else {
      __half q[4] = {};
      float d = 0.f;
      if (col < P.n) {
        const uint8_t* blk = static_cast<const uint8_t*>(P.X) + (j * (P.ldx / 32) + col / 32) * kQBlockBytes;
        const unsigned short* w = reinterpret_cast<const unsigned short*>(blk + 2 + at);
        d = f16_bits_to_f32(*reinterpret_cast<const unsigned short*>(blk));
#pragma unroll
        for (int e = 0; e < 4; ++e) q[e] = __int2half_rn((int)(int8_t)(w[e / 2] >> (8 * (e & 1))));
      }
      *reinterpret_cast<uint2*>(dst) = *reinterpret_cast<const uint2*>(q);
      if (at == 0) scale[(k * 4 + b) * mp + j] = d;
    }
  }
}

template <int MODE, int NG, int NS>
__global__ void __launch_bounds__(kThreads, 1) q4_kernel(const Q4Args A) {
  extern __shared__ __align__(16) uint8_t smem[];
  constexpr int kMp = NG * group_rows(MODE);     // rows of the batch that fit
  constexpr int kSlots = pass_slots(kMp);
  constexpr int kSums = MODE == kF32 ? 2 : 4;    // a lane and column group
  const Q4Params& P = A.P;
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int cluster = blockIdx.x / A.cs, rank = blockIdx.x - cluster * A.cs;
  const int strips = (int)((P.p + kQ4Rows - 1LL) / kQ4Rows), rec = q4_tile_bytes(P.group);
  const int u0 = (int)((long long)cluster * strips / A.ncl), u1 = (int)((cluster + 1LL) * strips / A.ncl);
  const int k0 = rank * A.kt / A.cs, ktl = (rank + 1) * A.kt / A.cs - k0;
  const int ktl_max = (A.kt + A.cs - 1) / A.cs;
  const Smem L = smem_layout(MODE, NG, ktl_max, A.ncol, A.cs > 1);
  __half* xf = reinterpret_cast<__half*>(smem);
  float* xs = reinterpret_cast<float*>(smem + L.scale);
  float* part = reinterpret_cast<float*>(smem + L.part);
  float* red = reinterpret_cast<float*>(smem + L.red);

  // The tiles of a pass: parts (a strip of one matrix) one behind the other.
  const auto address = [&](int unit0, int i) {
    const int sp = i / ktl, k = i - sp * ktl;
    const int unit = unit0 + (P.nmat == 2 ? sp >> 1 : sp);
    return (P.nmat == 2 && (sp & 1) ? P.w[1] : P.w[0]) + ((long long)unit * A.kt + k0 + k) * rec;
  };
  const auto pass_units = [&](int pass, int& a, int& b) {
    a = u0 + (int)((long long)pass * (u1 - u0) / A.passes);
    b = u0 + (int)((pass + 1LL) * (u1 - u0) / A.passes);
  };
  const auto range = [&](int n, int& a, int& b) {
    a = warp * n / kWarps;
    b = (warp + 1) * n / kWarps;
  };

  int ua, ub, i0, i1;
  pass_units(0, ua, ub);
  range((ub - ua) * P.nmat * ktl, i0, i1);
  griddep_launch_dependents();
  // (weights wait for nothing, but another kernel may be writing them: only the
  // L2 is asked for them before the work in front is done)
  for (int i = i0; i < min(i1, i0 + kAhead); ++i) {
    const uint8_t* p = address(ua, i) + lane * 128;
    if (lane * 128 < rec) asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
  }
  griddep_wait();

  Tile<NS> buf[kAhead];
  const uint8_t* next;  // the tile behind those in flight
  int next_i, next_k;   // its place in the pass and in its part
  const auto start = [&](int unit0) {
    next_i = i0;
    if (i0 >= i1) return;
    next = address(unit0, i0);
    next_k = i0 % ktl;
  };
  const auto fetch = [&](int unit0, Tile<NS>& b) {
    if (next_i >= i1) return;
    load_tile<NS>(next, lane, b);
    ++next_i;
    next += rec;
    if (++next_k == ktl) {
      next_k = 0;
      if (next_i < i1) next = address(unit0, next_i);
    }
  };
  start(ua);
#pragma unroll
  for (int d = 0; d < kAhead; ++d) fetch(ua, buf[d]);

  build_x<MODE>(A, k0, ktl, kMp, xf, xs);
  __syncthreads();

  for (int pass = 0; pass < A.passes; ++pass) {
    float acc[NG][kSums];
#pragma unroll
    for (int q = 0; q < NG; ++q)
#pragma unroll
      for (int e = 0; e < kSums; ++e) acc[q][e] = 0.f;
    int k = i0 < i1 ? i0 % ktl : 0, slot = 0;
    // a part's sums, [slot][row of the batch][16]
    const auto flush = [&]() {
      float* dst = part + (warp * kSlots + slot) * kMp * 16;
#pragma unroll
      for (int q = 0; q < NG; ++q) {
        if constexpr (MODE == kF32) {
          dst[(4 * q + t) * 16 + g] = acc[q][0];
          dst[(4 * q + t) * 16 + g + 8] = acc[q][1];
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) dst[(8 * q + 2 * t + (e & 1)) * 16 + g + 8 * (e >> 1)] = acc[q][e];
        }
#pragma unroll
        for (int e = 0; e < kSums; ++e) acc[q][e] = 0.f;
      }
      ++slot;
    };
    for (int i = i0; i < i1; i += kAhead) {
#pragma unroll
      for (int d = 0; d < kAhead; ++d) {
        if (i + d < i1) {
          const Tile<NS>& T = buf[d];
          float sum[NG][2];
          if constexpr (MODE == kF32) {
#pragma unroll
            for (int q = 0; q < NG; ++q) sum[q][0] = sum[q][1] = 0.f;
          }
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            const uint32_t w0 = b == 0 ? T.a[0].x : b == 1 ? T.a[0].y : b == 2 ? T.a[0].z : T.a[0].w;
            const uint32_t w1 = b == 0 ? T.a[1].x : b == 1 ? T.a[1].y : b == 2 ? T.a[1].z : T.a[1].w;
            uint32_t r0[4], r1[4];
            unpack(w0, r0);
            unpack(w1, r1);
            const float s0 = scale_of<NS>(T, 0, b), s1 = scale_of<NS>(T, 1, b);
#pragma unroll
            for (int q = 0; q < NG; ++q) {
              uint4 x = make_uint4(0, 0, 0, 0);
              if (8 * q + g < A.ncol)
                x = *reinterpret_cast<const uint4*>(xf + ((k * 4 + b) * A.ncol + 8 * q + g) * 32 + 8 * t);
              float c[4] = {0.f, 0.f, 0.f, 0.f};
              mma16816(c, r0[0], r1[0], r0[1], r1[1], x.x, x.y);
              mma16816(c, r0[2], r1[2], r0[3], r1[3], x.z, x.w);
              if constexpr (MODE == kF32) {
                sum[q][0] = fmaf(s0, c[0] + c[1], sum[q][0]);
                sum[q][1] = fmaf(s1, c[2] + c[3], sum[q][1]);
              } else if constexpr (MODE == kF16) {
                acc[q][0] = fmaf(s0, c[0], acc[q][0]);
                acc[q][1] = fmaf(s0, c[1], acc[q][1]);
                acc[q][2] = fmaf(s1, c[2], acc[q][2]);
                acc[q][3] = fmaf(s1, c[3], acc[q][3]);
              } else {
                const float2 d2 = *reinterpret_cast<const float2*>(xs + (k * 4 + b) * kMp + 8 * q + 2 * t);
                acc[q][0] = fmaf(s0 * d2.x, c[0], acc[q][0]);
                acc[q][1] = fmaf(s0 * d2.y, c[1], acc[q][1]);
                acc[q][2] = fmaf(s1 * d2.x, c[2], acc[q][2]);
                acc[q][3] = fmaf(s1 * d2.y, c[3], acc[q][3]);
              }
            }
          }
          if constexpr (MODE == kF32) {
#pragma unroll
            for (int q = 0; q < NG; ++q) {
              const float by = xs[k * kMp + 4 * q + t];
              acc[q][0] = fmaf(by, sum[q][0], acc[q][0]);
              acc[q][1] = fmaf(by, sum[q][1], acc[q][1]);
            }
          }
          fetch(ua, buf[d]);
          if (++k == ktl) {
            k = 0;
            flush();
          }
        }
      }
    }
    if (k != 0) flush();
    const int n = (ub - ua) * P.nmat * ktl, pa = ua, pu = ub - ua;
    const int first_n = n;
    if (pass + 1 < A.passes) {  // the next pass's first tiles
      pass_units(pass + 1, ua, ub);
      range((ub - ua) * P.nmat * ktl, i0, i1);
      start(ua);
#pragma unroll
      for (int d = 0; d < kAhead; ++d) fetch(ua, buf[d]);
    }
    __syncthreads();
    // a part's sum over the warps whose ranges meet it, in their order
    const auto cta_sum = [&](int sp, int j, int row) {
      const int a = ((sp * ktl + 1) * kWarps - 1) / first_n, b = ((sp + 1) * ktl * kWarps - 1) / first_n;
      float v = 0.f;
      for (int w = a; w <= b; ++w) {
        const int s0 = w * first_n / kWarps;
        if ((w + 1) * first_n / kWarps == s0) continue;  // (a warp without tiles)
        v += part[((w * kSlots + sp - s0 / ktl) * kMp + j) * 16 + row];
      }
      return v;
    };
    const auto finish = [&](int unit, int j, int row, float v, float up) {
      const int r = (pa + unit) * kQ4Rows + row;
      if (r >= P.p) return;
      if (P.nmat == 2) {
        v = v / (1.f + expf(-v)) * up;
      } else {
        if (P.bias) v += P.bias[r];
        if (P.residual) v += P.residual[j * P.ldr + r];
      }
      P.Y[j * P.ldy + r] = v;
    };
    if (A.cs == 1) {
      for (int o = threadIdx.x; o < pu * P.m * 16; o += kThreads) {
        const int row = o & 15, j = (o >> 4) % P.m, unit = (o >> 4) / P.m;
        if (P.nmat == 2)
          finish(unit, j, row, cta_sum(2 * unit, j, row), cta_sum(2 * unit + 1, j, row));
        else
          finish(unit, j, row, cta_sum(unit, j, row), 0.f);
      }
      __syncthreads();
    } else {
      for (int o = threadIdx.x; o < pu * P.nmat * P.m * 16; o += kThreads) {
        const int row = o & 15, j = (o >> 4) % P.m, sp = (o >> 4) / P.m;
        red[o] = cta_sum(sp, j, row);
      }
      cluster_sync();
      for (int o = rank * kThreads + threadIdx.x; o < pu * P.m * 16; o += A.cs * kThreads) {
        const int row = o & 15, j = (o >> 4) % P.m, unit = (o >> 4) / P.m;
        const int at = ((P.nmat * unit) * P.m + j) * 16 + row;
        float v = 0.f, up = 0.f;
        for (int c = 0; c < A.cs; ++c) {
          v += cluster_load(red + at, c);
          if (P.nmat == 2) up += cluster_load(red + at + P.m * 16, c);
        }
        finish(unit, j, row, v, up);
      }
      cluster_sync();  // (the sums are read before they change or their CTA leaves)
    }
  }
}

// ---- plan and launch --------------------------------------------------------
int max_clusters(const void* fn, int cs, int smem, int* out) {
  static std::mutex mu;
  static std::map<std::tuple<const void*, int, int>, int> known;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return record_cuda(e);
  std::lock_guard<std::mutex> lock(mu);
  const auto key = std::make_tuple(fn, cs, dev);
  const auto it = known.find(key);
  if (it != known.end()) {
    *out = it->second;
    return Q8D_OK;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(cs * 64);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cs;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  e = cudaOccupancyMaxActiveClusters(&n, fn, &cfg);
  if (e != cudaSuccess) return record_cuda(e);
  known[key] = *out = n;
  return Q8D_OK;
}

template <int MODE, int NG, int NS>
int launch(const Q4Params& P, cudaStream_t stream) {
  const auto kernel = q4_kernel<MODE, NG, NS>;
  const void* fn = reinterpret_cast<const void*>(kernel);
  int rc = configure_kernel(fn, kMaxSmem, false);
  if (rc) return rc;
  Q4Args A{};
  A.P = P;
  A.kt = q4_tiles(P.n);
  A.ncol = (MODE == kF32 ? 2 : 1) * P.m;
  const int strips = (int)q4_strips(P.p);
  // CTAs a cluster: a strip's columns in more parts fill the machine where it
  // has few strips or leaves a part of it idle in the last round, for two
  // meetings of the cluster; and many rows of activations need the parts to fit
  // shared memory.
  long long best = -1;
  int smem = 0;
  for (int cs = 1; cs <= 8 && cs <= A.kt; cs *= 2) {
    const int ktl = (A.kt + cs - 1) / cs;
    const Smem L = smem_layout(MODE, NG, ktl, A.ncol, cs > 1);
    if (L.total > kMaxSmem) continue;
    int most = sm_count();
    if (cs > 1) {
      rc = max_clusters(fn, cs, kMaxSmem, &most);
      if (rc) return rc;
      if (most < 1) continue;
    }
    const int ncl = std::min(most, strips);
    const long long cost = (long long)((strips + ncl - 1) / ncl) * P.nmat * ktl + (cs > 1 ? 40 : 0);
    if (best < 0 || cost < best) {
      best = cost;
      A.cs = cs;
      A.ncl = ncl;
      smem = L.total;
    }
  }
  if (best < 0) return Q8D_EUNSUPPORTED;
  const int units = (strips + A.ncl - 1) / A.ncl;
  constexpr int kParts = pass_parts(NG * group_rows(MODE));
  A.passes = (units * P.nmat + kParts - 1) / kParts;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(A.cs * A.ncl);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = A.cs;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, A);
  return e == cudaSuccess ? Q8D_OK : record_cuda(e);
}

template <int MODE, int NG>
int launch_g(const Q4Params& P, cudaStream_t stream) {
  switch (P.group) {
    case 32: return launch<MODE, NG, 4>(P, stream);
    case 64: return launch<MODE, NG, 2>(P, stream);
    default: return launch<MODE, NG, 1>(P, stream);
  }
}

template <int MODE>
int launch_m(const Q4Params& P, cudaStream_t stream) {
  return P.m <= group_rows(MODE) ? launch_g<MODE, 1>(P, stream) : launch_g<MODE, 2>(P, stream);
}

}  // namespace

int q4_launch(const Q4Params& P, cudaStream_t stream) {
  if (P.x_dtype == Q8D_KV_F16) return launch_m<kF16>(P, stream);
  if (P.x_dtype == Q8D_KV_Q8_0) return launch_m<kQ8>(P, stream);
  // f32 rows take two columns each: eight rows a launch
  Q4Params Q = P;
  for (int j = 0; j < P.m; j += 8) {
    Q.m = std::min(8, P.m - j);
    Q.X = static_cast<const float*>(P.X) + j * P.ldx;
    Q.Y = P.Y + j * P.ldy;
    Q.residual = P.residual ? P.residual + j * P.ldr : nullptr;
    const int rc = launch_m<kF32>(Q, stream);
    if (rc) return rc;
  }
  return Q8D_OK;
}

}  // namespace q8d
