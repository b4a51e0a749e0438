// Products with 4-bit weights and group scales for 1 to 16 activation rows:
//   Y[i][r] = sum_g s(r, g) sum_{j in g} (n(r, j) - 8) X[i][j]  (+ bias, + residual)
// and the gated pair silu(Wg x) * (Wu x).
//
// The weights' bytes bound it: an SM's share of HBM brings a tile of 16 rows by
// 128 columns (1056 to 1152 bytes) every 49 clocks, so that a tile has about
// 190 issue slots.  On CUDA cores its 2048 products alone take 64 (and their
// unpacking twice that); the tensor cores take them in eight mma.sync m16n8k16.
//  * The weights are the 16 x 16 operand, eight rows of the batch (four f32 ones
//    as f16 hi and lo) its 8 columns: 16 clocks of the tensor pipe a tile and column
//    group (counters of one and of sixteen rows), where a tcgen05.mma of as many
//    weights takes 93 for any number of columns up to 128 (q8d_mma.cu) and wants
//    them written out as f16 first.
//  * Tiles lie in memory in the order in which lanes feed them (q8d_layer.cuh):
//    two 16-byte reads a lane take a tile from shared memory, no byte twice and
//    no bank twice.  Each warp has a ring of its own there, filled by bulk copies
//    of two or four tiles that one lane issues: nothing but the warp itself waits
//    for them.  (Loads straight into registers, four tiles ahead, waited for the
//    newest of them too: 27.0 us for the gated pair 3584 -> 18944 of one token.)
//  * A pair of quants costs one LOP3 under the exponent of 1024 (1024 + n, or
//    1024 + 16 n of the half-byte above) and one exact f16 subtraction or fma
//    that leaves n - 8.
//  * An f32 row enters as f16 hi + 2^-12 lo under a power of two for every 128
//    columns (2^-22 relative, 2^-51 of the tile's largest at worst), f16 rows as
//    they are, Q8_0 rows as their whole numbers, their scales applied to the sums.
//    What that leaves of elements below 2^-32 of their tile's largest (kFar) is
//    added in 64 bits where the sums meet, so that an outlier on a weight of zero
//    costs its neighbours nothing.
//    The products are exact in f32; those of one scale, 128 columns at most, are
//    summed from zero on the tensor cores, the scales are applied outside and all
//    further sums are rounded f32 additions, because the tensor core cuts its own
//    off.
//  * A cluster of CTAs takes whole strips of 16 rows, each of its CTAs a part of
//    their columns; a CTA's tiles, strip after strip, are cut into equal ranges
//    for its warps.  The warps' sums of a strip meet in shared memory, the CTAs' in
//    that of the one that finishes them, both in a fixed order.
//
// us in a graph (and TB/s of weights): one row, 896 -> 151936 15.2 (4.8), gated 3584
// -> 18944 15.6 (4.9), 3584 -> 4608 5.8; gated, eight rows 23.5, sixteen f16 rows 27.6,
// Q8_0 34.5; 18944 -> 3584, sixteen rows 26.1.  A call spends about four
// microseconds starting and meeting; then a tile takes 50 to 55 clocks with one
// column group (150 instructions, 58 % of the issue slots), 80 with two (latency:
// sixteen warps of 128 registers).  Four groups keep 8 to 44 bytes a thread in local
// memory beside those registers; of 18944 -> 3584, sixteen rows, the tensor pipe is
// busy 30 % and the issue slots 47 %.
#include <algorithm>
#include <array>
#include <atomic>
#include <map>
#include <mutex>
#include <set>
#include <tuple>
#include <utility>

#include "q8d_layer.cuh"

namespace q8d {
namespace {

enum Mode { kF32 = 0, kF16 = 1, kQ8 = 2 };  // the rows of X

constexpr int kMaxCluster = 16;  // CTAs (more than eight are no portable size)
constexpr int kMaxStages = 4;    // copies of a warp in flight
// Tiles a copy.
__host__ __device__ constexpr int chunk_tiles(int mode, int ng) { return ng > 1 && mode == kF32 ? 2 : 4; }
// Strips (of either matrix) that a pass sums up at most, and how many of them a
// warp's range of a pass may touch.
constexpr int kMaxParts = 128;
__host__ __device__ constexpr int pass_slots(int warps, int parts) { return parts / warps + 2; }
constexpr int kMaxSmem = 232448;   // of a CTA alone on its SM
constexpr int kHalfSmem = 115712;  // of two (228 KB an SM, 1 KB of it for each CTA)

// Rows of the batch a column group of eight takes, and sums a lane keeps of it.
__host__ __device__ constexpr int group_rows(int mode) { return mode == kF32 ? 4 : 8; }

struct Q4Args {
  Q4Params P;
  int kt;        // tiles a strip
  int cs, ncl;   // CTAs a cluster, clusters
  int ncol;      // columns of the operand in use
  int passes, parts;  // strips a pass, at most
  int stages;         // of a warp's ring
  uint32_t polls;     // of a wait for a copy before it is given up
};

// The operand of the activations in shared memory: a column (a row of X, or its
// hi or lo part) is ktl tiles of 128 f16 and 64 bytes, so that two neighbouring
// columns lie in different halves of the banks.
__host__ __device__ constexpr int x_stride(int ktl) { return ktl * kQ4Cols + 32; }  // f16
// Scales of the activations: a power of two a row and tile, [row][tile], or one a
// row and block of 32, [block][row], so that a lane's two rows lie side by side.
__host__ __device__ constexpr int scale_floats(int mode, int mp, int ktl) {
  return mode == kF32 ? mp * ktl : mode == kQ8 ? mp * 4 * ktl : 0;
}
struct Smem {  // offsets
  int scale, far, part, red, meets, bars, ring;  // (the ring's stages take what is left)
};
__host__ __device__ inline Smem smem_layout(int warps, int mode, int ng, int ktl, int ncol, int parts,
                                            int cs) {
  const int mp = ng * group_rows(mode);
  Smem s;
  s.scale = ncol * x_stride(ktl) * 2;
  s.far = s.scale + ((scale_floats(mode, mp, ktl) * 4 + 15) & ~15);
  s.part = s.far + (mode == kF32 ? (mp * ktl + 15) & ~15 : 0);
  s.red = s.part + warps * pass_slots(warps, parts) * mp * 16 * 4;
  s.meets = s.red + (cs > 1 ? (parts * mp + 2 * cs) * 16 * 4 : 0);
  s.bars = s.meets + (parts * 4 + 4 + 15 & ~15);  // (and whether rows have far elements)
  s.ring = (s.bars + warps * kMaxStages * 8 + 127) & ~127;
  return s;
}

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same from zero.
__device__ __forceinline__ void mma16816_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{0f00000000,0f00000000,0f00000000,0f00000000};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Whole numbers under the exponent of 1024 become f16 by a mask and one exact
// operation (the conversion that Kim, Henry, Fahim and Awadalla, "Who Says Elephants
// Can't Run: Bringing Large Scale MoE Models into Cloud Scale Production", 2022,
// describe for 4- and 8-bit weights).
// Constants of unpack(), kept out of the compiler's sight: with them in
// registers (w & mask) | magic is one LOP3, as a constant it is two.
struct Magic {
  uint32_t k1024, off, sixteenth, off16;
  __device__ __forceinline__ Magic() {
    asm volatile("mov.b32 %0, 0x64006400;" : "=r"(k1024));      // 1024, twice
    asm volatile("mov.b32 %0, 0x64086408;" : "=r"(off));        // 1032
    asm volatile("mov.b32 %0, 0x2c002c00;" : "=r"(sixteenth));  // 1 / 16
    asm volatile("mov.b32 %0, 0xd480d480;" : "=r"(off16));      // -72
  }
};
// Eight quants of a word as four pairs of f16 n - 8, columns ascending.
__device__ __forceinline__ void unpack(uint32_t w, const Magic& m, uint32_t (&p)[4]) {
  const uint32_t v = w >> 8;
  uint32_t q[4];
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(q[0]) : "r"(w), "n"(0x000f000f), "r"(m.k1024));
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(q[1]) : "r"(w), "n"(0x00f000f0), "r"(m.k1024));
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(q[2]) : "r"(v), "n"(0x000f000f), "r"(m.k1024));
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(q[3]) : "r"(v), "n"(0x00f000f0), "r"(m.k1024));
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    asm("sub.f16x2 %0, %1, %2;" : "=r"(p[i]) : "r"(q[i]), "r"(m.off));
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(p[i + 1]) : "r"(q[i + 1]), "r"(m.sixteenth), "r"(m.off16));
  }
}

template <int NS>
struct Tile {
  uint4 a[2];  // rows g and g + 8: a word a block of 32 columns
  uint32_t s[NS];  // their scales: NS / 2 words each (one half word each for NS 1)
};
// NS: scales a row and tile (4, 2, 1): words of the two rows' scales
template <int NS>
__device__ __forceinline__ void read_tile(const uint8_t* tile, int lane, Tile<NS>& t) {
  t.a[0] = *reinterpret_cast<const uint4*>(tile + 16 * lane);
  t.a[1] = *reinterpret_cast<const uint4*>(tile + 512 + 16 * lane);
  const uint8_t* s = tile + kQ4QuantBytes + (lane >> 2) * (4 * NS);
  if constexpr (NS == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(s);
    t.s[0] = v.x, t.s[1] = v.y, t.s[2] = v.z, t.s[3] = v.w;
  } else if constexpr (NS == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(s);
    t.s[0] = v.x, t.s[1] = v.y;
  } else {
    t.s[0] = *reinterpret_cast<const uint32_t*>(s);
  }
}
// The scale of row g (h = 0) or g + 8 for block b of 32 columns.
template <int NS>
__device__ __forceinline__ float scale_of(const Tile<NS>& t, int h, int b) {
  const int i = h * NS + b * NS / 4;  // the half word
  const __half2 v = *reinterpret_cast<const __half2*>(&t.s[i / 2]);
  return i & 1 ? __high2float(v) : __low2float(v);
}

// The cluster's barrier in two halves: what a CTA wrote before it arrived is seen
// by those that have waited.
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Stores v at p's place in the shared memory of the cluster's CTA `rank`.
__device__ __forceinline__ void cluster_store(float* p, uint32_t rank, float v) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory");
}

// f32 elements below this under their tile's power of two are `far`: hi + 2^-12 lo,
// 2^-37 at best, is no longer within 2^-19 of them.
constexpr float kFar = 0x1p-18f;
// Two elements x times `by` as f16 hi and what that leaves (exactly, times 2^12 too).
__device__ __forceinline__ void split2(uint64_t x, float by, __half2& hi, __half2& lo) {
  float a, b;
  unpack2(mul2(x, pack2(by, by)), a, b);
  hi = __floats2half2_rn(a, b);
  const float2 h = __half22float2(hi);
  const float by12 = by * 0x1p12f;
  unpack2(fma2(pack2(h.x, h.y), pack2(-0x1p12f, -0x1p12f), mul2(x, pack2(by12, by12))), a, b);
  lo = __floats2half2_rn(a, b);
}
// Adds what the operand lacks of the far elements, times their weights, to the sums
// of a pass (its strips pa .. pa + pu - 1), into those of the first warp that met a
// part.  Its CTA's tiles of a strip are the ktl from k0 on.  (Rows seldom hold
// such elements; 3584 -> 18944, gated, one row: 15.4 us, of half zeros 15.8, with one
// of them 18.9, with one in every tile 73.)
template <int kWarps, int NG, int NS>
__device__ __noinline__ void add_far_terms(const Q4Args& A, uint8_t* smem, int pa, int pu, int k0, int ktl) {
  constexpr int kRec = kQ4QuantBytes + kQ4Rows * NS * 2, kMp = NG * group_rows(kF32);
  const Q4Params& P = A.P;
  const int most = (A.kt + A.cs - 1) / A.cs, parts = pu * P.nmat, cols = min(ktl * kQ4Cols, P.n - k0 * kQ4Cols);
  const Smem L = smem_layout(kWarps, kF32, NG, most, A.ncol, A.parts, A.cs);
  const int row = threadIdx.x & 15, h = row / 8, g = row & 7;
  const uint32_t half = 0xffffu << (threadIdx.x & 16);  // the sixteen threads of a strip and row of X
  const auto ballot = [&](bool yes) { return __ballot_sync(half, yes) >> (threadIdx.x & 16) & 0xffffu; };
  for (int o = threadIdx.x / 16; o < parts * P.m; o += kWarps * 2) {
    const int sp = o / P.m, j = o - sp * P.m, unit = pa + sp / P.nmat;
    const float* scale = reinterpret_cast<const float*>(smem + L.scale) + j * most;
    const float* x = static_cast<const float*>(P.X) + j * P.ldx + k0 * kQ4Cols;
    const uint8_t* tiles = P.w[sp % P.nmat] + ((long long)unit * A.kt + k0) * kRec;
    double sum = 0.0;
    const auto tile_terms = [&](int k) {
      const float back = scale[k], by = 1.f / back;  // (powers of two)
      const uint8_t* tile = tiles + (long long)k * kRec;
      float v[kQ4Cols / 16];
#pragma unroll
      for (int i = 0; i < kQ4Cols / 16; ++i) {
        const int c = k * kQ4Cols + 16 * i + row;
        v[i] = c < cols ? x[c] : 0.f;
      }
#pragma unroll
      for (int i = 0; i < kQ4Cols / 16; ++i) {
        for (uint32_t hits = ballot(v[i] != 0.f && fabsf(v[i]) < kFar * back); hits; hits &= hits - 1) {
          const int c = 16 * i + __ffs(hits) - 1, b = c / 32, t = c / 8 & 3, e = c & 7;
          const float f = __shfl_sync(half, v[i], c & 15, 16);
          __half2 hi, lo;
          split2(pack2(f, f), by, hi, lo);
          const double held = (double)__low2float(hi) + (double)__low2float(lo) * 0x1p-12;
          const uint32_t w = *reinterpret_cast<const uint32_t*>(tile + 512 * h + 16 * (4 * g + t) + 4 * b);
          const unsigned short s =
              *reinterpret_cast<const unsigned short*>(tile + kQ4QuantBytes + 2 * (NS * (2 * g + h) + b * NS / 4));
          sum += (f - held * back) * ((int)(w >> (4 * (e / 2 + 4 * (e & 1))) & 15u) - 8) * (double)f16_bits_to_f32(s);
        }
      }
    };
    for (int k = 0; k < ktl; k += 16)
      for (uint32_t far = ballot(k + row < ktl && smem[L.far + j * most + k + row]); far; far &= far - 1)
        tile_terms(k + __ffs(far) - 1);
    const uint32_t met = reinterpret_cast<const uint32_t*>(smem + L.meets)[sp];
    const int slot = (__ffs(met) - 1) * pass_slots(kWarps, A.parts) + (int)(met >> 24);
    reinterpret_cast<float*>(smem + L.part)[(slot * kMp + j) * 16 + row] += (float)sum;
  }
  __syncthreads();
}

// The activations' columns [128 k0, 128 (k0 + ktl)) as the MMA's second operand.
// xstep: x_stride; most: tiles of the largest part of a row.
// far: whether a tile of an f32 row has far elements, [row][tile];
// returns whether this thread met one.
// then(): what is to be started once the first loads are on their way.
template <int MODE, int kWarps, int kMp, typename Then>
__device__ __forceinline__ bool build_x(const Q4Args& A, int k0, int ktl, int most, int xstep, __half* xf,
                                        float* scale, uint8_t* far, Then then) {
  constexpr int kLoads = kWarps / 2;  // items a warp loads before it uses the first
  const Q4Params& P = A.P;
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const int at = (lane & 7) * 4;  // in the block of 32
  // (item 128 columns of a row; rows one behind the other)
  int j = 0, k = warp;
  const auto wrap = [&]() {
    while (k >= ktl && j < P.m) {
      k -= ktl;
      ++j;
    }
  };
  wrap();
  bool met_far = false;
  if (j >= P.m) then();
  for (bool started = false; j < P.m; started = true) {
    int js[kLoads], ks[kLoads];
    float4 f[kLoads];                // f32
    uint2 u[kLoads];                 // f16, or four quants
    unsigned short d[kLoads];        // the quants' scale
#pragma unroll
    for (int l = 0; l < kLoads; ++l) {
      js[l] = j;
      ks[l] = k;
      const int col = (k0 + k) * kQ4Cols + 4 * lane;
      f[l] = make_float4(0.f, 0.f, 0.f, 0.f);
      u[l] = make_uint2(0, 0);
      d[l] = 0;
      k += kWarps;
      wrap();
      const int j = js[l];
      if (j >= P.m || col >= P.n) continue;
      if constexpr (MODE == kF32) {
        f[l] = *reinterpret_cast<const float4*>(static_cast<const float*>(P.X) + j * P.ldx + col);
      } else if constexpr (MODE == kF16) {
        u[l] = *reinterpret_cast<const uint2*>(static_cast<const __half*>(P.X) + j * P.ldx + col);
      } else {
        const uint8_t* blk = static_cast<const uint8_t*>(P.X) + (j * (P.ldx / 32) + col / 32) * kQBlockBytes;
        const unsigned short* w = reinterpret_cast<const unsigned short*>(blk + 2 + at);
        d[l] = *reinterpret_cast<const unsigned short*>(blk);
        u[l].x = w[0] | (uint32_t)w[1] << 16;
      }
    }
    if (!started) then();
    uint32_t suspects = 0;  // items with elements that may be far
#pragma unroll
    for (int l = 0; l < kLoads; ++l) {
      const int j = js[l], k = ks[l];
      if (j >= P.m) break;  // (the whole warp)
      __half* dst = xf + (MODE == kF32 ? 2 * j : j) * xstep + k * kQ4Cols + 4 * lane;
      if constexpr (MODE == kF32) {
        const float v[4] = {f[l].x, f[l].y, f[l].z, f[l].w};
        // (bits of magnitudes are ordered as they are; infinities and NaN, the
        // largest, stay what they are and make the row's sums NaN)
        uint32_t top = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) top = max(top, __float_as_uint(v[e]) & 0x7fffffffu);
        top = __reduce_max_sync(0xffffffffu, top);
        const int up = top ? min(14 - ((int)(top >> 23) - 127), 114) : 0;  // largest into [2^14, 2^15)
        const float by = __uint_as_float((uint32_t)(up + 127) << 23);
        __half2 hi[2], lo[2];
        split2(pack2(v[0], v[1]), by, hi[0], lo[0]);
        split2(pack2(v[2], v[3]), by, hi[1], lo[1]);
        *reinterpret_cast<uint2*>(dst) = *reinterpret_cast<const uint2*>(hi);
        *reinterpret_cast<uint2*>(dst + xstep) = *reinterpret_cast<const uint2*>(lo);
        if (lane == 0) {
          scale[j * most + k] = __uint_as_float((uint32_t)(127 - up) << 23);
          far[j * most + k] = 0;
        }
        // (zeros are no far elements, but are told apart below)
        const __half2 least = __hmin2(__habs2(hi[0]), __habs2(hi[1]));
        const bool small = !__hbge2(least, __float2half2_rn(kFar));
        suspects |= (__any_sync(0xffffffffu, small) ? 1u : 0u) << l;
      } else if constexpr (MODE == kF16) {
        *reinterpret_cast<uint2*>(dst) = u[l];
      } else {
        // (a byte q + 128 under the exponent of 1024, less 1152)
        const uint32_t w = u[l].x ^ 0x80808080u;
        uint2 q;
        asm("sub.f16x2 %0, %1, %2;" : "=r"(q.x) : "r"(__byte_perm(w, 0x64646464u, 0x4140)), "r"(0x64806480u));
        asm("sub.f16x2 %0, %1, %2;" : "=r"(q.y) : "r"(__byte_perm(w, 0x64646464u, 0x4342)), "r"(0x64806480u));
        *reinterpret_cast<uint2*>(dst) = q;
        if (at == 0) scale[(k * 4 + lane / 8) * kMp + j] = f16_bits_to_f32(d[l]);
      }
    }
    if (MODE == kF32 && suspects) {
      __syncwarp();
#pragma unroll
      for (int l = 0; l < kLoads; ++l) {
        if (!(suspects >> l & 1u)) continue;
        const int at = js[l] * most + ks[l];
        const float limit = kFar * scale[at], v[4] = {f[l].x, f[l].y, f[l].z, f[l].w};
        bool out = false;
#pragma unroll
        for (int e = 0; e < 4; ++e) out |= v[e] != 0.f && fabsf(v[e]) < limit;
        out = __any_sync(0xffffffffu, out);
        met_far |= out;
        if (lane == 0 && out) far[at] = 1;
      }
    }
  }
  return met_far;
}

// The polls of a wait behind the first one, out of line: a limit in the loop's own
// registers costs eight rows, gated 3584 -> 18944, 0.6 us of 23.5.
__device__ __noinline__ bool wait_on(uint64_t* bar, uint32_t parity, uint32_t polls) {
  return mbar_wait(bar, parity, polls);
}

// kWarps warps a CTA, sixteen an SM
template <int kWarps, int MODE, int NG, int NS>
__global__ void __launch_bounds__(kWarps * 32, 16 / kWarps) q4_kernel(const __grid_constant__ Q4Args A) {
  extern __shared__ __align__(128) uint8_t smem[];
  constexpr int kMp = NG * group_rows(MODE);     // rows of the batch that fit
  constexpr int kThreads = kWarps * 32;
  constexpr int kSums = MODE == kF32 ? 2 : 4;  // a lane and column group
  constexpr int kRec = kQ4QuantBytes + kQ4Rows * NS * 2;
  constexpr int kChunk = chunk_tiles(MODE, NG), kStage = kChunk * kRec;
  const Q4Params& P = A.P;
  const int slot_floats = pass_slots(kWarps, A.parts) * kMp * 16;  // a warp's parts
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int cluster = blockIdx.x / A.cs, rank = blockIdx.x - cluster * A.cs;
  const int strips = (int)((P.p + kQ4Rows - 1LL) / kQ4Rows);
  const int u0 = (int)((long long)cluster * strips / A.ncl), u1 = (int)((cluster + 1LL) * strips / A.ncl);
  const int k0 = rank * A.kt / A.cs, ktl = (rank + 1) * A.kt / A.cs - k0;
  const int ktl_max = (A.kt + A.cs - 1) / A.cs;
  const Smem L = smem_layout(kWarps, MODE, NG, ktl_max, A.ncol, A.parts, A.cs);
  __half* xf = reinterpret_cast<__half*>(smem);
  float* xs = reinterpret_cast<float*>(smem + L.scale);
  uint8_t* far = smem + L.far;
  float* part = reinterpret_cast<float*>(smem + L.part);
  float* red = reinterpret_cast<float*>(smem + L.red);
  uint32_t* meets = reinterpret_cast<uint32_t*>(smem + L.meets);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L.bars) + warp * kMaxStages;
  uint8_t* ring = smem + L.ring + warp * A.stages * kStage;

  // The tiles of a pass: parts (a strip of one matrix) one behind the other.
  // This warp's range of them, cut where a part ends, is walked twice: by the
  // copies and, some stages behind, by the products.
  struct Walk {
    int pass, ua, ub;  // the pass and its strips
    int sp, k, n;      // the part; the next tile of it; tiles left of it here
    int left;          // tiles left of the range behind those
  };
  const auto enter = [&](Walk& w, int pass) {  // (n 0: a pass without tiles)
    w.pass = pass;
    w.ua = u0 + (int)((long long)pass * (u1 - u0) / A.passes);
    w.ub = u0 + (int)((pass + 1LL) * (u1 - u0) / A.passes);
    const int n = (w.ub - w.ua) * P.nmat * ktl, i0 = warp * n / kWarps;
    w.left = (warp + 1) * n / kWarps - i0;
    w.sp = i0 / ktl;
    w.k = i0 - w.sp * ktl;
    w.n = min(ktl - w.k, w.left);
    w.left -= w.n;
  };
  const auto next_part = [&](Walk& w) {
    ++w.sp;
    w.k = 0;
    w.n = min(ktl, w.left);
    w.left -= w.n;
  };

  Walk ahead{};  // where the next copy starts
  int issued = 0;
  const uint8_t* src = nullptr;
  const auto locate = [&]() {
    while (ahead.n == 0) {
      if (ahead.pass + 1 >= A.passes) return;
      enter(ahead, ahead.pass + 1);
    }
    const int unit = ahead.ua + (P.nmat == 2 ? ahead.sp >> 1 : ahead.sp);
    src = (P.nmat == 2 && (ahead.sp & 1) ? P.w[1] : P.w[0]) + ((long long)unit * A.kt + k0 + ahead.k) * kRec;
  };
  const uint64_t policy = policy_evict_first();
  const auto issue = [&](int stage) {
    const int n = min(kChunk, ahead.n);
    if (n == 0) return;
    if (lane == 0) {
      mbar_arrive_expect_tx(bars + stage, n * kRec);
      bulk_g2s(ring + stage * kStage, src, n * kRec, bars + stage, policy);
    }
    ++issued;
    ahead.n -= n;
    src += n * kRec;
    if (ahead.n == 0) {
      next_part(ahead);
      locate();
    }
  };
  griddep_launch_dependents();
  if (A.cs > 1) cluster_arrive();  // (waited for before the first store into another CTA)
  if (lane == 0)
    for (int s = 0; s < A.stages; ++s) mbar_init(bars + s, 1);
  fence_barrier_init();
  __syncwarp();
  enter(ahead, 0);
  locate();
  // (weights wait for nothing, but another kernel may be writing them: only the
  // L2 is asked for the first ones before the work in front is done)
  if (lane == 0 && ahead.n) bulk_prefetch_l2(src, min(A.stages * kChunk, ahead.n) * kRec);
  griddep_wait();
  const int xstep = x_stride(ktl_max);
  // One or two rows of X are asked for before the weights: every warp waits for
  // them, and all SMs' copies are microseconds of HBM (gated 3584 -> 18944, us with
  // the rows / the weights first: one row 15.6 / 16.3, four 17.4 / 17.1; 16 Q8_0
  // rows 3584 -> 4736 15.3 / 14.7).
  const auto start = [&]() {
    for (int s = 0; s < A.stages; ++s) issue(s);
  };
  const bool rows_first = P.m <= 2;
  if (!rows_first) start();
  const bool mine_far = build_x<MODE, kWarps, kMp>(A, k0, ktl, ktl_max, xstep, xf, xs, far, [&]() {
    if (rows_first) start();
  });
  const bool any_far = __syncthreads_or(mine_far);
  if (threadIdx.x == 0) meets[A.parts] = any_far;  // (read behind the next barrier)

  const Magic magic;
  int stage = 0, taken = 0;
  uint32_t parity = 0;
  bool dead = A.polls == 0;  // a copy did not land within the limit: the sums become NaN
  // (a lane whose column is not in use takes another one's values: its sums are
  // not looked at)
  const __half* xq[NG];
  const float* xsq[NG];  // of row 4 q + t, or of rows 8 q + 2 t and the next
#pragma unroll
  for (int q = 0; q < NG; ++q) {
    xq[q] = xf + min(8 * q + g, A.ncol - 1) * xstep + 8 * t;
    xsq[q] = xs + (MODE == kF32 ? (4 * q + t) * ktl_max : 8 * q + 2 * t);
  }
  for (int pass = 0; pass < A.passes; ++pass) {
    Walk w;
    enter(w, pass);
    float acc[NG][kSums];
#pragma unroll
    for (int q = 0; q < NG; ++q)
#pragma unroll
      for (int e = 0; e < kSums; ++e) acc[q][e] = 0.f;
    float* dst = part + warp * slot_floats;  // [part of this warp][row of the batch][16]
    while (w.n) {
      const int n = min(kChunk, w.n), k = w.k;
      // (all lanes see the copy, or the warp goes on without it)
      if (!dead) dead = !__all_sync(0xffffffffu, mbar_try_wait(bars + stage, parity) || wait_on(bars + stage, parity, A.polls - 1));
      if (dead) {
#pragma unroll
        for (int q = 0; q < NG; ++q)
#pragma unroll
          for (int e = 0; e < kSums; ++e) acc[q][e] = __int_as_float(0x7fc00000);
      } else {
        const uint8_t* tile = ring + stage * kStage;
        const auto work = [&](int c) {
            Tile<NS> T;
            read_tile<NS>(tile + c * kRec, lane, T);
            float sum[NG][2];  // (f32 rows: of a tile)
            float d[NG][4];    // (of a scale's columns)
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              const uint32_t w0 = b == 0 ? T.a[0].x : b == 1 ? T.a[0].y : b == 2 ? T.a[0].z : T.a[0].w;
              const uint32_t w1 = b == 0 ? T.a[1].x : b == 1 ? T.a[1].y : b == 2 ? T.a[1].z : T.a[1].w;
              uint32_t r0[4], r1[4];
              unpack(w0, magic, r0);
              unpack(w1, magic, r1);
              const float s0 = scale_of<NS>(T, 0, b), s1 = scale_of<NS>(T, 1, b);
#pragma unroll
              for (int q = 0; q < NG; ++q) {
                const uint4 v = *reinterpret_cast<const uint4*>(xq[q] + k * kQ4Cols + (4 * c + b) * 32);
                // (Q8_0 rows have a scale of their own every 32 columns)
                constexpr int kSame = MODE == kQ8 ? 1 : 4 / NS;
                if (b % kSame == 0)
                  mma16816_first(d[q], r0[0], r1[0], r0[1], r1[1], v.x, v.y);
                else
                  mma16816(d[q], r0[0], r1[0], r0[1], r1[1], v.x, v.y);
                mma16816(d[q], r0[2], r1[2], r0[3], r1[3], v.z, v.w);
                if (b % kSame != kSame - 1) continue;
                if constexpr (MODE == kF32) {
                  const float v0 = fmaf(d[q][1], 0x1p-12f, d[q][0]), v1 = fmaf(d[q][3], 0x1p-12f, d[q][2]);
                  sum[q][0] = b >= kSame ? fmaf(s0, v0, sum[q][0]) : s0 * v0;
                  sum[q][1] = b >= kSame ? fmaf(s1, v1, sum[q][1]) : s1 * v1;
                } else if constexpr (MODE == kF16) {
                  acc[q][0] = fmaf(s0, d[q][0], acc[q][0]);
                  acc[q][1] = fmaf(s0, d[q][1], acc[q][1]);
                  acc[q][2] = fmaf(s1, d[q][2], acc[q][2]);
                  acc[q][3] = fmaf(s1, d[q][3], acc[q][3]);
                } else {
                  const float2 e = *reinterpret_cast<const float2*>(xsq[q] + ((k + c) * 4 + b) * kMp);
                  acc[q][0] = fmaf(s0 * e.x, d[q][0], acc[q][0]);
                  acc[q][1] = fmaf(s0 * e.y, d[q][1], acc[q][1]);
                  acc[q][2] = fmaf(s1 * e.x, d[q][2], acc[q][2]);
                  acc[q][3] = fmaf(s1 * e.y, d[q][3], acc[q][3]);
                }
              }
            }
            if constexpr (MODE == kF32) {
#pragma unroll
              for (int q = 0; q < NG; ++q) {
                const float by = xsq[q][k + c];
                acc[q][0] = fmaf(by, sum[q][0], acc[q][0]);
                acc[q][1] = fmaf(by, sum[q][1], acc[q][1]);
              }
            }
        };
        // (us, whole copies unrolled / tiles unrolled with a branch each / a loop: one
        // row, gated 3584 -> 18944, 15.2 / 15.6 / -; eight 23.3 / 23.5 / 25.3; sixteen
        // Q8_0 rows 34.4 / 34.4 / 34.9, 3584 -> 4736 14.6 / 14.4 / 14.5; sixteen f16 rows in
        // groups of 32, 64, 128 27.9 / 27.8 / 27.5, 27.7 / 26.4 / 26.8, 26.6 / 25.9 / 26.3:
        // unrolled, those of 32 spill)
        if (MODE == kF16 && NG > 1 && NS == 4) {
#pragma unroll 1
          for (int c = 0; c < n; ++c) work(c);
        } else if (MODE != kF32 && NG > 1) {
#pragma unroll
          for (int c = 0; c < kChunk; ++c)
            if (c < n) work(c);
        } else if (n == kChunk) {
#pragma unroll
          for (int c = 0; c < kChunk; ++c) work(c);
        } else {
#pragma unroll 1
          for (int c = 0; c < n; ++c) work(c);
        }
        __syncwarp();  // (every lane has read the stage)
        ++taken;
        issue(stage);
        if (++stage == A.stages) {
          stage = 0;
          parity ^= 1;
        }
      }
      w.k += n;
      w.n -= n;
      if (w.n == 0) {
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
        dst += kMp * 16;
        next_part(w);
      }
    }
    // Which warps met a part (their ranges follow one another) and which of the
    // first one's parts it is; it is the others' first.
    const int pa = w.ua, pu = w.ub - w.ua, parts = pu * P.nmat, all = parts * ktl;
    for (int sp = threadIdx.x; sp < parts; sp += kThreads) {
      const int a = ((sp * ktl + 1) * kWarps - 1) / all, b = ((sp + 1) * ktl * kWarps - 1) / all;
      uint32_t met = 0;
      for (int v = a; v <= b; ++v)
        if ((v + 1) * all / kWarps > v * all / kWarps) met |= 1u << v;  // (a warp may have no tile)
      meets[sp] = met | (uint32_t)(sp - a * all / kWarps / ktl) << 24;
    }
    __syncthreads();
    const auto cta_sum = [&](int sp, int j, int row) {  // (in the warps' order)
      uint32_t met = meets[sp];
      const float* p = part + j * 16 + row;
      int v = __ffs(met) - 1;
      float sum = p[v * slot_floats + (met >> 24) * kMp * 16];
      met &= (met & 0xffffffu) - 1;
      while (met & 0xffffffu) {
        v = __ffs(met) - 1;
        sum += p[v * slot_floats];
        met &= met - 1;
      }
      return sum;
    };
    // pairs (strip, row of the batch) go to half warps; 2048 of them at most
    const uint32_t by_m = 65536u / P.m + 1;
    const auto over_m = [&](int x) { return (int)((uint32_t)x * by_m >> 16); };
    const int row = threadIdx.x & 15, first = threadIdx.x / 16;
    if constexpr (MODE == kF32)
      if (meets[A.parts]) add_far_terms<kWarps, NG, NS>(A, smem, pa, pu, k0, ktl);
    const auto finish = [&](int unit, int j, float v, float up) {
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
      for (int o = first; o < pu * P.m; o += kThreads / 16) {
        const int unit = over_m(o), j = o - unit * P.m;
        if (P.nmat == 2)
          finish(unit, j, cta_sum(2 * unit, j, row), cta_sum(2 * unit + 1, j, row));
        else
          finish(unit, j, cta_sum(unit, j, row), 0.f);
      }
      if (pass + 1 < A.passes) __syncthreads();
    } else {
      // pair o is finished by CTA o % cs, to which every CTA sends its sums: [CTA][its
      // pairs][matrix][16]
      const int pairs = pu * P.m, share = (pairs + A.cs - 1) / A.cs, mine = 16 * P.nmat;
      cluster_wait();  // (all of the cluster's CTAs run, and have read the last pass's)
      for (int o = first; o < pairs; o += kThreads / 16) {
        const int unit = over_m(o), j = o - unit * P.m, owner = o % A.cs;
        float* dst = red + (rank * share + o / A.cs) * mine + row;
        for (int e = 0; e < P.nmat; ++e) cluster_store(dst + 16 * e, owner, cta_sum(P.nmat * unit + e, j, row));
      }
      cluster_arrive();
      cluster_wait();
      for (int i = first; i < share; i += kThreads / 16) {
        const int o = i * A.cs + rank;
        if (o >= pairs) break;
        const int unit = over_m(o), j = o - unit * P.m;
        const float* src = red + i * mine + row;
        float v = 0.f, up = 0.f;
        for (int c = 0; c < A.cs; ++c) {
          v += src[c * share * mine];
          if (P.nmat == 2) up += src[c * share * mine + 16];
        }
        finish(unit, j, v, up);
      }
      if (pass + 1 < A.passes) cluster_arrive();
    }
  }
  // (no copy is left behind: one that did not land in time gets the whole limit)
  for (; taken < issued; ++taken) {
    mbar_wait(bars + stage, parity);
    if (++stage == A.stages) {
      stage = 0;
      parity ^= 1;
    }
  }
}

// ---- plan and launch --------------------------------------------------------
std::atomic<uint32_t> g_wait_limit{kWaitLimit};  // the poll at which a wait gives up

int max_clusters(const void* fn, int cs, int threads, int smem, int* out) {
  static std::mutex mu;
  static std::map<std::tuple<const void*, int, int, int>, int> known;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return record_cuda(e);
  std::lock_guard<std::mutex> lock(mu);
  const auto key = std::make_tuple(fn, cs, smem, dev);
  const auto it = known.find(key);
  if (it != known.end()) {
    *out = it->second;
    return Q8D_OK;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(cs * 64);
  cfg.blockDim = dim3(threads);
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

// Lets a kernel be launched in clusters of sixteen (once a device).
int allow_wide_clusters(const void* fn) {
  static std::mutex mu;
  static std::set<std::pair<const void*, int>> done;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return record_cuda(e);
  std::lock_guard<std::mutex> lock(mu);
  if (done.count({fn, dev})) return Q8D_OK;
  e = cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return record_cuda(e);
  done.insert({fn, dev});
  return Q8D_OK;
}

// A way of cutting a product up, and what it is expected to take.
struct Plan {
  int warps, cs, ncl, passes, parts, stages, smem;
  double ns;
};
// ns of an SM a tile, measured with calls of 400 and more: the issue slots bound
// them, and with many columns the operand's reads from shared memory.  (Of 396 ways of
// cutting up products of 9 to 16 f16 and Q8_0 rows one changes between 41 and 55, 60
// and 72 ns for the 45 and 65.)
constexpr double tile_ns(int mode, int ng, int scales) {
  return ng == 4 ? 70 + 6 * scales : ng == 2 ? (mode == kF32 ? 39 : mode == kF16 ? 45 : 65) : mode == kQ8 ? 35 : 27;
}
// Clusters of cs CTAs of kWarps warps, at most `most` of them, against the best
// way so far.
template <int kWarps, int MODE, int NG, int NS>
void weigh(const Q4Args& A, int strips, int cs, int most, Plan* best) {
  constexpr int kStage = chunk_tiles(MODE, NG) * (kQ4QuantBytes + kQ4Rows * NS * 2) * kWarps;
  constexpr int kLimit = kWarps == 8 ? kHalfSmem : kMaxSmem;
  const int ktl = (A.kt + cs - 1) / cs, ncl = std::min(most, strips), units = (strips + ncl - 1) / ncl;
  const int ctas = ncl * cs > sm_count() ? 16 / kWarps : 1;  // an SM
  // as few passes as leave the rings two copies a warp (or one)
  int stages = 0, passes = 0, parts = 0, ring = 0;
  for (int least = 2; least >= 1 && !stages; --least)
    for (int u = std::min(units, kMaxParts / A.P.nmat); u >= 1; u -= (u + 7) / 8) {
      passes = (units + u - 1) / u;
      parts = (units + passes - 1) / passes * A.P.nmat;
      ring = smem_layout(kWarps, MODE, NG, ktl, A.ncol, parts, cs).ring;
      if ((kLimit - ring) / kStage >= least) {
        stages = std::min(kMaxStages, (kLimit - ring) / kStage);
        break;
      }
    }
  if (!stages) return;
  // What an SM does, in ns: its CTAs' tiles; 128 columns of a row of X at a time
  // made into operands, several of them loaded by a warp at once; sixteen sums of a
  // strip and row brought together, in a cluster through another CTA; the passes'
  // ends; a cluster's meetings; and what sixteen warps take longer to start.
  const double tiles = (double)units * A.P.nmat * ktl * ctas;
  const int items = A.P.m * ktl, rounds = (items + kWarps * kWarps / 2 - 1) / (kWarps * kWarps / 2);
  const double ns = tiles * tile_ns(MODE, NG, NS) + items * ctas * 7.5 + rounds * 500 +
                    (double)passes * parts * A.P.m * (cs > 1 ? 6 : 5 * ctas) + (passes - 1) * 3000 +
                    (cs > 1 ? 1000 : 0) + (kWarps == 16 ? 300 : 0);
  if (best->cs == 0 || ns < best->ns)
    *best = {kWarps, cs, ncl, passes, parts, stages, ring + stages * kStage, ns};
}

// The ways with kWarps warps a CTA: clusters of every size.  Measured, us: 3584 ->
// 4608, one row, eight warps 5.6, sixteen 5.8, two CTAs a cluster 6.4; gated 3584
// -> 18944, eight rows, 27.6 (clusters of four), 23.2, 24.8; 18944 -> 3584, one
// row, 13.4 (clusters of eight), 15.1, 12.0.  (One CTA of eight warps an SM, beside
// which the next call's starts, takes 5.1 in a graph and 6.9 where single calls
// arrive one by one.)
template <int kWarps, int MODE, int NG, int NS>
int consider(const Q4Args& A, int strips, Plan* best) {
  const auto fn = reinterpret_cast<const void*>(q4_kernel<kWarps, MODE, NG, NS>);
  int rc = configure_kernel(fn, kMaxSmem, true);
  if (!rc) rc = allow_wide_clusters(fn);
  if (rc) return rc;
  weigh<kWarps, MODE, NG, NS>(A, strips, 1, 16 / kWarps * sm_count(), best);
  // (six and nine fit the GPCs three and two times, where eight does twice and
  // sixteen once: 18944 -> 3584, sixteen rows, 33.1, 31.8 and, with nine, 26.0 us)
  constexpr int kSizes[] = {2, 4, 6, 8, 9, kMaxCluster};
  for (const int cs : kSizes) {
    if (cs > A.kt) break;
    int most = 0;
    rc = max_clusters(fn, cs, kWarps * 32, kWarps == 8 ? kHalfSmem : kMaxSmem, &most);
    if (rc) return rc;
    if (most >= 1) weigh<kWarps, MODE, NG, NS>(A, strips, cs, most, best);
  }
  return Q8D_OK;
}

template <int kWarps, int MODE, int NG, int NS>
int launch_plan(const Q4Args& A, const Plan& plan, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(plan.cs * plan.ncl);
  cfg.blockDim = dim3(kWarps * 32);
  cfg.dynamicSmemBytes = plan.smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = plan.cs;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = plan.cs > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, q4_kernel<kWarps, MODE, NG, NS>, A);
  return e == cudaSuccess ? Q8D_OK : record_cuda(e);
}

// The best way for a product of P.m rows (plan.cs 0: none fits).  It depends on
// sizes alone and takes the host about as long as a launch: it is kept for them.
template <int MODE, int NG, int NS>
int make_plan(const Q4Params& P, Q4Args* A, Plan* plan) {
  static std::mutex mu;
  static std::map<std::array<int, 5>, Plan> known;
  *A = Q4Args{};
  A->P = P;
  A->kt = q4_tiles(P.n);
  A->ncol = (MODE == kF32 ? 2 : 1) * P.m;
  *plan = Plan{};
  const int strips = (int)q4_strips(P.p);
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return record_cuda(e);
  const std::array<int, 5> key = {dev, P.m, A->kt, strips, P.nmat};
  bool found = false;
  {
    std::lock_guard<std::mutex> lock(mu);
    const auto it = known.find(key);
    found = it != known.end();
    if (found) *plan = it->second;
  }
  if (!found) {
    int rc = consider<8, MODE, NG, NS>(*A, strips, plan);
    if (!rc) rc = consider<16, MODE, NG, NS>(*A, strips, plan);
    if (rc) return rc;
    std::lock_guard<std::mutex> lock(mu);
    if (known.size() >= 4096) known.clear();
    known[key] = *plan;
  }
  A->cs = plan->cs;
  A->ncl = plan->ncl;
  A->stages = plan->stages;
  A->passes = plan->passes;
  A->parts = plan->parts;
  A->polls = g_wait_limit - 1;
  return Q8D_OK;
}

template <int MODE, int NG, int NS>
int launch_made(const Q4Args& A, const Plan& plan, cudaStream_t stream) {
  if (plan.cs == 0) return Q8D_EUNSUPPORTED;
  return plan.warps == 8 ? launch_plan<8, MODE, NG, NS>(A, plan, stream) : launch_plan<16, MODE, NG, NS>(A, plan, stream);
}

template <int MODE, int NG, int NS>
int launch(const Q4Params& P, cudaStream_t stream) {
  Q4Args A;
  Plan plan;
  const int rc = make_plan<MODE, NG, NS>(P, &A, &plan);
  return rc ? rc : launch_made<MODE, NG, NS>(A, plan, stream);
}

// 9 to 16 f32 rows: in one launch, or as eight and the others, whichever is
// expected to be faster; both are planned before the first is launched (16 rows, us for one / two: 3584 -> 3584 11.3 / 16.8, 18944
// -> 3584 26.2 / 36.7, gated 3584 -> 18944 50.8 / 46.4).
template <int NS>
int launch_wide(const Q4Params& P, cudaStream_t stream) {
  Q4Args all, head;
  Plan pa, ph;
  int rc = make_plan<kF32, 4, NS>(P, &all, &pa);
  if (rc) return rc;
  Q4Params Q = P;
  Q.m = 8;
  rc = make_plan<kF32, 2, NS>(Q, &head, &ph);
  if (rc) return rc;
  // (eight rows take as long as five, and four about two thirds of that; a launch 4 us)
  if (pa.cs && (!ph.cs || pa.ns <= ph.ns * (P.m > 12 ? 2.0 : 1.7) + 4000)) return launch_made<kF32, 4, NS>(all, pa, stream);
  Q.m = P.m - 8;
  Q.X = static_cast<const float*>(P.X) + 8 * P.ldx;
  Q.Y = P.Y + 8 * P.ldy;
  Q.residual = P.residual ? P.residual + 8 * P.ldr : nullptr;
  Q4Args rest;
  Plan pr;
  rc = Q.m > 4 ? make_plan<kF32, 2, NS>(Q, &rest, &pr) : make_plan<kF32, 1, NS>(Q, &rest, &pr);
  if (!rc && (ph.cs == 0 || pr.cs == 0)) rc = Q8D_EUNSUPPORTED;
  if (!rc) rc = launch_made<kF32, 2, NS>(head, ph, stream);
  if (rc) return rc;
  return Q.m > 4 ? launch_made<kF32, 2, NS>(rest, pr, stream) : launch_made<kF32, 1, NS>(rest, pr, stream);
}

template <int MODE, int NG>
int launch_g(const Q4Params& P, cudaStream_t stream) {
  switch (P.group) {
    case 32: return launch<MODE, NG, 4>(P, stream);
    case 64: return launch<MODE, NG, 2>(P, stream);
    default: return launch<MODE, NG, 1>(P, stream);
  }
}

}  // namespace

static int launch_any(const Q4Params& P, cudaStream_t stream) {
  if (P.x_dtype == Q8D_KV_F16) return P.m <= 8 ? launch_g<kF16, 1>(P, stream) : launch_g<kF16, 2>(P, stream);
  if (P.x_dtype == Q8D_KV_Q8_0) return P.m <= 8 ? launch_g<kQ8, 1>(P, stream) : launch_g<kQ8, 2>(P, stream);
  // (f32 rows take two columns each)
  if (P.m <= 4) return launch_g<kF32, 1>(P, stream);
  if (P.m <= 8) return launch_g<kF32, 2>(P, stream);
  return P.group == 32 ? launch_wide<4>(P, stream) : P.group == 64 ? launch_wide<2>(P, stream) : launch_wide<1>(P, stream);
}

void q4_set_wait_limit(uint32_t polls) { g_wait_limit = polls ? polls : kWaitLimit; }

int q4_launch(const Q4Params& P, cudaStream_t stream) {
  try {
    return launch_any(P, stream);
  } catch (...) {  // (the host's memory ran out under the plans)
    return Q8D_ENOMEM;
  }
}

}  // namespace q8d
