// Rotary positions: the table of a model's angles, and rows of q, k and v
// turned by it on their way to attention, k and v into the KV caches.
//
// Element pairs (a, b) of a head at position pos become
//   (a cos - b sin, a sin + b cos),  angle = pos * f_i,
// for the pairs (i, i + rot / 2) or (2 i, 2 i + 1) of the head's first rot
// elements; before that the bias is added and the head normed, where given.
//
// f_i = theta^(-2 i / rot), scaled for contexts longer than the trained one:
//   linear: f_i / factor
//   NTK:    theta * factor^(rot / (rot - 2)) in theta's place
//   YaRN (Peng et al., "YaRN: Efficient Context Window Extension of Large
//           Language Models"): f_i / factor * ramp_i + f_i * (1 - ramp_i), ramp
//           rising from 0 to 1 between the pairs that turn beta_fast and
//           beta_slow times in the trained context.
// An angle is a 64-bit product: at position 131071 an f32 one is off by 0.004.
// Cosine and sine are rounded once and kept in a table [max_pos][rot], which a
// model's layers share: the row of a position is read by all its heads, where
// working it out in 64 bits would take longer than moving the row.
//
// The rows are memory bound, but for the instructions that norms and packed
// caches add: a warp takes up to four heads (or pairs of narrow ones) of q, of k
// or of v and walks several rows with them, the next row's values and angles in
// flight while it turns one; a lane has four consecutive elements (eight of heads
// wider than 128), so that 16 bytes an access fill the sectors, and eight (four)
// neighbours make a packed block.  Each step of the arithmetic is rounded to f32 by
// itself, so that the packed caches' codes are those of the plain formulas whatever
// the compiler contracts.
//
// us in a graph (and TB/s): 4096 rows of 16 / 8 heads of 128 from f32 into f16 22.5
// (5.3), with norms 28.9, into Q8_0 24.8, with norms and YaRN 33.8; 28 / 4 heads
// 26.7 (5.4); 8 sequences of up to 1999 f16 rows of 14 / 2 heads of 64 into f16 17.3
// (3.3: short rows, a kilobyte a warp), into 4 bits 19.4; one token of 64 sequences
// 3.3.  (A row a warp, loaded when it was due: 46.3, 64.2 and 70.0 for the first,
// second and fourth.)
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "q8d_kv_rows.cuh"
#include "q8d_layer.cuh"
#include "q8d_rms.cuh"

namespace q8d {
namespace {

// ---- the table --------------------------------------------------------------
struct TableArgs {
  float* table;
  int max_pos, half, scaling;
  double theta, factor, mscale, low, high;  // low, high: YaRN's ramp in pairs
};

// The angle of an entry is the rounded product pos * f, as the plain formula has
// it, and each is handed to the functions: turning a neighbour's angle on, two to
// four times as fast, is as near to the true value but rounds elsewhere, and one of
// 3000 entries at positions near 131072 came out a unit apart (0.9 to 1.1 ms for
// 131072 positions of 128, 0.15 for 8192, once a model; every thread works out its
// frequency, and the FP64 pipe bounds it).
__global__ void __launch_bounds__(256) rope_positions_kernel(const TableArgs A) {
  griddep_launch_dependents();
  griddep_wait();
  const int i = blockIdx.y * 32 + threadIdx.x;
  if (i >= A.half) return;
  const double rot = 2.0 * A.half;
  const double base = A.scaling == Q8D_ROPE_NTK ? A.theta * pow(A.factor, rot / (rot - 2.0)) : A.theta;
  double f = pow(base, -2.0 * i / rot);
  if (A.scaling == Q8D_ROPE_LINEAR) {
    f /= A.factor;
  } else if (A.scaling == Q8D_ROPE_YARN) {
    const double ramp = fmin(fmax((i - A.low) / fmax(A.high - A.low, 0.001), 0.0), 1.0);
    f = f / A.factor * ramp + f * (1.0 - ramp);
  }
  for (long long pos = blockIdx.x * 8 + threadIdx.y; pos < A.max_pos; pos += gridDim.x * 8) {
    double s, c;
    sincos((double)pos * f, &s, &c);
    float* row = A.table + pos * 2 * A.half;
    row[i] = (float)(c * A.mscale);
    row[A.half + i] = (float)(s * A.mscale);
  }
}

// ---- the rows ---------------------------------------------------------------
constexpr int kWarps = 8;
// Steps a warp at most: 64 bytes of f32 a lane (heads wider than 128 with four
// steps spilled: 4 x 1000 ragged rows of 8 / 4 heads of 256 43.3 us, now 17.1).
constexpr int steps_of(int e) { return 16 / e; }

// A row's work is steps of one head each (several narrow ones).  A warp takes
// several of q, of k or of v.
struct RopeArgs {
  RopeRowsParams P;
  FastDiv chunks;  // warps a row
  int cq, ck;      // of them for q, and for each of k and v
  int per;         // steps a warp
  int rpw;         // rows a warp, one after the other
  int lph;         // lanes a head: a power of two
  Pair inv_n;
};

// How rows are moved and turned: 16 bytes (8 of f16) at once with a lane's
// partners in one other lane (kHalves) or beside them (kPairs); or element by
// element, partners through shared memory, which serves every case.
enum Way { kHalves, kPairs, kAny };

// kE elements of a row as they lie in memory.
template <typename T, int kE, bool vec>
__device__ __forceinline__ void get_raw(const T* p, uint32_t (&w)[kE * sizeof(T) / 4]) {
  if constexpr (vec) {
#pragma unroll
    for (int e = 0; e < kE; e += 4) {
      if constexpr (sizeof(T) == 4) {
        const uint4 a = __ldcs(reinterpret_cast<const uint4*>(p + e));
        w[e] = a.x, w[e + 1] = a.y, w[e + 2] = a.z, w[e + 3] = a.w;
      } else {
        const uint2 a = __ldcs(reinterpret_cast<const uint2*>(p + e));
        w[e / 2] = a.x, w[e / 2 + 1] = a.y;
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < kE; ++e) {
      if constexpr (sizeof(T) == 4)
        w[e] = reinterpret_cast<const uint32_t*>(p)[e];
      else
        w[e / 2] = e & 1 ? w[e / 2] | (uint32_t) reinterpret_cast<const unsigned short*>(p)[e] << 16
                         : reinterpret_cast<const unsigned short*>(p)[e];
    }
  }
}
template <typename T, int kE>
__device__ __forceinline__ void expand(const uint32_t (&w)[kE * sizeof(T) / 4], uint64_t (&f)[kE / 2]) {
#pragma unroll
  for (int i = 0; i < kE / 2; ++i) {
    if constexpr (sizeof(T) == 4) {
      f[i] = pack2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    } else {
      const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      f[i] = pack2(t.x, t.y);
    }
  }
}
template <typename T, int kE, bool vec>
__device__ __forceinline__ void put(T* p, const uint64_t (&f)[kE / 2]) {
  float v[kE];
#pragma unroll
  for (int i = 0; i < kE / 2; ++i) unpack2(f[i], v[2 * i], v[2 * i + 1]);
#pragma unroll
  for (int e = 0; e < kE; e += 4) {
    if constexpr (!vec) {
#pragma unroll
      for (int i = 0; i < 4; ++i) p[e + i] = (T)v[e + i];
    } else if constexpr (sizeof(T) == 4) {
      *reinterpret_cast<float4*>(p + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
    } else {
      const __half2 a = __floats2half2_rn(v[e], v[e + 1]), b = __floats2half2_rn(v[e + 2], v[e + 3]);
      *reinterpret_cast<uint2*>(p + e) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    }
  }
}
// f32 vectors that every row reads.
template <int kE, bool vec>
__device__ __forceinline__ void get_shared(const float* p, uint64_t (&f)[kE / 2]) {
#pragma unroll
  for (int e = 0; e < kE; e += 4) {
    const float4 a = vec ? __ldg(reinterpret_cast<const float4*>(p + e))
                         : make_float4(__ldg(p + e), __ldg(p + e + 1), __ldg(p + e + 2), __ldg(p + e + 3));
    f[e / 2] = pack2(a.x, a.y);
    f[e / 2 + 1] = pack2(a.z, a.w);
  }
}

// cos and signed sin of kE elements from el on of the rotated part: element e
// becomes c[e] x[e] + s[e] partner[e].
template <int kE, int WAY>
__device__ __forceinline__ void angles(const float* row, int half, int layout, int el, uint64_t (&c)[kE / 2],
                                       uint64_t (&s)[kE / 2]) {
  if constexpr (WAY == kHalves) {
    const bool up = el >= half;
    const float* p = row + (up ? el - half : el);
    const float sign = up ? 1.f : -1.f;
    get_shared<kE, true>(p, c);
    get_shared<kE, true>(p + half, s);
#pragma unroll
    for (int e = 0; e < kE / 2; ++e) s[e] = mul2(s[e], pack2(sign, sign));
  } else {
#pragma unroll
    for (int e = 0; e < kE; e += 2) {
      if (WAY == kPairs || layout == Q8D_ROPE_PAIRS) {
        const int i = (el + e) / 2;
        const float cv = i < half ? __ldg(row + i) : 1.f, sv = i < half ? __ldg(row + half + i) : 0.f;
        c[e / 2] = pack2(cv, cv);
        s[e / 2] = pack2(-sv, sv);
        continue;
      }
      float cv[2] = {1.f, 1.f}, sv[2] = {0.f, 0.f};
#pragma unroll
      for (int o = 0; o < 2; ++o) {
        const int j = el + e + o;
        if (j >= 2 * half) continue;
        const bool up = j >= half;
        const int i = up ? j - half : j;
        cv[o] = __ldg(row + i);
        sv[o] = __ldg(row + half + i);
        if (!up) sv[o] = -sv[o];
      }
      c[e / 2] = pack2(cv[0], cv[1]);
      s[e / 2] = pack2(sv[0], sv[1]);
    }
  }
}

// The factors of a warp's steps' norms.  ss: this lane's squares of each step;
// valid(u): whether step u of this lane's head is normed.  The sums of four
// steps are folded together: lanes that differ in bit 0 exchange two of them
// each, in bit 1 one, and from there on lane l carries step l & 3, so that a
// warp adds six times where one step after the other would take twenty.  (Two
// steps: one exchange, lane l carries step l & 1.)
template <int kE, typename Valid>
__device__ __forceinline__ void head_factors(const Pair (&ss)[steps_of(kE)],
                                             const uint64_t (&f)[steps_of(kE)][kE / 2], const RopeArgs& A,
                                             int lane, Valid valid, float (&inv)[steps_of(kE)]) {
  constexpr int kSteps = steps_of(kE);
  static_assert(kSteps == 4 || kSteps == 2, "");
  const auto meet = [](const Pair& keep, const Pair& send, int o) {
    return pair_meet(keep, pair_shfl_xor(send, o, 0xffffffffu));
  };
  const bool b0 = lane & 1;
  Pair p = meet(b0 ? ss[1] : ss[0], b0 ? ss[0] : ss[1], 1);
  if constexpr (kSteps == 4) {
    const bool b1 = lane & 2;
    const Pair q = meet(b0 ? ss[3] : ss[2], b0 ? ss[2] : ss[3], 1);
    p = meet(b1 ? q : p, b1 ? p : q, 2);
  }
#pragma unroll
  for (int o = kSteps; o < 32; o <<= 1)
    if (o < A.lph) p = meet(p, p, o);
  const float eps = A.P.d.eps;
  const int mine = lane & (kSteps - 1);
  float r = rms_factor(p, A.inv_n, eps);
  const bool good = !valid(mine) || rms_in_range(p, eps);
  if (!__all_sync(0xffffffffu, good)) {
    double d[kSteps];
#pragma unroll
    for (int u = 0; u < kSteps; ++u) {
      d[u] = 0.0;
#pragma unroll
      for (int e = 0; e < kE / 2; ++e) {
        float x, y;
        unpack2(f[u][e], x, y);
        d[u] += (double)x * (double)x;
        d[u] += (double)y * (double)y;
      }
      for (int o = 1; o < A.lph; o <<= 1) d[u] += __shfl_xor_sync(0xffffffffu, d[u], o);
    }
    double all = d[0];
#pragma unroll
    for (int u = 1; u < kSteps; ++u) all = mine == u ? d[u] : all;
    if (!good) r = rms_factor_wide(all, A.P.d.head_dim, eps);
  }
#pragma unroll
  for (int u = 0; u < kSteps; ++u) inv[u] = __shfl_sync(0xffffffffu, r, (lane & ~(kSteps - 1)) | u);
}

// (three CTAs an SM, us for 4096 rows of 16 / 8 heads of 128 from f32 into f16: two
// 27.5, three 25.6, four 31.7.  With the norms, and into packed caches, the 80
// registers of three do not hold a lane's four steps: the instances with norms keep
// 24 to 108 bytes a thread in local memory, from f16 rows 24 to 44, those without at
// most 60; two CTAs were not measured for these.)
template <typename T, int KV, int kE, bool kNorm, int WAY>
__global__ void __launch_bounds__(kWarps * 32, kE == 4 ? 3 : 2) rope_rows_kernel(const RopeArgs A) {
  constexpr int kP = kE / 2, kW = kE * sizeof(T) / 4, kSteps = steps_of(kE);
  constexpr bool kVec = WAY != kAny;
  __shared__ float turn[WAY == kAny ? kWarps : 1][32 * kE];
  griddep_launch_dependents();
  griddep_wait();
  const RopeRowsParams& P = A.P;
  const q8d_rope_desc& D = P.d;
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const int sub = lane / A.lph, hpw = 32 / A.lph, el = (lane & (A.lph - 1)) * kE;
  const int half = D.rot_dim / 2;
  const uint32_t item = blockIdx.x * kWarps + warp;
  const int row0 = (int)A.chunks.div(item), chunk = (int)(item - (uint32_t)row0 * A.chunks.d);
  // the segment (0 q, 1 k, 2 v), this lane's first head and how many steps have one
  const int g = chunk < A.cq ? 0 : chunk < A.cq + A.ck ? 1 : 2;
  const int first = (chunk - (g == 0 ? 0 : g == 1 ? A.cq : A.cq + A.ck)) * A.per * hpw;
  const int heads = g ? D.n_kv_heads : D.n_heads, head = first + sub;
  const int steps = min(A.per, (heads - first + hpw - 1) / hpw);  // (the warp's)
  const int mine = el < D.head_dim ? min(steps, (heads - head + hpw - 1) / hpw) : 0;
  const int col = head * D.head_dim + el, stride = hpw * D.head_dim;  // a step's elements
  const int width = D.n_kv_heads * D.head_dim;
  const bool turns = g < 2 && el < D.rot_dim;
  const float* bias = g == 0 ? D.bq : g == 1 ? D.bk : D.bv;
  const long long ld = g ? D.ldkv : D.ldq;
  uint64_t wn[kP];  // the heads' norm weights
#pragma unroll
  for (int e = 0; e < kP; ++e) wn[e] = 0;
  if (kNorm && g < 2 && el < D.head_dim) get_shared<kE, kVec>((g ? D.k_norm : D.q_norm) + el, wn);
  for (int s = blockIdx.y; s < P.batch; s += gridDim.y) {
    const int pos = P.d_pos[s], rpos = P.d_rope_pos ? P.d_rope_pos[s] : pos;
    const int count = P.d_counts ? P.d_counts[s] : P.rows;
    int bad = 0;
    if (count < 0 || count > P.rows)
      bad = Q8D_DERR_LEN_RANGE;
    else if (count > 0 && ((P.k && (pos < 0 || pos > D.cap - count)) || rpos < 0 || rpos > D.max_pos - count))
      bad = Q8D_DERR_POS_RANGE;
    if (bad && P.d_err && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(P.d_err, bad);
    // (a refused sequence: its q rows become NaN, nothing is stored)
    if (bad && g) continue;
    int row = row0 * A.rpw;
    const int end = min(bad ? P.rows : count, row + A.rpw);
    if (row >= end) continue;  // (the whole warp)
    long long r = (long long)s * P.rows + row;
    const T* src = static_cast<const T*>(g == 0 ? P.q : g == 1 ? P.k : P.v) + r * ld + col;
    const float* table = D.table + (bad ? 0 : ((long long)rpos + row) * D.rot_dim);
    // the next row's values and angles are on their way while a row is worked on
    uint32_t raw[kSteps][kW];
    uint64_t c[kP], sn[kP];
    const auto fetch = [&]() {
#pragma unroll
      for (int u = 0; u < kSteps; ++u) {
#pragma unroll
        for (int e = 0; e < kW; ++e) raw[u][e] = 0;
        if (u < mine) get_raw<T, kE, kVec>(src + u * stride, raw[u]);
      }
#pragma unroll
      for (int e = 0; e < kP; ++e) c[e] = sn[e] = 0;
      if (turns && !bad) angles<kE, WAY>(table, half, D.layout, el, c, sn);
    };
    fetch();
    for (;; ++row, ++r) {
      uint64_t f[kSteps][kP], cc[kP], cs[kP];
#pragma unroll
      for (int u = 0; u < kSteps; ++u) expand<T, kE>(raw[u], f[u]);
#pragma unroll
      for (int e = 0; e < kP; ++e) cc[e] = c[e], cs[e] = sn[e];
      if (row + 1 < end) {
        src += ld;
        if (!bad) table += D.rot_dim;
        fetch();
      }
      if (bias) {
#pragma unroll
        for (int u = 0; u < kSteps; ++u) {
          if (u >= mine) continue;
          uint64_t b[kP];
          get_shared<kE, kVec>(bias + col + u * stride, b);
#pragma unroll
          for (int e = 0; e < kP; ++e) f[u][e] = add2(f[u][e], b[e]);
        }
      }
      if constexpr (kNorm) {
        if (g < 2) {
          Pair ss[kSteps];
#pragma unroll
          for (int u = 0; u < kSteps; ++u) {
            Pair2 both{0, 0};
#pragma unroll
            for (int e = 0; e < kP; ++e) pair2_add_square(both, f[u][e]);
            ss[u] = pair2_join(both);
          }
          float inv[kSteps];
          head_factors<kE>(ss, f, A, lane, [&](int u) { return head + u * hpw < heads && u < steps; }, inv);
#pragma unroll
          for (int u = 0; u < kSteps; ++u)
#pragma unroll
            for (int e = 0; e < kP; ++e) f[u][e] = mul2(mul2(f[u][e], pack2(inv[u], inv[u])), wn[e]);
        }
      }
      if (g < 2 && half) {
        const int by = half / kE, from = turns ? (el < half ? lane + by : lane - by) : lane;
#pragma unroll
        for (int u = 0; u < kSteps; ++u) {
          if (u >= steps) break;
          float p[kE];  // the partners
          if constexpr (WAY == kPairs) {
#pragma unroll
            for (int e = 0; e < kP; ++e) unpack2(f[u][e], p[2 * e + 1], p[2 * e]);
          } else if constexpr (WAY == kHalves) {
#pragma unroll
            for (int e = 0; e < kP; ++e) unpack2(__shfl_sync(0xffffffffu, f[u][e], from), p[2 * e], p[2 * e + 1]);
          } else {
            float* t = turn[warp] + lane * kE;
            __syncwarp();
#pragma unroll
            for (int e = 0; e < kP; ++e) unpack2(f[u][e], t[2 * e], t[2 * e + 1]);
            __syncwarp();
#pragma unroll
            for (int e = 0; e < kE; ++e) {
              const int j = el + e;
              p[e] = t[e + (j >= 2 * half                    ? 0
                            : D.layout == Q8D_ROPE_PAIRS     ? 1 - 2 * (j & 1)
                            : j < half                       ? half
                                                             : -half)];
            }
          }
          // (elements behind rot_dim, which may end inside a lane's, are as they were;
          // scalar steps, each rounded: packed products are contracted into the sum)
          if (turns) {
#pragma unroll
            for (int e = 0; e < kP; ++e) {
              if (el + 2 * e >= 2 * half) break;
              float x[2], cv[2], sv[2];
              unpack2(f[u][e], x[0], x[1]);
              unpack2(cc[e], cv[0], cv[1]);
              unpack2(cs[e], sv[0], sv[1]);
              f[u][e] = pack2(__fadd_rn(__fmul_rn(x[0], cv[0]), __fmul_rn(p[2 * e], sv[0])),
                              __fadd_rn(__fmul_rn(x[1], cv[1]), __fmul_rn(p[2 * e + 1], sv[1])));
            }
          }
        }
      }
      if (g == 0) {
        if (bad) {
#pragma unroll
          for (int u = 0; u < kSteps; ++u)
#pragma unroll
            for (int e = 0; e < kP; ++e) f[u][e] = 0x7fc000007fc00000ull;
        }
        const long long at = r * D.ldo + col;
#pragma unroll
        for (int u = 0; u < kSteps; ++u) {
          if (u >= mine) break;
          if (D.q_dtype == Q8D_KV_F16)
            put<__half, kE, kVec>(static_cast<__half*>(P.q_out) + at + u * stride, f[u]);
          else
            put<float, kE, kVec>(static_cast<float*>(P.q_out) + at + u * stride, f[u]);
        }
        if (row + 1 >= end) break;
        continue;
      }
      uint8_t* cache = (g == 1 ? P.kc : P.vc) + P.seq_bytes * s;
      const long long cr = (long long)pos + row;
      if constexpr (KV == Q8D_KV_Q4 || KV == Q8D_KV_Q8_0) {
        uint8_t* blk = KV == Q8D_KV_Q4 ? cache + cr * (width / 2) + col / 32 * 16
                                       : cache + (cr * (width / kQBlock) + col / 32) * kQBlockBytes;
        uint8_t* scale = cache + q4_scale_plane(D.cap, width) + cr * (width / 16) + col / 32 * 2;
#pragma unroll
        for (int u = 0; u < kSteps; ++u) {
          if (u >= steps) break;
          float v[kE];
#pragma unroll
          for (int e = 0; e < kP; ++e) unpack2(f[u][e], v[2 * e], v[2 * e + 1]);
          if constexpr (KV == Q8D_KV_Q4)
            put_q4<kE>(blk + u * (stride / 2), scale + u * (stride / 16), lane & (32 / kE - 1), v, u < mine);
          else
            put_q8_0<kE>(blk + u * (stride / 32 * kQBlockBytes), lane & (32 / kE - 1), v, u < mine);
        }
      } else {
        using C = typename std::conditional<KV == Q8D_KV_F16, __half, float>::type;
        C* dst = reinterpret_cast<C*>(cache) + cr * width + col;
#pragma unroll
        for (int u = 0; u < kSteps; ++u)
          if (u < mine) put<C, kE, true>(dst + u * stride, f[u]);
      }
      if (row + 1 >= end) break;
    }
  }
}

template <typename T, int KV, int kE>
int launch_rope(const RopeRowsParams& P, cudaStream_t stream) {
  const q8d_rope_desc& D = P.d;
  RopeArgs A{};
  A.P = P;
  A.lph = 1;
  while (A.lph * kE < D.head_dim) A.lph *= 2;
  if (A.lph < 32 / kE) A.lph = 32 / kE;  // (a packed block's lanes)
  const int hpw = 32 / A.lph;
  const int sq = P.q ? (D.n_heads + hpw - 1) / hpw : 0, sk = P.k ? (D.n_kv_heads + hpw - 1) / hpw : 0;
  // as many steps a warp as it may take once that leaves two full machines of
  // warps, else one, for the latency
  constexpr int kSteps = steps_of(kE);
  A.per = (long long)P.batch * P.rows * (sq + 2 * sk) >= kSteps * 2LL * 64 * sm_count() ? kSteps : 1;
  A.cq = (sq + A.per - 1) / A.per;
  A.ck = (sk + A.per - 1) / A.per;
  A.chunks = fast_div((uint32_t)(A.cq + 2 * A.ck));
  A.inv_n = pair_inverse(D.head_dim);
  // Rows a warp: whole rounds of resident CTAs, of which one costs its rows and
  // about one and a half for starting (4096 rows of 16 / 8 heads: 8 rows make 512
  // CTAs, a round and an eighth of them).
  const long long slots = (kE == 4 ? 3LL : 2LL) * sm_count();
  double best = 0.0;
  for (int r = 1; r <= 32; ++r) {
    long long ctas = ((P.rows + r - 1LL) / r * A.chunks.d + kWarps - 1) / kWarps * P.batch;
    if (P.batch > 1 && P.d_counts) ctas = ctas * 5 / 8;  // (what a ragged batch's may be)
    const double cost = (double)((ctas + slots - 1) / slots) * (r + 1.5);
    if (r == 1 || cost < best) {
      best = cost;
      A.rpw = r;
    }
  }
  const long long items = (P.rows + A.rpw - 1LL) / A.rpw * A.chunks.d;
  if (items > 0xffff0000LL) return Q8D_EUNSUPPORTED;  // (item numbers are 32 bits)
  // 16-byte accesses (8 of f16) where every row allows them
  const uintptr_t in = 4 * sizeof(T), out = D.q_dtype == Q8D_KV_F16 ? 8 : 16;
  const auto on = [](const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; };
  const bool vec = (!P.q || (on(P.q, in) && D.ldq % 4 == 0 && on(P.q_out, out) && D.ldo % 4 == 0)) &&
                   (!P.k || (on(P.k, in) && on(P.v, in) && D.ldkv % 4 == 0)) && on(D.bq, 16) && on(D.bk, 16) &&
                   on(D.bv, 16) && on(D.q_norm, 16) && on(D.k_norm, 16);
  const bool whole = D.layout == Q8D_ROPE_PAIRS || D.rot_dim % (2 * kE) == 0;
  const dim3 grid((unsigned)((items + kWarps - 1) / kWarps), (unsigned)std::min(P.batch, 65535));
  const auto run = [&](auto* kernel) { return launch_ex(kernel, grid, dim3(kWarps * 32), 0, stream, true, A); };
  if (D.q_norm) {
    if (!vec || !whole) return run(rope_rows_kernel<T, KV, kE, true, kAny>);
    return D.layout == Q8D_ROPE_PAIRS ? run(rope_rows_kernel<T, KV, kE, true, kPairs>)
                                      : run(rope_rows_kernel<T, KV, kE, true, kHalves>);
  }
  if (!vec || !whole) return run(rope_rows_kernel<T, KV, kE, false, kAny>);
  return D.layout == Q8D_ROPE_PAIRS ? run(rope_rows_kernel<T, KV, kE, false, kPairs>)
                                    : run(rope_rows_kernel<T, KV, kE, false, kHalves>);
}

template <typename T, int KV>
int launch_e(const RopeRowsParams& P, cudaStream_t stream) {
  return P.d.head_dim <= 128 ? launch_rope<T, KV, 4>(P, stream) : launch_rope<T, KV, 8>(P, stream);
}

template <typename T>
int launch_kv(const RopeRowsParams& P, cudaStream_t stream) {
  switch (P.d.kv_dtype) {
    case Q8D_KV_F32: return launch_e<T, Q8D_KV_F32>(P, stream);
    case Q8D_KV_F16: return launch_e<T, Q8D_KV_F16>(P, stream);
    case Q8D_KV_Q8_0: return launch_e<T, Q8D_KV_Q8_0>(P, stream);
    default: return launch_e<T, Q8D_KV_Q4>(P, stream);
  }
}

}  // namespace

int rope_table_launch(float* table, int max_pos, int rot_dim, double theta, int scaling, double factor,
                      double orig_ctx, double beta_fast, double beta_slow, double mscale,
                      cudaStream_t stream) {
  TableArgs A{table, max_pos, rot_dim / 2, scaling, theta, factor, mscale, 0.0, 0.0};
  if (scaling == Q8D_ROPE_YARN) {
    // the pair that turns `t` times in the trained context
    const auto at = [&](double t) {
      return rot_dim * std::log(orig_ctx / (t * 2.0 * 3.14159265358979323846)) / (2.0 * std::log(theta));
    };
    A.low = std::max(std::floor(at(beta_fast)), 0.0);
    A.high = std::min(std::ceil(at(beta_slow)), rot_dim - 1.0);
  }
  const dim3 grid((unsigned)std::min((max_pos + 7LL) / 8, 4096LL), (unsigned)((A.half + 31) / 32));
  return launch_ex(rope_positions_kernel, grid, dim3(32, 8), 0, stream, true, A);
}

int rope_rows_launch(const RopeRowsParams& P, cudaStream_t stream) {
  return P.d.row_dtype == Q8D_KV_F16 ? launch_kv<__half>(P, stream) : launch_kv<float>(P, stream);
}

}  // namespace q8d
