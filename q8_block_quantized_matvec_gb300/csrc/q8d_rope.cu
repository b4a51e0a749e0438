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
// The rows are memory bound: a warp takes up to four heads (or pairs of narrow
// heads) of one row and segment, with the angles in registers and all loads in
// flight before any is used; a lane has four consecutive elements (eight of
// heads wider than 128), so that 16 bytes an access fill the sectors, and eight
// (four) neighbours make a packed block.  Each step of the arithmetic is
// rounded to f32 by itself, so that the packed caches' codes are those of the
// plain formulas whatever the compiler contracts.
#include <algorithm>
#include <cmath>

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

__global__ void __launch_bounds__(256) rope_table_kernel(const TableArgs A) {
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
  for (int pos = blockIdx.x * 8 + threadIdx.y; pos < A.max_pos; pos += gridDim.x * 8) {
    double s, c;
    sincos((double)pos * f, &s, &c);
    float* row = A.table + (long long)pos * 2 * A.half;
    row[i] = (float)(c * A.mscale);
    row[A.half + i] = (float)(s * A.mscale);
  }
}

// ---- the rows ---------------------------------------------------------------
constexpr int kWarps = 8;
constexpr int kHeads = 4;  // heads (or groups of narrow ones) a warp at most

struct RopeArgs {
  RopeRowsParams P;
  FastDiv chunks;  // warps a row
  int cq, ck;      // of them for q and for each of k and v
  int per;         // heads (groups) a warp
  int lph;         // lanes a head: a power of two
  Pair inv_n;
  bool vec_in, vec_out;
};

template <typename T, int kE>
__device__ __forceinline__ void get(const T* p, bool vec, float (&f)[kE]) {
  if (!vec) {
#pragma unroll
    for (int e = 0; e < kE; ++e) f[e] = (float)p[e];
    return;
  }
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int e = 0; e < kE; e += 4) {
      const float4 a = *reinterpret_cast<const float4*>(p + e);
      f[e] = a.x, f[e + 1] = a.y, f[e + 2] = a.z, f[e + 3] = a.w;
    }
  } else {
#pragma unroll
    for (int e = 0; e < kE; e += 4) {
      const uint2 u = *reinterpret_cast<const uint2*>(p + e);
      const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&u.x));
      const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&u.y));
      f[e] = a.x, f[e + 1] = a.y, f[e + 2] = b.x, f[e + 3] = b.y;
    }
  }
}
template <typename T, int kE>
__device__ __forceinline__ void put(T* p, bool vec, const float (&f)[kE]) {
  if (!vec) {
#pragma unroll
    for (int e = 0; e < kE; ++e) p[e] = (T)f[e];
    return;
  }
#pragma unroll
  for (int e = 0; e < kE; e += 4) {
    if constexpr (sizeof(T) == 4) {
      *reinterpret_cast<float4*>(p + e) = make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]);
    } else {
      const __half2 a = __floats2half2_rn(f[e], f[e + 1]), b = __floats2half2_rn(f[e + 2], f[e + 3]);
      *reinterpret_cast<uint2*>(p + e) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    }
  }
}
// f32 vectors that every row reads.
template <int kE>
__device__ __forceinline__ void get_shared(const float* p, float (&f)[kE]) {
#pragma unroll
  for (int e = 0; e < kE; ++e) f[e] = __ldg(p + e);
}

// cos and signed sin of kE elements from el on of the rotated part: element e
// becomes c[e] x[e] + s[e] partner[e].
template <int kE>
__device__ __forceinline__ void angles(const float* row, int half, int layout, int el, float (&c)[kE],
                                       float (&s)[kE]) {
  if (layout == Q8D_ROPE_HALF && half % kE == 0) {
    const bool up = el >= half;
    const float* p = row + (up ? el - half : el);
#pragma unroll
    for (int e = 0; e < kE; e += 4) {
      const float4 a = __ldg(reinterpret_cast<const float4*>(p + e));
      const float4 b = __ldg(reinterpret_cast<const float4*>(p + half + e));
      c[e] = a.x, c[e + 1] = a.y, c[e + 2] = a.z, c[e + 3] = a.w;
      s[e] = b.x, s[e + 1] = b.y, s[e + 2] = b.z, s[e + 3] = b.w;
    }
#pragma unroll
    for (int e = 0; e < kE; ++e) s[e] = up ? s[e] : -s[e];
  } else {
#pragma unroll
    for (int e = 0; e < kE; ++e) {
      const int j = el + e;
      c[e] = 1.f;
      s[e] = 0.f;
      if (j >= 2 * half) continue;
      const bool up = layout == Q8D_ROPE_HALF ? j >= half : (j & 1);
      const int i = layout == Q8D_ROPE_HALF ? (up ? j - half : j) : j / 2;
      c[e] = __ldg(row + i);
      s[e] = __ldg(row + half + i);
      s[e] = up ? s[e] : -s[e];
    }
  }
}

template <typename T, int KV, int kE>
__global__ void __launch_bounds__(kWarps * 32) rope_rows_kernel(const RopeArgs A) {
  __shared__ float turn[kWarps][32 * kE];  // (half layouts whose halves cut a lane's elements)
  griddep_launch_dependents();
  griddep_wait();
  const RopeRowsParams& P = A.P;
  const q8d_rope_desc& D = P.d;
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const int sub = lane / A.lph, hpw = 32 / A.lph, el = (lane & (A.lph - 1)) * kE;
  const int half = D.rot_dim / 2;
  const uint32_t item = blockIdx.x * kWarps + warp;
  const int width = D.n_kv_heads * D.head_dim;
  for (int s = blockIdx.y; s < P.batch; s += gridDim.y) {
    const int pos = P.d_pos[s], rpos = P.d_rope_pos ? P.d_rope_pos[s] : pos;
    int count = P.d_counts ? P.d_counts[s] : P.rows;
    int bad = 0;
    if (count < 0 || count > P.rows)
      bad = Q8D_DERR_LEN_RANGE;
    else if (count > 0 && ((P.k && (pos < 0 || pos > D.cap - count)) || rpos < 0 || rpos > D.max_pos - count))
      bad = Q8D_DERR_POS_RANGE;
    if (bad && P.d_err && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(P.d_err, bad);
    // (a refused sequence: its q rows become NaN, nothing of it is stored)
    if (bad) count = P.rows;
    if (item >= (uint32_t)count * A.chunks.d) continue;  // (the whole warp)
    const int row = (int)A.chunks.div(item), chunk = (int)(item - (uint32_t)row * A.chunks.d);
    const int seg = chunk < A.cq ? 0 : chunk < A.cq + A.ck ? 1 : 2;
    if (bad && seg) continue;
    const int heads = seg ? D.n_kv_heads : D.n_heads;
    const int h0 = (chunk - (seg == 0 ? 0 : seg == 1 ? A.cq : A.cq + A.ck)) * A.per * hpw + sub;
    const long long ld = seg ? D.ldkv : D.ldq, r = (long long)s * P.rows + row;
    const T* src = static_cast<const T*>(seg == 0 ? P.q : seg == 1 ? P.k : P.v) + r * ld + el;
    const float* bias = seg == 0 ? D.bq : seg == 1 ? D.bk : D.bv;
    const float* norm = seg == 0 ? D.q_norm : seg == 1 ? D.k_norm : nullptr;
    const bool in = el < D.head_dim;
    float f[kHeads][kE], c[kE], sn[kE], wn[kE];
#pragma unroll
    for (int u = 0; u < kHeads; ++u) {
      const int head = h0 + u * hpw;
#pragma unroll
      for (int e = 0; e < kE; ++e) f[u][e] = 0.f;
      if (u < A.per && head < heads && in) get<T, kE>(src + head * D.head_dim, A.vec_in, f[u]);
    }
    const bool turns = seg < 2 && el < D.rot_dim && !bad;
#pragma unroll
    for (int e = 0; e < kE; ++e) c[e] = 1.f, sn[e] = 0.f, wn[e] = 0.f;
    if (turns) angles<kE>(D.table + ((long long)rpos + row) * D.rot_dim, half, D.layout, el, c, sn);
    if (norm && in) get_shared<kE>(norm + el, wn);
#pragma unroll
    for (int u = 0; u < kHeads; ++u) {
      if (u >= A.per) break;
      const int head = h0 + u * hpw;
      const bool live = head < heads && in;
      if (bias && live) {
        float b[kE];
        get_shared<kE>(bias + head * D.head_dim + el, b);
#pragma unroll
        for (int e = 0; e < kE; ++e) f[u][e] = __fadd_rn(f[u][e], b[e]);
      }
      if (norm) {
        Pair ss{0.f, 0.f};
#pragma unroll
        for (int e = 0; e < kE; ++e) pair_add_square(ss, f[u][e]);
        ss = pair_sum(ss, A.lph, 0xffffffffu);
        float inv = rms_factor(ss, A.inv_n, D.eps);
        const bool good = head >= heads || rms_in_range(ss);
        if (!__all_sync(0xffffffffu, good)) {
          double d = 0.0;
#pragma unroll
          for (int e = 0; e < kE; ++e) d += (double)f[u][e] * (double)f[u][e];
          for (int o = 1; o < A.lph; o <<= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
          if (!good) inv = rms_factor_wide(d, D.head_dim, D.eps);
        }
#pragma unroll
        for (int e = 0; e < kE; ++e) f[u][e] = __fmul_rn(__fmul_rn(f[u][e], inv), wn[e]);
      }
      if (seg < 2 && half) {
        float g[kE];
        if (D.layout == Q8D_ROPE_PAIRS) {
#pragma unroll
          for (int e = 0; e < kE; ++e) g[e] = f[u][e ^ 1];
        } else if (half % kE == 0) {
          const int by = half / kE, from = turns ? (el < half ? lane + by : lane - by) : lane;
#pragma unroll
          for (int e = 0; e < kE; ++e) g[e] = __shfl_sync(0xffffffffu, f[u][e], from);
        } else {
          __syncwarp();
#pragma unroll
          for (int e = 0; e < kE; ++e) turn[warp][lane * kE + e] = f[u][e];
          __syncwarp();
#pragma unroll
          for (int e = 0; e < kE; ++e) {
            const int j = el + e;
            g[e] = turn[warp][lane * kE + e + (j < half ? half : j < 2 * half ? -half : 0)];
          }
        }
        if (turns) {
#pragma unroll
          for (int e = 0; e < kE; ++e)
            if (el + e < 2 * half) f[u][e] = __fadd_rn(__fmul_rn(f[u][e], c[e]), __fmul_rn(g[e], sn[e]));
        }
      }
      if (seg == 0) {
        if (bad) {
#pragma unroll
          for (int e = 0; e < kE; ++e) f[u][e] = __int_as_float(0x7fc00000);
        }
        const long long at = r * D.ldo + head * D.head_dim + el;
        if (live) {
          if (D.q_dtype == Q8D_KV_F16)
            put<__half, kE>(static_cast<__half*>(P.q_out) + at, A.vec_out, f[u]);
          else
            put<float, kE>(static_cast<float*>(P.q_out) + at, A.vec_out, f[u]);
        }
        continue;
      }
      uint8_t* cache = (seg == 1 ? P.kc : P.vc) + P.seq_bytes * s;
      const long long cr = (long long)pos + row;
      const int col = head * D.head_dim + el;
      if constexpr (KV == Q8D_KV_Q4) {
        put_q4<kE>(cache + cr * (width / 2) + col / 32 * 16,
                   cache + q4_scale_plane(D.cap, width) + cr * (width / 16) + col / 32 * 2,
                   lane & (32 / kE - 1), f[u], live);
      } else if constexpr (KV == Q8D_KV_Q8_0) {
        put_q8_0<kE>(cache + (cr * (width / kQBlock) + col / 32) * kQBlockBytes, lane & (32 / kE - 1), f[u], live);
      } else if constexpr (KV == Q8D_KV_F16) {
        if (live) put<__half, kE>(reinterpret_cast<__half*>(cache) + cr * width + col, true, f[u]);
      } else {
        if (live) put<float, kE>(reinterpret_cast<float*>(cache) + cr * width + col, true, f[u]);
      }
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
  // four heads a warp once that leaves two full machines of warps, else one,
  // for the latency
  A.per = (long long)P.batch * P.rows * (sq + 2 * sk) >= 4LL * 2 * 64 * sm_count() ? kHeads : 1;
  A.cq = (sq + A.per - 1) / A.per;
  A.ck = (sk + A.per - 1) / A.per;
  A.chunks = fast_div((uint32_t)(A.cq + 2 * A.ck));
  A.inv_n = pair_inverse(D.head_dim);
  const long long items = (long long)P.rows * A.chunks.d;
  if (items > 0xffff0000LL) return Q8D_EUNSUPPORTED;  // (item numbers are 32 bits)
  // 16-byte accesses (8 of f16) where every row allows them
  const uintptr_t in = 4 * sizeof(T), out = D.q_dtype == Q8D_KV_F16 ? 8 : 16;
  const auto on = [](const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; };
  A.vec_in = (!P.q || (on(P.q, in) && D.ldq % 4 == 0)) &&
             (!P.k || (on(P.k, in) && on(P.v, in) && D.ldkv % 4 == 0));
  A.vec_out = !P.q || (on(P.q_out, out) && D.ldo % 4 == 0);
  const dim3 grid((unsigned)((items + kWarps - 1) / kWarps), (unsigned)std::min(P.batch, 65535));
  return launch_ex(rope_rows_kernel<T, KV, kE>, grid, dim3(kWarps * 32), 0, stream, true, A);
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
  const dim3 grid((unsigned)std::min((max_pos + 7) / 8, 4096), (unsigned)((A.half + 31) / 32));
  return launch_ex(rope_table_kernel, grid, dim3(32, 8), 0, stream, true, A);
}

int rope_rows_launch(const RopeRowsParams& P, cudaStream_t stream) {
  return P.d.row_dtype == Q8D_KV_F16 ? launch_kv<__half>(P, stream) : launch_kv<float>(P, stream);
}

}  // namespace q8d
