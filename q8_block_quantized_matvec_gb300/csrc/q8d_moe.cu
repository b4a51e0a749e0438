// A mixture-of-experts feed-forward layer over Q8_0 experts for a few tokens,
// in three launches that overlap (programmatic dependents):
//  1. router: logits, choice and weights, and the tokens' operand image;
//  2. gate / up: h = silu(Wg x) * (Wu x) of every (token, chosen expert);
//  3. down: y = residual + sum over a token's experts of w * Wd h.
//
// What bounds it is reading the chosen experts' matrices once from HBM: with
// m tokens choosing k of E, 2 and 3 stream about E (1 - (1 - k/E)^m) experts
// of 34 bytes a block of 32, and a token adds only a column to each product.
// So both are streaming kernels: one producer warp keeps a ring of shared
// memory stages filled by bulk copies (every row of a stage in a slot of its
// own, slots 4 (mod 8) words apart so that eight rows' words lie in distinct
// banks), a second one the tokens' values, and up to sixteen consumer warps
// multiply with mma.sync m16n8k16:
//  * A: sixteen weight rows, a lane's word of four quants made two exact f16
//    pairs (one PRMT and one subtraction a pair); B: up to eight tokens of
//    the expert; the warps split the blocks of a row.
//  * The tokens' values are f16 hi + lo under a power-of-two scale for each
//    block of 32 (the scheme of q8d_mma_frag.cuh): products are exact in f32
//    and a block's sum is scaled once by weight scale * inverse scale, so
//    results are f32-accurate.
//  * Whoever makes the values writes them in the operand's order: the router
//    kernel for x, the gate / up epilogue for h (it owns whole blocks of 32
//    rows), 16 bytes {hi01, hi23, lo01, lo23} a word, 128 a block, so the
//    products fetch them with bulk copies and never convert.
//  * An expert's tokens are taken eight at a time (fewer where long rows
//    leave no room); experts nobody chose are not touched.
//  * gate / up: a work unit is 32 rows of an expert (32 gate and 32 up rows:
//    64 slots, four A tiles that share every B load), units dealt to the CTAs
//    in contiguous ranges.  down: a CTA owns a few output rows of every
//    expert, so the weighted sum over experts needs no other CTA; each warp
//    adds its share of every expert into a table of its own, and the tables
//    are added once, in order.  No atomics on results anywhere: the same
//    bits every time.
#include <algorithm>
#include <cmath>

#include "q8d_gemv.cuh"
#include "q8d_internal.cuh"
#include "q8d_mma_frag.cuh"
#include "q8d_moe.cuh"

namespace q8d {
namespace {

using namespace mv;

constexpr int kImgBlock = 128;  // image bytes a block
constexpr int kMaxSmem = 222 * 1024;

__host__ __device__ constexpr int inv_pitch(int bpr) { return (bpr + 3) & ~3; }

// ---- 1. router --------------------------------------------------------------
constexpr int kRtThreads = 256;
constexpr int kRtCluster = 8;
constexpr int kRtTokens = 4;  // tokens a cluster, at most

__device__ __forceinline__ uint64_t neg2(uint64_t a) { return a ^ 0x8000000080000000ull; }

// (s, c) += a * b as an unevaluated sum: the product's rounding error (one
// FMA) and the sum's (TwoSum) go to c, so s + c carries about 48 bits.  f64
// arithmetic would be exact enough as well, but this GPU has next to none.
__device__ __forceinline__ void dot2(uint64_t& s, uint64_t& c, uint64_t a, uint64_t b) {
  const uint64_t m1 = pack2(-1.f, -1.f);
  const uint64_t p = mul2(a, b);
  const uint64_t e = fma2(a, b, neg2(p));
  const uint64_t t = add2(s, p);
  const uint64_t z = fma2(s, m1, t);                      // t - s
  const uint64_t x = fma2(fma2(z, m1, t), m1, s);         // s - (t - z)
  const uint64_t y = fma2(z, m1, p);                      // p - z
  c = add2(c, add2(add2(x, y), e));
  s = t;
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Stores v at p's place in the shared memory of the cluster's CTA 0.
__device__ __forceinline__ void store_leader(double* p, double v) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(smem_u32(p)));
  asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(a), "d"(v) : "memory");
}

// Orders doubles as integers; NaN below every number, 0 free for "taken".
__device__ __forceinline__ uint64_t rank_key(double v) {
  if (isnan(v)) return 1ull;
  const long long b = __double_as_longlong(v + 0.0);  // (-0 and 0 tie)
  return b < 0 ? ~(uint64_t)b : (uint64_t)b | 0x8000000000000000ull;
}

// Choice and weights of one token by a warp; kPer: experts a lane.
template <int kPer>
__device__ void choose(const MoeParams& P, int t, const double* logits, int lane) {
  const int E = P.n_experts;
  uint64_t key[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) key[i] = lane + 32 * i < E ? rank_key(logits[lane + 32 * i]) : 0ull;
  int mine = 0;
  double top = 0.0;  // the largest logit
  for (int k = 0; k < P.top_k; ++k) {
    uint64_t best = 0;
    int at = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (key[i] > best) best = key[i], at = lane + 32 * i;
    const uint32_t hi = (uint32_t)(best >> 32), lo = (uint32_t)best;
    const uint32_t mhi = __reduce_max_sync(0xffffffffu, hi);
    const uint32_t mlo = __reduce_max_sync(0xffffffffu, hi == mhi ? lo : 0u);
    const int e = (int)__reduce_min_sync(0xffffffffu, hi == mhi && lo == mlo ? (unsigned)at : 0xffffu);
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (e == lane + 32 * i) key[i] = 0ull;
    if (k == 0) top = logits[e];
    if (lane == k) mine = e;
  }
  // exp of the difference in two f32 parts (its rounding to one would cost up
  // to 2^-24 of the difference)
  const auto ex = [&](int e) {
    const double d = logits[e] - top;
    const float dh = (float)d;
    const float x = expf(dh), dl = (float)(d - (double)dh);
    return isinf(dh) ? x : fmaf(x, dl, x);
  };
  double all = 0.0;
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (lane + 32 * i < E) all += (double)ex(lane + 32 * i);
  const float w = lane < P.top_k ? ex(mine) : 0.f;
  double chosen = (double)w;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    all += __shfl_xor_sync(0xffffffffu, all, o);
    chosen += __shfl_xor_sync(0xffffffffu, chosen, o);
  }
  if (lane < P.top_k) {
    P.experts[t * P.top_k + lane] = mine;
    const float r = (float)((double)w / (P.norm ? chosen : all));
    P.weights[t * P.top_k + lane] = isnan(all) ? __int_as_float(0x7fc00000) : r;
  }
}

// One image word: the four values (already in operand order) of word w of a
// block, the block's eight words in eight neighbouring lanes.  Every lane of
// the warp calls; live: the word exists.
__device__ __forceinline__ void image_word(const float (&v)[4], bool live, uint8_t* blk, float* inv, int w) {
  float m = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
  m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
  m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
  // m < 2^(field - 126); the scale 2^e brings it below 2^15, e in [-113, 125]
  const int e = min(125, 15 + 126 - (int)(__float_as_uint(m) >> 23));
  if (!live) return;
  const float sc = __int_as_float((127 + e) << 23);
  const float t[4] = {v[0] * sc, v[1] * sc, v[2] * sc, v[3] * sc};
  tc::store_x_word(blk + 16 * w, t);
  if (w == 0) *inv = __int_as_float((127 - e) << 23);
}

template <int kT>
__global__ void __launch_bounds__(kRtThreads) moe_router_kernel(const MoeParams P, int per_cluster, bool perm) {
  __shared__ double logits[kRtTokens][kMoeMaxExperts];
  const int rank = (int)cluster_rank(), lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t0 = (blockIdx.x / kRtCluster) * per_cluster;
  const int nt = min(per_cluster, P.m - t0);
  const int ep = (P.n_experts + kRtCluster - 1) / kRtCluster;
  const int e0 = rank * ep, e1 = min(P.n_experts, e0 + ep);
  griddep_launch_dependents();
  // the router's rows depend on nothing in flight: into L2 meanwhile
  for (int e = e0 + warp; e < e1; e += kRtThreads / 32) {
    const char* r = reinterpret_cast<const char*>(P.router + (size_t)e * P.hidden);
    for (int o = lane * 4096; o < P.hidden * 4; o += 32 * 4096)
      bulk_prefetch_l2(r + o, (uint32_t)min(4096, P.hidden * 4 - o));
  }
  griddep_wait();
  // every CTA of the cluster is running before one stores to another's memory
  cluster_sync();
  for (int e = e0 + warp; e < e1; e += kRtThreads / 32) {
    const float4* r = reinterpret_cast<const float4*>(P.router + (size_t)e * P.hidden);
    uint64_t s[kT][2], c[kT][2];
#pragma unroll
    for (int t = 0; t < kT; ++t) s[t][0] = s[t][1] = c[t][0] = c[t][1] = pack2(0.f, 0.f);
#pragma unroll 4
    for (int i = lane; i < P.hidden / 4; i += 32) {
      const float4 a = __ldg(r + i);
#pragma unroll
      for (int t = 0; t < kT; ++t) {
        const float4 b = *(reinterpret_cast<const float4*>(P.X + (size_t)(t0 + min(t, nt - 1)) * P.ldx) + i);
        dot2(s[t][0], c[t][0], pack2(a.x, a.y), pack2(b.x, b.y));
        dot2(s[t][1], c[t][1], pack2(a.z, a.w), pack2(b.z, b.w));
      }
    }
#pragma unroll
    for (int t = 0; t < kT; ++t) {
      float x[8];
      unpack2(s[t][0], x[0], x[1]);
      unpack2(s[t][1], x[2], x[3]);
      unpack2(c[t][0], x[4], x[5]);
      unpack2(c[t][1], x[6], x[7]);
      // (the error terms of an overflowed or NaN sum mean nothing)
      const float plain = (x[0] + x[1]) + (x[2] + x[3]);
      double v = isfinite(plain) ? (((double)x[0] + x[1]) + ((double)x[2] + x[3])) +
                                       (((double)x[4] + x[5]) + ((double)x[6] + x[7]))
                                 : (double)plain;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (lane == 0 && t < nt) store_leader(&logits[t][e], v);
    }
  }
  // the tokens' operand images, a word a thread, blocks dealt over the cluster
  const int bpr = P.hidden / kQBlock, words = nt * bpr * 8;
  for (int i0 = (rank * kRtThreads + warp * 32); i0 < words; i0 += kRtCluster * kRtThreads) {
    const int i = i0 + lane, ii = min(i, words - 1);
    const int t = ii / (bpr * 8), b = (ii >> 3) % bpr, w = ii & 7;
    float v[4];
    const float* x = P.X + (size_t)(t0 + t) * P.ldx + (size_t)b * kQBlock;
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = x[tc::word_quant(perm && !(b & 1), w, k)];
    image_word(v, i < words, P.ximg + ((size_t)(t0 + t) * bpr + b) * kImgBlock,
               P.xinv + (size_t)(t0 + t) * inv_pitch(bpr) + b, w);
  }
  cluster_sync();  // the logits are complete
  if (rank == 0 && warp < nt) {
    const double* l = logits[warp];
    if (P.n_experts <= 64)
      choose<2>(P, t0 + warp, l, lane);
    else if (P.n_experts <= 128)
      choose<4>(P, t0 + warp, l, lane);
    else
      choose<kMoeMaxExperts / 32>(P, t0 + warp, l, lane);
  }
}

// ---- 2, 3. the products -----------------------------------------------------

// How a product kernel lays out its shared memory (host plan).
struct MoePlan {
  int bpr;          // blocks a row
  int S, nsl;       // blocks a slice, slices a row
  int SR;           // slot bytes
  int slots;        // row slots of a stage
  int stage_bytes, nst;
  int tg;           // tokens a group (1, 2, 4 or 8)
  int XS, XI;       // image bytes and inverse scales a token in a buffer
  int xbuf_bytes, nbuf;
  int W, KW;        // consumer warps, warps over the blocks of a row
  int rows, mt;     // down: output rows a CTA takes at once, A tiles of 16
  int items;        // (expert, token group) pairs at most
  int o_x, o_part, o_hq, o_mask, o_ebase, o_item, o_tok, o_bar;  // offsets
  int smem;
};

struct MoeShared {
  uint8_t* smem;
  float* part;
  unsigned long long* mask;  // [E] tokens of an expert
  int* ebase;                // [E] first item (low half) and first pair row (high half)
  int2* item;                // (expert | tokens << 16, first pair row)
  float* pw;                 // [pairs] weight of a pair row
  uint8_t* ptok;             // [pairs] token of a pair row
  uint64_t *full, *empty, *xfull, *xempty;
  int n_items;
};

__device__ __forceinline__ MoeShared carve(const MoePlan& L, uint8_t* smem, int pairs) {
  MoeShared S;
  S.smem = smem;
  S.part = reinterpret_cast<float*>(smem + L.o_part);
  S.mask = reinterpret_cast<unsigned long long*>(smem + L.o_mask);
  S.ebase = reinterpret_cast<int*>(smem + L.o_ebase);
  S.item = reinterpret_cast<int2*>(smem + L.o_item);
  S.pw = reinterpret_cast<float*>(smem + L.o_tok);
  S.ptok = smem + L.o_tok + 4 * pairs;
  S.full = reinterpret_cast<uint64_t*>(smem + L.o_bar);
  S.empty = S.full + L.nst;
  S.xfull = S.empty + L.nst;
  S.xempty = S.xfull + L.nbuf;
  S.n_items = 0;
  return S;
}

// Groups the (token, slot) pairs by expert, in every CTA alike: experts in
// order, an expert's tokens in order; a pair's row is its place in that
// order.  The whole CTA calls.
__device__ void group_pairs(const MoeParams& P, const MoePlan& L, MoeShared& S) {
  __shared__ int s_items;
  const int pairs = P.m * P.top_k, E = P.n_experts, nthr = blockDim.x;
  for (int e = threadIdx.x; e < E; e += nthr) S.mask[e] = 0ull;
  if (threadIdx.x == 0) {
    for (int i = 0; i < L.nst; ++i) {
      mbar_init(&S.full[i], 1);
      mbar_init(&S.empty[i], L.W);
    }
    for (int i = 0; i < L.nbuf; ++i) {
      mbar_init(&S.xfull[i], 1);
      mbar_init(&S.xempty[i], L.W);
    }
    fence_barrier_init();
  }
  __syncthreads();
  for (int p = threadIdx.x; p < pairs; p += nthr)
    atomicOr(&S.mask[__ldcg(P.experts + p)], 1ull << (p / P.top_k));
  __syncthreads();
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x, per = (E + 31) / 32;
    int items = 0, rows = 0;
    for (int e = lane * per; e < min(E, (lane + 1) * per); ++e) {
      const int c = __popcll(S.mask[e]);
      items += (c + L.tg - 1) / L.tg;
      rows += c;
    }
    int x = items | rows << 16, incl = x;  // (both fit 12 bits)
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    x = incl - x;
    for (int e = lane * per; e < min(E, (lane + 1) * per); ++e) {
      S.ebase[e] = x;
      const int c = __popcll(S.mask[e]);
      for (int g = 0; g < c; g += L.tg) {
        S.item[x & 0xffff] = make_int2(e | min(L.tg, c - g) << 16, (x >> 16));
        x += 1 + (min(L.tg, c - g) << 16);
      }
    }
    if (lane == 31) s_items = incl & 0xffff;
  }
  __syncthreads();
  for (int p = threadIdx.x; p < pairs; p += nthr) {
    const int e = __ldcg(P.experts + p), t = p / P.top_k;
    const int row = (S.ebase[e] >> 16) + __popcll(S.mask[e] & ((1ull << t) - 1ull));
    S.ptok[row] = (uint8_t)t;
    S.pw[row] = __ldcg(P.weights + p);
  }
  __syncthreads();
  S.n_items = s_items;
}

// One warp fills stage `st` with blocks [c0, c0 + nb) of `n` rows: row(i)
// gives slot i's matrix and row in it.  Rows start on any even byte unless
// kAl: the copy covers the 16-byte lines the row touches, and the last bytes
// of a matrix, when its end is no line's end, come by plain stores.
template <bool kAl, typename RowFn>
__device__ __forceinline__ void fill_stage(const MoePlan& L, uint8_t* st, uint64_t* full, int n, int c0, int nb,
                                           long long mat_bytes, RowFn row, uint64_t pol, int lane) {
  uint32_t bytes[2] = {0u, 0u};
  const uint8_t* src[2] = {nullptr, nullptr};
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int i = lane + 32 * u;
    if (i >= n) continue;
    const uint8_t* base;
    long long r;
    row(i, base, r);
    const long long a = r * (long long)(L.bpr * kQBlockBytes) + (long long)c0 * kQBlockBytes;
    if constexpr (kAl) {
      src[u] = base + a;
      bytes[u] = (uint32_t)nb * kQBlockBytes;
    } else {
      const long long lo = a & ~15LL, end = a + (long long)nb * kQBlockBytes;
      const long long hi = min((end + 15) & ~15LL, mat_bytes & ~15LL);
      src[u] = base + lo;
      bytes[u] = (uint32_t)(hi - lo);
      for (long long x = hi; x < end; x += 2)  // (the matrix ends inside its last line)
        *reinterpret_cast<unsigned short*>(st + (size_t)i * L.SR + (x - lo)) =
            *reinterpret_cast<const unsigned short*>(base + x);
    }
  }
  if constexpr (!kAl) {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // (plain stores before later copies)
    __syncwarp();
  }
  const uint32_t total = __reduce_add_sync(0xffffffffu, bytes[0] + bytes[1]);
  if (lane == 0) mbar_arrive_expect_tx(full, total);
  __syncwarp();
#pragma unroll
  for (int u = 0; u < 2; ++u)
    if (bytes[u]) bulk_g2s(st + (size_t)(lane + 32 * u) * L.SR, src[u], bytes[u], full, pol);
}

// Buffers `n` tokens' images and inverse scales (token i's at rows(i)).
template <typename RowFn>
__device__ __forceinline__ void fill_x(const MoePlan& L, uint8_t* xb, uint64_t* full, const uint8_t* img,
                                       const float* inv, int n, RowFn rows, uint64_t pol, int lane) {
  const uint32_t ib = (uint32_t)L.bpr * kImgBlock, vb = (uint32_t)L.XI * 4;
  if (lane == 0) mbar_arrive_expect_tx(full, (uint32_t)n * (ib + vb));
  __syncwarp();
  if (lane < n) {
    const size_t r = (size_t)rows(lane);
    bulk_g2s(xb + (size_t)lane * L.XS, img + r * ib, ib, full, pol);
    bulk_g2s(xb + (size_t)L.tg * L.XS + (size_t)lane * vb, inv + r * L.XI, vb, full, pol);
  }
}

// The word of four quants w = 4 step + c of a block at smem address ba.
// kAl: words are aligned in odd blocks; an even block's word 7 is its first
// two and last two quants (tc::word_quant).  Otherwise any even address,
// quants in order.
template <bool kAl>
__device__ __forceinline__ uint32_t quant_word(uint32_t ba, bool even, int step, int c) {
  if constexpr (kAl) {
    if (!even) return tc::lds32a(ba + 2u + 16u * step + 4u * c);
    if (step == 0) return tc::lds32a(ba + 4u + 4u * c);
    const uint32_t l0 = tc::lds32a(ba), l1 = tc::lds32a(ba + (c == 3 ? 32u : 20u + 4u * c));
    return __byte_perm(l0, l1, c == 3 ? 0x5432u : 0x7654u);
  } else {
    const uint32_t q = ba + 2u + 16u * step + 4u * c, a = q & ~3u;
    return __byte_perm(tc::lds32a(a), tc::lds32a(a + 4u), (q & 2u) ? 0x5432u : 0x3210u);
  }
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}

// y[t] += the products of one block: kTiles A tiles whose rows g and g + 8 of
// tile t start (this block) at ra[t][0] and ra[t][1]; xa: this lane's image
// words, xi: the inverse scales of its two tokens.
template <bool kAl, int kTiles>
__device__ __forceinline__ void block_mma(const uint32_t (&ra)[kTiles][2], bool even, int c, uint32_t xa, float xi0,
                                          float xi1, float (&y)[kTiles][4]) {
  const uint4 b0 = lds128(xa), b1 = lds128(xa + 64u);
#pragma unroll
  for (int t = 0; t < kTiles; ++t) {
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    uint32_t a0, a1, a2, a3;
    tc::quant_pairs(quant_word<kAl>(ra[t][0], even, 0, c), a0, a2);
    tc::quant_pairs(quant_word<kAl>(ra[t][1], even, 0, c), a1, a3);
    tc::mma_f16(acc, a0, a1, a2, a3, b0.x, b0.y);
    tc::mma_f16(acc, a0, a1, a2, a3, b0.z, b0.w);
    tc::quant_pairs(quant_word<kAl>(ra[t][0], even, 1, c), a0, a2);
    tc::quant_pairs(quant_word<kAl>(ra[t][1], even, 1, c), a1, a3);
    tc::mma_f16(acc, a0, a1, a2, a3, b1.x, b1.y);
    tc::mma_f16(acc, a0, a1, a2, a3, b1.z, b1.w);
    const float d0 = f16_bits_to_f32(tc::lds16a(ra[t][0])), d1 = f16_bits_to_f32(tc::lds16a(ra[t][1]));
    y[t][0] = fmaf(d0 * xi0, acc[0], y[t][0]);
    y[t][1] = fmaf(d0 * xi1, acc[1], y[t][1]);
    y[t][2] = fmaf(d1 * xi0, acc[2], y[t][2]);
    y[t][3] = fmaf(d1 * xi1, acc[3], y[t][3]);
  }
}

// One warp's wait on a barrier that lane 0 polls.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort, int lane) {
  const int ok = lane ? 1 : (wait_or_abort(bar, parity, abort) ? 1 : 0);
  return __all_sync(0xffffffffu, ok);
}

// Ends a product kernel: reports a wait that gave up, and has a producer
// warp (of `issued` fills of the n buffers behind `full`) wait for its copies
// in flight before the CTA leaves.
__device__ __forceinline__ void finish(const MoeParams& P, uint64_t* full, int n, volatile int* abort, int issued) {
  if (*abort)
    for (int j = max(0, issued - n); j < issued; ++j) mbar_wait(&full[j % n], (uint32_t)(j / n) & 1u);
  __syncthreads();
  if (threadIdx.x == 0 && *abort && P.d_err) atomicOr(P.d_err, Q8D_DERR_WAIT);
}

constexpr int kGuWarps = 16, kGuK = 8;  // consumer warps; over the blocks of a row
constexpr int kGuRows = 32;             // h rows a unit
constexpr int kGuTiles = 2;             // A tiles (8 gate + 8 up rows) a warp

template <bool kAl>
__global__ void __launch_bounds__((kGuWarps + 2) * 32, 1)
    moe_gate_up_kernel(const MoeParams P, const MoePlan L, bool hperm) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int s_abort;
  MoeShared S = carve(L, smem, P.m * P.top_k);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) s_abort = 0;
  griddep_wait();
  griddep_launch_dependents();  // (after the wait: the next kernel may read the choice at once)
  group_pairs(P, L, S);
  const int nq = P.ffn / kGuRows;                // units an item
  const long long units = (long long)S.n_items * nq;
  const int q0 = (int)(units * blockIdx.x / gridDim.x), q1 = (int)(units * (blockIdx.x + 1) / gridDim.x);
  int issued = 0;
  if (warp == kGuWarps) {
    const uint64_t pol = policy_evict_first();
    const long long mat = (long long)P.n_experts * P.ffn * L.bpr * kQBlockBytes;
    bool ok = true;
    for (int q = q0; q < q1 && ok; ++q) {
      const int it = q / nq;
      const long long r0 = (long long)(S.item[it].x & 0xffff) * P.ffn + (long long)(q - it * nq) * kGuRows;
      for (int sl = 0; sl < L.nsl; ++sl, ++issued) {
        const int s = issued % L.nst;
        if (issued >= L.nst) ok = warp_wait(&S.empty[s], (uint32_t)(issued / L.nst - 1) & 1u, &s_abort, lane);
        if (!ok) break;
        fill_stage<kAl>(L, smem + (size_t)s * L.stage_bytes, &S.full[s], 2 * kGuRows, sl * L.S,
                        min(L.S, L.bpr - sl * L.S), mat,
                        [&](int i, const uint8_t*& base, long long& r) {
                          base = i < kGuRows ? P.wg : P.wu;
                          r = r0 + (i & (kGuRows - 1));
                        },
                        pol, lane);
      }
    }
  } else if (warp == kGuWarps + 1) {
    const uint64_t keep = policy_evict_last();
    fence_proxy_async_global();  // (the images were written by ordinary stores)
    for (int it = q0 / nq; it * nq < q1; ++it, ++issued) {
      const int s = issued % L.nbuf;
      if (issued >= L.nbuf && !warp_wait(&S.xempty[s], (uint32_t)(issued / L.nbuf - 1) & 1u, &s_abort, lane)) break;
      const int2 I = S.item[it];
      fill_x(L, smem + L.o_x + s * L.xbuf_bytes, &S.xfull[s], P.ximg, P.xinv, I.x >> 16,
             [&](int i) { return (int)S.ptok[I.y + i]; }, keep, lane);
    }
  } else {
    const int gq = lane >> 2, cq = lane & 3;
    const int kb = warp % kGuK, th = warp / kGuK;  // blocks kb, kb + 8, ..; tiles 2 th, 2 th + 1
    const uint32_t smem32 = smem_u32(smem);
    const uint32_t xl = (uint32_t)(min(gq, L.tg - 1) * L.XS + cq * 16);
    float* hq = reinterpret_cast<float*>(smem + L.o_hq);  // [32 rows][8 tokens + 1]
    int item = -1, xuse = -1, stage = 0;
    bool ok = true;
    uint32_t xb = 0;
    const float* xiv = nullptr;
    for (int q = q0; q < q1; ++q) {
      const int it = q / nq;
      if (it != item) {
        if (xuse >= 0) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&S.xempty[xuse % L.nbuf]);
        }
        item = it;
        ++xuse;
        ok = wait_or_abort(&S.xfull[xuse % L.nbuf], (uint32_t)(xuse / L.nbuf) & 1u, &s_abort) && ok;
        const uint32_t off = (uint32_t)(L.o_x + (xuse % L.nbuf) * L.xbuf_bytes);
        xb = after_wait(smem32 + off) + xl;
        xiv = reinterpret_cast<const float*>(smem + off + (size_t)L.tg * L.XS);
      }
      const int2 I = S.item[it];
      const int ntok = I.x >> 16;
      const long long r0 = (long long)(I.x & 0xffff) * P.ffn + (long long)(q - it * nq) * kGuRows;
      const float* xi0 = xiv + min(2 * cq, L.tg - 1) * L.XI;
      const float* xi1 = xiv + min(2 * cq + 1, L.tg - 1) * L.XI;
      float y[kGuTiles][4];
#pragma unroll
      for (int t = 0; t < kGuTiles; ++t) y[t][0] = y[t][1] = y[t][2] = y[t][3] = 0.f;
      // where this lane's rows start in their slots
      uint32_t ro[kGuTiles][2];
#pragma unroll
      for (int t = 0; t < kGuTiles; ++t) {
        const int r = (2 * th + t) * 8 + gq;
        const uint32_t mis = kAl ? 0u : (uint32_t)(((r0 + r) * (L.bpr * kQBlockBytes)) & 15);
        ro[t][0] = (uint32_t)(r * L.SR) + mis;
        ro[t][1] = (uint32_t)((kGuRows + r) * L.SR) + mis;
      }
      for (int sl = 0; sl < L.nsl; ++sl, ++stage) {
        const int s = stage % L.nst;
        ok = wait_or_abort(&S.full[s], (uint32_t)(stage / L.nst) & 1u, &s_abort) && ok;
        const uint32_t st = after_wait(smem32 + (uint32_t)s * (uint32_t)L.stage_bytes);
        const int c0 = sl * L.S, nb = min(L.S, L.bpr - c0);
        // (a slice's own misalignment: c0 * 34 beyond the row's)
        for (int j = kb; j < nb; j += kGuK) {
          uint32_t ra[kGuTiles][2];
#pragma unroll
          for (int t = 0; t < kGuTiles; ++t)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if constexpr (kAl) {
                ra[t][h] = st + ro[t][h] + (uint32_t)j * kQBlockBytes;
              } else {
                const uint32_t slot = (uint32_t)((h * kGuRows + (2 * th + t) * 8 + gq) * L.SR);
                ra[t][h] = st + slot + ((ro[t][h] - slot + (uint32_t)c0 * kQBlockBytes) & 15u) +
                           (uint32_t)j * kQBlockBytes;
              }
            }
          const int blk = c0 + j;
          block_mma<kAl, kGuTiles>(ra, !(blk & 1), cq, xb + (uint32_t)blk * kImgBlock, xi0[blk], xi1[blk], y);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.empty[s]);
      }
      // the warps' shares of the unit: [kb][tile][row of 16][token]
#pragma unroll
      for (int t = 0; t < kGuTiles; ++t) {
        float* p = S.part + ((kb * 4 + 2 * th + t) * 16 + gq) * 8 + 2 * cq;
        *reinterpret_cast<float2*>(p) = make_float2(y[t][0], y[t][1]);
        *reinterpret_cast<float2*>(p + 64) = make_float2(y[t][2], y[t][3]);
      }
      consumer_sync(kGuWarps * 32);
      if (threadIdx.x < 256) {
        const int tile = threadIdx.x >> 6, r = (threadIdx.x >> 3) & 7, n = threadIdx.x & 7;
        float g = 0.f, u = 0.f;
#pragma unroll
        for (int k = 0; k < kGuK; ++k) {
          g += S.part[((k * 4 + tile) * 16 + r) * 8 + n];
          u += S.part[((k * 4 + tile) * 16 + r + 8) * 8 + n];
        }
        hq[(tile * 8 + r) * 9 + n] = g / (1.f + expf(-g)) * u;
      }
      consumer_sync(kGuWarps * 32);
      if (threadIdx.x < 64) {  // the unit is block q - it * nq of its tokens' h: token n, word w
        const int n = threadIdx.x >> 3, w = threadIdx.x & 7, b = q - it * nq;
        float v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = hq[tc::word_quant(hperm && !(b & 1), w, k) * 9 + n];
        image_word(v, n < ntok, P.himg + ((size_t)(I.y + n) * nq + b) * kImgBlock,
                   P.hinv + (size_t)(I.y + n) * inv_pitch(nq) + b, w);
      }
    }
  }
  finish(P, warp == kGuWarps ? S.full : S.xfull, warp == kGuWarps ? L.nst : L.nbuf, &s_abort, issued);
}

constexpr int kDnMaxWarps = 16;

template <bool kAl, int kTiles>
__global__ void __launch_bounds__((kDnMaxWarps + 2) * 32, 1) moe_down_kernel(const MoeParams P, const MoePlan L) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int s_abort;
  MoeShared S = carve(L, smem, P.m * P.top_k);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, W = L.W;
  if (threadIdx.x == 0) s_abort = 0;
  group_pairs(P, L, S);  // (the choice is complete: the gate / up kernel started behind it)
  const int chunks = (P.hidden + L.rows - 1) / L.rows;
  int issued = 0;
  if (warp == W) {
    // Weights depend on nothing in flight: they fill the ring while the gate /
    // up kernel ends.
    const uint64_t pol = policy_evict_first();
    const long long mat = (long long)P.n_experts * P.hidden * L.bpr * kQBlockBytes;
    bool ok = true;
    for (int ch = blockIdx.x; ch < chunks && ok; ch += gridDim.x) {
      const int r0 = ch * L.rows, nr = min(L.rows, P.hidden - r0);
      for (int it = 0; it < S.n_items && ok; ++it) {
        const long long e0 = (long long)(S.item[it].x & 0xffff) * P.hidden + r0;
        for (int sl = 0; sl < L.nsl; ++sl, ++issued) {
          const int s = issued % L.nst;
          if (issued >= L.nst) ok = warp_wait(&S.empty[s], (uint32_t)(issued / L.nst - 1) & 1u, &s_abort, lane);
          if (!ok) break;
          fill_stage<kAl>(L, smem + (size_t)s * L.stage_bytes, &S.full[s], nr, sl * L.S,
                          min(L.S, L.bpr - sl * L.S), mat,
                          [&](int i, const uint8_t*& base, long long& r) {
                            base = P.wd;
                            r = e0 + i;
                          },
                          pol, lane);
        }
      }
    }
  } else if (warp == W + 1) {
    const uint64_t keep = policy_evict_last();
    griddep_wait();
    fence_proxy_async_global();
    bool ok = true;
    for (int ch = blockIdx.x; ch < chunks && ok; ch += gridDim.x)
      for (int it = 0; it < S.n_items; ++it, ++issued) {
        const int s = issued % L.nbuf;
        if (issued >= L.nbuf) ok = warp_wait(&S.xempty[s], (uint32_t)(issued / L.nbuf - 1) & 1u, &s_abort, lane);
        if (!ok) break;
        const int2 I = S.item[it];
        fill_x(L, smem + L.o_x + s * L.xbuf_bytes, &S.xfull[s], P.himg, P.hinv, I.x >> 16,
               [&](int i) { return I.y + i; }, keep, lane);
      }
  } else {
    griddep_wait();
    const int gq = lane >> 2, cq = lane & 3;
    const uint32_t smem32 = smem_u32(smem);
    const uint32_t xl = (uint32_t)(min(gq, L.tg - 1) * L.XS + cq * 16);
    const int yp = P.m | 1;                                 // table pitch (odd: rows in distinct banks)
    float* tab = S.part + (size_t)warp * L.mt * 16 * yp;    // this warp's [rows][tokens]
    int xuse = 0, stage = 0;
    bool ok = true;
    for (int ch = blockIdx.x; ch < chunks; ch += gridDim.x) {
      const int r0 = ch * L.rows, nr = min(L.rows, P.hidden - r0);
      for (int i = lane; i < L.mt * 16 * yp; i += 32) tab[i] = 0.f;
      __syncwarp();
      for (int it = 0; it < S.n_items; ++it, ++xuse) {
        const int2 I = S.item[it];
        const int ntok = I.x >> 16;
        const long long e0 = (long long)(I.x & 0xffff) * P.hidden + r0;
        ok = wait_or_abort(&S.xfull[xuse % L.nbuf], (uint32_t)(xuse / L.nbuf) & 1u, &s_abort) && ok;
        const uint32_t off = (uint32_t)(L.o_x + (xuse % L.nbuf) * L.xbuf_bytes);
        const uint32_t xb = after_wait(smem32 + off) + xl;
        const float* xiv = reinterpret_cast<const float*>(smem + off + (size_t)L.tg * L.XS);
        const float* xi0 = xiv + min(2 * cq, L.tg - 1) * L.XI;
        const float* xi1 = xiv + min(2 * cq + 1, L.tg - 1) * L.XI;
        float y[kTiles][4];
#pragma unroll
        for (int t = 0; t < kTiles; ++t) y[t][0] = y[t][1] = y[t][2] = y[t][3] = 0.f;
        for (int sl = 0; sl < L.nsl; ++sl, ++stage) {
          const int s = stage % L.nst;
          ok = wait_or_abort(&S.full[s], (uint32_t)(stage / L.nst) & 1u, &s_abort) && ok;
          const uint32_t st = after_wait(smem32 + (uint32_t)s * (uint32_t)L.stage_bytes);
          const int c0 = sl * L.S, nb = min(L.S, L.bpr - c0);
          uint32_t ro[kTiles][2];
#pragma unroll
          for (int t = 0; t < kTiles; ++t)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int r = 16 * t + 8 * h + gq;
              const uint32_t mis =
                  kAl ? 0u : (uint32_t)(((e0 + r) * (L.bpr * kQBlockBytes) + c0 * kQBlockBytes) & 15);
              ro[t][h] = st + (uint32_t)(r * L.SR) + mis;
            }
          for (int j = warp; j < nb; j += W) {
            uint32_t ra[kTiles][2];
#pragma unroll
            for (int t = 0; t < kTiles; ++t)
#pragma unroll
              for (int h = 0; h < 2; ++h) ra[t][h] = ro[t][h] + (uint32_t)j * kQBlockBytes;
            const int blk = c0 + j;
            block_mma<kAl, kTiles>(ra, !(blk & 1), cq, xb + (uint32_t)blk * kImgBlock, xi0[blk], xi1[blk], y);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&S.empty[s]);
        }
        if (lane == 0) mbar_arrive(&S.xempty[xuse % L.nbuf]);
        // weighted into the warp's table: lane (g, c) alone owns these entries
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int n = 2 * cq + k;
          if (n < ntok) {
            const float w = S.pw[I.y + n];
            float* col = tab + S.ptok[I.y + n];
#pragma unroll
            for (int t = 0; t < kTiles; ++t) {
              float* a = col + (16 * t + gq) * yp;
              float* b = a + 8 * yp;
              *a = fmaf(w, y[t][k], *a);
              *b = fmaf(w, y[t][2 + k], *b);
            }
          }
        }
        __syncwarp();
      }
      consumer_sync(W * 32);
      for (int i = threadIdx.x; i < nr * P.m; i += W * 32) {
        const int r = i % nr, t = i / nr;
        float sum = P.residual ? P.residual[(long long)t * P.ldr + r0 + r] : 0.f;
        for (int w = 0; w < W; ++w) sum += S.part[((size_t)w * L.mt * 16 + r) * yp + t];
        P.Y[(long long)t * P.ldy + r0 + r] = sum;
      }
      consumer_sync(W * 32);  // (the tables are cleared next)
    }
  }
  finish(P, warp == W ? S.full : S.xfull, warp == W ? L.nst : L.nbuf, &s_abort, issued);
  griddep_launch_dependents();
}

int up16i(int n) { return (n + 15) / 16 * 16; }
size_t up16(size_t n) { return (n + 15) / 16 * 16; }

// A slot of n blocks: a multiple of 16 bytes, 4 (mod 8) words long; rows off
// the 16-byte boundaries may start 14 bytes in and are read 4 bytes past.
int slot_bytes(int n, bool aligned) {
  int b = up16i(n * kQBlockBytes + (aligned ? 0 : 18));
  while ((b / 4) % 8 != 4) b += 16;
  return b;
}

// Token groups and their buffers: as many tokens as can share an expert (up
// to 8, a power of two), several buffers where they leave the ring its room.
void plan_x(const MoeParams& P, int bpr, int most, int most_buf, MoePlan* L) {
  L->bpr = bpr;
  L->XI = inv_pitch(bpr);
  // token rows half a bank cycle apart: the two tokens of a quarter warp's
  // 16-byte loads lie in distinct banks
  L->XS = bpr * kImgBlock + 64;
  const int a_token = L->XS + L->XI * 4;
  L->tg = 8;
  while (L->tg > 1 && (L->tg / 2 >= P.m || L->tg * a_token > most)) L->tg /= 2;
  L->xbuf_bytes = up16i(L->tg * a_token);
  L->nbuf = std::max(1, std::min(most_buf, most / L->xbuf_bytes));
  const int pairs = P.m * P.top_k;
  L->items = std::min(pairs, P.n_experts + pairs / L->tg);
}

// Offsets behind the ring; returns the bytes used without the ring.
int plan_rest(const MoeParams& P, int part_floats, int hq_floats, MoePlan* L) {
  const int pairs = P.m * P.top_k;
  int o = L->nst * L->stage_bytes;
  L->o_x = o;
  o += L->nbuf * L->xbuf_bytes;
  L->o_part = o;
  o += up16i(4 * part_floats);
  L->o_hq = o;
  o += up16i(4 * hq_floats);
  L->o_mask = o;
  o += 8 * P.n_experts;
  L->o_ebase = o;
  o += up16i(4 * P.n_experts);
  o = up16i(o);
  L->o_item = o;
  o += 8 * L->items;
  L->o_tok = o = up16i(o);
  o += up16i(5 * pairs);
  L->o_bar = o = up16i(o);
  o += 16 * L->nst + 16 * L->nbuf;
  L->smem = o;
  return o - L->nst * L->stage_bytes;
}

int plan_gate_up(const MoeParams& P, MoePlan* L) {
  const int bpr = P.hidden / kQBlock;
  const bool al = bpr % 8 == 0;
  plan_x(P, bpr, 120 * 1024, 2, L);
  L->W = kGuWarps;
  L->KW = kGuK;
  L->slots = 2 * kGuRows;
  L->rows = kGuRows;
  L->mt = 4;
  for (int nbuf = L->nbuf; nbuf >= 1; --nbuf) {
    L->nbuf = nbuf;
    // two blocks a warp in a stage, or one where that leaves too few stages
    for (int s = std::min(16, bpr); s >= 1; s = s > 8 ? 8 : s / 2) {
      L->S = s;
      L->nsl = (bpr + s - 1) / s;
      L->SR = slot_bytes(s, al);
      L->stage_bytes = L->slots * L->SR;
      L->nst = 0;
      const int rest = plan_rest(P, kGuK * 4 * 128, kGuRows * 9, L) + 16 * 8;
      L->nst = std::min(8, (kMaxSmem - rest) / L->stage_bytes);
      if (L->nst >= 3) {
        plan_rest(P, kGuK * 4 * 128, kGuRows * 9, L);
        return Q8D_OK;
      }
      if (al && s <= 8) break;  // (aligned slices are whole groups of 8 blocks)
    }
  }
  return Q8D_EUNSUPPORTED;
}

int plan_down(const MoeParams& P, int sms, MoePlan* L) {
  const int bpr = P.ffn / kQBlock;
  const bool al = bpr % 8 == 0;
  plan_x(P, bpr, 80 * 1024, 4, L);
  // the warp count in 8 .. 16 that splits a row's blocks most evenly
  double best = 0.0;
  for (int w = kDnMaxWarps; w >= 8; --w) {
    const double eff = (double)bpr / (w * ((bpr + w - 1) / w));
    if (eff > best + 1e-9) {
      best = eff;
      L->W = w;
    }
  }
  for (int w = L->W;; w = 8) {
    L->W = L->KW = w;
    // rows a CTA: an equal share of the output, in as few passes as 32 rows
    // at a time allow
    for (int most = 32; most >= 16; most -= 16) {
      const int passes = (P.hidden + sms * most - 1) / (sms * most);
      L->rows = std::min(most, (P.hidden + sms * passes - 1) / (sms * passes));
      L->mt = L->rows > 16 ? 2 : 1;
      L->slots = L->mt * 16;
      const int table = w * L->mt * 16 * (P.m | 1);
      for (int s = std::min(bpr, 64); s >= 1; s = al ? s - 8 : s - std::max(1, s / 8)) {
        L->S = al ? s / 8 * 8 : s;
        L->nsl = (bpr + L->S - 1) / L->S;
        L->S = (bpr + L->nsl - 1) / L->nsl;  // (equal slices)
        if (al) L->S = (L->S + 7) / 8 * 8;
        L->SR = slot_bytes(L->S, al);
        L->stage_bytes = L->slots * L->SR;
        L->nst = 0;
        const int rest = plan_rest(P, table, 0, L) + 16 * 12;
        if (rest < kMaxSmem) L->nst = std::min(12, (kMaxSmem - rest) / L->stage_bytes);
        if (L->nst >= 4) {
          plan_rest(P, table, 0, L);
          return Q8D_OK;
        }
      }
    }
    if (w == 8) return Q8D_EUNSUPPORTED;
  }
}

}  // namespace

size_t moe_workspace_bytes(int m, int hidden, int ffn, int n_experts, int top_k) {
  (void)n_experts;
  const size_t pairs = (size_t)m * top_k;
  return up16(4 * pairs) * 2 + (size_t)m * (hidden / kQBlock) * kImgBlock +
         4 * (size_t)m * inv_pitch(hidden / kQBlock) + pairs * (ffn / kQBlock) * kImgBlock +
         4 * pairs * inv_pitch(ffn / kQBlock);
}

int moe_launch(MoeParams P, void* workspace, cudaStream_t stream) {
  const size_t pairs = (size_t)P.m * P.top_k;
  const int bx = P.hidden / kQBlock, bh = P.ffn / kQBlock;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  P.ximg = ws;
  ws += (size_t)P.m * bx * kImgBlock;
  P.himg = ws;
  ws += pairs * bh * kImgBlock;
  P.xinv = reinterpret_cast<float*>(ws);
  ws += 4 * (size_t)P.m * inv_pitch(bx);
  P.hinv = reinterpret_cast<float*>(ws);
  ws += 4 * pairs * inv_pitch(bh);
  if (!P.experts) P.experts = reinterpret_cast<int*>(ws);
  ws += up16(4 * pairs);
  if (!P.weights) P.weights = reinterpret_cast<float*>(ws);

  const int sms = sm_count();
  MoePlan gu{}, dn{};
  int rc = plan_gate_up(P, &gu);
  if (!rc) rc = plan_down(P, sms, &dn);
  if (rc) return rc;
  const bool gal = bx % 8 == 0, dal = bh % 8 == 0;
  void (*const gu_fn)(MoeParams, MoePlan, bool) = gal ? moe_gate_up_kernel<true> : moe_gate_up_kernel<false>;
  void (*const dn_fns[2][2])(MoeParams, MoePlan) = {{moe_down_kernel<false, 1>, moe_down_kernel<false, 2>},
                                                    {moe_down_kernel<true, 1>, moe_down_kernel<true, 2>}};
  const auto dn_fn = dn_fns[dal][dn.mt - 1];
  rc = configure_kernel(reinterpret_cast<const void*>(gu_fn), kMaxSmem, true);
  if (!rc) rc = configure_kernel(reinterpret_cast<const void*>(dn_fn), kMaxSmem, true);
  if (rc) return rc;

  // the router: clusters of 8 CTAs, up to 4 tokens each, at most 16 clusters
  const int per = (P.m + 15) / 16;
  const int clusters = (P.m + per - 1) / per;
  void (*const rt_fns[4])(MoeParams, int, bool) = {moe_router_kernel<1>, moe_router_kernel<2>, moe_router_kernel<3>,
                                                   moe_router_kernel<4>};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(clusters * kRtCluster);
  cfg.blockDim = dim3(kRtThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kRtCluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, rt_fns[per - 1], P, per, gal);
  if (e != cudaSuccess) return record_cuda(e);
  rc = launch_ex(gu_fn, dim3(sms), dim3((gu.W + 2) * 32), (size_t)gu.smem, stream, true, P, gu, dal);
  if (rc) return rc;
  const int chunks = (P.hidden + dn.rows - 1) / dn.rows;
  return launch_ex(dn_fn, dim3(std::min(sms, chunks)), dim3((dn.W + 2) * 32), (size_t)dn.smem, stream, true, P, dn);
}

}  // namespace q8d
