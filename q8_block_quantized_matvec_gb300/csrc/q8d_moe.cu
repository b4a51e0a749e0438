// A mixture-of-experts feed-forward layer over Q8_0 experts for a few tokens,
// in three launches that overlap (programmatic dependents):
//  1. router: logits, choice and weights, and the tokens' operand image;
//  2. gate / up: h = silu(Wg x) * (Wu x) of every (token, chosen expert);
//  3. down: y = residual + sum over a token's experts of w * Wd h.
//
// What bounds it is reading the chosen experts' matrices once from HBM: with
// m tokens choosing k of E, 2 and 3 stream about E (1 - (1 - k/E)^m) experts
// of 34 bytes a block of 32, and a token adds only a column to each product.
// So both are streaming kernels: four producer warps keep a ring of shared
// memory stages filled with 16-byte cp.async copies (every row of a stage in a
// slot of its own, slots 4 (mod 8) words apart so that eight rows' words lie in
// distinct banks; bulk copies of such short pieces issue a lane at a time and
// held the stream to 6 bytes a cycle and SM), and up to sixteen consumer warps
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
//    rows), 16 bytes {hi01, hi23, lo01, lo23} a word, 144 a block with its
//    inverse scale, so the products copy them beside the weights and never
//    convert.
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

constexpr int kImgBlock = 144;  // image bytes a block: 8 words of 16, the inverse scale, 12 unused
constexpr int kMaxSmem = 222 * 1024;

// ---- 1. router --------------------------------------------------------------
constexpr int kRtThreads = 512;
constexpr int kRtCluster = 8;

__device__ __forceinline__ uint64_t neg2(uint64_t a) { return a ^ 0x8000000080000000ull; }

// (s, c) += a * b as an unevaluated sum: the product's rounding error (one
// FMA) and the sum's (TwoSum) go to c, so s + c carries about 48 bits.  (f64
// arithmetic would do as well, but an SM of this GPU does two a cycle.)
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
// (h, l) += (a, b), pairs as above.
__device__ __forceinline__ void add_pair(float& h, float& l, float a, float b) {
  const float t = __fadd_rn(h, a), z = __fsub_rn(t, h);
  const float e = __fadd_rn(__fsub_rn(h, __fsub_rn(t, z)), __fsub_rn(a, z));
  h = t;
  l = __fadd_rn(l, __fadd_rn(b, e));
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
__device__ __forceinline__ void store_leader(float2* p, float2 v) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(smem_u32(p)));
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(a), "f"(v.x), "f"(v.y) : "memory");
}

// Orders logits (h, l), l at most half a unit of h's last place, as integers;
// NaN below every number, 0 free for "taken".
__device__ __forceinline__ uint32_t order32(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);  // (-0 and 0 tie)
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ uint64_t rank_key(float2 v) {
  return isnan(v.x) ? 1ull : (uint64_t)order32(v.x) << 32 | order32(v.y);
}

// Choice and weights of one token by a warp; kPer: experts a lane.
template <int kPer>
__device__ void choose(const MoeParams& P, int t, const float2* logits, int lane) {
  const int E = P.n_experts;
  uint64_t key[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) key[i] = lane + 32 * i < E ? rank_key(logits[lane + 32 * i]) : 0ull;
  int mine = 0;
  float2 top = make_float2(0.f, 0.f);  // the largest logit
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
  // exp(l - top), the difference in two parts (rounded to one it would be off
  // by up to 2^-24 of itself)
  const auto ex = [&](int e) {
    const float2 v = logits[e];
    float d = v.x, r = v.y;
    add_pair(d, r, -top.x, -top.y);
    const float x = expf(d);
    return isinf(d) ? x : fmaf(x, r, x);
  };
  float all = 0.f, all2 = 0.f;
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (lane + 32 * i < E) add_pair(all, all2, ex(lane + 32 * i), 0.f);
  const float w = lane < P.top_k ? ex(mine) : 0.f;
  float chosen = w, chosen2 = 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float a = __shfl_xor_sync(0xffffffffu, all, o), a2 = __shfl_xor_sync(0xffffffffu, all2, o);
    const float c = __shfl_xor_sync(0xffffffffu, chosen, o), c2 = __shfl_xor_sync(0xffffffffu, chosen2, o);
    add_pair(all, all2, a, a2);
    add_pair(chosen, chosen2, c, c2);
  }
  if (lane < P.top_k) {
    P.experts[t * P.top_k + lane] = mine;
    P.weights[t * P.top_k + lane] =
        isnan(all) ? __int_as_float(0x7fc00000) : __fdiv_rn(w, P.norm ? chosen + chosen2 : all + all2);
  }
}

// One image word: the four values (already in operand order) of word w of a
// block, the block's eight words in eight neighbouring lanes.  Every lane of
// the warp calls; live: the word exists.
__device__ __forceinline__ void image_word(const float (&v)[4], bool live, uint8_t* blk, int w) {
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
  if (w == 0) *reinterpret_cast<float*>(blk + 128) = __int_as_float((127 - e) << 23);
}

// Logits of kE experts e, e + stride, .. for kT tokens by a warp, to the
// leader's table.
template <int kT, int kE>
__device__ __forceinline__ void logits_of(const MoeParams& P, int t0, int nt, int e, int stride, int e1,
                                          float2 (*table)[kMoeMaxExperts], int lane) {
  uint64_t s[kE][kT][2], c[kE][kT][2];
#pragma unroll
  for (int x = 0; x < kE; ++x)
#pragma unroll
    for (int t = 0; t < kT; ++t) s[x][t][0] = s[x][t][1] = c[x][t][0] = c[x][t][1] = pack2(0.f, 0.f);
  constexpr int kAhead = kT * kE == 1 ? 8 : kT * kE <= 4 ? 4 : 2;  // loads in flight
  const int n = P.hidden / 4;
  for (int i0 = lane; i0 < n; i0 += 32 * kAhead) {
    float4 a[kAhead][kE], b[kAhead][kT];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int i = i0 + 32 * u;
      const bool ok = i < n;
#pragma unroll
      for (int x = 0; x < kE; ++x)
        a[u][x] = ok ? __ldg(reinterpret_cast<const float4*>(
                                 P.router + (size_t)min(e + x * stride, e1 - 1) * P.hidden) + i)
                     : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int t = 0; t < kT; ++t)
        b[u][t] = ok ? *(reinterpret_cast<const float4*>(P.X + (size_t)(t0 + min(t, nt - 1)) * P.ldx) + i)
                     : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
#pragma unroll
      for (int x = 0; x < kE; ++x)
#pragma unroll
        for (int t = 0; t < kT; ++t) {
          dot2(s[x][t][0], c[x][t][0], pack2(a[u][x].x, a[u][x].y), pack2(b[u][t].x, b[u][t].y));
          dot2(s[x][t][1], c[x][t][1], pack2(a[u][x].z, a[u][x].w), pack2(b[u][t].z, b[u][t].w));
        }
  }
#pragma unroll
  for (int x = 0; x < kE; ++x)
#pragma unroll
    for (int t = 0; t < kT; ++t) {
      float v[4], r[4];
      unpack2(s[x][t][0], v[0], v[1]);
      unpack2(s[x][t][1], v[2], v[3]);
      unpack2(c[x][t][0], r[0], r[1]);
      unpack2(c[x][t][1], r[2], r[3]);
      float plain = (v[0] + v[1]) + (v[2] + v[3]);
#pragma unroll
      for (int k = 1; k < 4; ++k) add_pair(v[0], r[0], v[k], r[k]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const float a = __shfl_xor_sync(0xffffffffu, v[0], o), b = __shfl_xor_sync(0xffffffffu, r[0], o);
        plain += __shfl_xor_sync(0xffffffffu, plain, o);
        add_pair(v[0], r[0], a, b);
      }
      // normalise; the error terms of an overflowed or NaN sum mean nothing
      const float h = v[0] + r[0];
      const float2 l = isfinite(h) ? make_float2(h, __fsub_rn(r[0], __fsub_rn(h, v[0]))) : make_float2(plain, 0.f);
      if (lane == 0 && t < nt && e + x * stride < e1) store_leader(&table[t][e + x * stride], l);
    }
}

template <int kT>
__global__ void __launch_bounds__(kRtThreads) moe_router_kernel(const MoeParams P, int per_cluster, bool perm) {
  __shared__ float2 logits[kT][kMoeMaxExperts];
  constexpr int kWarps = kRtThreads / 32;
  const int rank = (int)cluster_rank(), lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t0 = (blockIdx.x / kRtCluster) * per_cluster;
  const int nt = min(per_cluster, P.m - t0);
  const int ep = (P.n_experts + kRtCluster - 1) / kRtCluster;
  const int e0 = rank * ep, e1 = min(P.n_experts, e0 + ep);
  griddep_launch_dependents();
  // the router's rows depend on nothing in flight: into L2 meanwhile
  for (int e = e0 + warp; e < e1; e += kWarps) {
    const char* r = reinterpret_cast<const char*>(P.router + (size_t)e * P.hidden);
    for (int o = lane * 4096; o < P.hidden * 4; o += 32 * 4096)
      bulk_prefetch_l2(r + o, (uint32_t)min(4096, P.hidden * 4 - o));
  }
  griddep_wait();
  // every CTA of the cluster is running before one stores to another's memory
  cluster_sync();
  int e = e0 + warp;
  for (; e + kWarps < e1; e += 2 * kWarps) logits_of<kT, 2>(P, t0, nt, e, kWarps, e1, logits, lane);
  if (e < e1) logits_of<kT, 1>(P, t0, nt, e, kWarps, e1, logits, lane);
  // the tokens' operand images, a word a thread, blocks dealt over the cluster
  const int bpr = P.hidden / kQBlock, words = nt * bpr * 8;
  for (int i0 = (rank * kRtThreads + warp * 32); i0 < words; i0 += kRtCluster * kRtThreads) {
    const int i = i0 + lane, ii = min(i, words - 1);
    const int t = ii / (bpr * 8), b = (ii >> 3) % bpr, w = ii & 7;
    float v[4];
    const float* x = P.X + (size_t)(t0 + t) * P.ldx + (size_t)b * kQBlock;
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = x[tc::word_quant(perm && !(b & 1), w, k)];
    image_word(v, i < words, P.ximg + ((size_t)(t0 + t) * bpr + b) * kImgBlock, w);
  }
  cluster_sync();  // the logits are complete
  if (rank == 0 && warp < nt) {
    const float2* l = logits[warp];
    if (P.n_experts <= 64)
      choose<2>(P, t0 + warp, l, lane);
    else if (P.n_experts <= 128)
      choose<4>(P, t0 + warp, l, lane);
    else
      choose<kMoeMaxExperts / 32>(P, t0 + warp, l, lane);
  }
}

// ---- 2, 3. the products -----------------------------------------------------

constexpr int kProducers = 4;  // producer warps (the first brings the images too)

// How a product kernel lays out its shared memory (host plan).
struct MoePlan {
  int bpr;          // blocks a row
  int S, nsl;       // blocks a slice, slices a row
  int SR;           // slot bytes
  int slots;        // row slots of a stage
  int tg;           // tokens a group (1, 2, 4 or 8)
  int XR;           // image bytes a token of a stage
  int stage_bytes, nst;
  int W;            // consumer warps
  int rows, mt;     // down: output rows a CTA takes at once, A tiles of 16
  int items;        // (expert, token group) pairs at most
  int o_part, o_hq, o_mask, o_ebase, o_item, o_tok, o_bar;  // offsets
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
  uint64_t *full, *empty;
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
      mbar_init(&S.full[i], kProducers * 32 + 1);
      mbar_init(&S.empty[i], L.W);
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

// 16 bytes, of which n exist (the others become zeros).
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, int n) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
// Arrives on bar once this thread's copies so far have landed.
__device__ __forceinline__ void cp_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// A producer thread's share of a stage's rows: 16-byte line c of rows rg,
// rg + step, ..  (Fixed for the kernel: the copy loops only add.)
struct FillLane {
  int c, rg, step;
};
template <bool kAl>
__device__ __forceinline__ FillLane fill_lane(const MoePlan& L, int tid) {
  const int len = L.S * kQBlockBytes;
  const int cpr = kAl ? len / 16 : (len + 29) / 16;  // lines a row, at most
  FillLane F;
  F.step = kProducers * 32 / cpr;
  F.rg = tid / cpr;
  F.c = tid - F.rg * cpr;
  if (F.rg >= F.step) F.rg = 1 << 20;  // (no rows)
  return F;
}

// Copies blocks [c0, c0 + nb) of n consecutive rows, the first at byte `off`
// of its matrix, into slots from `dst` on.  Rows start on any even byte
// unless kAl, so the copy covers the 16-byte lines a row touches (no byte
// past the matrix).
template <bool kAl>
__device__ __forceinline__ void fill_rows(const MoePlan& L, const FillLane& F, uint32_t dst, const uint8_t* base,
                                          long long off, int n, int c0, int nb, long long mat_bytes) {
  const int rb = L.bpr * kQBlockBytes, len = nb * kQBlockBytes;
  if (F.c * 16 >= (kAl ? len : len + 14)) return;
  const long long step = (long long)F.step * rb;
  const uint32_t dstep = (uint32_t)(F.step * L.SR);
  long long a = off + (long long)F.rg * rb + (long long)c0 * kQBlockBytes;
  dst += (uint32_t)(F.rg * L.SR + F.c * 16);
  if constexpr (kAl) {
    const uint8_t* src = base + a + F.c * 16;
#pragma unroll 4
    for (int r = F.rg; r < n; r += F.step) {
      cp16(dst, src, 16);
      src += step;
      dst += dstep;
    }
  } else {
    const long long last = mat_bytes - F.c * 16;
#pragma unroll 2
    for (int r = F.rg; r < n; r += F.step) {
      const long long lo = a & ~15LL, left = last - lo;
      if (left > 0) cp16(dst, base + lo + F.c * 16, left < 16 ? (int)left : 16);
      a += step;
      dst += dstep;
    }
  }
}

// One warp: blocks [c0, c0 + nb) of n <= 8 tokens' images (token i's at
// img(i)), a bulk copy each.
template <typename ImgFn>
__device__ __forceinline__ void fill_images(const MoePlan& L, uint8_t* dst, uint64_t* full, int n, int c0, int nb,
                                            ImgFn img, uint64_t pol, int lane) {
  const uint32_t bytes = (uint32_t)nb * kImgBlock;
  if (lane == 0) mbar_arrive_expect_tx(full, bytes * n);
  __syncwarp();
  if (lane < n) bulk_g2s(dst + lane * L.XR, img(lane) + (size_t)c0 * kImgBlock, bytes, full, pol);
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}

// What a lane reads of one block: its words of kTiles A tiles, their scales,
// its columns' operand and inverse scales.  All loads of a block are issued
// before its arithmetic (asm volatile keeps their order), and two blocks'
// before either's.
template <int kTiles>
struct BlockIn {
  uint32_t w[kTiles][2][3];  // row g or g + 8: word of step 0, words of step 1
  uint32_t d[kTiles][2];
  uint4 b0, b1;
  float xi0, xi1;
};

// kAl: words are aligned in odd blocks; an even block's word 7 is its first
// two and last two quants (tc::word_quant).  Otherwise a block starts at any
// even address, quants in order.
template <bool kAl, int kTiles>
__device__ __forceinline__ void load_block(const uint32_t (&ra)[kTiles][2], bool even, int c, uint32_t xa, uint32_t x0,
                                           uint32_t x1, BlockIn<kTiles>& B) {
  B.b0 = lds128(xa);
  B.b1 = lds128(xa + 64u);
#pragma unroll
  for (int t = 0; t < kTiles; ++t)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t ba = ra[t][h];
      B.d[t][h] = tc::lds16a(ba);
      if constexpr (kAl) {
        if (even) {
          B.w[t][h][0] = tc::lds32a(ba + 4u + 4u * c);
          B.w[t][h][1] = tc::lds32a(ba);
          B.w[t][h][2] = tc::lds32a(ba + (c == 3 ? 32u : 20u + 4u * c));
        } else {
          B.w[t][h][0] = tc::lds32a(ba + 2u + 4u * c);
          B.w[t][h][1] = tc::lds32a(ba + 18u + 4u * c);
        }
      } else {
        const uint32_t q = ba + 2u + 4u * c, a = q & ~3u, sel = (q & 2u) ? 0x5432u : 0x3210u;
        B.w[t][h][0] = __byte_perm(tc::lds32a(a), tc::lds32a(a + 4u), sel);
        B.w[t][h][1] = __byte_perm(tc::lds32a(a + 16u), tc::lds32a(a + 20u), sel);
      }
    }
  B.xi0 = tc::lds32f(x0 + 128u);
  B.xi1 = tc::lds32f(x1 + 128u);
}

// y[t] += the products of a loaded block: columns 2c and 2c + 1 of rows g
// ([0], [1]) and g + 8 ([2], [3]) of tile t.
template <bool kAl, int kTiles>
__device__ __forceinline__ void block_mma(const BlockIn<kTiles>& B, bool even, int c, float (&y)[kTiles][4]) {
#pragma unroll
  for (int t = 0; t < kTiles; ++t) {
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    uint32_t a0, a1, a2, a3;
    tc::quant_pairs(B.w[t][0][0], a0, a2);
    tc::quant_pairs(B.w[t][1][0], a1, a3);
    tc::mma_f16(acc, a0, a1, a2, a3, B.b0.x, B.b0.y);
    tc::mma_f16(acc, a0, a1, a2, a3, B.b0.z, B.b0.w);
    uint32_t w0 = B.w[t][0][1], w1 = B.w[t][1][1];
    if (kAl && even) {
      const uint32_t sel = c == 3 ? 0x5432u : 0x7654u;
      w0 = __byte_perm(w0, B.w[t][0][2], sel);
      w1 = __byte_perm(w1, B.w[t][1][2], sel);
    }
    tc::quant_pairs(w0, a0, a2);
    tc::quant_pairs(w1, a1, a3);
    tc::mma_f16(acc, a0, a1, a2, a3, B.b1.x, B.b1.y);
    tc::mma_f16(acc, a0, a1, a2, a3, B.b1.z, B.b1.w);
    const float d0 = f16_bits_to_f32(B.d[t][0]), d1 = f16_bits_to_f32(B.d[t][1]);
    y[t][0] = fmaf(d0 * B.xi0, acc[0], y[t][0]);
    y[t][1] = fmaf(d0 * B.xi1, acc[1], y[t][1]);
    y[t][2] = fmaf(d1 * B.xi0, acc[2], y[t][2]);
    y[t][3] = fmaf(d1 * B.xi1, acc[3], y[t][3]);
  }
}

// A warp's blocks first, first + step, .. < nb of a stage, two at a time.
// ro: where this lane's rows' blocks start (block 0), xl, x0, x1: its image
// words and its columns' images (block 0).
template <bool kAl, int kTiles>
__device__ __forceinline__ void stage_blocks(const uint32_t (&ro)[kTiles][2], uint32_t xl, uint32_t x0, uint32_t x1,
                                             int first, int step, int nb, int c, float (&y)[kTiles][4]) {
  const auto load = [&](int j, BlockIn<kTiles>& B) {
    uint32_t ra[kTiles][2];
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
      for (int h = 0; h < 2; ++h) ra[t][h] = ro[t][h] + (uint32_t)j * kQBlockBytes;
    const uint32_t xo = (uint32_t)j * kImgBlock;
    load_block<kAl, kTiles>(ra, !(j & 1), c, xl + xo, x0 + xo, x1 + xo, B);
  };
  for (int j = first; j < nb; j += 2 * step) {
    BlockIn<kTiles> A, B;
    const int j1 = j + step;
    load(j, A);
    if (j1 < nb) load(j1, B);
    block_mma<kAl, kTiles>(A, !(j & 1), c, y);
    if (j1 < nb) block_mma<kAl, kTiles>(B, !(j1 & 1), c, y);
  }
}

// Bounded wait that gives up when another thread of the CTA has.  (try_wait
// without a time hint: with one it polls through nanosleep, and twenty
// waiting warps then take the issue slots of those that work.)
__device__ __forceinline__ bool ring_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  for (uint32_t i = 0; i < kWaitLimit; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort) return false;
  }
  *abort = 1;
  return false;
}

// A place in the ring: stage s, filled for the ph-th time (parity).
struct Cursor {
  int s = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void next(int nst) {
    if (++s == nst) {
      s = 0;
      ph ^= 1u;
    }
  }
};

// One warp's wait on a barrier that lane 0 polls.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort, int lane) {
  const int ok = lane ? 1 : (ring_wait(bar, parity, abort) ? 1 : 0);
  return __all_sync(0xffffffffu, ok);
}

// After a wait gave up: the bulk copies of the last fills (of i) have landed.
__device__ __forceinline__ void drain(const MoePlan& L, const MoeShared& S, int i, volatile int* abort) {
  if (*abort)
    for (int j = max(0, i - L.nst); j < i; ++j) mbar_wait(&S.full[j % L.nst], (uint32_t)(j / L.nst) & 1u);
}

// Ends a product kernel: no copy is in flight when the CTA leaves, and a wait
// that gave up is reported.
__device__ __forceinline__ void finish(const MoeParams& P, volatile int* abort) {
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
  if (threadIdx.x == 0 && *abort && P.d_err) atomicOr(P.d_err, Q8D_DERR_WAIT);
}

constexpr int kGuWarps = 16, kGuK = 8;  // consumer warps; over the blocks of a row
constexpr int kGuRows = 32;             // h rows a unit
constexpr int kGuTiles = 2;             // A tiles (8 gate + 8 up rows) a warp

template <bool kAl>
__global__ void __launch_bounds__((kGuWarps + kProducers) * 32, 1)
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
  if (warp >= kGuWarps) {
    const int tid = threadIdx.x - kGuWarps * 32;
    const int rb = L.bpr * kQBlockBytes;
    const long long mat = (long long)P.n_experts * P.ffn * rb;
    const uint32_t smem32 = smem_u32(smem);
    const FillLane F = fill_lane<kAl>(L, tid);
    const bool first = warp == kGuWarps;
    const uint64_t keep = policy_evict_last();
    fence_proxy_async_global();  // (the images were written by ordinary stores)
    Cursor R;
    int issued = 0;
    bool ok = true;
    for (int q = q0, it = q0 / nq; q < q1 && ok; ++q) {
      if (q >= (it + 1) * nq) ++it;
      const int2 I = S.item[it];
      const long long r0 = ((long long)(I.x & 0xffff) * P.ffn + (long long)(q - it * nq) * kGuRows) * rb;
      for (int sl = 0; sl < L.nsl; ++sl, ++issued, R.next(L.nst)) {
        const int s = R.s;
        if (issued >= L.nst) ok = warp_wait(&S.empty[s], R.ph ^ 1u, &s_abort, lane);
        if (!ok) break;
        const uint32_t st = smem32 + (uint32_t)s * (uint32_t)L.stage_bytes;
        const int c0 = sl * L.S, nb = min(L.S, L.bpr - c0);
        if (first)
          fill_images(L, smem + (size_t)s * L.stage_bytes + L.slots * L.SR, &S.full[s], I.x >> 16, c0, nb,
                      [&](int n) { return P.ximg + (size_t)S.ptok[I.y + n] * L.bpr * kImgBlock; }, keep, lane);
        fill_rows<kAl>(L, F, st, P.wg, r0, kGuRows, c0, nb, mat);
        fill_rows<kAl>(L, F, st + (uint32_t)(kGuRows * L.SR), P.wu, r0, kGuRows, c0, nb, mat);
        cp_arrive(&S.full[s]);
      }
    }
    if (first) drain(L, S, issued, &s_abort);
  } else {
    const int gq = lane >> 2, cq = lane & 3;
    const int kb = warp % kGuK, th = warp / kGuK;  // blocks kb, kb + 8, ..; tiles 2 th, 2 th + 1
    const uint32_t smem32 = smem_u32(smem);
    const uint32_t xoff = (uint32_t)(L.slots * L.SR);
    const uint32_t xl = xoff + (uint32_t)(min(gq, L.tg - 1) * L.XR + cq * 16);
    const uint32_t x0 = xoff + (uint32_t)(min(2 * cq, L.tg - 1) * L.XR);
    const uint32_t x1 = xoff + (uint32_t)(min(2 * cq + 1, L.tg - 1) * L.XR);
    float* hq = reinterpret_cast<float*>(smem + L.o_hq);  // [32 rows][8 tokens + 1]
    Cursor R;
    for (int q = q0, it = q0 / nq; q < q1; ++q) {
      if (q >= (it + 1) * nq) ++it;
      const int2 I = S.item[it];
      const int ntok = I.x >> 16;
      const long long r0 = (long long)(I.x & 0xffff) * P.ffn + (long long)(q - it * nq) * kGuRows;
      float y[kGuTiles][4];
#pragma unroll
      for (int t = 0; t < kGuTiles; ++t) y[t][0] = y[t][1] = y[t][2] = y[t][3] = 0.f;
      // this lane's slots, and how far into its first line each row starts
      uint32_t ro[kGuTiles][2], mis[kGuTiles];
#pragma unroll
      for (int t = 0; t < kGuTiles; ++t) {
        const int r = (2 * th + t) * 8 + gq;
        mis[t] = kAl ? 0u : (uint32_t)(((r0 + r) * (L.bpr * kQBlockBytes)) & 15);
        ro[t][0] = (uint32_t)(r * L.SR);
        ro[t][1] = (uint32_t)((kGuRows + r) * L.SR);
      }
      for (int sl = 0; sl < L.nsl; ++sl, R.next(L.nst)) {
        const int s = R.s;
        ring_wait(&S.full[s], R.ph, &s_abort);
        const uint32_t st = after_wait(smem32 + (uint32_t)s * (uint32_t)L.stage_bytes);
        const int c0 = sl * L.S, nb = min(L.S, L.bpr - c0);
        uint32_t ra[kGuTiles][2];
#pragma unroll
        for (int t = 0; t < kGuTiles; ++t) {
          const uint32_t o = st + (kAl ? 0u : (mis[t] + (uint32_t)c0 * kQBlockBytes) & 15u);
          ra[t][0] = ro[t][0] + o;
          ra[t][1] = ro[t][1] + o;
        }
        stage_blocks<kAl, kGuTiles>(ra, st + xl, st + x0, st + x1, kb, kGuK, nb, cq, y);
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
        image_word(v, n < ntok, P.himg + ((size_t)(I.y + n) * nq + b) * kImgBlock, w);
      }
    }
  }
  finish(P, &s_abort);
}

constexpr int kDnMaxWarps = 16;

template <bool kAl, int kTiles>
__global__ void __launch_bounds__((kDnMaxWarps + kProducers) * 32, 1) moe_down_kernel(const MoeParams P, const MoePlan L) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int s_abort;
  MoeShared S = carve(L, smem, P.m * P.top_k);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, W = L.W;
  if (threadIdx.x == 0) s_abort = 0;
  group_pairs(P, L, S);  // (the choice is complete: the gate / up kernel started behind it)
  const int chunks = (P.hidden + L.rows - 1) / L.rows;
  const int per = S.n_items * L.nsl;  // stages a chunk of rows
  const int mine = blockIdx.x < chunks ? (chunks - blockIdx.x + gridDim.x - 1) / gridDim.x : 0;
  const int total = mine * per;
  if (warp >= W) {
    const int tid = threadIdx.x - W * 32;
    const int rb = L.bpr * kQBlockBytes;
    const long long mat = (long long)P.n_experts * P.hidden * rb;
    const uint32_t smem32 = smem_u32(smem);
    const FillLane F = fill_lane<kAl>(L, tid);
    const bool first = warp == W;
    const uint64_t keep = policy_evict_last();
    // a place in this CTA's sequence of stages: chunk of rows, item, slice
    struct Place {
      Cursor R;
      int ch, it = 0, sl = 0;
      __device__ void next(const MoePlan& L, int items) {
        R.next(L.nst);
        if (++sl == L.nsl) {
          sl = 0;
          if (++it == items) {
            it = 0;
            ch += gridDim.x;
          }
        }
      }
    };
    const auto weights = [&](const Place& p) {
      const int c0 = p.sl * L.S, r0 = p.ch * L.rows;
      fill_rows<kAl>(L, F, smem32 + (uint32_t)p.R.s * (uint32_t)L.stage_bytes, P.wd,
                     ((long long)(S.item[p.it].x & 0xffff) * P.hidden + r0) * rb, min(L.rows, P.hidden - r0), c0,
                     min(L.S, L.bpr - c0), mat);
      cp_arrive(&S.full[p.R.s]);
    };
    const auto images = [&](const Place& p) {
      const int c0 = p.sl * L.S;
      const int2 I = S.item[p.it];
      fill_images(L, smem + (size_t)p.R.s * L.stage_bytes + L.slots * L.SR, &S.full[p.R.s], I.x >> 16, c0,
                  min(L.S, L.bpr - c0),
                  [&](int n) { return P.himg + (size_t)(I.y + n) * L.bpr * kImgBlock; }, keep, lane);
    };
    // Weights depend on nothing in flight: the first ring of them comes while
    // the gate / up kernel ends.
    const int ring = min(total, L.nst);
    Place w, x;
    w.ch = x.ch = blockIdx.x;
    int i = 0;
    for (; i < ring; ++i, w.next(L, S.n_items)) weights(w);
    griddep_wait();  // (h)
    fence_proxy_async_global();
    if (first)
      for (int k = 0; k < ring; ++k, x.next(L, S.n_items)) images(x);
    for (; i < total; ++i, w.next(L, S.n_items)) {
      if (!warp_wait(&S.empty[w.R.s], w.R.ph ^ 1u, &s_abort, lane)) break;
      if (first) images(w);
      weights(w);
    }
    if (first) drain(L, S, i, &s_abort);
  } else {
    griddep_wait();
    const int gq = lane >> 2, cq = lane & 3;
    const uint32_t smem32 = smem_u32(smem);
    const uint32_t xoff = (uint32_t)(L.slots * L.SR);
    const uint32_t xl = xoff + (uint32_t)(min(gq, L.tg - 1) * L.XR + cq * 16);
    const uint32_t x0 = xoff + (uint32_t)(min(2 * cq, L.tg - 1) * L.XR);
    const uint32_t x1 = xoff + (uint32_t)(min(2 * cq + 1, L.tg - 1) * L.XR);
    const int yp = P.m | 1;                                 // table pitch (odd: rows in distinct banks)
    float* tab = S.part + (size_t)warp * L.mt * 16 * yp;    // this warp's [rows][tokens]
    Cursor R;
    for (int ch = blockIdx.x; ch < chunks; ch += gridDim.x) {
      const int r0 = ch * L.rows, nr = min(L.rows, P.hidden - r0);
      for (int i = lane; i < L.mt * 16 * yp; i += 32) tab[i] = 0.f;
      __syncwarp();
      for (int it = 0; it < S.n_items; ++it) {
        const int2 I = S.item[it];
        const int ntok = I.x >> 16;
        const long long e0 = (long long)(I.x & 0xffff) * P.hidden + r0;
        float y[kTiles][4];
#pragma unroll
        for (int t = 0; t < kTiles; ++t) y[t][0] = y[t][1] = y[t][2] = y[t][3] = 0.f;
        for (int sl = 0; sl < L.nsl; ++sl, R.next(L.nst)) {
          const int s = R.s;
          ring_wait(&S.full[s], R.ph, &s_abort);
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
          stage_blocks<kAl, kTiles>(ro, st + xl, st + x0, st + x1, warp, W, nb, cq, y);
          __syncwarp();
          if (lane == 0) mbar_arrive(&S.empty[s]);
        }
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
  finish(P, &s_abort);
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

// Tokens a group: about twice an expert's share of the (token, slot) pairs,
// a power of two up to 8 (an expert with more is read once a group; with
// fewer, its stage space idles).
int group_tokens(const MoeParams& P) {
  const int want = std::min(P.m, 2 * P.m * P.top_k / P.n_experts + 2);
  int tg = 1;
  while (tg < 8 && tg < want) tg *= 2;
  return tg;
}

// Slices of S blocks, tokens and stage of a plan whose slots are set.
void plan_stage(const MoeParams& P, int S, bool al, int tg, MoePlan* L) {
  L->S = S;
  L->nsl = (L->bpr + S - 1) / S;
  L->S = (L->bpr + L->nsl - 1) / L->nsl;  // (equal slices; whole groups of 8 blocks where rows are aligned)
  if (al) L->S = (L->S + 7) / 8 * 8;
  L->SR = slot_bytes(L->S, al);
  // token rows half a bank cycle apart: the two tokens of a quarter warp's
  // 16-byte loads lie in distinct banks
  L->XR = (L->S * kImgBlock + 127) / 128 * 128 + 64;
  L->tg = tg;
  L->stage_bytes = L->slots * L->SR + tg * L->XR;
  const int pairs = P.m * P.top_k;
  L->items = std::min(pairs, P.n_experts + pairs / tg);
}

// Offsets behind a ring of nst stages; sets smem.
void plan_rest(const MoeParams& P, int nst, int part_floats, int hq_floats, MoePlan* L) {
  const int pairs = P.m * P.top_k;
  L->nst = nst;
  int o = nst * L->stage_bytes;
  L->o_part = o;
  o += up16i(4 * part_floats);
  L->o_hq = o;
  o += up16i(4 * hq_floats);
  L->o_mask = o;
  o += 8 * P.n_experts;
  L->o_ebase = o;
  o = up16i(o + 4 * P.n_experts);
  L->o_item = o;
  o += 8 * L->items;
  L->o_tok = o = up16i(o);
  o += up16i(5 * pairs);
  L->o_bar = o;
  L->smem = o + 16 * nst;
}

// As many stages as fit, at least `least`.
bool plan_ring(const MoeParams& P, int least, int most, int part_floats, int hq_floats, MoePlan* L) {
  plan_rest(P, 0, part_floats, hq_floats, L);
  const int n = L->smem < kMaxSmem ? std::min(most, (kMaxSmem - L->smem) / (L->stage_bytes + 16)) : 0;
  if (n < least) return false;
  plan_rest(P, n, part_floats, hq_floats, L);
  return true;
}

int plan_gate_up(const MoeParams& P, MoePlan* L) {
  const bool al = P.hidden / kQBlock % 8 == 0;
  L->bpr = P.hidden / kQBlock;
  L->W = kGuWarps;
  L->slots = 2 * kGuRows;
  L->rows = kGuRows;
  L->mt = 4;
  // two blocks a warp in a stage, or one where that leaves fewer than three
  // stages
  for (int tg = group_tokens(P); tg >= 1; tg /= 2)
    for (int s = std::min(16, L->bpr); s >= std::min(8, L->bpr); s = s > 8 ? 8 : s - 1) {
      plan_stage(P, s, al, tg, L);
      if (plan_ring(P, 3, 8, kGuK * 4 * 128, kGuRows * 9, L)) return Q8D_OK;
    }
  return Q8D_EUNSUPPORTED;
}

int plan_down(const MoeParams& P, int sms, MoePlan* L) {
  const bool al = P.ffn / kQBlock % 8 == 0;
  L->bpr = P.ffn / kQBlock;
  // Few blocks a row: eight warps, since every warp pays for an item's
  // bookkeeping; long rows: as many as split them evenly.
  const int bpr = L->bpr;
  int W = 8;
  double best = 0.0;
  if (bpr >= 48)
    for (int w = kDnMaxWarps; w >= 12; --w) {
      const double eff = (double)bpr / (w * ((bpr + w - 1) / w));
      if (eff > best + 1e-9) {
        best = eff;
        W = w;
      }
    }
  for (int tg = group_tokens(P); tg >= 1; tg /= 2)
    for (int w = W; w >= 8; w -= w > 8 ? w - 8 : 1)
      for (int most = 32; most >= 16; most -= 16) {
        // rows a CTA: an equal share of the output, in as few passes as
        // `most` rows at a time allow
        const int passes = (P.hidden + sms * most - 1) / (sms * most);
        L->W = w;
        L->rows = std::min(most, (P.hidden + sms * passes - 1) / (sms * passes));
        L->mt = L->rows > 16 ? 2 : 1;
        L->slots = L->mt * 16;
        const int table = w * L->slots * (P.m | 1);
        for (int s = std::min(bpr, 56); s >= std::min(bpr, 8); s -= 8) {  // (a row's lines: a producer thread each)
          plan_stage(P, s, al, tg, L);
          if (plan_ring(P, 4, 12, table, 0, L)) return Q8D_OK;
        }
      }
  return Q8D_EUNSUPPORTED;
}

}  // namespace

size_t moe_workspace_bytes(int m, int hidden, int ffn, int n_experts, int top_k) {
  (void)n_experts;
  const size_t pairs = (size_t)m * top_k;
  return up16(4 * pairs) * 2 + (size_t)m * (hidden / kQBlock) * kImgBlock + pairs * (ffn / kQBlock) * kImgBlock;
}

int moe_launch(MoeParams P, void* workspace, cudaStream_t stream) {
  const size_t pairs = (size_t)P.m * P.top_k;
  const int bx = P.hidden / kQBlock, bh = P.ffn / kQBlock;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  P.ximg = ws;
  ws += (size_t)P.m * bx * kImgBlock;
  P.himg = ws;
  ws += pairs * bh * kImgBlock;
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
  rc = launch_ex(gu_fn, dim3(sms), dim3((gu.W + kProducers) * 32), (size_t)gu.smem, stream, true, P, gu, dal);
  if (rc) return rc;
  const int chunks = (P.hidden + dn.rows - 1) / dn.rows;
  return launch_ex(dn_fn, dim3(std::min(sms, chunks)), dim3((dn.W + kProducers) * 32), (size_t)dn.smem, stream, true, P, dn);
}

}  // namespace q8d
