// A mixture-of-experts feed-forward layer over Q8_0 experts for a few tokens,
// in four launches that overlap (programmatic dependents):
//  1. router: logits, choice and weights, and the tokens' operand image;
//  2. gate / up: h = silu(Wg x) * (Wu x) of every (token, chosen expert);
//  3. down: w * Wd h of every (token, chosen expert);
//  4. y = residual + the sum of a token's experts' rows.
//
// What bounds it is reading the chosen experts' matrices once from HBM: with
// m tokens choosing k of E, 2 and 3 stream about E (1 - (1 - k/E)^m) experts
// of 34 bytes a block of 32, and a token adds only a column to each product.
// So both are streaming kernels: producer warps keep a ring of shared memory
// stages filled, and sixteen consumer warps multiply with mma.sync m16n8k16.
//  * A: sixteen weight rows, a lane's word of four quants made two exact f16
//    pairs (one PRMT and one subtraction a pair); B: the expert's tokens;
//    the warps split the blocks of a row.
//  * The tokens' values are f16 hi + lo under a power-of-two scale for each
//    block of 32 (the scheme of q8d_mma_frag.cuh): products are exact in f32
//    and a block's sum is scaled once by weight scale * inverse scale, so
//    results are f32-accurate.
//  * Whoever makes the values writes them in the operand's order: the router
//    kernel for x, the gate / up epilogue for h (it owns whole blocks of 32
//    rows), 16 bytes {hi01, hi23, lo01, lo23} a word, 144 a block with its
//    inverse scale, so the products copy them beside the weights and never
//    convert.
//  * A work unit is 64 slots of rows of one expert (32 gate and 32 up rows,
//    or 64 down rows) for a group of its tokens: four A tiles.  Units are
//    dealt to the CTAs in contiguous ranges; experts nobody chose are not
//    touched (but for the rows behind a last down unit of half the rows, which
//    a tensor copy brings along).  (Giving each CTA a few output rows of every expert instead
//    saves launch 4 but has every CTA fetch every h, 2.3 bytes for one of
//    weights at 64 tokens, and one tile per B load: 118 against 62 us for
//    the down products of 128 experts of 2048 x 768.)
//  * How rows come depends on where they lie.  Whole 16-byte lines (a
//    multiple of 8 blocks): a TMA tensor copy brings 8 blocks of 32 or 64
//    rows, 272 bytes a row, so rows lie 4 (mod 32) banks apart and eight
//    rows' words in distinct banks without padding; an image's slice comes
//    with them.  Else, up to 64 blocks: rows are contiguous, so a stage's are
//    one bulk copy a matrix, and the images stay in shared memory for all
//    units of an item (fetched with every stage they were up to twice the
//    weights' bytes, and rows copied singly were bound by the copies' issue:
//    21 tokens, 2560 x 1120, 7 of 64 experts, 183 us for the layer, now 137;
//    27 tokens, 1376 x 160, 6 of 128, 81, now 47).  Longer rows: a bulk copy
//    each into padded slots, in slices whose images serve four tiles.
//  * Sums are taken in a fixed order throughout and nothing is added to
//    memory atomically: the same bits every time.
// 64 tokens, 2048 x 768, 8 of 128 experts (630 MB of weights): router 14, gate
// / up 104, down and sum 53 us.  The gate / up products alone would take 82 us
// (55 percent of the issue slots at 20 warps an SM) and their copies alone 75
// (weights and images, 650 MB through L2); they share shared memory and the
// issue slots, and 104 is what both take.
#include <cuda.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <mutex>
#include <type_traits>

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
// FMA) and the sum's (Knuth's TwoSum) go to c, the compensated dot product of
// Ogita, Rump and Oishi, so s + c carries about 48 bits.  (f64
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
  const float w = lane < P.top_k ? ex(mine) : 0.f;
  // the sum of the chosen, or of all, in two parts
  float sum = P.norm ? w : 0.f, sum2 = 0.f;
  bool bad = isnan(top.x) || isinf(top.x);
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (lane + 32 * i < E) {
      if (!P.norm) add_pair(sum, sum2, ex(lane + 32 * i), 0.f);
      bad = bad || isnan(logits[lane + 32 * i].x);
    }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float a = __shfl_xor_sync(0xffffffffu, sum, o), a2 = __shfl_xor_sync(0xffffffffu, sum2, o);
    add_pair(sum, sum2, a, a2);
  }
  bad = __any_sync(0xffffffffu, bad);  // (then the softmax is NaN throughout)
  if (lane < P.top_k) {
    P.experts[t * P.top_k + lane] = mine;
    P.weights[t * P.top_k + lane] = bad ? __int_as_float(0x7fc00000) : __fdiv_rn(w, sum + sum2);
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
  constexpr int kAhead = kT * kE == 1 ? 4 : kT * kE == 2 ? 2 : 1;  // loads in flight (64 registers)
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
__global__ void __launch_bounds__(kRtThreads, 2) moe_router_kernel(const MoeParams P, int per_cluster, bool perm) {
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
  if constexpr (kT == 1)  // (two experts at once share a token's loads; with two tokens they spill)
    for (; e + kWarps < e1; e += 2 * kWarps) logits_of<kT, 2>(P, t0, nt, e, kWarps, e1, logits, lane);
  for (; e < e1; e += kWarps) logits_of<kT, 1>(P, t0, nt, e, kWarps, e1, logits, lane);
  cluster_sync();  // the logits are complete
  if (rank > 0) {
    // meanwhile the others make the tokens' operand images, a word a thread
    const int bpr = P.hidden / kQBlock, words = nt * bpr * 8;
    for (int i0 = (rank - 1) * kRtThreads + warp * 32; i0 < words; i0 += (kRtCluster - 1) * kRtThreads) {
      const int i = i0 + lane, ii = min(i, words - 1);
      const int t = ii / (bpr * 8), b = (ii >> 3) - t * bpr, w = ii & 7;
      float v[4];
      const float* x = P.X + (size_t)(t0 + t) * P.ldx + (size_t)b * kQBlock;
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = x[tc::word_quant(perm && !(b & 1), w, k)];
      image_word(v, i < words, P.ximg + ((size_t)(t0 + t) * bpr + b) * kImgBlock, w);
    }
  } else if (warp < nt) {
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

// Producer warps.  With tensor copies the first brings the weights, the others
// the images; else each brings a quarter of the rows and of the images.
constexpr int kProducers = 4;
constexpr int kSlots = 64;   // row slots of a stage
constexpr int kTiles = 4;    // A tiles of a unit: a warp multiplies all four with its blocks
constexpr int kGuRows = 32;  // h rows of a gate / up unit: one block of the down products' rows
constexpr int kSubBytes = kSlots * 8 * kQBlockBytes;  // 64 row slots of 8 blocks

// How a matrix's rows come.
constexpr int kRowCopies = 0;   // a bulk copy a row and slice, into padded slots
constexpr int kTensor = 1;      // tensor copies of 8 blocks by 32 or 64 rows
constexpr int kContiguous = 2;  // whole rows, one bulk copy a matrix and stage

// How a product kernel lays out its shared memory (host plan).
struct MoePlan {
  int mode;         // kRowCopies ..
  int bpr;          // blocks a row
  int S, nsl;       // blocks a slice, slices a row
  int stages;       // of a unit: a slice each (tensor copies), a tile and slice each (rows), or `tr` tiles each
  int tr, lq;       // tiles a stage; log2 of the rows between a tile's rows g and g + 1
  int SR;           // slot bytes (tensor copies: of 8 blocks)
  int x_off;        // the images' offset in a stage
  int tg, lg;       // tokens a group (1, 2, 4, 8 or 16), log2 of it
  float inv_k;      // 1 / top_k
  int XR;           // image bytes a token of a stage, or of a buffer
  int img_bytes;    // an image buffer beside the ring (0: images lie in the stages)
  int stage_bytes, nst;
  int items;        // (expert, token group) pairs at most
  int o_img, o_part, o_hq, o_mask, o_ebase, o_item, o_tok, o_bar;  // offsets
  int smem;
};

struct MoeShared {
  uint8_t* smem;
  float* part;
  unsigned long long* mask;  // [E] tokens of an expert
  int* ebase;                // [E] first item (low half) and first row (high half)
  int2* item;                // (expert | tokens << 16, first row)
  float* pw;                 // [pairs] weight of a row
  unsigned short* ppair;     // [pairs] pair (token * top_k + slot) of a row
  unsigned short* ptok;      // [pairs] its token
  uint64_t *full, *empty;    // [nst]
  uint64_t *ifull, *iempty;  // [4] image buffers beside the ring
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
  S.ppair = reinterpret_cast<unsigned short*>(S.pw + pairs);
  S.ptok = S.ppair + pairs;
  S.full = reinterpret_cast<uint64_t*>(smem + L.o_bar);
  S.empty = S.full + L.nst;
  S.ifull = S.empty + L.nst;
  S.iempty = S.ifull + 4;
  S.n_items = 0;
  return S;
}

constexpr int kConsumers = 16;                              // consumer warps
// Two groups of eight warps work on two units at a time, each with its own
// sums and barriers: warps of one unit load, decode and multiply at about the
// same time, so the other group's keep the pipes they do not use busy, and
// one group's epilogue overlaps the other's products.  The stages of the two
// units alternate, so a stage of the ring always belongs to the same group (a
// barrier's parity tells two neighbouring phases apart, no more).
constexpr int kGroups = 2, kGroupWarps = kConsumers / kGroups, kGroupThreads = kGroupWarps * 32;
constexpr int kThreads = (kConsumers + kProducers) * 32;
static_assert(2 * kMoeMaxTokens * kMoeMaxTop <= kConsumers * kSlots * 8, "the pairs fit the sums' space");

// The barriers and the experts' masks, before anything is waited for.  The
// whole CTA calls.
__device__ __forceinline__ void start(const MoeParams& P, const MoePlan& L, const MoeShared& S) {
  for (int e = threadIdx.x; e < P.n_experts; e += kThreads) S.mask[e] = 0ull;
  // (the barriers lie one behind the other: a thread each)
  const int i = threadIdx.x, full = L.mode == kContiguous ? 1 : kProducers;
  if (i < 2 * L.nst + 8) {
    const int group = L.mode == kContiguous && i >= 2 * L.nst ? kConsumers : kGroupWarps;
    mbar_init(&S.full[i], i < L.nst || (i >= 2 * L.nst && i < 2 * L.nst + 4) ? full : group);
    fence_barrier_init();
  }
  __syncthreads();
}

// Groups the (token, slot) pairs by expert, in every CTA alike: experts in
// order, an expert's tokens in order; a pair's row is its place in that
// order.  (One token: a pair is an item, in the order of the choice.)  The
// whole CTA calls.
__device__ void group_pairs(const MoeParams& P, const MoePlan& L, MoeShared& S) {
  __shared__ int s_items;
  const int pairs = P.m * P.top_k, E = P.n_experts;
  if (P.m == 1) {
    const int p = threadIdx.x;
    if (p < pairs) {
      S.item[p] = make_int2(__ldcg(P.experts + p) | 1 << 16, p);
      S.pw[p] = __ldcg(P.weights + p);
      S.ppair[p] = (unsigned short)p;
      S.ptok[p] = 0;
    }
    __syncthreads();
    S.n_items = pairs;
    return;
  }
  // (loops are kept rolled: code that runs once costs its fetch)
  const auto token = [&](int p) { return (int)(((float)p + 0.5f) * L.inv_k); };
  int* pe = reinterpret_cast<int*>(S.part);  // (the sums' space is free so far)
  float* pw = S.part + pairs;
#pragma unroll 1
  for (int p = threadIdx.x; p < pairs; p += kThreads) {
    const int e = __ldcg(P.experts + p);
    pw[p] = __ldcg(P.weights + p);
    pe[p] = e;
    atomicOr(&S.mask[e], 1ull << token(p));
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x, per = (E + 31) / 32, e0 = lane * per, e1 = min(E, e0 + per);
    int x = 0;  // items | rows << 16 (both fit 12 bits)
#pragma unroll 1
    for (int e = e0; e < e1; ++e) {
      const int c = __popcll(S.mask[e]);
      x += ((c + L.tg - 1) >> L.lg) | c << 16;
    }
    int incl = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    x = incl - x;
#pragma unroll 1
    for (int e = e0; e < e1; ++e) {
      S.ebase[e] = x;
#pragma unroll 1
      for (int c = __popcll(S.mask[e]); c > 0; c -= L.tg) {
        const int n = min(L.tg, c);
        S.item[x & 0xffff] = make_int2(e | n << 16, x >> 16);
        x += 1 | n << 16;
      }
    }
    if (lane == 31) s_items = incl & 0xffff;
  }
  __syncthreads();
#pragma unroll 1
  for (int p = threadIdx.x; p < pairs; p += kThreads) {
    const int e = pe[p], tok = token(p);
    const int row = (S.ebase[e] >> 16) + __popcll(S.mask[e] & ((1ull << tok) - 1ull));
    S.ptok[row] = (unsigned short)tok;
    S.ppair[row] = (unsigned short)p;
    S.pw[row] = pw[p];
  }
  __syncthreads();
  S.n_items = s_items;
}

__device__ __forceinline__ uint32_t token_off(int XR, int t) { return (uint32_t)(t * XR + (t >> 1) * 16); }

// Rows [y, y + box) of blocks x / 68 .. of a matrix (box: the tensor map's).
__device__ __forceinline__ void tensor_g2s(uint32_t dst, const CUtensorMap* map, int x, int y, uint64_t* bar,
                                           uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint "
      "[%0], [%1, {%2, %3}], [%4], %5;" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}

// One warp: blocks [c0, c0 + nb) of the images of tokens first, first + step,
// .. < n (token i's at img(i)), a bulk copy each, announced by the caller.
template <typename ImgFn>
__device__ __forceinline__ void bulk_images(const MoePlan& L, uint8_t* dst, uint64_t* full, int first, int step, int n,
                                            int c0, int nb, ImgFn img, uint64_t pol, int lane) {
  const int i = first + lane * step;
  if (i < n)
    bulk_g2s(dst + token_off(L.XR, i), img(i) + (size_t)c0 * kImgBlock, (uint32_t)nb * kImgBlock, full, pol);
}

// The 16-byte lines that blocks [c0, c0 + nb) of a row touch: rows start on
// any even byte (off: the row's start in its matrix).  A matrix of 32 n rows
// ends with a line.
struct RowLines {
  long long lo;    // the first line's start
  uint32_t bytes;
};
__device__ __forceinline__ RowLines row_lines(long long off, int c0, int nb) {
  RowLines R;
  const long long a = off + (long long)c0 * kQBlockBytes;
  R.lo = a & ~15LL;
  R.bytes = (uint32_t)(((a + (long long)nb * kQBlockBytes + 15) & ~15LL) - R.lo);
  return R;
}

// Shared loads at an immediate offset: the blocks' words lie at constant
// distances, and an address register each would cost an addition a load.
template <int OFF>
__device__ __forceinline__ uint4 lds128i(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4+%5];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a), "n"(OFF));
  return v;
}
template <int OFF>
__device__ __forceinline__ uint2 lds64i(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0,%1}, [%2+%3];" : "=r"(v.x), "=r"(v.y) : "r"(a), "n"(OFF));
  return v;
}
template <int OFF>
__device__ __forceinline__ uint32_t lds32i(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1+%2];" : "=r"(v) : "r"(a), "n"(OFF));
  return v;
}
template <int OFF>
__device__ __forceinline__ uint32_t lds16i(uint32_t a) {
  unsigned short v;
  asm volatile("ld.shared.b16 %0, [%1+%2];" : "=h"(v) : "r"(a), "n"(OFF));
  return v;
}

// How a product's columns hold an item's tokens.
constexpr int kPacked = 0;  // up to four: columns 0-3 their hi parts, 4-7 their lo parts
constexpr int kEight = 1;   // up to eight, hi and lo an MMA each
constexpr int kSixteen = 2; // up to sixteen: two column tiles share every decoded A
constexpr int col_tiles(int cols) { return cols == kSixteen ? 2 : 1; }

// What a lane reads of one block: words and scales of kN A tiles; and its
// columns' operand and inverse scales.  All loads of a piece are issued
// before its arithmetic (asm volatile keeps their order).
template <int kN>
struct RowsIn {
  uint32_t w[kN][2][3];  // row g or g + 8: words of steps 0 and 1, the scale (even blocks: and quants 0, 1)
};
template <int kCols>
struct ColsIn {
  uint32_t b[col_tiles(kCols)][2][kCols == kPacked ? 2 : 4];
  float xi[col_tiles(kCols)][2];
};

// xa: this lane's column's words, x0 and x1: the images whose inverse scales
// its results take; of each column tile.
template <int kCols>
__device__ __forceinline__ void load_x(uint32_t xo, const uint32_t (&xa)[col_tiles(kCols)],
                                       const uint32_t (&x0)[col_tiles(kCols)], const uint32_t (&x1)[col_tiles(kCols)],
                                       ColsIn<kCols>& B) {
#pragma unroll
  for (int i = 0; i < col_tiles(kCols); ++i) {
    if constexpr (kCols == kPacked) {
      const uint2 u = lds64i<0>(xo + xa[i]), v = lds64i<64>(xo + xa[i]);
      B.b[i][0][0] = u.x, B.b[i][0][1] = u.y;
      B.b[i][1][0] = v.x, B.b[i][1][1] = v.y;
    } else {
      const uint4 u = lds128i<0>(xo + xa[i]), v = lds128i<64>(xo + xa[i]);
      B.b[i][0][0] = u.x, B.b[i][0][1] = u.y, B.b[i][0][2] = u.z, B.b[i][0][3] = u.w;
      B.b[i][1][0] = v.x, B.b[i][1][1] = v.y, B.b[i][1][2] = v.z, B.b[i][1][3] = v.w;
    }
    B.xi[i][0] = __uint_as_float(lds32i<128>(xo + x0[i]));
    B.xi[i][1] = __uint_as_float(lds32i<128>(xo + x1[i]));
  }
}

// Slot of row g + 8 h of tile t, less g.
template <bool kGate>
__host__ __device__ constexpr int slot_of(int t, int h) {
  return kGate ? kGuRows * h + 8 * t : 16 * t + 8 * h;
}

// Rows from tensor copies: 272 bytes a slot, so that a slot is an immediate
// offset.  bg: block start in slot g.  Words are aligned in odd blocks; an
// even block's word 7 is its first two and last two quants (tc::word_quant).
// Tiles T0 .. T0 + kN - 1.
template <bool kGate, int T0, int kN, int I = 0>
__device__ __forceinline__ void load_aligned(uint32_t bg, bool even, int c, RowsIn<kN>& B) {
  if constexpr (I < 2 * kN) {
    constexpr int t = I / 2, h = I % 2, so = slot_of<kGate>(T0 + t, h) * 8 * kQBlockBytes;
    if (even) {
      B.w[t][h][0] = lds32i<so + 4>(bg + 4u * c);
      B.w[t][h][1] = lds32i<so>(bg + (c == 3 ? 32u : 20u + 4u * c));
      B.w[t][h][2] = lds32i<so>(bg);
    } else {
      B.w[t][h][0] = lds32i<so + 2>(bg + 4u * c);
      B.w[t][h][1] = lds32i<so + 18>(bg + 4u * c);
      B.w[t][h][2] = lds16i<so>(bg);
    }
    load_aligned<kGate, T0, kN, I + 1>(bg, even, c, B);
  }
}
// Other rows: a block starts at any even address, quants in order.
__device__ __forceinline__ void load_unaligned(uint32_t ba, int h, int c, RowsIn<1>& B) {
  const uint32_t q = ba + 2u + 4u * c, a = q & ~3u, sel = (q & 2u) ? 0x5432u : 0x3210u;
  const uint32_t w0 = lds32i<0>(a), w1 = lds32i<4>(a), w4 = lds32i<16>(a), w5 = lds32i<20>(a);
  B.w[0][h][2] = lds16i<0>(ba);
  B.w[0][h][0] = __byte_perm(w0, w1, sel);
  B.w[0][h][1] = __byte_perm(w4, w5, sel);
}

// The unit's row that slot (tile t, half h, row g) holds.  Tensor and row
// copies: in order (gate: h is the matrix).  Whole rows lie bpr * 34 bytes
// apart, which puts eight rows' words into few banks for many widths, so
// there a tile takes every 2^lq-th row of the stage.
template <bool kGate>
__device__ __forceinline__ int slot_row(const MoePlan& L, int t, int h, int g) {
  const int tt = t & (L.tr - 1), s = kGate ? tt : 2 * tt + h;
  return (t - tt) * (kGate ? 8 : 16) + ((s >> L.lq) << (3 + L.lq)) + (g << L.lq) + (s & ((1 << L.lq) - 1));
}

__device__ __forceinline__ void mma_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// y[t] += the products of a loaded block: columns 2c and 2c + 1 of rows g
// ([0]) and g + 8 ([1]) of tile t, of each column tile.
template <bool kAl, int kCols, int T0, int kN, int kT>
__device__ __forceinline__ void block_mma(const RowsIn<kN>& A, const ColsIn<kCols>& B, bool even, int c,
                                          uint64_t (&y)[col_tiles(kCols)][kT][2]) {
  const uint32_t sel = c == 3 ? 0x5432u : 0x7654u;
#pragma unroll
  for (int t = 0; t < kN; ++t) {
    uint32_t a0, a1, a2, a3, e0, e1, e2, e3;
    tc::quant_pairs(A.w[t][0][0], a0, a2);
    tc::quant_pairs(A.w[t][1][0], a1, a3);
    uint32_t w0 = A.w[t][0][1], w1 = A.w[t][1][1];
    if (kAl && even) {
      w0 = __byte_perm(A.w[t][0][2], w0, sel);
      w1 = __byte_perm(A.w[t][1][2], w1, sel);
    }
    const float d0 = __low2float(*reinterpret_cast<const __half2*>(&A.w[t][0][2]));
    const float d1 = __low2float(*reinterpret_cast<const __half2*>(&A.w[t][1][2]));
    float acc[col_tiles(kCols)][4];
#pragma unroll
    for (int i = 0; i < col_tiles(kCols); ++i) {
      mma_zero(acc[i], a0, a1, a2, a3, B.b[i][0][0], B.b[i][0][1]);
      if constexpr (kCols != kPacked) tc::mma_f16(acc[i], a0, a1, a2, a3, B.b[i][0][2], B.b[i][0][3]);
    }
    tc::quant_pairs(w0, e0, e2);
    tc::quant_pairs(w1, e1, e3);
#pragma unroll
    for (int i = 0; i < col_tiles(kCols); ++i) {
      tc::mma_f16(acc[i], e0, e1, e2, e3, B.b[i][1][0], B.b[i][1][1]);
      if constexpr (kCols != kPacked) tc::mma_f16(acc[i], e0, e1, e2, e3, B.b[i][1][2], B.b[i][1][3]);
      const uint64_t xi = pack2(B.xi[i][0], B.xi[i][1]);
      uint64_t(&yy)[2] = y[i][T0 + t];
      yy[0] = fma2(mul2(pack2(d0, d0), xi), pack2(acc[i][0], acc[i][1]), yy[0]);
      yy[1] = fma2(mul2(pack2(d1, d1), xi), pack2(acc[i][2], acc[i][3]), yy[1]);
    }
  }
}

// f of 0 .. kTiles - 1 as constants.
template <typename F>
__device__ __forceinline__ void each_tile(F f) {
  f(std::integral_constant<int, 0>{});
  f(std::integral_constant<int, 1>{});
  f(std::integral_constant<int, 2>{});
  f(std::integral_constant<int, 3>{});
}
static_assert(kTiles == 4, "");

// Bounded wait (limit - 1 polls) that gives up when another thread of the CTA
// has.  (try_wait without a time hint: with one it polls through nanosleep, and
// twenty waiting warps then take the issue slots of those that work.)
__device__ __forceinline__ bool ring_wait(uint64_t* bar, uint32_t parity, uint32_t limit, volatile int* abort) {
  for (uint32_t i = 1; i < limit; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort) return false;
  }
  *abort = 1;
  return false;
}

// The producers' place in the CTA's sequence of stages: the units q0 .. q1
// in pairs, a pair's slices in turn (group 0's, group 1's); a last unit
// without a partner leaves the other group's stages out.
struct Place {
  int s = 0, ph = 0;  // stage of the ring; parity of its next fill
  bool again = false; // filled before
  int q, sl = 0, half = 0;  // the pair's first unit, slice, unit of the pair
  __device__ __forceinline__ int unit() const { return q + half; }
  __device__ __forceinline__ void next(const MoePlan& L, int q1) {
    int step = 1;
    if (half == 0 && q + 1 < q1) {
      half = 1;
    } else {
      step = 1 + (half == 0 ? 1 : 0);
      half = 0;
      if (++sl == L.stages) {
        sl = 0;
        q += 2;
      }
    }
    s += step;
    if (s >= L.nst) {
      s -= L.nst;
      ph ^= 1;
      again = true;
    }
  }
};

// Barrier of the whole CTA, which its roles reach at places of their own.
__device__ __forceinline__ void cta_sync() { asm volatile("bar.sync 0;" ::: "memory"); }
// Barrier among one group's threads.
__device__ __forceinline__ void group_sync(int group) {
  asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(kGroupThreads) : "memory");
}

// Launches 2 (kGate) and 3.  P.ypart row p = token * top_k + slot receives
// that pair's weighted down product.
//
// A wait that gives up ends every wait of its CTA.  A consumer then makes the
// sums it could not finish NaN, here and in the units to come, and hands no
// stage back; producers start no more copies, and settle those in flight before
// the CTA ends.
template <int kMode, bool kGate, int kCols>
__global__ void __launch_bounds__(kThreads, 1)
    moe_product_kernel(const MoeParams P, const MoePlan L, bool hperm,
                                                                  const __grid_constant__ CUtensorMap map0,
                                                                  const __grid_constant__ CUtensorMap map1) {
  constexpr bool kAl = kMode == kTensor;
  constexpr int kCt = col_tiles(kCols);
  constexpr bool kResident = kMode == kContiguous;  // images stay for an item, in two buffers
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int s_abort, s_fills, s_ifills;
  MoeShared S = carve(L, smem, P.m * P.top_k);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) s_abort = s_fills = s_ifills = 0;
  // The gate / up kernel lets the down kernel start once it has itself waited
  // for the router, so the down kernel may read the choice, and fill its ring
  // with weights, before it waits for h.
  start(P, L, S);
  if (kGate) griddep_wait();
  griddep_launch_dependents();
  group_pairs(P, L, S);
  constexpr int kRows = kGate ? kGuRows : kSlots;  // rows of a unit
  const int rows = kGate ? P.ffn : P.hidden;       // rows of a matrix
  const int nq = (rows + kRows - 1) / kRows;       // units an item
  const unsigned units = (unsigned)S.n_items * (unsigned)nq;  // (at most 2048 x 512)
  const int q0 = (int)(units * blockIdx.x / gridDim.x), q1 = (int)(units * (blockIdx.x + 1) / gridDim.x);
  const int it0 = kResident ? q0 / nq : 0, n_it = kResident && q1 > q0 ? (q1 - 1) / nq - it0 + 1 : 0;  // the CTA's items
  if (warp >= kConsumers) {
    const int rb = L.bpr * kQBlockBytes;
    const uint32_t smem32 = smem_u32(smem);
    const auto img = [&](int row) {
      return kGate ? P.ximg + (size_t)S.ptok[row] * L.bpr * kImgBlock : P.himg + (size_t)row * L.bpr * kImgBlock;
    };
    const int pw = warp - kConsumers;
    const uint64_t pol = policy_evict_first(), keep = policy_evict_last();
    uint32_t filled = 0, parity = 0;
    int images = 0;  // whole rows: items whose images this warp fetched
    uint32_t ifilled = 0, iparity = 0;  // rows in slices: image buffers filled, parity of the last fill
    int fills = 0, ifills = 0;  // stages, image buffers this warp arrived at
    bool have = false;          // rows in slices: the slice's images are asked for
    Place w;
    w.q = q0;
    const auto announced = [&]() {  // this warp's arrival at the stage is due
      filled |= 1u << w.s;
      parity = (parity & ~(1u << w.s)) | (uint32_t)w.ph << w.s;
      ++fills;
    };
    const auto ready = [&]() {  // the stage may be filled
      const bool ok = !w.again || ring_wait(&S.empty[w.s], (uint32_t)w.ph ^ 1u, P.wait_limit, &s_abort);
      if (!__all_sync(0xffffffffu, ok)) return false;
      announced();
      return true;
    };
    // rows in slices: the buffer of the slice's images, and how often it was filled before
    const auto image_buffer = [&](int& buf) {
      const int c = (w.q - q0) / 2 * L.nsl + w.sl / kTiles;
      buf = 2 * w.half + (c & 1);
      return c / 2;
    };
    const auto images_announced = [&](int buf, int turn) {
      ifilled |= 1u << buf;
      iparity = (iparity & ~(1u << buf)) | (uint32_t)(turn & 1) << buf;
      ++ifills;
      have = true;
    };
    // Weights depend on nothing in flight, so the down kernel fills its ring
    // with them before it waits for h.
    if (kAl && pw == 0) {
      for (; w.q < q1; w.next(L, q1)) {
        if (!ready()) break;
        if (lane == 0) {
          const int subs = min(L.S, L.bpr - w.sl * L.S) / 8, x0 = w.sl * L.S / 8 * (8 * kQBlockBytes / 4);
          const int it = w.unit() / nq, y0 = (S.item[it].x & 0xffff) * rows + (w.unit() - it * nq) * kRows;
          const uint32_t st = smem32 + (uint32_t)w.s * (uint32_t)L.stage_bytes;
          uint64_t* full = &S.full[w.s];
          mbar_arrive_expect_tx(full, (uint32_t)(subs * kSubBytes));
          for (int s = 0; s < subs; ++s) {
            const uint32_t d = st + (uint32_t)(s * kSubBytes);
            const int xs = x0 + s * (8 * kQBlockBytes / 4);
            tensor_g2s(d, &map0, xs, y0, full, pol);
            if (kGate) tensor_g2s(d + kSubBytes / 2, &map1, xs, y0, full, pol);
          }
        }
        __syncwarp();
      }
    } else if (kMode == kContiguous && pw == 0) {
      constexpr int kTileRows = kGate ? 8 : 16;
      for (; w.q < q1; w.next(L, q1)) {
        if (!ready()) break;
        if (lane == 0) {
          const int it = w.unit() / nq, r0 = (w.unit() - it * nq) * kRows + w.sl * L.tr * kTileRows;
          // (rows are a multiple of 32: every piece starts and ends on 16 bytes)
          const uint32_t bytes = (uint32_t)max(0, min(L.tr * kTileRows, rows - r0)) * (uint32_t)rb;
          const long long off = ((long long)(S.item[it].x & 0xffff) * rows + r0) * rb;
          uint8_t* st = smem + (size_t)w.s * L.stage_bytes;
          uint64_t* full = &S.full[w.s];
          mbar_arrive_expect_tx(full, (kGate ? 2u : 1u) * bytes);
          if (bytes) {
            bulk_g2s(st, (kGate ? P.wg : P.wd) + off, bytes, full, pol);
            if (kGate) bulk_g2s(st + L.tr * kTileRows * L.SR, P.wu + off, bytes, full, pol);
          }
        }
        __syncwarp();
      }
    } else if (kResident) {
      if (pw == 1) {
        if (!kGate) griddep_wait();  // (h)
        fence_proxy_async_global();  // (the images were written by ordinary stores)
        for (; images < n_it; ++images) {
          uint64_t* full = &S.ifull[images & 1];
          const bool ok = images < 2 || ring_wait(&S.iempty[images & 1], (uint32_t)(images / 2 - 1) & 1u, P.wait_limit, &s_abort);
          if (!__all_sync(0xffffffffu, ok)) break;
          const int2 I = S.item[it0 + images];
          const int n = I.x >> 16;
          if (lane == 0) mbar_arrive_expect_tx(full, (uint32_t)(n * L.bpr * kImgBlock));
          __syncwarp();
          bulk_images(L, smem + L.o_img + (size_t)(images & 1) * L.img_bytes, full, 0, 1, n, 0, L.bpr,
                      [&](int k) { return img(I.y + k); }, keep, lane);
        }
      }
    } else if (kAl) {
      if (!kGate) griddep_wait();  // (h)
      fence_proxy_async_global();  // (the images were written by ordinary stores)
      for (; w.q < q1; w.next(L, q1)) {
        if (!ready()) break;
        const int2 I = S.item[w.unit() / nq];
        const int n = I.x >> 16, c0 = w.sl * L.S, nb = min(L.S, L.bpr - c0), f = pw - 1;
        const int mine = f < n ? (n - f + kProducers - 2) / (kProducers - 1) : 0;  // tokens f, f + 3, ..
        if (lane == 0) mbar_arrive_expect_tx(&S.full[w.s], (uint32_t)(mine * nb * kImgBlock));
        __syncwarp();
        bulk_images(L, smem + (size_t)w.s * L.stage_bytes + L.x_off, &S.full[w.s], f, kProducers - 1, n, c0, nb,
                    [&](int k) { return img(I.y + k); }, keep, lane);
      }
    } else {
      if (!kGate) griddep_wait();
      fence_proxy_async_global();
      for (; w.q < q1; w.next(L, q1)) {
        const int it = w.unit() / nq;
        const int2 I = S.item[it];
        const int tile = w.sl % kTiles, c0 = w.sl / kTiles * L.S, nb = min(L.S, L.bpr - c0);
        const int r0 = (w.unit() - it * nq) * kRows;
        if (tile == 0) {  // the slice's images, for its four tiles
          int buf;
          const int n = I.x >> 16, turn = image_buffer(buf);
          const bool ok = turn < 1 || ring_wait(&S.iempty[buf], (uint32_t)(turn - 1) & 1u, P.wait_limit, &s_abort);
          if (!__all_sync(0xffffffffu, ok)) break;
          images_announced(buf, turn);
          const int mine = pw < n ? (n - pw + kProducers - 1) / kProducers : 0;  // tokens pw, pw + 4, ..
          if (lane == 0) mbar_arrive_expect_tx(&S.ifull[buf], (uint32_t)(mine * nb * kImgBlock));
          __syncwarp();
          bulk_images(L, smem + L.o_img + (size_t)buf * L.img_bytes, &S.ifull[buf], pw, kProducers, n, c0, nb,
                      [&](int k) { return img(I.y + k); }, keep, lane);
        }
        if (!ready()) break;
        have = false;
        uint8_t* st = smem + (size_t)w.s * L.stage_bytes;
        uint64_t* full = &S.full[w.s];
        // lanes 0-3: a row of the tile's sixteen each; a warp's rows are one matrix's
        constexpr int kMine = 16 / kProducers;
        const int slot = pw * kMine + (lane & (kMine - 1));
        const uint8_t* base = kGate ? (slot < 8 ? P.wg : P.wu) : P.wd;
        const int r = kGate ? 8 * tile + (slot & 7) : 16 * tile + slot;
        const bool live = lane < kMine && r0 + r < rows;
        RowLines R{};
        if (live) R = row_lines(((long long)(I.x & 0xffff) * rows + r0 + r) * rb, c0, nb);
        const uint32_t sum = __reduce_add_sync(0xffffffffu, live ? R.bytes : 0u);
        if (lane == 0) mbar_arrive_expect_tx(full, sum);
        __syncwarp();
        if (live) bulk_g2s(st + (size_t)slot * L.SR, base + R.lo, R.bytes, full, pol);
      }
    }
    cta_sync();
    if (*(volatile int*)&s_abort) {
      // a barrier's phase ends when all its producers have arrived: those that
      // gave up earlier than others make up for it, without copies
      if (kMode != kContiguous) {
        if (lane == 0) atomicMax(&s_fills, fills), atomicMax(&s_ifills, ifills);
        asm volatile("bar.sync 3, %0;" ::"n"(kProducers * 32) : "memory");
        const int all = *(volatile int*)&s_fills, iall = *(volatile int*)&s_ifills;
        for (;; w.next(L, q1), have = false) {
          if (kMode == kRowCopies && w.sl % kTiles == 0 && !have && ifills < iall) {
            int buf;
            const int turn = image_buffer(buf);
            if (lane == 0) mbar_arrive(&S.ifull[buf]);
            images_announced(buf, turn);
          }
          if (fills == all) break;
          if (lane == 0) mbar_arrive(&S.full[w.s]);
          announced();
        }
      }
      for (int s = 0; s < L.nst; ++s)
        if (filled >> s & 1u) mbar_wait(&S.full[s], parity >> s & 1u);
      for (int i = 0; i < 4; ++i)
        if (ifilled >> i & 1u) mbar_wait(&S.ifull[i], iparity >> i & 1u);
      for (int i = max(0, images - 2); i < images; ++i) mbar_wait(&S.ifull[i & 1], (uint32_t)(i / 2) & 1u);
    }
  } else {
    if (!kGate) griddep_wait();
    const int gq = lane >> 2, cq = lane & 3;
    const uint32_t smem32 = smem_u32(smem);
    const uint32_t xoff = !kAl ? 0u : (uint32_t)L.x_off;
    // column g of tile i is token 8 i + g (packed: token g % 4, hi or lo)
    uint32_t xl[kCt], x0[kCt], x1[kCt];
#pragma unroll
    for (int i = 0; i < kCt; ++i) {
      const auto col = [&](int n) {
        return xoff + token_off(L.XR, min(kCols == kPacked ? n & 3 : 8 * i + n, L.tg - 1));
      };
      xl[i] = col(gq) + (uint32_t)(cq * 16 + (kCols == kPacked ? 8 * (gq >> 2) : 0));
      x0[i] = col(2 * cq);
      x1[i] = col(2 * cq + 1);
    }
    const int group = warp / kGroupWarps, member = warp % kGroupWarps, tid = threadIdx.x - group * kGroupThreads;
    float* part = S.part + group * kGroupWarps * kSlots * 8;                                 // [warp][slot][token]
    float* hq = reinterpret_cast<float*>(smem + L.o_hq) + group * kGuRows * 9;  // gate: [32 rows][8 tokens + 1]
    int s = group;
    uint32_t ph = 0;
    int chunk = 0;  // rows in slices: this group's slices so far
    int held = -1;  // resident images: the item whose buffer this group holds
    bool ok = true; // no wait of this lane gave up
    const auto next_images = [&]() {  // every item in turn, also those without a unit of this group
      if (held >= 0) {
        __syncwarp();
        if (lane == 0 && ok) mbar_arrive(&S.iempty[held & 1]);
      }
      ++held;
      ok = ok && ring_wait(&S.ifull[held & 1], (uint32_t)(held >> 1) & 1u, P.wait_limit, &s_abort);
    };
    for (int q = q0 + group; q < q1; q += kGroups) {
      const int it = q / nq;
      const int2 I = S.item[it];
      const int ntok = I.x >> 16, u = q - it * nq, r0 = u * kRows;
      if (kResident)
        while (held < it - it0) next_images();
      const uint32_t xres = smem32 + (uint32_t)(L.o_img + (held & 1) * L.img_bytes);
      uint64_t y[kCt][kTiles][2];
#pragma unroll
      for (int i = 0; i < kCt; ++i)
#pragma unroll
        for (int t = 0; t < kTiles; ++t) y[i][t][0] = y[i][t][1] = pack2(0.f, 0.f);
      const auto stage = [&]() {  // the group's next stage
        ok = ok && ring_wait(&S.full[s], ph, P.wait_limit, &s_abort);
        return after_wait(smem32 + (uint32_t)s * (uint32_t)L.stage_bytes);
      };
      const auto release = [&]() {
        __syncwarp();
        if (lane == 0 && ok) mbar_arrive(&S.empty[s]);
        s += kGroups;
        if (s >= L.nst) {
          s -= L.nst;
          ph ^= 1u;
        }
      };
      if constexpr (kAl) {
        for (int sl = 0; sl < L.nsl; ++sl) {
          const uint32_t st = stage();
          const int nb = min(L.S, L.bpr - sl * L.S);
          for (int j = member; j < nb; j += kGroupWarps) {
            ColsIn<kCols> B;
            load_x<kCols>(st + (uint32_t)(j * kImgBlock), xl, x0, x1, B);
            // (sub-stages of 8 blocks)
            const uint32_t bg = st + (uint32_t)((j >> 3) * kSubBytes + (j & 7) * kQBlockBytes + gq * 8 * kQBlockBytes);
            if constexpr (kCt == 1) {
              RowsIn<kTiles> A;
              load_aligned<kGate, 0>(bg, !(j & 1), cq, A);
              block_mma<kAl, kCols, 0>(A, B, !(j & 1), cq, y);
            } else {  // (four tiles' words at once would spill)
              RowsIn<2> A;
              load_aligned<kGate, 0>(bg, !(j & 1), cq, A);
              block_mma<kAl, kCols, 0>(A, B, !(j & 1), cq, y);
              load_aligned<kGate, 2>(bg, !(j & 1), cq, A);
              block_mma<kAl, kCols, 2>(A, B, !(j & 1), cq, y);
            }
          }
          release();
        }
      } else if (kMode == kContiguous) {
        const uint32_t base = (uint32_t)((gq << L.lq) * L.SR + member * kQBlockBytes);
        // tile t of the stage into y[T]
        const auto tile = [&](uint32_t ba, int t, const ColsIn<kCols>& B, auto T) {
          const int s0 = kGate ? t : 2 * t, s1 = 2 * t + 1;
          const uint32_t at = ba + (uint32_t)((((s0 >> L.lq) << (3 + L.lq)) + (s0 & ((1 << L.lq) - 1))) * L.SR);
          const uint32_t at1 = kGate ? at + (uint32_t)(L.tr * 8 * L.SR)
                                     : ba + (uint32_t)((((s1 >> L.lq) << (3 + L.lq)) + (s1 & ((1 << L.lq) - 1))) * L.SR);
          RowsIn<1> A;
          load_unaligned(at, 0, cq, A);
          load_unaligned(at1, 1, cq, A);
          block_mma<kAl, kCols, decltype(T)::value>(A, B, false, cq, y);
        };
        if (L.tr == kTiles) {
          const uint32_t st = stage();
          for (int j = member; j < L.bpr; j += kGroupWarps) {
            const uint32_t ba = st + base + (uint32_t)((j - member) * kQBlockBytes);
            ColsIn<kCols> B;
            load_x<kCols>(xres + (uint32_t)(j * kImgBlock), xl, x0, x1, B);
            each_tile([&](auto T) { tile(ba, T.value, B, T); });
          }
          release();
        } else {
          each_tile([&](auto T) {
            const uint32_t st = stage();
            for (int j = member; j < L.bpr; j += kGroupWarps) {
              ColsIn<kCols> B;
              load_x<kCols>(xres + (uint32_t)(j * kImgBlock), xl, x0, x1, B);
              tile(st + base + (uint32_t)((j - member) * kQBlockBytes), 0, B, T);
            }
            release();
          });
        }
      } else {
        for (int sl = 0; sl < L.nsl; ++sl, ++chunk) {
          const int buf = 2 * group + (chunk & 1), c0 = sl * L.S, nb = min(L.S, L.bpr - c0);
          ok = ok && ring_wait(&S.ifull[buf], (uint32_t)(chunk >> 1) & 1u, P.wait_limit, &s_abort);
          const uint32_t xs = smem32 + (uint32_t)(L.o_img + buf * L.img_bytes);
          each_tile([&](auto T) {
            const uint32_t st = stage();
            // where row g's slice starts in its slot (row g + 8's, 8 * 272
            // bytes of the matrix on or in the other one: as far into a line)
            const uint32_t r = (uint32_t)(r0 + (kGate ? 8 : 16) * T.value + gq);
            const uint32_t mis = (((uint32_t)(I.x & 0xffff) * (uint32_t)rows + r) * (uint32_t)L.bpr + (uint32_t)c0) *
                                 (uint32_t)kQBlockBytes & 15u;
            for (int j = member; j < nb; j += kGroupWarps) {
              const uint32_t ba = st + (uint32_t)(gq * L.SR) + mis + (uint32_t)(j * kQBlockBytes);
              ColsIn<kCols> B;
              load_x<kCols>(xs + (uint32_t)(j * kImgBlock), xl, x0, x1, B);
              RowsIn<1> A;
              load_unaligned(ba, 0, cq, A);
              load_unaligned(ba + (uint32_t)(8 * L.SR), 1, cq, A);
              block_mma<kAl, kCols, decltype(T)::value>(A, B, false, cq, y);
            }
            release();
          });
          if (lane == 0 && ok) mbar_arrive(&S.iempty[buf]);  // (every lane is past its loads: release())
        }
      }
      if (!ok) {
        const float nan = __int_as_float(0x7fc00000);
#pragma unroll
        for (int i = 0; i < kCt; ++i)
#pragma unroll
          for (int t = 0; t < kTiles; ++t) y[i][t][0] = y[i][t][1] = pack2(nan, nan);
      }
#pragma unroll
      for (int i = 0; i < kCt; ++i) {
        const int n0 = 8 * i, nt = min(ntok - n0, 8);  // the tile's tokens
        if (nt <= 0) break;
        // the warps' shares of the unit
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
          float* p = part + ((member * kTiles + t) * 16 + gq) * 8 + 2 * cq;
          *reinterpret_cast<uint64_t*>(p) = y[i][t][0];
          *reinterpret_cast<uint64_t*>(p + 64) = y[i][t][1];
        }
        group_sync(group);
        const int n = tid & 7;
        const auto total = [&](int row) {  // of slot `row` of the unit's A tiles, column n
          float v = 0.f;
#pragma unroll
          for (int k = 0; k < kGroupWarps; ++k) {
            const float* p = part + (k * kSlots + row) * 8;
            v += kCols == kPacked ? p[n & 3] + p[(n & 3) | 4] : p[n];
          }
          return v;
        };
        if constexpr (kGate) {
          const int t = tid >> 6, r = (tid >> 3) & 7;
          const float g = total(16 * t + r), v = total(16 * t + r + 8);
          hq[(kResident ? slot_row<true>(L, t, 0, r) : t * 8 + r) * 9 + n] = g / (1.f + expf(-g)) * v;
          group_sync(group);
          if (tid < 64) {  // the unit is block u of its tokens' h: token x, word w
            const int x = tid >> 3, w = tid & 7;
            float v4[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) v4[k] = hq[tc::word_quant(hperm && !(u & 1), w, k) * 9 + x];
            image_word(v4, x < nt, P.himg + ((size_t)(I.y + n0 + x) * nq + u) * kImgBlock, w);
          }
        } else {
#pragma unroll
          for (int k = 0; k < 2; ++k) {  // 64 rows x 8 tokens
            const int slot = (tid >> 3) + 32 * k, r = kResident ? slot_row<false>(L, slot >> 4, slot >> 3 & 1, slot & 7) : slot;
            const float v = total(slot);
            if (n < nt && r0 + r < rows)
              P.ypart[(size_t)S.ppair[I.y + n0 + n] * P.hidden + r0 + r] = S.pw[I.y + n0 + n] * v;
          }
          group_sync(group);  // (the shares are rewritten next)
        }
      }
    }
    if (kResident)
      while (held < n_it - 1) next_images();
    cta_sync();
    if (threadIdx.x == 0 && *(volatile int*)&s_abort && P.d_err) atomicOr(P.d_err, Q8D_DERR_WAIT);
  }
}

// 4. A thread an output: the experts' rows in the order of the choice.
__global__ void __launch_bounds__(256) moe_sum_kernel(const MoeParams P) {
  griddep_launch_dependents();
  const int r = blockIdx.x * 256 + threadIdx.x, t = blockIdx.y;
  griddep_wait();
  if (r >= P.hidden) return;
  float y = P.residual ? P.residual[(long long)t * P.ldr + r] : 0.f;
  const float* p = P.ypart + (size_t)t * P.top_k * P.hidden + r;
#pragma unroll 8
  for (int k = 0; k < P.top_k; ++k) y += p[(size_t)k * P.hidden];
  P.Y[(long long)t * P.ldy + r] = y;
}

int up16i(int n) { return (n + 15) / 16 * 16; }
size_t up16(size_t n) { return (n + 15) / 16 * 16; }

// A slot of n blocks of rows off the 16-byte boundaries: they start up to 14
// bytes in and are read 4 bytes past; 4 (mod 8) words long, so that eight
// slots' words lie in distinct banks.
int slot_bytes(int n) {
  int b = up16i(n * kQBlockBytes + 18);
  while ((b / 4) % 8 != 4) b += 16;
  return b;
}

// The map of n_rows rows of bpr blocks (a multiple of 8) as 32-bit words,
// in boxes of box_rows rows by 8 blocks.
int weight_map(const uint8_t* w, int bpr, long long n_rows, int box_rows, CUtensorMap* map) {
  typedef CUresult (*Encode)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                             const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                             CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static std::mutex mu;
  static Encode encode = nullptr;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!encode) {
      void* fn = nullptr;
      cudaDriverEntryPointQueryResult found;
      const cudaError_t e =
          cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found);
      if (e != cudaSuccess) return record_cuda(e);
      if (found != cudaDriverEntryPointSuccess || !fn) return record_cuda(cudaErrorNotSupported);
      encode = reinterpret_cast<Encode>(fn);
    }
  }
  const cuuint64_t dim[2] = {(cuuint64_t)bpr * kQBlockBytes / 4, (cuuint64_t)n_rows};
  const cuuint64_t stride[1] = {(cuuint64_t)bpr * kQBlockBytes};
  const cuuint32_t box[2] = {8 * kQBlockBytes / 4, (cuuint32_t)box_rows}, one[2] = {1, 1};
  const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<uint8_t*>(w), dim, stride, box, one,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? Q8D_OK : record_cuda(cudaErrorInvalidValue);
}

// Tokens a group: about twice an expert's share of the (token, slot) pairs,
// a power of two up to 8 (an expert with more is read once a group; with
// fewer, its stage space idles).  The mean decides, so where the choice is
// lopsided a popular expert is read more often: 64 tokens that all ask for one
// of 512 experts are 32 groups of two.  Sixteen where that is clearly fewer units
// (nq an item; the two groups of every SM take one each a turn): by 1.35 for
// tensor copies and two turns or more, else by 1.7.  Measured, eight /
// sixteen, us: 64 tokens, 4096 x 4096, 2 of 8 experts, 268 / 215, 1 of 8, 174 /
// 153; 64, 2048 x 1024, 6 of 16, 106 / 90; 32, 2048 x 1024, 2 of 8 (one turn),
// 37.2 / 35.1; but 64, 2048 x 1024, 2 of 16, 54 / 56; 40, 3360 x 1120, 3 of 8,
// 107 / 116; 33, 2944 x 704, 4 of 16, 79 / 89; 64, 2048 x 768, 8 of 128, 174 /
// 207.
int group_tokens(const MoeParams& P, int nq, bool al) {
  const double share = (double)P.m * P.top_k / P.n_experts;
  const int want = std::min(P.m, (int)(2 * share) + 2);
  int tg = 1;
  while (tg < 8 && tg < want) tg *= 2;
  const auto turns = [&](int n) {  // (an expert's last group is half full on average)
    return std::max(1.0, share / n + 0.5) * P.n_experts * nq / (kGroups * sm_count());
  };
  const double few = turns(16), many = turns(8);
  return share >= 8 && ((al && few >= 2 ? 1.35 : 1.7) * few < many || (few <= 1 && many > 1)) ? 16 : tg;
}

// Banks: the most of eight rows' words (rows `step` bytes apart) that one
// bank holds.
int bank_rows(int step) {
  int n[32] = {}, most = 0;
  for (int g = 0; g < 8; ++g)
    for (int c = 0; c < 4; ++c) most = std::max(most, ++n[(g * step / 4 + c) % 32]);
  return most;
}

// Lays out a product kernel over rows of bpr blocks.  Where rows are whole
// 16-byte lines: tensor copies of slices of 16 or 8 blocks.  Else, up to 64
// blocks, whole rows, 64 of them a stage while they are short, and the images
// of two items beside the ring.  Longer rows, or where those leave no four
// stages: a tile's rows in slices of up to 64 blocks.
int plan_product(const MoeParams& P, int bpr, bool gate, MoePlan* L) {
  const bool al = bpr % 8 == 0;
  const int pairs = P.m * P.top_k;
  L->bpr = bpr;
  const int nq = gate ? P.ffn / kGuRows : (P.hidden + kSlots - 1) / kSlots;
  for (int tg = group_tokens(P, nq, al); tg >= 1; tg /= 2) {
    L->tg = tg;
    for (L->lg = 0; 1 << L->lg < tg;) ++L->lg;
    L->inv_k = 1.f / (float)P.top_k;
    L->items = std::min(pairs, P.n_experts + pairs / tg);
    int o = 0;  // behind the ring
    L->o_part = o;
    o += kConsumers * kSlots * 8 * 4;
    L->o_hq = o;
    o += up16i(kGroups * kGuRows * 9 * 4);
    L->o_mask = o;
    o += 8 * P.n_experts;
    L->o_ebase = o;
    o = up16i(o + 4 * P.n_experts);
    L->o_item = o;
    o = up16i(o + 8 * L->items);
    L->o_tok = o;
    o = up16i(o + 8 * pairs);
    L->o_bar = o;
    const int behind = o;
    // of at most s blocks; false if four stages, or a ring of `least` bytes, do not fit
    const auto slices = [&](int mode, int s, int least) {
      const bool whole = mode == kContiguous;
      L->mode = mode;
      L->nsl = whole ? 1 : (bpr + s - 1) / s;
      L->S = (bpr + L->nsl - 1) / L->nsl;  // (equal slices; whole groups of 8 blocks for tensor copies)
      if (mode == kTensor) L->S = (L->S + 7) / 8 * 8;
      L->tr = mode == kRowCopies || (whole && bpr > 16) ? 1 : kTiles;
      L->lq = 0;
      if (whole) {
        int least_rows = bank_rows(bpr * kQBlockBytes);
        for (int lq = 1; 1 << lq <= L->tr * (gate ? 1 : 2); ++lq) {
          const int n = bank_rows((bpr * kQBlockBytes) << lq);
          if (n < least_rows) least_rows = n, L->lq = lq;
        }
      }
      L->stages = mode == kTensor ? L->nsl : whole ? kTiles / L->tr : kTiles * L->nsl;
      L->SR = mode == kTensor ? 8 * kQBlockBytes : whole ? bpr * kQBlockBytes : slot_bytes(L->S);
      L->x_off = mode == kTensor ? L->S / 8 * kSubBytes : 16 * L->tr * L->SR;
      // token rows half a bank cycle apart: the two tokens of a quarter warp's
      // 16-byte loads lie in distinct banks
      L->XR = (L->S * kImgBlock + 127) / 128 * 128 + 64;
      const int images = up16i(tg * L->XR + 8 * tg);
      L->img_bytes = mode == kTensor ? 0 : images;
      const int bufs = whole ? 2 : 4;  // two items', or two slices' of each group
      // (tensor copies land on 128 bytes; a row's last word is read 4 bytes past)
      L->stage_bytes = (L->x_off + (mode != kTensor ? 16 : images) + 127) / 128 * 128;
      L->o_img = up16i(behind + 64);
      L->smem = L->o_img + bufs * L->img_bytes;
      L->nst = std::min(12, (kMaxSmem - L->smem) / (L->stage_bytes + 16)) / kGroups * kGroups;
      if (L->nst < 2 * kGroups || L->nst * L->stage_bytes < least) return false;
      const int ring = L->nst * L->stage_bytes;
      for (int* f : {&L->o_part, &L->o_hq, &L->o_mask, &L->o_ebase, &L->o_item, &L->o_tok, &L->o_bar, &L->o_img})
        *f += ring;
      L->o_img += 16 * L->nst;  // (the barriers: 16 bytes a stage and the images' 64)
      L->smem += ring + 16 * L->nst;
      return true;
    };
    if (!al && bpr <= 64 && slices(kContiguous, bpr, 0)) return Q8D_OK;
    for (int least : {al ? 0 : 64 * 1024, 0})
      for (int s = al ? 16 : 64; s >= 8; s -= 8)
        if (slices(al ? kTensor : kRowCopies, s, least)) return Q8D_OK;
  }
  return Q8D_EUNSUPPORTED;
}

}  // namespace

static std::atomic<uint32_t> g_wait_limit{kWaitLimit};
void moe_set_wait_limit(uint32_t polls) { g_wait_limit = polls ? polls : kWaitLimit; }

size_t moe_workspace_bytes(int m, int hidden, int ffn, int n_experts, int top_k) {
  (void)n_experts;
  const size_t pairs = (size_t)m * top_k;
  return up16(4 * pairs) * 2 + (size_t)m * (hidden / kQBlock) * kImgBlock + pairs * (ffn / kQBlock) * kImgBlock +
         4 * pairs * hidden;
}

int moe_launch(MoeParams P, void* workspace, cudaStream_t stream) {
  const size_t pairs = (size_t)P.m * P.top_k;
  const int bx = P.hidden / kQBlock, bh = P.ffn / kQBlock;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  P.ximg = ws;
  ws += (size_t)P.m * bx * kImgBlock;
  P.himg = ws;
  ws += pairs * bh * kImgBlock;
  P.ypart = reinterpret_cast<float*>(ws);
  ws += 4 * pairs * P.hidden;
  if (!P.experts) P.experts = reinterpret_cast<int*>(ws);
  ws += up16(4 * pairs);
  if (!P.weights) P.weights = reinterpret_cast<float*>(ws);
  P.wait_limit = g_wait_limit;

  MoePlan gu{}, dn{};
  int rc = plan_product(P, bx, true, &gu);
  if (!rc) rc = plan_product(P, bh, false, &dn);
  if (rc) return rc;
  const bool gal = bx % 8 == 0, dal = bh % 8 == 0;
  typedef void (*Product)(MoeParams, MoePlan, bool, CUtensorMap, CUtensorMap);
  const auto fn = [](const MoePlan& L, auto gate) -> Product {
    constexpr bool kGate = decltype(gate)::value;
    static const Product fns[3][3] = {
        {moe_product_kernel<kRowCopies, kGate, kPacked>, moe_product_kernel<kRowCopies, kGate, kEight>,
         moe_product_kernel<kRowCopies, kGate, kSixteen>},
        {moe_product_kernel<kTensor, kGate, kPacked>, moe_product_kernel<kTensor, kGate, kEight>,
         moe_product_kernel<kTensor, kGate, kSixteen>},
        {moe_product_kernel<kContiguous, kGate, kPacked>, moe_product_kernel<kContiguous, kGate, kEight>,
         moe_product_kernel<kContiguous, kGate, kSixteen>}};
    return fns[L.mode][L.tg <= 4 ? kPacked : L.tg == 8 ? kEight : kSixteen];
  };
  const Product gu_fn = fn(gu, std::true_type{}), dn_fn = fn(dn, std::false_type{});
  CUtensorMap mg{}, mu{}, md{};
  if (gal) {
    rc = weight_map(P.wg, bx, (long long)P.n_experts * P.ffn, kGuRows, &mg);
    if (!rc) rc = weight_map(P.wu, bx, (long long)P.n_experts * P.ffn, kGuRows, &mu);
  }
  if (!rc && dal) rc = weight_map(P.wd, bh, (long long)P.n_experts * P.hidden, kSlots, &md);
  if (!rc) rc = configure_kernel(reinterpret_cast<const void*>(gu_fn), kMaxSmem, true);
  if (!rc) rc = configure_kernel(reinterpret_cast<const void*>(dn_fn), kMaxSmem, true);
  if (rc) return rc;

  // The router: clusters of 8 CTAs, two CTAs an SM at once, a token each as
  // long as that is one wave, else two (four a cluster at one CTA an SM left
  // too few warps to cover the loads: 22 us at 64 tokens).
  const int per = P.m * kRtCluster <= 2 * sm_count() ? 1 : 2;
  const int clusters = (P.m + per - 1) / per;
  void (*const rt_fns[2])(MoeParams, int, bool) = {moe_router_kernel<1>, moe_router_kernel<2>};
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
  const int sms = sm_count();
  rc = launch_ex(gu_fn, dim3(sms), dim3(kThreads), (size_t)gu.smem, stream, true, P, gu, dal, mg, mu);
  if (!rc) rc = launch_ex(dn_fn, dim3(sms), dim3(kThreads), (size_t)dn.smem, stream, true, P, dn, dal, md, md);
  if (rc) return rc;
  return launch_ex(moe_sum_kernel, dim3((P.hidden + 255) / 256, P.m), dim3(256), 0, stream, true, P);
}

}  // namespace q8d
