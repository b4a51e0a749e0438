// Split-K decode attention over a 4-bit KV cache (Q8D_KV_Q4) on the tensor
// cores: the contract of the other decode-attention kernels.
//
// At 9/16 byte an element the arithmetic, not HBM, is what such a kernel runs
// out of first: at the copy rate an SM gets one token of one KV head (144
// bytes at head_dim 128) every 6 cycles, 780 issue slots for a tile of 32
// tokens; the tile takes 800 warp instructions with up to four heads a KV
// head, 1000 with five to eight, 320 of them to unpack its quants, and sixteen
// warps an SM (128 registers each) fill 51 to 58 percent of the slots.  So
// the layout saves instructions:
//  * A half-byte n put under the exponent of 1024 is the f16 1024 + n (1024 +
//    16 n for the upper one): one LOP3 a pair, and one sub.f16x2 leaves the
//    exact n - 8 (16 (n - 8)).  (Masked out alone it would be the subnormal
//    n * 2^-24, without a subtraction; but the tensor core aligns products by
//    the operands' exponent fields, and a subnormal's loses it 7 bits.)
//  * Rows of A are what the cache holds (16 tokens for K.Q^T, 16 dims for
//    V.P^T) and columns of B the heads, so the few heads of a KV head fill
//    the short side.  q is f16 hi + lo parts.  With at most four heads a KV
//    head, parts are neighbouring columns and one MMA does two; else each takes
//    its own.
//    (Heads as rows of A, hi and lo in rows g and g + 8, took 920
//    instructions a tile with two heads, against 740 so, P in two parts both
//    times: 62 and 45 us for 32 sequences of up to 8192 tokens, 16 query and 8
//    KV heads of 128.)
//  * A lane's scores are tokens g, g + 8, .. of heads 2c, 2c + 1 (packed: of
//    head c), so a token's scale and a head's factors are loaded or kept
//    once.  V's scale depends on the token and the block, so it multiplies P
//    once per block before the split; movmatrix turns the parts into the B
//    operand; ldmatrix.trans hands a lane the same two bytes of V of tokens 2c
//    and 2c + 1.
//  * P times V's scale is three bf16 parts, exactly the f32 product, and the
//    quants are bf16 (n under the exponent of 128).  Its terms may lie far
//    apart within a head: the token that takes the softmax may have no V, one
//    block's scales lie far above another's.  f16 hi + lo under one power of two
//    a warp (a third fewer MMAs, upper half-bytes without their shift: 42.0 us
//    for that batch, 46.3 so; 29.4 and 32.6 for 8 sequences of up to 32768, 28
//    and 4 heads) is off by 2^-32 of the largest P times the largest scale, and
//    outputs made of terms 2^-15 below that leave f32's accuracy.
//  * A tile's products are summed from zero and added to O with rounded f32
//    additions.  The tensor core cuts its running sums off, always towards zero:
//    over 16384 rows a warp of V of one sign, 3 to 5e-5 of the output, 4e-7 so
//    (46.3 and 32.6 us for the batches above with O as the accumulators, 47.4 and
//    33.3 so).  For the same reason lo stands beside mid: added to hi, it would
//    be a small remainder of one sign that every rounding drops.
//  * The running maximum moves only when a score exceeds it by 2^8, so an
//    ordinary tile does no reduction across lanes.
//  * Eight warps, each with its own softmax over 32-token tiles and its own
//    two-stage cp.async ring (16-byte chunks, XOR-swizzled for ldmatrix),
//    merge once; partials are combined as in the other kernels.  Short caches
//    are not cut, and then there is nothing to combine.
#include <cuda_fp16.h>

#include <algorithm>

#include "q8d_attn.cuh"
#include "q8d_attn_common.cuh"
#include "q8d_internal.cuh"
#include "q8d_kv_rows.cuh"

namespace q8d {
namespace {

constexpr int kWarps4 = 8;
constexpr int kThreads4 = kWarps4 * 32;
constexpr float kLog2e4 = 1.4426950408889634f;
constexpr int kTile4 = 32;        // tokens a warp step
constexpr int kStages4 = 2;
constexpr float kSlack4 = 8.f;    // the running maximum may lag by this (log2)
constexpr int kSeqCost4 = 16;     // a sequence's fixed work, in tiles
// Caches of up to this many rows: sequences are not cut, so the attention
// kernel writes the outputs itself and there is no second launch.  Graph /
// single call, us, cut and combined against whole: 28 / 4 heads of 128, 256
// rows, 6.1 / 8.6 against 4.9 / 6.6; 512 rows, 6.1 / 8.4 against 6.9 / 7.0; 1024
// rows, 6.2 / 8.4 against 10.5 / 10.7; 32 ragged sequences of 16 / 8 heads, 512
// rows, 13.2 / 13.6 against 11.2 / 11.5; 1024 rows, 16.3 / 16.7 against 17.4 /
// 17.9.
constexpr int kWholeCap4 = 512;

template <int D, int NH>
struct Cfg4 {
  static constexpr int kNB = D / 32;                      // blocks of a head row
  static constexpr int kRow = D / 2;                      // quant bytes of a head row
  static constexpr int kSRow = D / 16;                    // scale bytes of a head row
  static constexpr int kQuants = kTile4 * kRow;
  static constexpr int kScales = kTile4 * kSRow;
  static constexpr int kStage = 2 * (kQuants + kScales);  // K, V quants, K, V scales
  static constexpr int kOffQf = kWarps4 * kStages4 * kStage;      // A fragments of q
  static constexpr int kQf = NH * (D / 16) * 32 * 16;
  static constexpr int kOffQs = kOffQf + kQf;             // f32 q [8 NH][D], power-of-two scaled
  static constexpr int kOffF = kOffQs + 8 * NH * D * 4;   // score factors 2^-sh [8 NH]
  static constexpr int kSmem = kOffF + 8 * NH * 4;
  static constexpr int kOStride = D + 4;  // merge rows: a half warp's pairs in distinct banks
  static_assert(kWarps4 * 8 * NH * (kOStride + 2) * 4 <= kOffQf + kQf, "merge buffer fits");
};

template <int N>
__device__ __forceinline__ void cp4(uint32_t dst, const void* src, bool live) {
  const int n = live ? N : 0;  // (0: the destination is filled with zeros)
  if constexpr (N == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N), "r"(n)
                 : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void mma4(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                     uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same from zero.
__device__ __forceinline__ void mma4z(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                      uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// The same with bf16 operands.
__device__ __forceinline__ void mma4b(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                      uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same from zero.
__device__ __forceinline__ void mma4bz(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                       uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// d += v, rounded.
__device__ __forceinline__ void add4(float (&d)[4], const float (&v)[4]) {
  unpack2(add2(pack2(d[0], d[1]), pack2(v[0], v[1])), d[0], d[1]);
  unpack2(add2(pack2(d[2], d[3]), pack2(v[2], v[3])), d[2], d[3]);
}
// 2^x to two units in the last place; results below 2^-126 are 0 (a weight
// that small next to 1 is beyond every sum's accuracy).
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// The NB halves of a token's scales.
template <int NB>
__device__ __forceinline__ void scales4(const uint8_t* p, uint32_t (&w)[NB / 2]) {
  if constexpr (NB == 4) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x;
    w[1] = v.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}
__device__ __forceinline__ float half_of(uint32_t w, int i) {
  const __half2 h = *reinterpret_cast<const __half2*>(&w);
  return i ? __high2float(h) : __low2float(h);
}
// An 8 x 8 matrix of halves (lane (g, c): row g, columns 2c, 2c+1), transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
  return r;
}
// n - 8 of the low half-bytes n of bytes 0 and 2 of w as an exact f16 pair
// (kHi: 16 (n - 8) of the high half-bytes).
template <bool kHi>
__device__ __forceinline__ uint32_t nib8(uint32_t w, uint32_t k1024) {
  uint32_t x;  // (w & mask) | k1024: one LOP3 while k1024 is a register
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(x) : "r"(w), "n"(kHi ? 0x00f000f0 : 0x000f000f), "r"(k1024));
  uint32_t r;
  asm("sub.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(kHi ? 0x64806480u : 0x64086408u));
  return r;
}
// n - 8 of the low half-bytes n of bytes 0 and 2 of w as an exact bf16 pair
// (under the exponent of 128: 128 + n).
__device__ __forceinline__ uint32_t nib8b(uint32_t w, uint32_t k128) {
  uint32_t x;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(x) : "r"(w), "n"(0x000f000f), "r"(k128));
  uint32_t r;
  asm("sub.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(0x43084308u));
  return r;
}
// A pair of f32 values as three bf16 each, which add up to it exactly: a bf16
// is the upper half of an f32, eight leading bits.  hi and mid hold the value
// and what its upper half leaves; their upper halves are the parts.
struct Parts3 {
  float hi[2], mid[2], lo[2];
  __device__ __forceinline__ explicit Parts3(uint64_t a) {
    unpack2(a, hi[0], hi[1]);
    const uint64_t m = add2(a, upper_neg(hi));
    unpack2(m, mid[0], mid[1]);
    unpack2(add2(m, upper_neg(mid)), lo[0], lo[1]);
  }
  static __device__ __forceinline__ uint64_t upper_neg(const float (&v)[2]) {  // (one LOP3 each)
    return pack2(__uint_as_float((__float_as_uint(v[0]) & 0xffff0000u) ^ 0x80000000u),
                 __uint_as_float((__float_as_uint(v[1]) & 0xffff0000u) ^ 0x80000000u));
  }
};
// The upper halves of a and b.
__device__ __forceinline__ uint32_t upper2(float a, float b) {
  return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
}

// ---- the split ----
// The batch's tiles of kTile4 rows, sequence after sequence, are cut into
// pieces of equal length, one a CTA (of each KV head), whatever sequences
// they lie in: one wave of CTAs that end together.  A sequence counts
// kSeqCost4 tiles more than it has (its queries, the first loads, the merge),
// in front of its rows.  The lengths live in device memory, so every CTA and
// the combine derive the same cut from them.  (Chunks of one sequence each,
// four a sequence on average and 3.4 waves: 62 us in the case above, 54 so
// with the same tile; kSeqCost4 of 6, 12, 16, 28: 47.7, 47.1, 47.4, 49.3 us
// there and 34.4, 33.5, 33.3, 34.0 for 8 sequences of up to 32768, 28 query
// and 4 KV heads.)
__device__ __forceinline__ int window_len4(const AttnParams& P, int b) {
  if (!P.d_runs) {
    const int L = __ldcg(P.d_lens + b);
    return (L >= 1 && L <= P.cap) ? L : -1;
  }
  const int L = attn_window_len(P, b);
  return L <= kAttnQ4MaxRows ? L : -1;
}
__device__ __forceinline__ int tiles4(int L) { return L < 1 ? 0 : (L + kTile4 - 1) / kTile4; }

struct Split4 {
  int piece;  // tiles a CTA
  int total;  // tiles of the batch
  bool bad;   // an invalid length
  int len;    // of sequence `lane`
};
// Every lane of a warp calls.  kWhole: a sequence goes whole to the CTA in
// whose piece it starts.
template <bool kWhole>
__device__ __forceinline__ Split4 split4(const AttnParams& P, int lane) {
  Split4 S;
  if (P.batch == 1) {  // (no sums to wait for)
    S.len = window_len4(P, 0);
    S.bad = S.len < 1;
    const int ctas = kWhole ? 1 : min(P.nct, P.nc);
    S.total = tiles4(S.len);
    S.piece = max(kMinChunk / kTile4, (S.total + ctas - 1) / ctas);
    return S;
  }
  int sum = 0, most = 0;
  bool bad = false;
  S.len = -1;
  for (int s = lane; s < P.batch; s += 32) {
    const int L = window_len4(P, s), n = tiles4(L);
    if (s < 32) S.len = L;
    bad = bad || n == 0;
    sum += n ? n + kSeqCost4 : 0;
    most = max(most, n);
  }
  sum = __reduce_add_sync(0xffffffffu, sum);
  most = __reduce_max_sync(0xffffffffu, most);
  S.bad = __any_sync(0xffffffffu, bad);
  S.total = sum;
  S.piece = max(kMinChunk / kTile4, (sum + P.nct - 1) / P.nct);
  // a sequence's pieces fit its slots (two or more: batches of caches that are
  // cut have them): with rows that start anywhere in a piece, k pieces' length
  // touches k + 1
  if (!kWhole) S.piece = max(S.piece, (most + P.nc - 2) / (P.nc - 1));
  return S;
}

// The length of sequence b and where its rows start.  Every lane of a warp
// calls.
__device__ __forceinline__ int seq_of4(const AttnParams& P, const Split4& S, int b, int lane, int& L) {
  L = S.len;
  if (P.batch == 1) return 0;
  int sum = 0;
  for (int s = lane; s < b; s += 32) {
    const int n = tiles4(s < 32 ? S.len : window_len4(P, s));
    sum += n ? n + kSeqCost4 : 0;
  }
  L = b < 32 ? __shfl_sync(0xffffffffu, S.len, b) : window_len4(P, b);
  return (int)__reduce_add_sync(0xffffffffu, sum) + kSeqCost4;
}

// A sequence with rows in a CTA's piece, and where its first row lies.
struct Seq4 {
  int b, L, at;
};
// The first sequence with rows at or after tile `from` (kWhole: that starts
// there); false if there is none.  Every lane of a warp calls.
template <bool kWhole>
__device__ __forceinline__ bool seq_from4(const AttnParams& P, const Split4& S, int from, int lane, Seq4& q) {
  if (P.batch == 1) {
    q.b = q.at = 0;
    q.L = S.len;
    return from < tiles4(S.len);
  }
  int before = 0;
  for (int s0 = 0; s0 < P.batch; s0 += 32) {
    const int s = s0 + lane;
    const int L = s0 == 0 ? S.len : s < P.batch ? window_len4(P, s) : -1;
    const int n = tiles4(L);
    int end = n ? n + kSeqCost4 : 0;  // inclusive prefix sum
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, end, o);
      if (lane >= o) end += v;
    }
    end += before;
    const uint32_t hit = __ballot_sync(0xffffffffu, n && (kWhole ? end - n >= from : end > from));
    if (hit) {
      const int x = __ffs(hit) - 1;
      q.b = s0 + x;
      q.L = __shfl_sync(0xffffffffu, L, x);
      q.at = __shfl_sync(0xffffffffu, end - n, x);
      return true;
    }
    before = __shfl_sync(0xffffffffu, end, 31);
  }
  return false;
}
// The next sequence with rows; false if there is none.
__device__ __forceinline__ bool seq_next4(const AttnParams& P, Seq4& q) {
  q.at += tiles4(q.L) + kSeqCost4;
  while (++q.b < P.batch) {
    q.L = window_len4(P, q.b);
    if (q.L >= 1) return true;
  }
  return false;
}

// NH: column tiles (2 for nine to sixteen heads).  kPack: at most four heads,
// a head's hi and lo parts in columns 2h and 2h + 1 of one tile; else a tile
// is eight heads and hi and lo take an MMA each.
template <int D, int NH, bool kPack, bool kWhole>
__global__ void __launch_bounds__(kThreads4, NH == 1 ? 2 : 1) gqa_q4kv_kernel(const AttnParams P) {
  using C = Cfg4<D, NH>;
  constexpr int NB = C::kNB;
  constexpr int KS = D / 16;
  constexpr int NT = kTile4 / 8;      // groups of eight tokens of a tile
  constexpr int HC = kPack ? 1 : 2;   // heads a lane keeps scores of, of each column tile
  constexpr int kHeads = kPack ? 4 : 8 * NH;
  extern __shared__ __align__(128) uint8_t smem[];
  float* qs = reinterpret_cast<float*>(smem + C::kOffQs);
  float* fh = reinterpret_cast<float*>(smem + C::kOffF);
  __shared__ AttnWindow s_win;

  const int g = blockIdx.y;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int gq = lane >> 2, cq = lane & 3;
  const int G = P.n_heads / P.n_kv_heads;
  griddep_wait();  // (a programmatic dependent: the previous work is complete)
  // after the wait: the combine, scheduled from here on, may read the lengths
  // before this grid is done
  griddep_launch_dependents();
  const Split4 sp = split4<kWhole>(P, lane);
  if (sp.bad && blockIdx.x == 0 && g == 0 && tid == 0 && P.d_err) atomicOr(P.d_err, Q8D_DERR_LEN_RANGE);
  if (kWhole && sp.bad && blockIdx.x == 0)  // (else the combine does)
    for (int b = 0; b < P.batch; ++b)
      if (window_len4(P, b) < 1)
        for (int e = tid; e < G * D; e += kThreads4)
          P.out[((long long)b * P.n_heads + (long long)g * G) * D + e] = __int_as_float(0x7fc00000);
  if ((long long)blockIdx.x * sp.piece >= sp.total) return;
  const int p_begin = blockIdx.x * sp.piece;
  Seq4 sq;
  if (!seq_from4<kWhole>(P, sp, p_begin, lane, sq)) return;

  const int width = P.n_kv_heads * D;
  const long long splane = q4_scale_plane(P.cap, width);
  const uint32_t rowq = (uint32_t)width / 2, rows = (uint32_t)width / 16;  // bytes a row
  const uint32_t ring = smem_u32(smem) + warp * kStages4 * C::kStage;
  constexpr int kCh = C::kRow / 16;          // 16-byte chunks of a head row
  constexpr int kRowsPass = 32 / kCh;        // rows the lanes copy at once
  const int ld_r = lane / kCh, ld_c = lane % kCh;
  // (the swizzle repeats every 8 rows: it does not depend on the pass)
  constexpr int kSwz = D == 128 ? 1 : 2;
  const uint32_t ld_dst = ld_r * C::kRow + ((ld_c ^ ((ld_r >> kSwz) & (kCh - 1))) << 4);
  uint32_t k1024;  // (1024, 1024), kept out of the compiler's sight as a constant
  asm volatile("mov.b32 %0, 0x64006400;" : "=r"(k1024));
  uint32_t k128;  // (128, 128) in bf16, as well
  asm volatile("mov.b32 %0, 0x43004300;" : "=r"(k128));
  // ldmatrix row addresses.  K (x4): 8 tokens, blocks 0-3 (head_dim 64: 8
  // tokens each of two groups, blocks 0-1); V (x4, transposed): tokens 0-7
  // and 8-15 of block 2 i, then of block 2 i + 1.
  const int mi = lane >> 3, mr = lane & 7;
  const uint32_t k_row = D == 128 ? mr : (mi >> 1) * 8 + mr, k_blk = D == 128 ? mi : mi & 1;
  const uint32_t k_off = k_row * C::kRow + ((k_blk ^ ((k_row >> kSwz) & (kCh - 1))) << 4);
  const uint32_t v_row = (mi & 1) * 8 + mr;
  uint32_t v_off[NB / 2];
#pragma unroll
  for (int i = 0; i < NB / 2; ++i)
    v_off[i] = C::kQuants + v_row * C::kRow + (((2 * i + (mi >> 1)) ^ ((v_row >> kSwz) & (kCh - 1))) << 4);

  for (bool first = true; sq.at < p_begin + sp.piece; first = false) {  // the piece's sequences
    const int b = sq.b, L = sq.L;
    int t_begin = 0, t_end = L, c = 0;
    if (!kWhole) {
      t_begin = max(p_begin - sq.at, 0) * kTile4;
      t_end = min(L, min(tiles4(L), p_begin + sp.piece - sq.at) * kTile4);  // (below 2^31)
      c = blockIdx.x - (P.batch == 1 ? 0 : sq.at / sp.piece);
    }
    if (!first) __syncthreads();  // (the merge buffer lies over the ring)
    const long long seq_off = (long long)b * (P.batch_stride / kQBlock) * 18;
    uint8_t* kq = static_cast<uint8_t*>(P.kcache) + seq_off + g * C::kRow;
    uint8_t* vq = static_cast<uint8_t*>(P.vcache) + seq_off + g * C::kRow;
    uint8_t* ks = static_cast<uint8_t*>(P.kcache) + seq_off + splane + g * C::kSRow;
    uint8_t* vs = static_cast<uint8_t*>(P.vcache) + seq_off + splane + g * C::kSRow;

    // In-kernel append of row L-1 by the CTA that owns it; read back below.
    if (P.k_new != nullptr && t_end == L && warp < 2) {
      const float* src = (warp ? P.v_new : P.k_new) + (long long)b * width + (long long)g * D;
      const long long row = attn_cell(P, b, L - 1);
#pragma unroll
      for (int t = 0; t < NB; ++t)
        quantize_q4_warp(src[lane + 32 * t], (warp ? vq : kq) + row * rowq + 16 * t,
                         (warp ? vs : ks) + row * rows + 2 * t, lane);
    }
    // a causal window is the one run (0, L): only run maps and the appended row
    // need the CTA's threads to meet here
    int run0_len = L, run0_cell = 0;
    if (P.d_runs) {
      if (tid == 0) attn_window_store(P, b, &s_win);
      __syncthreads();
      run0_len = s_win.len[0];
      run0_cell = s_win.cell[0];
    } else if (P.k_new != nullptr && t_end == L) {
      __syncthreads();
    }
    const auto cell_of = [&](int t) { return t < run0_len ? run0_cell + t : s_win.cell_of(t); };

    // ---- this warp's ring over its tiles (tile i: tokens t_begin + 32 (warp + 8 i)) ----
    const int ntiles = (t_end - t_begin + kTile4 - 1) / kTile4;
    const int my_tiles = ntiles > warp ? (ntiles - warp + kWarps4 - 1) / kWarps4 : 0;
    auto load_tile = [&](int i) {
      if (i < my_tiles) {
        const int t0 = t_begin + (warp + kWarps4 * i) * kTile4;
        const int nr = min(kTile4, t_end - t0);
        const uint32_t st = ring + (i % kStages4) * C::kStage;
        if (nr == kTile4 && t0 + kTile4 <= run0_len) {
          const long long row = run0_cell + t0 + ld_r;
          const uint8_t* kp = kq + row * rowq + ld_c * 16;
          const uint8_t* vp = vq + row * rowq + ld_c * 16;
#pragma unroll
          for (int k = 0; k < kTile4 / kRowsPass; ++k) {
            cp4<16>(st + ld_dst + k * kRowsPass * C::kRow, kp + k * kRowsPass * rowq, true);
            cp4<16>(st + C::kQuants + ld_dst + k * kRowsPass * C::kRow, vp + k * kRowsPass * rowq, true);
          }
          const long long sr = run0_cell + t0 + lane;
          cp4<C::kSRow>(st + 2 * C::kQuants + lane * C::kSRow, ks + sr * rows, true);
          cp4<C::kSRow>(st + 2 * C::kQuants + C::kScales + lane * C::kSRow, vs + sr * rows, true);
        } else {
          // rows past the chunk become zeros: scale 0, so they add nothing
          for (int k = 0; k < kTile4 / kRowsPass; ++k) {
            const int r = k * kRowsPass + ld_r;
            const bool live = r < nr;
            const long long off = (long long)cell_of(t0 + (live ? r : 0)) * rowq + ld_c * 16;
            cp4<16>(st + ld_dst + k * kRowsPass * C::kRow, kq + off, live);
            cp4<16>(st + C::kQuants + ld_dst + k * kRowsPass * C::kRow, vq + off, live);
          }
          const bool live = lane < nr;
          const long long off = (long long)cell_of(t0 + (live ? lane : 0)) * rows;
          cp4<C::kSRow>(st + 2 * C::kQuants + lane * C::kSRow, ks + off, live);
          cp4<C::kSRow>(st + 2 * C::kQuants + C::kScales + lane * C::kSRow, vs + off, live);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");  // (possibly empty: a uniform count)
    };
#pragma unroll
    for (int i = 0; i < kStages4 - 1; ++i) load_tile(i);

    // ---- q * scale * log2(e), rows times 2^sh into [2^14, 2^15), 2^-sh ----
#pragma unroll
    for (int u = 0; u < NH; ++u) {
      const int hh = warp + 8 * u;
      if (hh >= kHeads) break;
      float v[NB];
      float mx = 0.f;
#pragma unroll
      for (int t = 0; t < NB; ++t) {
        v[t] = hh < G ? P.q[((long long)b * P.n_heads + g * G + hh) * D + lane + 32 * t] * (P.scale * kLog2e4) : 0.f;
        mx = fmaxf(mx, fabsf(v[t]));
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      // mx < 2^(field - 126); sh in [-126, 126] keeps 2^sh and 2^-sh normal
      const int field = (int)(__float_as_uint(mx) >> 23);
      const int sh = max(-126, min(126, 15 + 126 - field));
      const float up = __int_as_float((127 + sh) << 23);
#pragma unroll
      for (int t = 0; t < NB; ++t) qs[hh * D + lane + 32 * t] = v[t] * up;
      if (lane == 0) fh[hh] = __int_as_float((127 - sh) << 23);
    }
    __syncthreads();
    // B fragments: lane (g, c) of k-step kk = 2 blk + half holds, of column g,
    // dims 32 blk + 16 half + 4c + {0, 2} (k slots 2c, 2c+1) and + {1, 3} (slots
    // 2c+8, 2c+9), hi and lo (packed: the column's part); the upper half-bytes
    // count 16-fold, so theirs are divided by 16.
    uint4* qf = reinterpret_cast<uint4*>(smem + C::kOffQf);
    for (int i = tid; i < NH * KS * 32; i += kThreads4) {
      const int ln = i & 31, kk = (i >> 5) % KS, ht = i / (32 * KS);
      const int head = kPack ? ln >> 3 : ht * 8 + (ln >> 2);
      const float* q = qs + head * D + 16 * kk + 4 * (ln & 3);
      const float f = kk & 1 ? 0.0625f : 1.f;
      uint4 a;  // {hi, hi, lo, lo}
      attn_split2(q[0] * f, q[2] * f, a.x, a.z);
      attn_split2(q[1] * f, q[3] * f, a.y, a.w);
      if constexpr (kPack)
        reinterpret_cast<uint2*>(qf)[i] = ln & 4 ? make_uint2(a.z, a.w) : make_uint2(a.x, a.y);
      else
        qf[i] = a;
    }
    __syncthreads();
    float fac[NH][HC];
#pragma unroll
    for (int u = 0; u < NH; ++u)
#pragma unroll
      for (int x = 0; x < HC; ++x) fac[u][x] = fh[u * 8 + HC * cq + x];

    // o[u][2 blk + half]: dims 32 blk + 16 half + 2 gq + {0 ([0], [1]), 1 ([2], [3])}, columns 2cq, 2cq+1
    float o[NH][2 * NB][4];
    // this lane's heads: the running maximum m (log2), the raw score that
    // moves it, and this lane's sum of P
    float m[NH][HC], top[NH][HC], l[NH][HC];
#pragma unroll
    for (int u = 0; u < NH; ++u) {
#pragma unroll
      for (int x = 0; x < HC; ++x) {
        m[u][x] = top[u][x] = -INFINITY;
        l[u][x] = 0.f;
      }
#pragma unroll
      for (int t = 0; t < 2 * NB; ++t) o[u][t][0] = o[u][t][1] = o[u][t][2] = o[u][t][3] = 0.f;
    }

    for (int i = 0; i < my_tiles; ++i) {
      load_tile(i + kStages4 - 1);
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages4 - 1) : "memory");
      __syncwarp();
      const int nr = min(kTile4, t_end - (t_begin + (warp + kWarps4 * i) * kTile4));
      const uint32_t st = ring + (i % kStages4) * C::kStage;
      const uint8_t* sc = smem + (st - smem_u32(smem)) + 2 * C::kQuants + gq * C::kSRow;  // token gq's scales

      // ---- S = K.Q^T ----
      uint32_t kw[NT][NB];
      if constexpr (D == 128) {
#pragma unroll
        for (int j = 0; j < NT; ++j) ldsm4(st + k_off + j * 8 * C::kRow, kw[j]);
      } else {
#pragma unroll
        for (int j = 0; j < NT; j += 2) {
          uint32_t r[4];
          ldsm4(st + k_off + j * 8 * C::kRow, r);
          kw[j][0] = r[0];
          kw[j][1] = r[1];
          kw[j + 1][0] = r[2];
          kw[j + 1][1] = r[3];
        }
      }
      uint32_t ksc[NT][NB / 2];
#pragma unroll
      for (int j = 0; j < NT; ++j) scales4<NB>(sc + j * 8 * C::kSRow, ksc[j]);
      // raw scores of tokens 8j + gq, columns 2cq, 2cq+1 of each tile, in units of fac
      float s[NH][NT][2];
#pragma unroll
      for (int bb = 0; bb < NB; ++bb) {
        uint32_t a[NT / 2][8];  // A fragments of 16 tokens: k-steps 2 bb and 2 bb + 1
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const uint32_t w = kw[j][bb], w8 = w >> 8;
          uint32_t* f = a[j / 2] + j % 2;
          f[0] = nib8<false>(w, k1024);
          f[2] = nib8<false>(w8, k1024);
          f[4] = nib8<true>(w, k1024);
          f[6] = nib8<true>(w8, k1024);
        }
#pragma unroll
        for (int u = 0; u < NH; ++u) {
          uint4 q0, q1;
          if constexpr (kPack) {
            const uint2* f = reinterpret_cast<const uint2*>(qf) + 2 * bb * 32 + lane;
            const uint2 x0 = f[0], x1 = f[32];
            q0 = make_uint4(x0.x, x0.y, 0u, 0u);
            q1 = make_uint4(x1.x, x1.y, 0u, 0u);
          } else {
            const uint4* f = qf + (u * KS + 2 * bb) * 32 + lane;
            q0 = f[0];
            q1 = f[32];
          }
#pragma unroll
          for (int h = 0; h < NT / 2; ++h) {
            float acc[4];
            mma4z(acc, a[h][0], a[h][1], a[h][2], a[h][3], q0.x, q0.y);
            if constexpr (!kPack) mma4(acc, a[h][0], a[h][1], a[h][2], a[h][3], q0.z, q0.w);
            mma4(acc, a[h][4], a[h][5], a[h][6], a[h][7], q1.x, q1.y);
            if constexpr (!kPack) mma4(acc, a[h][4], a[h][5], a[h][6], a[h][7], q1.z, q1.w);
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const float d = half_of(ksc[2 * h + y][bb / 2], bb & 1);
              float* r = s[u][2 * h + y];
              r[0] = bb ? fmaf(d, acc[2 * y], r[0]) : d * acc[2 * y];
              r[1] = bb ? fmaf(d, acc[2 * y + 1], r[1]) : d * acc[2 * y + 1];
            }
          }
        }
      }

      // ---- the running maximum ----
      float mx[NH][HC];
      bool above = false;
#pragma unroll
      for (int u = 0; u < NH; ++u) {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          if constexpr (kPack) s[u][j][0] += s[u][j][1];
          if (nr < kTile4 && 8 * j + gq >= nr) s[u][j][0] = s[u][j][1] = -INFINITY;
        }
#pragma unroll
        for (int x = 0; x < HC; ++x) {
          mx[u][x] = fmaxf(fmaxf(s[u][0][x], s[u][1][x]), fmaxf(s[u][2][x], s[u][3][x]));
          above = above || mx[u][x] > top[u][x];
        }
      }
      if (__any_sync(0xffffffffu, above)) {  // (rare after the first tiles)
#pragma unroll
        for (int u = 0; u < NH; ++u) {
          float cr[HC];
#pragma unroll
          for (int x = 0; x < HC; ++x) {
            float z = mx[u][x];
#pragma unroll
            for (int of = 4; of < 32; of <<= 1) z = fmaxf(z, __shfl_xor_sync(0xffffffffu, z, of));
            const float mn = fmaxf(m[u][x], z * fac[u][x]);
            cr[x] = m[u][x] == -INFINITY ? 0.f : ex2(m[u][x] - mn);
            m[u][x] = mn;
            // (fac is a power of two: its inverse, exactly)
            top[u][x] = (mn + kSlack4) * __uint_as_float(0x7f000000u - __float_as_uint(fac[u][x]));
            l[u][x] *= cr[x];
          }
#pragma unroll
          for (int t = 0; t < 2 * NB; ++t) {
            o[u][t][0] *= cr[0];
            o[u][t][1] *= cr[HC - 1];
            o[u][t][2] *= cr[0];
            o[u][t][3] *= cr[HC - 1];
          }
        }
      }

      // ---- P, then O += (P * scale) . V per block; a block's products of the
      // tile from zero ----
      float p[NT / 2][NH][2][HC];
#pragma unroll
      for (int h = 0; h < NT / 2; ++h)
#pragma unroll
        for (int u = 0; u < NH; ++u)
#pragma unroll
          for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int x = 0; x < HC; ++x)
              p[h][u][y][x] = ex2(fmaf(s[u][2 * h + y][x], fac[u][x], -m[u][x]));
#pragma unroll
      for (int u = 0; u < NH; ++u)
#pragma unroll
        for (int x = 0; x < HC; ++x) l[u][x] += (p[0][u][0][x] + p[0][u][1][x]) + (p[1][u][0][x] + p[1][u][1][x]);
      static_assert(NT == 4, "");
#pragma unroll
      for (int bp = 0; bp < NB / 2; ++bp) {
        uint32_t vw[NT / 2][4], vsc[NT];  // 16 tokens' words each; the scales of tokens gq, gq + 8, ..
#pragma unroll
        for (int h = 0; h < NT / 2; ++h) ldsm4t(st + v_off[bp] + h * 16 * C::kRow, vw[h]);
#pragma unroll
        for (int j = 0; j < NT; ++j)
          vsc[j] = *reinterpret_cast<const uint32_t*>(sc + C::kScales + j * 8 * C::kSRow + 4 * bp);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int bb = 2 * bp + x;
          float lo[NH][4], up[NH][4];
#pragma unroll
          for (int h = 0; h < NT / 2; ++h) {
            const uint32_t w0 = vw[h][2 * x], w1 = vw[h][2 * x + 1];
            const uint32_t l0 = nib8b(w0, k128), l1 = nib8b(w0 >> 8, k128), l2 = nib8b(w1, k128),
                           l3 = nib8b(w1 >> 8, k128);
            const uint32_t u0 = nib8b(w0 >> 4, k128), u1 = nib8b(w0 >> 12, k128), u2 = nib8b(w1 >> 4, k128),
                           u3 = nib8b(w1 >> 12, k128);
            const float d0 = half_of(vsc[2 * h], x), d1 = half_of(vsc[2 * h + 1], x);
#pragma unroll
            for (int u = 0; u < NH; ++u) {
              // tokens gq and gq + 8 of the columns 2cq, 2cq+1, transposed into
              // B fragments
              const float(&ph)[2][HC] = p[h][u];
              uint32_t b[3][2];
              if constexpr (kPack) {  // columns (hi, mid), then (0, lo)
                const Parts3 a(mul2(pack2(ph[0][0], ph[1][0]), pack2(d0, d1)));
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                  b[0][y] = transpose8(upper2(a.hi[y], a.mid[y]));
                  b[1][y] = transpose8(__float_as_uint(a.lo[y]) & 0xffff0000u);
                }
              } else {
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                  const float d = y ? d1 : d0;
                  const Parts3 a(mul2(pack2(ph[y][0], ph[y][HC - 1]), pack2(d, d)));
                  b[0][y] = transpose8(upper2(a.hi[0], a.hi[1]));
                  b[1][y] = transpose8(upper2(a.mid[0], a.mid[1]));
                  b[2][y] = transpose8(upper2(a.lo[0], a.lo[1]));
                }
              }
#pragma unroll
              for (int i = 0; i < (kPack ? 2 : 3); ++i) {
                if (h == 0 && i == 0) {
                  mma4bz(lo[u], l0, l1, l2, l3, b[i][0], b[i][1]);
                  mma4bz(up[u], u0, u1, u2, u3, b[i][0], b[i][1]);
                } else {
                  mma4b(lo[u], l0, l1, l2, l3, b[i][0], b[i][1]);
                  mma4b(up[u], u0, u1, u2, u3, b[i][0], b[i][1]);
                }
              }
            }
          }
#pragma unroll
          for (int u = 0; u < NH; ++u) {
            add4(o[u][2 * bb], lo[u]);
            add4(o[u][2 * bb + 1], up[u]);
          }
        }
      }
      __syncwarp();  // the stage is rewritten next
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");

    // ---- merge the warps' {m, l, O}; write the chunk's partial ----
    __syncthreads();
    float* mm = reinterpret_cast<float*>(smem);
    float* ll = mm + kWarps4 * kHeads;
    float* oo = ll + kWarps4 * kHeads;
#pragma unroll
    for (int u = 0; u < NH; ++u) {
#pragma unroll
      for (int x = 0; x < HC; ++x) {
        const int row = warp * kHeads + 8 * u + HC * cq + x;
        float sum = l[u][x];
#pragma unroll
        for (int of = 4; of < 32; of <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, of);
        if (gq == 0) {
          mm[row] = m[u][x];
          ll[row] = sum;
        }
#pragma unroll
        for (int t = 0; t < 2 * NB; ++t) {
          const float* v = o[u][t];
          *reinterpret_cast<float2*>(oo + row * C::kOStride + 16 * t + 2 * gq) =
              kPack ? make_float2(v[0] + v[1], v[2] + v[3]) : make_float2(v[x], v[2 + x]);
        }
      }
    }
    __syncthreads();
    // head h's weights of the warps (each replaces its maximum), its sum
    if (tid < G) {
      const int h = tid;
      float M = -INFINITY, lsum = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps4; ++w) M = fmaxf(M, mm[w * kHeads + h]);
#pragma unroll
      for (int w = 0; w < kWarps4; ++w) {
        const float mw = mm[w * kHeads + h];
        const float wgt = mw == -INFINITY ? 0.f : ex2(mw - M);  // (a warp without a tile)
        mm[w * kHeads + h] = wgt;
        lsum = fmaf(ll[w * kHeads + h], wgt, lsum);
      }
      if (kWhole) {
        ll[h] = lsum;  // (its own column's first entry)
      } else {
        const long long hq = (long long)b * P.n_heads + (long long)g * G + h;
        P.ws_m[hq * P.nc + c] = M;
        P.ws_l[hq * P.nc + c] = lsum;
      }
    }
    __syncthreads();
    for (int e = tid; e < G * (D / 4); e += kThreads4) {
      const int h = e / (D / 4), j = e % (D / 4) * 4;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps4; ++w) {
        const float wgt = mm[w * kHeads + h];
        const float4 x = *reinterpret_cast<const float4*>(oo + (w * kHeads + h) * C::kOStride + j);
        acc.x = fmaf(x.x, wgt, acc.x);
        acc.y = fmaf(x.y, wgt, acc.y);
        acc.z = fmaf(x.z, wgt, acc.z);
        acc.w = fmaf(x.w, wgt, acc.w);
      }
      const long long hq = (long long)b * P.n_heads + (long long)g * G + h;
      if (kWhole) {
        float* o1 = P.out + hq * D + j;
        const float sum = ll[h];
        o1[0] = acc.x / sum, o1[1] = acc.y / sum, o1[2] = acc.z / sum, o1[3] = acc.w / sum;
      } else {
        *reinterpret_cast<float4*>(P.ws_o + (hq * P.nc + c) * D + j) = acc;
      }
    }
    if (!seq_next4(P, sq)) break;
  }
}

// out = sum_c 2^(m_c - M) O_c / sum_c 2^(m_c - M) l_c over the chunks of one
// (sequence, query head).  The kernel is all latency (one dependent launch),
// so it asks for everything at once: the lengths before it waits for the
// partials, then D/4 lanes a chunk keep up to kMine4 16-byte pieces of O in
// flight while the first threads fetch m and l and work out the weights.
constexpr int kCombThreads4 = 512;  // and chunks at most: a thread has one's m and l
constexpr int kMine4 = 5;  // chunks a thread, at a time

template <int D>
__global__ void __launch_bounds__(kCombThreads4) gqa_q4kv_combine_kernel(const AttnParams P) {
  constexpr int kLanes = D / 4, kGroups = kCombThreads4 / kLanes;
  __shared__ float wt[kCombThreads4], red[2][kCombThreads4 / 32];
  __shared__ float4 so[kGroups][kLanes];
  const int hq = blockIdx.x, b = hq / P.n_heads;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int j = tid % kLanes, grp = tid / kLanes;
  // the attention grid released this one after its own wait: the lengths are
  // readable
  const Split4 sp = split4<false>(P, lane);
  int L;
  const int at = seq_of4(P, sp, b, lane, L);
  const int nact = (at + tiles4(L) - 1) / sp.piece - at / sp.piece + 1;
  griddep_wait();               // the partials are complete and visible
  griddep_launch_dependents();  // (not earlier: the next kernel would take SMs from this one)
  float* o = P.out + (long long)hq * D;
  if (L < 1) {
    if (grp == 0) {
      const float q = __int_as_float(0x7fc00000);
      for (int i = 0; i < 4; ++i) o[4 * j + i] = q;
    }
    return;
  }
  const float* O = P.ws_o + (long long)hq * P.nc * D;
  float4 v[kMine4];
#pragma unroll
  for (int u = 0; u < kMine4; ++u) {
    const int c = grp + u * kGroups;
    v[u] = c < nact ? __ldcg(reinterpret_cast<const float4*>(O + (long long)c * D) + j)
                    : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  const float mc = tid < nact ? __ldcg(P.ws_m + (long long)hq * P.nc + tid) : -INFINITY;
  const float lc = tid < nact ? __ldcg(P.ws_l + (long long)hq * P.nc + tid) : 0.f;
  float M = mc;
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, s));
  if (lane == 0) red[0][warp] = M;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kCombThreads4 / 32; ++w) M = fmaxf(M, red[0][w]);
  const float w = mc == -INFINITY ? 0.f : ex2(mc - M);
  wt[tid] = w;
  float ls = lc * w;
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, s);
  if (lane == 0) red[1][warp] = ls;
  __syncthreads();
  float lsum = 0.f;
#pragma unroll
  for (int x = 0; x < kCombThreads4 / 32; ++x) lsum += red[1][x];
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int u0 = 0; grp + u0 * kGroups < nact; u0 += kMine4) {
#pragma unroll
    for (int u = 0; u < kMine4; ++u) {
      const int c = grp + (u0 + u) * kGroups;
      if (c >= nact) break;
      const float4 x = u0 == 0 ? v[u] : __ldcg(reinterpret_cast<const float4*>(O + (long long)c * D) + j);
      const float g = wt[c];
      acc.x = fmaf(x.x, g, acc.x);
      acc.y = fmaf(x.y, g, acc.y);
      acc.z = fmaf(x.z, g, acc.z);
      acc.w = fmaf(x.w, g, acc.w);
    }
  }
  so[grp][j] = acc;
  __syncthreads();
  if (tid < D) {
    float s = 0.f;
#pragma unroll
    for (int x = 0; x < kGroups; ++x) s += reinterpret_cast<const float*>(so[x])[tid];
    o[tid] = s / lsum;
  }
}

// The same by a warp a (sequence, query head), lanes holding D/32 dims, for
// many heads, which as blocks of their own would take several waves.  The
// whole call, blocks / warps: 32 ragged sequences of 16 heads up to 8192 rows,
// 50.0 / 47.4 us; 20 of 32 heads up to 1000 rows, 19.2 / 15.8.  With many
// chunks and few heads its loads are too few at a time: 8 ragged of 28 heads
// up to 32768 rows, 33.3 / 37.9; 6 of 24 heads, 2000 rows, 9.4 / 13.5.
constexpr int kFewThreads4 = 256;

template <int D>
__global__ void __launch_bounds__(kFewThreads4) gqa_q4kv_combine_few_kernel(const AttnParams P) {
  constexpr int kV = D / 32;
  const int lane = threadIdx.x & 31;
  const int hq = blockIdx.x * (kFewThreads4 / 32) + (threadIdx.x >> 5);
  const Split4 sp = split4<false>(P, lane);  // (readable, as above)
  const bool live = hq < P.batch * P.n_heads;
  int L;
  const int b = live ? hq / P.n_heads : 0, at = seq_of4(P, sp, b, lane, L);
  const int nact = (at + tiles4(L) - 1) / sp.piece - at / sp.piece + 1;
  griddep_wait();
  griddep_launch_dependents();
  if (!live) return;
  float* o = P.out + (long long)hq * D + kV * lane;
  const float* O = P.ws_o + (long long)hq * P.nc * D + kV * lane;
  const float *wm = P.ws_m + (long long)hq * P.nc, *wl = P.ws_l + (long long)hq * P.nc;
  float acc[kV], M = -INFINITY, lsum = 0.f;
#pragma unroll
  for (int i = 0; i < kV; ++i) acc[i] = 0.f;
  if (L < 1) lsum = __int_as_float(0x7fc00000);
  for (int c0 = 0; L >= 1 && c0 < nact; c0 += 32) {
    const int nc = min(32, nact - c0);
    const float mc = lane < nc ? __ldcg(wm + c0 + lane) : -INFINITY;
    const float lc = lane < nc ? __ldcg(wl + c0 + lane) : 0.f;
    float mx = mc;
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
    mx = fmaxf(M, mx);
    const float old = M == -INFINITY ? 0.f : ex2(M - mx);
    M = mx;
    const float w = mc == -INFINITY ? 0.f : ex2(mc - M);
    float ls = lc * w;
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, s);
    lsum = fmaf(lsum, old, ls);
#pragma unroll
    for (int i = 0; i < kV; ++i) acc[i] *= old;
#pragma unroll 4
    for (int c = 0; c < nc; ++c) {
      const float g = __shfl_sync(0xffffffffu, w, c);
      const float* r = O + (long long)(c0 + c) * D;
      if constexpr (kV == 4) {
        const float4 v = __ldcg(reinterpret_cast<const float4*>(r));
        acc[0] = fmaf(v.x, g, acc[0]), acc[1] = fmaf(v.y, g, acc[1]);
        acc[2] = fmaf(v.z, g, acc[2]), acc[3] = fmaf(v.w, g, acc[3]);
      } else {
        const float2 v = __ldcg(reinterpret_cast<const float2*>(r));
        acc[0] = fmaf(v.x, g, acc[0]), acc[1] = fmaf(v.y, g, acc[1]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kV; ++i) o[i] = acc[i] / lsum;
}

template <int D, int NH, bool kPack, bool kWhole>
int launch_q4kv(AttnParams P, cudaStream_t stream) {
  using C = Cfg4<D, NH>;
  const auto fn = gqa_q4kv_kernel<D, NH, kPack, kWhole>;
  // (no carveout preference: a change of carveout between this kernel and
  // the next drains the SMs, 2 us a call)
  int rc = configure_kernel(reinterpret_cast<const void*>(fn), C::kSmem, false);
  if (rc) return rc;
  // one wave (two column tiles: a CTA an SM), and no more pieces than the
  // combine has threads
  const int wave = std::max(1, (NH == 1 ? 2 : 1) * sm_count() / P.n_kv_heads);
  P.nct = !kWhole ? std::min({P.nct, wave, kCombThreads4}) : P.batch == 1 ? 1 : wave;
  rc = launch_ex(fn, dim3(P.nct, P.n_kv_heads), dim3(kThreads4), (size_t)C::kSmem, stream, true, P);
  if (rc || kWhole) return rc;
  const long long heads = (long long)P.batch * P.n_heads;
  if (heads > 2LL * sm_count()) {
    constexpr int kPer = kFewThreads4 / 32;
    return launch_ex(gqa_q4kv_combine_few_kernel<D>, dim3((unsigned)((heads + kPer - 1) / kPer)),
                     dim3(kFewThreads4), 0, stream, true, P);
  }
  return launch_ex(gqa_q4kv_combine_kernel<D>, dim3((unsigned)heads), dim3(kCombThreads4), 0, stream, true, P);
}

template <int D, bool kWhole>
int launch_q4kv_g(const AttnParams& P, cudaStream_t stream) {
  const int G = P.n_heads / P.n_kv_heads;
  if (G <= 4) return launch_q4kv<D, 1, true, kWhole>(P, stream);
  if (G <= 8) return launch_q4kv<D, 1, false, kWhole>(P, stream);
  return launch_q4kv<D, 2, false, kWhole>(P, stream);
}

}  // namespace

int attn_q4kv_launch(const AttnParams& P, cudaStream_t stream) {
  if (P.cap <= kWholeCap4)
    return P.head_dim == 128 ? launch_q4kv_g<128, true>(P, stream) : launch_q4kv_g<64, true>(P, stream);
  return P.head_dim == 128 ? launch_q4kv_g<128, false>(P, stream) : launch_q4kv_g<64, false>(P, stream);
}

}  // namespace q8d
