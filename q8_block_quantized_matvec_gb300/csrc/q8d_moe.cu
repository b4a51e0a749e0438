// A mixture-of-experts feed-forward layer over Q8_0 experts for a few
// tokens: router, choice of experts, gate and up products with SiLU, down
// products with the weighted sum over a token's experts.
#include <algorithm>
#include <cmath>

#include "q8d_internal.cuh"
#include "q8d_moe.cuh"

namespace q8d {
namespace {

constexpr int kMoeThreads = 256;

// scale * quant . x over one Q8_0 row, by a warp.
__device__ __forceinline__ float row_dot(const uint8_t* row, const float* x, int n, int lane) {
  float s = 0.f;
  for (int b = 0; b < n / kQBlock; ++b) {
    const uint8_t* blk = row + (size_t)b * kQBlockBytes;
    const float d = f16_bits_to_f32(*reinterpret_cast<const unsigned short*>(blk));
    s = fmaf(d * (float)(int8_t)blk[2 + lane], x[b * kQBlock + lane], s);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// Router logits in f64: the choice among experts of nearly equal rank must
// not depend on the order of a sum.  A warp per (token, expert).
__global__ void moe_router_kernel(const MoeParams P) {
  griddep_launch_dependents();
  griddep_wait();
  const int w = (blockIdx.x * blockDim.x + threadIdx.x) >> 5, lane = threadIdx.x & 31;
  if (w >= P.m * P.n_experts) return;
  const int t = w / P.n_experts, e = w % P.n_experts;
  double s = 0.0;
  for (int i = lane; i < P.hidden; i += 32)
    s = fma((double)P.X[(long long)t * P.ldx + i], (double)P.router[(long long)e * P.hidden + i], s);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) P.logits[w] = s;
}

// The top_k experts of a token, largest logit first (ties: the lower
// index; NaN last), and their weights.  A warp per token.
__global__ void moe_choose_kernel(const MoeParams P) {
  griddep_launch_dependents();
  griddep_wait();
  const int t = blockIdx.x, lane = threadIdx.x;
  constexpr int kPer = kMoeMaxExperts / 32;
  double l[kPer];
  double mx = -INFINITY, sum = 0.0;
  for (int i = 0; i < kPer; ++i) {
    const int e = lane + 32 * i;
    l[i] = e < P.n_experts ? P.logits[t * P.n_experts + e] : -INFINITY;
    mx = fmax(mx, l[i]);
  }
  for (int o = 16; o > 0; o >>= 1) mx = fmax(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  for (int i = 0; i < kPer; ++i)
    if (lane + 32 * i < P.n_experts) sum += exp(l[i] - mx);
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  uint32_t taken = 0;
  double chosen = 0.0, mine = 0.0;
  for (int k = 0; k < P.top_k; ++k) {
    double best = -INFINITY;
    int at = 0x7fffffff;
    for (int i = 0; i < kPer; ++i) {
      const int e = lane + 32 * i;
      if (e >= P.n_experts || (taken >> i & 1u)) continue;
      const double v = isnan(l[i]) ? -INFINITY : l[i];
      if (v > best || (v == best && e < at)) best = v, at = e;
    }
    for (int o = 16; o > 0; o >>= 1) {
      const double ob = __shfl_xor_sync(0xffffffffu, best, o);
      const int oa = __shfl_xor_sync(0xffffffffu, at, o);
      if (ob > best || (ob == best && oa < at)) best = ob, at = oa;
    }
    if ((at & 31) == lane) taken |= 1u << (at >> 5);
    const double p = exp(P.logits[t * P.n_experts + at] - mx) / sum;
    chosen += p;
    if (lane == k) mine = p, P.experts[t * P.top_k + k] = at;
  }
  if (lane < P.top_k) P.weights[t * P.top_k + lane] = (float)(P.norm ? mine / chosen : mine);
}

// h[t][k][r] = silu(gate) * up: a warp per (token, slot, row).
__global__ void moe_gate_up_kernel(const MoeParams P) {
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, pair = blockIdx.y;
  const int r = (blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  if (r >= P.ffn) return;
  const size_t row = ((size_t)P.experts[pair] * P.ffn + r) * (P.hidden / kQBlock) * kQBlockBytes;
  const float* x = P.X + (long long)(pair / P.top_k) * P.ldx;
  const float g = row_dot(P.wg + row, x, P.hidden, lane), u = row_dot(P.wu + row, x, P.hidden, lane);
  if (lane == 0) P.h[(size_t)pair * P.ffn + r] = g / (1.f + expf(-g)) * u;
}

// y[t][r] = residual + sum_k w_k Wd_k[r] . h[t][k]: a warp per (token, row).
__global__ void moe_down_kernel(const MoeParams P) {
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, t = blockIdx.y;
  const int r = (blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  if (r >= P.hidden) return;
  float y = 0.f;
  for (int k = 0; k < P.top_k; ++k) {
    const int pair = t * P.top_k + k;
    const size_t row = ((size_t)P.experts[pair] * P.hidden + r) * (P.ffn / kQBlock) * kQBlockBytes;
    y = fmaf(P.weights[pair], row_dot(P.wd + row, P.h + (size_t)pair * P.ffn, P.ffn, lane), y);
  }
  if (P.residual) y += P.residual[(long long)t * P.ldr + r];
  if (lane == 0) P.Y[(long long)t * P.ldy + r] = y;
}

size_t up16(size_t n) { return (n + 15) / 16 * 16; }

}  // namespace

size_t moe_workspace_bytes(int m, int hidden, int ffn, int n_experts, int top_k) {
  (void)hidden;
  return up16(sizeof(double) * (size_t)m * n_experts) + up16(4 * (size_t)m * top_k) * 2 +
         4 * (size_t)m * top_k * ffn;
}

int moe_launch(MoeParams P, void* workspace, cudaStream_t stream) {
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  P.logits = reinterpret_cast<double*>(ws);
  ws += up16(sizeof(double) * (size_t)P.m * P.n_experts);
  if (!P.experts) P.experts = reinterpret_cast<int*>(ws);
  ws += up16(4 * (size_t)P.m * P.top_k);
  if (!P.weights) P.weights = reinterpret_cast<float*>(ws);
  ws += up16(4 * (size_t)P.m * P.top_k);
  P.h = reinterpret_cast<float*>(ws);
  const int warps = kMoeThreads / 32;
  const dim3 block(kMoeThreads);
  int rc = launch_ex(moe_router_kernel, dim3((P.m * P.n_experts + warps - 1) / warps), block, 0, stream, true, P);
  if (rc) return rc;
  rc = launch_ex(moe_choose_kernel, dim3(P.m), dim3(32), 0, stream, true, P);
  if (rc) return rc;
  rc = launch_ex(moe_gate_up_kernel, dim3((P.ffn + warps - 1) / warps, P.m * P.top_k), block, 0, stream, true, P);
  if (rc) return rc;
  return launch_ex(moe_down_kernel, dim3((P.hidden + warps - 1) / warps, P.m), block, 0, stream, true, P);
}

}  // namespace q8d
