// Parameters of the mixture-of-experts feed-forward kernels.
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace q8d {

constexpr int kMoeMaxTokens = 64;
constexpr int kMoeMaxExperts = 512;
constexpr int kMoeMaxTop = 32;

struct MoeParams {
  const float* X;  // token t at X + t * ldx
  int ldx;
  const float* router;  // [E][hidden]
  const uint8_t *wg, *wu, *wd;  // Q8_0 [E][ffn][hidden] x2, [E][hidden][ffn]
  const float* residual;  // or nullptr; token t at residual + t * ldr
  int ldr;
  float* Y;
  int ldy;
  int m, hidden, ffn, n_experts, top_k, norm;
  int* experts;    // [m][top_k] (the caller's, or in the workspace)
  float* weights;  // [m][top_k]
  int* d_err;
  // activation images in the workspace (q8d_moe.cu): rows of 144 bytes a
  // block of 32
  uint8_t *ximg, *himg;  // [m], [m * top_k]
  float* ypart;          // [m * top_k][hidden]
  uint32_t wait_limit;   // of the products' waits
};

size_t moe_workspace_bytes(int m, int hidden, int ffn, int n_experts, int top_k);
int moe_launch(MoeParams P, void* workspace, cudaStream_t stream);
void moe_set_wait_limit(uint32_t polls);  // of launches from now on; 0: the default

}  // namespace q8d
