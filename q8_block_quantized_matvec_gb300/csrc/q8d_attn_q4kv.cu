// Split-K decode attention over a 4-bit KV cache (Q8D_KV_Q4): the contract
// and the split of the other decode-attention kernels.
//
// One CTA per (sequence, KV head, chunk); its warps take tokens in turn with
// their own online softmax, lane j holding element j of every block, and
// merge once.
#include "q8d_attn.cuh"
#include "q8d_attn_common.cuh"
#include "q8d_internal.cuh"
#include "q8d_kv_rows.cuh"

namespace q8d {
namespace {

constexpr int kWarps4 = 4;
constexpr float kLog2e4 = 1.4426950408889634f;

template <int D, int GMAX>
__global__ void __launch_bounds__(kWarps4 * 32) gqa_q4kv_kernel(const AttnParams P) {
  constexpr int NB = D / 32;
  __shared__ AttnWindow s_win;
  __shared__ float sm[kWarps4][GMAX], sl[kWarps4][GMAX];
  __shared__ float so[kWarps4][GMAX][D];
  const int g = blockIdx.y;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int G = P.n_heads / P.n_kv_heads;
  griddep_launch_dependents();
  griddep_wait();
  int b, c, n;
  if (!attn_chunk_of(P, blockIdx.x, b, c, n)) return;
  const int L = attn_window_len(P, b);
  if (L < 1) {
    if (g == 0 && tid == 0 && P.d_err) atomicOr(P.d_err, Q8D_DERR_LEN_RANGE);
    return;
  }
  const int tpc = (L + n - 1) / n;
  const int t_begin = c * tpc;
  if (t_begin >= L) return;
  const int t_end = min(L, t_begin + tpc);
  if (tid == 0) attn_window_store(P, b, &s_win);
  const int width = P.n_kv_heads * D;
  const long long seq_off = (long long)b * (P.batch_stride / kQBlock) * 18;
  const long long splane = q4_scale_plane(P.cap, width);
  uint8_t* kq = static_cast<uint8_t*>(P.kcache) + seq_off + g * (D / 2);
  uint8_t* vq = static_cast<uint8_t*>(P.vcache) + seq_off + g * (D / 2);
  uint8_t* ks = static_cast<uint8_t*>(P.kcache) + seq_off + splane + g * (D / 16);
  uint8_t* vs = static_cast<uint8_t*>(P.vcache) + seq_off + splane + g * (D / 16);
  if (P.k_new != nullptr && t_end == L && warp < 2) {
    const float* src = (warp ? P.v_new : P.k_new) + (long long)b * width + (long long)g * D;
    const long long row = attn_cell(P, b, L - 1);
    for (int t = 0; t < NB; ++t)
      quantize_q4_warp(src[lane + 32 * t], (warp ? vq : kq) + row * (width / 2) + 16 * t,
                       (warp ? vs : ks) + row * (width / 16) + 2 * t, lane);
  }
  __syncthreads();
  float q[GMAX][NB], o[GMAX][NB], m[GMAX], l[GMAX];
#pragma unroll
  for (int h = 0; h < GMAX; ++h) {
    m[h] = -INFINITY;
    l[h] = 0.f;
#pragma unroll
    for (int t = 0; t < NB; ++t) {
      q[h][t] = h < G ? P.q[((long long)b * P.n_heads + g * G + h) * D + lane + 32 * t] *
                            (P.scale * kLog2e4)
                      : 0.f;
      o[h][t] = 0.f;
    }
  }
  for (int t = t_begin + warp; t < t_end; t += kWarps4) {
    const long long row = s_win.cell_of(t);
    float k[NB], v[NB];
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int sh = lane & 16 ? 4 : 0;
      const uint32_t nk = kq[row * (width / 2) + 16 * i + (lane & 15)] >> sh & 15u;
      const uint32_t nv = vq[row * (width / 2) + 16 * i + (lane & 15)] >> sh & 15u;
      k[i] = ((float)nk - 8.f) *
             f16_bits_to_f32(*reinterpret_cast<unsigned short*>(ks + row * (width / 16) + 2 * i));
      v[i] = ((float)nv - 8.f) *
             f16_bits_to_f32(*reinterpret_cast<unsigned short*>(vs + row * (width / 16) + 2 * i));
    }
#pragma unroll
    for (int h = 0; h < GMAX; ++h) {
      if (h >= G) break;
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < NB; ++i) s = fmaf(q[h][i], k[i], s);
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
      const float mn = fmaxf(m[h], s);
      const float r = m[h] == -INFINITY ? 0.f : exp2f(m[h] - mn), p = exp2f(s - mn);
      l[h] = l[h] * r + p;
#pragma unroll
      for (int i = 0; i < NB; ++i) o[h][i] = fmaf(o[h][i], r, p * v[i]);
      m[h] = mn;
    }
  }
#pragma unroll
  for (int h = 0; h < GMAX; ++h) {
    if (lane == 0) sm[warp][h] = m[h], sl[warp][h] = l[h];
#pragma unroll
    for (int i = 0; i < NB; ++i) so[warp][h][lane + 32 * i] = o[h][i];
  }
  __syncthreads();
  for (int e = tid; e < G * D; e += kWarps4 * 32) {
    const int h = e / D, j = e % D;
    float M = -INFINITY, acc = 0.f, lsum = 0.f;
    for (int w = 0; w < kWarps4; ++w) M = fmaxf(M, sm[w][h]);
    for (int w = 0; w < kWarps4; ++w) {
      if (sm[w][h] == -INFINITY) continue;
      const float wgt = exp2f(sm[w][h] - M);
      acc = fmaf(so[w][h][j], wgt, acc);
      lsum = fmaf(sl[w][h], wgt, lsum);
    }
    const long long hq = (long long)b * P.n_heads + (long long)g * G + h;
    P.ws_o[(hq * P.nc + c) * D + j] = acc;
    if (j == 0) {
      P.ws_m[hq * P.nc + c] = M;
      P.ws_l[hq * P.nc + c] = lsum;
    }
  }
}

template <int D, int GMAX>
int launch_q4kv(const AttnParams& P, cudaStream_t stream) {
  const int rc = launch_ex(gqa_q4kv_kernel<D, GMAX>, dim3(P.nct, P.n_kv_heads), dim3(kWarps4 * 32),
                           0, stream, true, P);
  return rc ? rc : attn_combine_launch(P, stream);
}

}  // namespace

int attn_q4kv_launch(const AttnParams& P, cudaStream_t stream) {
  const bool small = P.n_heads / P.n_kv_heads <= 8;
  if (P.head_dim == 128)
    return small ? launch_q4kv<128, 8>(P, stream) : launch_q4kv<128, 16>(P, stream);
  return small ? launch_q4kv<64, 8>(P, stream) : launch_q4kv<64, 16>(P, stream);
}

}  // namespace q8d
