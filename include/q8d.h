/*
 * q8d — Q8_0 single-token decode hot path for NVIDIA GB300 (sm_103a).
 *
 * C ABI.  Every pointer named d_* or documented as "device" is a device
 * pointer owned by the caller (the library never frees it).  Every compute
 * entry point is asynchronous on the CUDA stream passed as `stream`
 * (a cudaStream_t cast to void*; NULL means the legacy default stream) and
 * returns an int status:
 *     0               success (work enqueued)
 *     Q8D_EINVAL      null pointer or impossible size/shape
 *     Q8D_EALIGN      a pointer or stride breaks the stated alignment
 *     Q8D_EUNSUPPORTED a valid shape this build does not run
 *                     (n % 32 != 0, head_dim not 64/128, H % Hk != 0, ...)
 *     Q8D_ERANGE      an index/length outside its buffer (host-visible args)
 *     Q8D_ECUDA       a CUDA call failed; q8d_last_cuda_error() has the code
 *     Q8D_ETIMEOUT    a bounded host wait ran out
 *     Q8D_ENOMEM      the library's own allocation failed (step create; the
 *                     host's memory under a product's plan)
 * On any non-zero status nothing was launched (but where a call of several
 * launches gets Q8D_ECUDA for one behind the first).  There is no fallback path:
 * an unsupported case is refused, never computed another way.
 *
 * Quantities that live in device memory (positions, lengths, token ids) are
 * checked on the device: a bad value sets a bit in the caller's int error
 * word (Q8D_DERR_*), the affected write is skipped and the affected outputs
 * are set to NaN, so a silent no-write cannot pass for a result.
 *
 * Formats (from "IV.4: One command buffer per token", sections "Eight
 * kernels" and "The decoder: kernels and helpers"):
 *   Q8_0 block  34 bytes: little-endian IEEE binary16 scale (bytes 0-1) then
 *               32 two's-complement int8 quants (bytes 2-33); value of quant
 *               j is scale * q_j.
 *   Q8_0 matrix [p][n], row-major, n % 32 == 0: row r is n/32 consecutive
 *               blocks starting at byte r * (n/32) * 34 (no padding).
 *               The base must be 16-byte aligned.
 *   KV cache    per layer [cap][n_kv_heads * head_dim] of f32 or f16
 *               (Q8D_KV_F32 / Q8D_KV_F16); KV head g occupies columns
 *               [g*head_dim, (g+1)*head_dim) of every row ("minfer Metal
 *               Backend Design" / "Metal Backend Optimizations", the
 *               [nkv][nk*hd] layout shared with llama.cpp).
 *   Packed KV   Q8D_KV_Q8_0 ("minfer Metal Backend Design", "Execution
 *               dispatch": packed q8_0 KV): the same [cap][kv_width] cache
 *               stored as a Q8_0 matrix, row t = kv_width/32 consecutive
 *               34-byte blocks starting at byte t * kv_width/32 * 34, so
 *               KV head g is blocks [g*head_dim/32, (g+1)*head_dim/32).
 *               Rows are written by the Q8_0 quantizer: per block
 *               d = max|x| / 127, q_j = x_j * (1/d) rounded to nearest with
 *               halves away from zero, scale = d rounded to binary16, all in
 *               f32 (an all-zero block stores zeros); inputs must be finite
 *               (a NaN or an infinity leaves a block whose scale is NaN or
 *               infinite).
 *   4-bit KV    Q8D_KV_Q4: blocks of 32 elements as 16 bytes of quants and
 *               one binary16 scale, kept as two planes: row t's quants are
 *               the kv_width/2 bytes from byte t * kv_width/2 of the
 *               sequence's cache, its scales the kv_width/16 bytes from byte
 *               cap * kv_width/2 + t * kv_width/16 (9/16 bytes an element in
 *               all).  Byte i of a block holds element i in its low half and
 *               element i + 16 in its high half; value = scale * (n - 8) of
 *               the half-byte n.  The quantizer: m = the block's element of
 *               largest magnitude (the first of them), d = m / -8, id = 1/d
 *               (0 where that is not finite), n_j = floor(x_j * id + 8.5)
 *               limited to [0, 15], scale = d rounded to binary16, all in
 *               f32; inputs must be finite, and below 524160 in magnitude for
 *               a finite scale (65520 and more round to infinity).
 */
#ifndef Q8D_H
#define Q8D_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define Q8D_OK 0
#define Q8D_EINVAL (-1)
#define Q8D_EALIGN (-2)
#define Q8D_EUNSUPPORTED (-3)
#define Q8D_ERANGE (-4)
#define Q8D_ECUDA (-5)
#define Q8D_ETIMEOUT (-6)
#define Q8D_ENOMEM (-7)

#define Q8D_KV_F32 0
#define Q8D_KV_F16 1
#define Q8D_KV_Q8_0 2 /* packed: every cache row is kv_width/32 Q8_0 blocks */
#define Q8D_KV_Q4 4   /* 4-bit: a plane of quants, then a plane of scales (3 is no type) */

/* Bits of the device-side error word. */
#define Q8D_DERR_POS_RANGE 0x1   /* append position outside [0, cap)          */
#define Q8D_DERR_LEN_RANGE 0x2   /* attended length outside [1, cap]          */
#define Q8D_DERR_TOKEN_RANGE 0x4 /* token id outside [0, vocab)               */
#define Q8D_DERR_WAIT 0x8        /* a bounded in-kernel wait gave up          */

/* Library version (major*10000 + minor*100 + patch). */
int q8d_version(void);

/* Static text for a status code. */
const char* q8d_strerror(int status);

/* The cudaError_t of the last Q8D_ECUDA returned on this thread (0 if none). */
int q8d_last_cuda_error(void);

/* ------------------------------------------------------------------------
 * q8d_matvec — Q8_0 dequantising matrix-vector product
 * ("IV.4: One command buffer per token", "Eight kernels": q8_matvec).
 *   out[r] = sum_{b < n/32} scale(r,b) * sum_{j < 32} q(r,b,j) * x[32b + j]
 * x: device f32[n]; w_q8: device Q8_0 [p][n] (16-byte aligned);
 * out: device f32[p], fully overwritten, must not overlap x or w.
 * n % 32 == 0 (else Q8D_EUNSUPPORTED); n == 0 writes zeros; p == 0 is a
 * no-op.  f32 accumulation; x is used as given (never quantised).
 * ---------------------------------------------------------------------- */
int q8d_matvec(const float* x, const void* w_q8, float* out, int n, int p, void* stream);

/* ------------------------------------------------------------------------
 * q8d_matmul_small_m — the same weight matrix applied to m activations
 * ("Metal Backend Optimizations": the nt in [2, 8] batched-matvec gap and
 * the quantised GEMM tier for nt >= 2).
 *   Y[i][r] = sum_k X[i][k] * W[r][k],   i < m, r < p
 * X: device f32, row i at X + i*ldx (ldx >= n); Y: device f32, row i at
 * Y + i*ldy (ldy >= p), only the first p entries of each row are written.
 * m <= 8: f32-accurate paths (within 1e-5 of sum|terms| per output): the
 * tensor-core matvec with up to four activation rows per pass sharing every
 * decoded weight block (exact f16 quants, activations split into f16 hi +
 * lo, f32 accumulation) where the shape suits it (n % 256 == 0, n >= 2048,
 * p >= 16 rows per SM, the rows' activation fragments in shared memory),
 * else CUDA cores with the weights read once for up to four rows.
 * m >= 9 and n % 256 == 0: tensor-core path (tcgen05.mma, f16 operands:
 * the weights as f16 of scale * q, rounded once; the activations as f16
 * under a power-of-two scale per row, rounded once; f32 accumulation):
 * relative accuracy ~2^-11 per product, i.e. within 2e-3 of sum|terms|
 * per output (plus 2^-25 * sum|x| where scale * q is below 2^-14).  Block
 * scales above 511.75 (scale * q beyond f16) make the outputs of their
 * 128-row tile NaN.  It first writes the activations, rounded to f16, into
 * a workspace laid out as the MMA's B operand, with the rows' scales
 * (q8d_matmul_small_m_workspace_bytes(m, n) bytes); this entry point takes
 * that workspace from the stream's memory pool (cudaMallocAsync) and frees
 * it stream-ordered behind the kernels; q8d_matmul_small_m_ws uses the
 * caller's.  Other m >= 9 shapes run the f32 CUDA-core path.
 * 1 <= m <= 256; n % 32 == 0; X and w_q8 16-byte aligned, ldx % 4 == 0,
 * Y 4-byte aligned (Q8D_EALIGN otherwise); Y must not overlap X or w_q8
 * (Q8D_EINVAL).  m == 0 or p == 0: Q8D_OK, nothing written.
 * ---------------------------------------------------------------------- */
int q8d_matmul_small_m(const float* X, int ldx, const void* w_q8, float* Y, int ldy, int m,
                       int n, int p, void* stream);

/* Bytes of the workspace q8d_matmul_small_m_ws needs for m activation rows of
 * n elements: 2 * n * (m rounded up to 16 per block of 128 rows) + 16 *
 * ceil(m / 4) when the tensor-core path takes the shape (9 <= m <= 256,
 * n % 256 == 0), else 0. */
size_t q8d_matmul_small_m_workspace_bytes(int m, int n);

/* q8d_matmul_small_m with a caller-owned workspace: device memory of at
 * least q8d_matmul_small_m_workspace_bytes(m, n) bytes, 16-byte aligned,
 * overlapping none of X, w_q8 and Y, not in use by other work until the
 * call's kernels on `stream` have completed (the call writes it, then
 * reads it).  Q8D_EINVAL if it is needed and null or too small, or
 * overlaps an operand; Q8D_EALIGN if misaligned.  Unused (may be null)
 * when the size is 0. */
int q8d_matmul_small_m_ws(const float* X, int ldx, const void* w_q8, float* Y, int ldy, int m,
                          int n, int p, void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------
 * q8d_kv_append — write one token's K and V rows into the caches
 * ("IV.4: One command buffer per token", "Eight kernels": append_kv).
 *   kcache[pos][i] = cvt(k[i]), vcache[pos][i] = cvt(v[i]), i < kv_width
 * cvt is the identity for an f32 cache, round-to-nearest-even to binary16
 * for an f16 cache and the quantizer of each 32-element block for a packed
 * Q8_0 or a 4-bit cache (kv_width % 32 == 0, else Q8D_EUNSUPPORTED; the
 * stored bytes equal a scalar CPU quantizer's).  pos is read from device memory (*d_pos)
 * so a captured graph replays unchanged; pos outside [0, cap) sets
 * Q8D_DERR_POS_RANGE in *d_err and writes nothing.  k, v: device
 * f32[kv_width]; caches: device, cap rows (a packed or 4-bit cache 16-byte
 * aligned, else Q8D_EALIGN); d_err: device int (OR-ed into, never cleared).
 * ---------------------------------------------------------------------- */
int q8d_kv_append(const float* k, const float* v, void* kcache, void* vcache, int kv_dtype,
                  int kv_width, int cap, const int* d_pos, int* d_err, void* stream);

/* Bytes of one sequence's K (or V) cache of cap rows of kv_width elements;
 * 0 for a type, width or capacity that no cache has (kv_width % 32 != 0 for
 * a packed or 4-bit cache). */
size_t q8d_kv_cache_bytes(int kv_dtype, int kv_width, int cap);

/* ------------------------------------------------------------------------
 * q8d_kv_append_rows — store up to `rows` rows of every sequence of a batch
 * (a prompt, or one token of each sequence) into the caches.
 *   kcache[s][d_pos[s] + i] = cvt(k[s][i]), vcache likewise,
 *   s < batch, i < d_counts[s] (`rows` for every sequence if d_counts is
 *   NULL), with q8d_kv_append's cvt (f16 rows are exact in f32 first).
 * k, v: device rows of kv_width elements of row_dtype (Q8D_KV_F32 or
 *   Q8D_KV_F16); row i of sequence s starts at element (s * rows + i) * ld
 *   (ld >= kv_width: k and v may be columns of one projection's output);
 *   element-aligned, read 16 bytes at a time where the pointers and ld allow.
 * kcache, vcache: device, every kv_dtype; sequence s's cache of cap rows
 *   starts at element s * cache_batch_stride (at least cap * kv_width when
 *   batch > 1; starts must be 16-byte aligned: a multiple of 256 elements
 *   suits every type), and must not overlap k, v or each other.
 * d_pos, d_counts: device int[batch].  A count outside [0, rows] sets
 *   Q8D_DERR_LEN_RANGE, a row outside [0, cap) Q8D_DERR_POS_RANGE in *d_err
 *   (may be NULL), and nothing of that sequence is written; a count of 0
 *   writes nothing whatever the position.
 * kv_width % 32 == 0 for a packed or 4-bit cache; rows * (kv_width / 4,
 *   rounded up) at most 2^32 - 2^16, else Q8D_EUNSUPPORTED (above that, types
 *   that move eight elements at once still run).  rows == 0: no-op.
 * ---------------------------------------------------------------------- */
int q8d_kv_append_rows(const void* k, const void* v, int row_dtype, int ld, void* kcache,
                       void* vcache, int kv_dtype, int batch, int rows, int kv_width, int cap,
                       long long cache_batch_stride, const int* d_pos, const int* d_counts,
                       int* d_err, void* stream);

/* ------------------------------------------------------------------------
 * q8d_kv_read_rows — the values of cache rows (q8d_kv_append_rows reversed):
 *   k_out[s][i] = value of kcache[s][d_pos[s] + i], v_out likewise,
 *   s < batch, i < d_counts[s],
 * as f32 or f16 rows (row_dtype; f16 rounds to nearest even once).  Rows
 * i >= d_counts[s] of the outputs are left as they were; the rows of a
 * sequence whose count or position is refused (as above) are set to NaN,
 * all `rows` of them.  Other arguments as for q8d_kv_append_rows.
 * ---------------------------------------------------------------------- */
int q8d_kv_read_rows(const void* kcache, const void* vcache, int kv_dtype, void* k_out,
                     void* v_out, int row_dtype, int ld, int batch, int rows, int kv_width,
                     int cap, long long cache_batch_stride, const int* d_pos,
                     const int* d_counts, int* d_err, void* stream);

/* Bytes of scratch q8d_gqa_decode_attn needs for these sizes: the split-K
 * partials {m, l, O} of up to a fixed number of chunk slots per sequence
 * and query head (chunk CTAs are split over a batch in proportion to the
 * lengths, on the device).  Pass the cache capacity `cap` as max_len: the
 * call checks ws_bytes against the size for its cap. */
size_t q8d_gqa_workspace_bytes(int batch, int n_heads, int n_kv_heads, int head_dim, int max_len);

/* ------------------------------------------------------------------------
 * q8d_gqa_decode_attn — grouped-query attention of one query token per
 * sequence over a resident KV cache, split over the context ("IV.4: One
 * command buffer per token", "Eight kernels": attention_decode; "Metal
 * Backend Optimizations" 3.3, split-attention partial + combine).
 * For sequence s with length L = d_lens[s] (read on the device) and query
 * head h, KV head g = h / (n_heads / n_kv_heads):
 *   s_t = scale * q[s,h,:] . K[s][t][g*hd : (g+1)*hd],   t < L
 *   out[s,h,:] = sum_t softmax(s)_t * V[s][t][g*hd : (g+1)*hd]
 * If k_new/v_new are non-NULL, row L-1 of sequence s is first written with
 * cvt(k_new[s]), cvt(v_new[s]) (as q8d_kv_append) and the rounded values
 * are the ones attended to.
 *   q, out:  device f32 [batch][n_heads*head_dim]
 *   k_new, v_new: device f32 [batch][n_kv_heads*head_dim] or both NULL
 *   kcache, vcache: device; sequence s's cache starts at element
 *            s*cache_batch_stride, rows of n_kv_heads*head_dim elements,
 *            16-byte aligned, cap rows
 *   d_lens:  device int[batch]; 1 <= L <= cap, else Q8D_DERR_LEN_RANGE is
 *            set in *d_err and that sequence's outputs are NaN
 *   workspace: device scratch of at least
 *            q8d_gqa_workspace_bytes(batch, n_heads, n_kv_heads, head_dim, cap)
 *            bytes (contents need no initialisation)
 * head_dim in {64, 128}; n_heads % n_kv_heads == 0; n_heads/n_kv_heads <= 16;
 * every kv_dtype (a packed or 4-bit cache's stride is still in elements:
 * a multiple of 256, so that sequences start on 16-byte boundaries);
 * for a 4-bit cache cap at most 2^30 and batch * (cap / 32 + 17) below 2^30
 * (with run maps 4 cap), else Q8D_EUNSUPPORTED.
 * Over a 4-bit cache a score is off by at most 2^-21 of scale * sum_i
 * max(|q_i|, 2^-18 max |q|) |K_i|, in natural units, and given the scores an
 * output by 1e-5 of sum_t p_t |V_t|, however far apart the p_t and V's scales
 * lie (weights below 2^-126 of the largest are 0), for up to 2^20 rows a
 * sequence.
 * ---------------------------------------------------------------------- */
int q8d_gqa_decode_attn(const float* q, const float* k_new, const float* v_new, void* kcache,
                        void* vcache, int kv_dtype, float* out, int batch, int n_heads,
                        int n_kv_heads, int head_dim, int cap, long long cache_batch_stride,
                        const int* d_lens, float scale, void* workspace, size_t ws_bytes,
                        int* d_err, void* stream);

/* ------------------------------------------------------------------------
 * q8d_gqa_decode_attn_window — q8d_gqa_decode_attn over explicit KV windows
 * ("minfer Metal Backend Design", "Execution dispatch", window modes: an
 * explicit [lo, hi) span per query, or a map of up to four (cell, len) runs
 * per query, e.g. a prefix shared by several sequences plus a private run).
 * Sequence s attends exactly the cache rows of its runs, in run order:
 *   d_runs:  device int [batch][Q8D_MAX_RUNS][2], run r of sequence s is
 *            (cell, len) = (d_runs[s][r][0], d_runs[s][r][1]), the rows
 *            [cell, cell + len) of sequence s's cache; unused runs have
 *            len 0.  A span [lo, hi) is the single run (lo, hi - lo).
 *            Every run must lie in [0, cap) (0 <= cell, 0 <= len,
 *            cell + len <= cap) and the runs must hold at least one row in
 *            all and at most 2^31 - 1 (2^30 over a 4-bit cache), else
 *            Q8D_DERR_LEN_RANGE is set in *d_err and the sequence's outputs
 *            are NaN.
 *   cache_batch_stride: as for q8d_gqa_decode_attn, or 0: every sequence
 *            reads the same cache (shared cells, e.g. a common prefix).
 * With k_new/v_new the rounded new rows are first written at the LAST row
 * of each sequence's window (the last row of its last non-empty run) and
 * attended to; that row must not be read by another sequence of the same
 * call, nor lie in another run of its own window (writes and reads would
 * race).
 * Other arguments, the workspace and the results are those of
 * q8d_gqa_decode_attn (f32, f16, packed Q8_0 and 4-bit caches).
 * ---------------------------------------------------------------------- */
#define Q8D_MAX_RUNS 4
int q8d_gqa_decode_attn_window(const float* q, const float* k_new, const float* v_new,
                               void* kcache, void* vcache, int kv_dtype, float* out, int batch,
                               int n_heads, int n_kv_heads, int head_dim, int cap,
                               long long cache_batch_stride, const int* d_runs, float scale,
                               void* workspace, size_t ws_bytes, int* d_err, void* stream);

/* ------------------------------------------------------------------------
 * q8d_gqa_decode_attn_noalloc — q8d_gqa_decode_attn without a caller
 * workspace.  The pages have no counterpart to this entry point.
 * It exists for callers that cannot allocate device memory: code whose
 * device memory is owned by a host framework's allocator or pool that
 * forbids side allocations, and latency-sensitive loops that cannot afford
 * cudaMalloc's implicit device-wide synchronisation.  The split-K scratch
 * lives instead in one fixed array inside libq8d, of
 * q8d_noalloc_scratch_bytes() bytes (4 MiB) on every GPU that loads the
 * library, held until the process exits.  Arguments and results are those
 * of q8d_gqa_decode_attn (the caller still passes q, caches, out, lengths
 * and the error word); sizes whose scratch would exceed the array,
 * i.e. q8d_gqa_workspace_bytes(batch, n_heads, n_kv_heads, head_dim, cap)
 * > q8d_noalloc_scratch_bytes(), are refused with Q8D_ERANGE.
 * The call allocates nothing.  Its first call on a device looks up the
 * array's device address (cudaGetSymbolAddress, with that device current)
 * and caches it; make that first call before any stream capture.
 * All calls on a device share the one array, and it keeps the last call's
 * contents (nothing in it needs to start at zero): calls that overlap on the
 * GPU (different streams, or concurrent host threads) race on it.
 * ---------------------------------------------------------------------- */
size_t q8d_noalloc_scratch_bytes(void);
int q8d_gqa_decode_attn_noalloc(const float* q, const float* k_new, const float* v_new,
                                void* kcache, void* vcache, int kv_dtype, float* out, int batch,
                                int n_heads, int n_kv_heads, int head_dim, int cap,
                                long long cache_batch_stride, const int* d_lens, float scale,
                                int* d_err, void* stream);

/* ------------------------------------------------------------------------
 * q8d_moe_ffn — a mixture-of-experts feed-forward layer over Q8_0 experts
 * for a few tokens (the expert form of the dense gate / up / down products
 * of the decode step).  For token t with x = X[t]:
 *   l_e = sum_i router[e][i] * x[i],   p = softmax(l) over all experts
 *   the top_k experts of largest l (ties: the lower index; NaN last),
 *   largest first; w_k = p of the k-th, divided by their sum if norm_topk
 *   Y[t] = residual[t] + sum_k w_k * Wd_k (silu(Wg_k x) * (Wu_k x))
 * The logits and the choice are computed in pairs of f32 (about 48 bits), so
 * that neighbours in rank whose logits an f32 sum would confuse are told
 * apart; the weights w are f32 results, within 2^-21 of the softmax's.
 * The products are f32-accurate (within 1e-5 of their sums of |terms|).
 * Matrices of experts that no token chose are not read (but for up to 32 rows
 * behind an asked expert's down matrix); an expert's are read once for every
 * group of its tokens.  A group is 1, 2, 4, 8 or 16 tokens for the whole call,
 * about twice the mean m * top_k / n_experts and fewer where the experts' rows
 * leave no room: few experts that most tokens ask for are read several times.
 * Nothing depends on the order in which threads finish.
 *   X: device f32, token t at X + t*ldx (ldx >= hidden, ldx % 4 == 0),
 *      16-byte aligned
 *   router: device f32 [n_experts][hidden], 16-byte aligned
 *   wg, wu: device Q8_0 [n_experts][ffn][hidden], wd: [n_experts][hidden]
 *      [ffn], the experts' matrices one behind the other, 16-byte aligned
 *   residual: device f32, token t at residual + t*ldr (ldr >= hidden), or
 *      NULL; may be Y itself (same pointer, ldr == ldy)
 *   Y: device f32, token t at Y + t*ldy (ldy >= hidden); only the first
 *      hidden entries of a row are written
 *   experts, weights: device int / f32 [m][top_k], the choice made and its
 *      weights, or NULL
 *   workspace: device scratch of q8d_moe_workspace_bytes(m, hidden, ffn,
 *      n_experts, top_k) bytes, 16-byte aligned; its contents need no
 *      initialisation and belong to the call until its work on `stream` is
 *      done (calls that may overlap, or graphs replayed at the same time,
 *      need one each)
 *   d_err: device int error word (OR-ed into) or NULL; a wait that ran out
 *      sets Q8D_DERR_WAIT and makes the entries of Y it concerns NaN
 * 0 <= m <= 64 (m == 0: no-op), hidden % 32 == 0, ffn % 32 == 0,
 * 1 <= n_experts <= 512, 1 <= top_k <= min(n_experts, 32), hidden and ffn
 * at most 16384; else Q8D_EUNSUPPORTED.  Outputs must not overlap inputs
 * (but Y may be residual), the workspace or each other, a strided operand
 * counted whole from its first row's start to its last row's end.
 * ---------------------------------------------------------------------- */
size_t q8d_moe_workspace_bytes(int m, int hidden, int ffn, int n_experts, int top_k);
int q8d_moe_ffn(const float* X, int ldx, const float* router, const void* wg, const void* wu,
                const void* wd, const float* residual, int ldr, float* Y, int ldy, int m,
                int hidden, int ffn, int n_experts, int top_k, int norm_topk, int* experts,
                float* weights, void* workspace, size_t ws_bytes, int* d_err, void* stream);

/* Sets at which poll a wait inside the expert layer's products gives up (1:
 * without waiting; 0: the default, 2^24), for every later call of the process
 * and the graphs that capture it.  On expiry the call sets Q8D_DERR_WAIT, the
 * outputs that the unfinished products enter are NaN, the copies in flight are
 * waited for, and the CUDA context stays usable.  A small value is a way to
 * check that a caller's error handling sees such a call. */
int q8d_moe_set_wait_limit(unsigned polls);

/* ------------------------------------------------------------------------
 * The operators between the products of a dense layer, and products with
 * 4-bit weights: norm -> projections -> rotary positions and cache ->
 * attention -> projection + residual -> norm -> gated projections ->
 * projection + residual.  None needs a workspace.
 *   Operands that must not overlap may be columns of one buffer, where their
 * rows are the same number of bytes apart and share none; operands whose rows
 * are not count whole, from the first row's start to the last one's end.
 * ---------------------------------------------------------------------- */

/* ------------------------------------------------------------------------
 * q8d_rmsnorm_rows - root-mean-square norm of rows, with the residual's
 * addition before it:
 *   h = x + residual (h = x without one),  sum_out = h,
 *   y = h / sqrt(mean(h^2) + eps) * weight
 * in f32: h is rounded to f32 (and for sum_out to the rows' type; the norm
 * takes the f32 value), the mean is that of 64-bit arithmetic (within 2^-40),
 * the factor 1 / sqrt(...) is rounded to f32 once, and each product once, so
 * that an 8-bit output is that of the plain formula.
 *   x, residual, sum_out: device rows of row_dtype (Q8D_KV_F32 or Q8D_KV_F16),
 *      ldx, ldr, lds elements apart (>= n); residual and sum_out may be NULL,
 *      sum_out may be x or residual itself (same pointer and distance)
 *   weight: device f32[n]
 *   y: device rows of y_dtype, ldy elements apart (>= n): Q8D_KV_F32,
 *      Q8D_KV_F16, or Q8D_KV_Q8_0: rows of Q8_0 blocks, quantized as in a packed
 *      cache (n % 32 == 0; ldy % 32 == 0, row i at byte i * ldy / 32 * 34)
 * 1 <= n <= 16384 (else Q8D_EUNSUPPORTED), eps >= 0, rows >= 0 (0: no-op).
 * Pointers are aligned to their elements (y as Q8_0 to 2 bytes); 16-byte
 * accesses where all pointers and distances allow them.  y must not overlap
 * any other operand, nor sum_out one that it is not.  A row that holds a NaN or
 * an infinity gives what the formula gives in 64 bits (NaN or zeros; as Q8_0 a
 * block with a NaN among its values has the scale NaN).
 * ---------------------------------------------------------------------- */
int q8d_rmsnorm_rows(const void* x, const void* residual, void* sum_out, int row_dtype,
                     long long ldx, long long ldr, long long lds, const float* weight, float eps,
                     void* y, int y_dtype, long long ldy, int rows, int n, void* stream);

/* How the angles of rotary positions are scaled for long contexts. */
#define Q8D_ROPE_PLAIN 0
#define Q8D_ROPE_LINEAR 1 /* every angle / factor */
#define Q8D_ROPE_NTK 2    /* theta * factor^(rot_dim / (rot_dim - 2)) for theta */
#define Q8D_ROPE_YARN 3   /* fast pairs as they are, slow ones / factor, a ramp between */

/* Which elements of a head make a pair. */
#define Q8D_ROPE_HALF 0  /* i and i + rot_dim / 2 */
#define Q8D_ROPE_PAIRS 1 /* 2 i and 2 i + 1       */

/* ------------------------------------------------------------------------
 * q8d_rope_table - the cosines and sines of a model's rotary positions:
 *   table[pos][i] = mscale * cos(pos * f_i),
 *   table[pos][rot_dim / 2 + i] = mscale * sin(pos * f_i),
 *   pos < max_pos, i < rot_dim / 2, f_i = theta^(-2 i / rot_dim), scaled:
 *   linear f_i / factor; NTK as above; YaRN f_i / factor * r_i + f_i * (1 - r_i)
 *   with r_i = (i - low) / (high - low) limited to [0, 1], low and high the
 *   pairs that turn beta_fast and beta_slow times in orig_ctx positions
 *   (rot_dim ln(orig_ctx / (2 pi beta)) / (2 ln theta), low rounded down to at
 *   least 0, high up to at most rot_dim - 1, apart by at least 0.001)
 * worked out in 64 bits and rounded to f32 once.  table: device
 * f32[max_pos][rot_dim], 16-byte aligned.  rot_dim even and positive, theta > 1,
 * factor > 0, mscale finite (1 for none; YaRN's is 0.1 ln(factor) + 1);
 * orig_ctx, beta_fast and beta_slow > 0 are read for YaRN only; NTK needs
 * rot_dim > 2.
 * ---------------------------------------------------------------------- */
int q8d_rope_table(float* table, int max_pos, int rot_dim, double theta, int scaling,
                   double factor, double orig_ctx, double beta_fast, double beta_slow,
                   double mscale, void* stream);

/* What does not change from call to call of q8d_rope_append_rows (a host
 * struct, read during the call). */
typedef struct q8d_rope_desc {
  int n_heads, n_kv_heads, head_dim;
  int rot_dim;      /* elements of a head that turn: even, 0 .. head_dim */
  int layout;       /* Q8D_ROPE_HALF or Q8D_ROPE_PAIRS                   */
  int max_pos;      /* rows of the table                                */
  int row_dtype;    /* of q, k, v: Q8D_KV_F32 or Q8D_KV_F16             */
  int q_dtype;      /* of q_out: Q8D_KV_F32 or Q8D_KV_F16               */
  int kv_dtype;     /* of the caches: any Q8D_KV_*                      */
  int cap;          /* rows of a sequence's cache                       */
  float eps;        /* of the heads' norms                              */
  long long ldq;    /* elements from a row of q to the next             */
  long long ldkv;   /* of k and of v                                    */
  long long ldo;    /* of q_out                                         */
  long long cache_batch_stride; /* elements, as for q8d_kv_append_rows  */
  const float* table;           /* q8d_rope_table's; NULL if rot_dim is 0 */
  const float *bq, *bk, *bv;    /* f32 [heads * head_dim], or all NULL  */
  const float *q_norm, *k_norm; /* f32 [head_dim], or both NULL         */
} q8d_rope_desc;

/* ------------------------------------------------------------------------
 * q8d_rope_append_rows - up to `rows` rows of q, k and v of every sequence of
 * a batch (a prompt, or a token each) made ready for attention: the bias is
 * added, each q and k head normed (x / sqrt(mean(x^2) + eps) * q_norm or
 * k_norm), its first rot_dim elements turned by the row's position
 *   (a, b) -> (a cos - b sin, a sin + b cos),
 * q written to q_out, k and v stored in the caches as q8d_kv_append_rows
 * stores them.  Each step is one f32 rounding.
 *   Row i of sequence s, i < d_counts[s] (`rows` for every one if NULL), is row
 *   s * rows + i of q, k, v and q_out, goes to cache row d_pos[s] + i and is
 *   turned by position d_rope_pos[s] + i (d_pos[s] + i if d_rope_pos is NULL).
 *   q, k, v: device, row_dtype; they may be columns of one projection's output.
 *   q_out: device rows of q_dtype; may be q itself (same pointer, type and
 *      distance).  q and q_out may be NULL (k and v alone), or k, v, kcache and
 *      vcache (q alone; then d_pos gives the position only, unless d_rope_pos
 *      does).
 *   A count outside [0, rows] sets Q8D_DERR_LEN_RANGE, a row outside [0, cap) or
 *   a position outside [0, max_pos) Q8D_DERR_POS_RANGE in *d_err (may be NULL);
 *   nothing of that sequence is stored and all its `rows` rows of q_out become
 *   NaN.  Rows behind a count are left as they were.
 * head_dim a multiple of 8 (of 32 for a packed or 4-bit cache) up to 256,
 * else Q8D_EUNSUPPORTED; the caches' alignment and overlaps are those of
 * q8d_kv_append_rows, table 16-byte aligned.  rows == 0: no-op.
 * ---------------------------------------------------------------------- */
int q8d_rope_append_rows(const q8d_rope_desc* desc, const void* q, const void* k, const void* v,
                         void* q_out, void* kcache, void* vcache, int batch, int rows,
                         const int* d_pos, const int* d_rope_pos, const int* d_counts, int* d_err,
                         void* stream);

/* ------------------------------------------------------------------------
 * 4-bit weight matrices [p][n], n % 32 == 0, with a binary16 scale for every
 * group of 32, 64 or 128 neighbours of a row (the last group of a row may be
 * shorter): value = scale * (n_j - 8), n_j in 0..15.  The quantizer is the
 * 4-bit cache's, over a group: scale = the element of largest magnitude (the
 * first of them) / -8, n_j = floor(x_j / scale + 8.5) limited to [0, 15]; inputs
 * must be finite and below 524160 in magnitude.  The bytes are laid out for the
 * products (q8d_q4_pack makes them, once for a model):
 *   q8d_q4_matrix_bytes(p, n, group) bytes, 16-byte aligned: tiles of 16 rows by
 *   128 columns (filled up with zeros), those of 16 rows one behind the other;
 *   a tile is 1024 bytes of quants, then 16 * 128 / group scales.
 * ---------------------------------------------------------------------- */

/* Bytes of such a matrix; 0 for sizes that none has. */
size_t q8d_q4_matrix_bytes(int p, int n, int group);

/* Quantizes rows into a matrix.  src: device rows of src_dtype (Q8D_KV_F32,
 * Q8D_KV_F16, or Q8D_KV_Q8_0: rows of Q8_0 blocks), ld elements apart (>= n; for
 * Q8_0 ld % 32 == 0), aligned to their elements (Q8_0: 2 bytes); w_q4 must not
 * overlap it.  p == 0: no-op. */
int q8d_q4_pack(const void* src, int src_dtype, long long ld, void* w_q4, int p, int n, int group,
                void* stream);

/* The values of a matrix as rows of dst_dtype (Q8D_KV_F32, exact, or
 * Q8D_KV_F16, rounded to nearest even once), ld elements apart. */
int q8d_q4_unpack(const void* w_q4, void* dst, int dst_dtype, long long ld, int p, int n,
                  int group, void* stream);

/* ------------------------------------------------------------------------
 * q8d_q4_matmul - a 4-bit matrix applied to m rows of activations:
 *   Y[i][r] = sum_k X[i][k] * W[r][k] (+ bias[r]) (+ residual[i][r])
 * within 1e-5 of the sum of |terms| (and 2^-126, below f32's normal range),
 * however far the elements of a row lie apart; where that sum passes f32's range,
 * infinite or NaN.
 *   X: device rows of x_dtype, ldx elements apart (>= n): Q8D_KV_F32 or
 *      Q8D_KV_F16 (16-byte aligned, ldx % 4 == 0, f16 % 8 == 0), or Q8D_KV_Q8_0:
 *      rows of Q8_0 blocks as q8d_rmsnorm_rows writes them (2-byte aligned,
 *      ldx % 32 == 0).  A row with an infinity or NaN makes its row of Y NaN or
 *      infinite.
 *   bias: device f32[p] or NULL; residual: device f32 rows ldr apart (>= p) or
 *      NULL, may be Y itself (same pointer, ldr == ldy)
 *   Y: device f32 rows, ldy apart (>= p); only the first p entries of a row are
 *      written; must not overlap any other operand
 * 0 <= m <= 16, 32 <= n <= 32768, n % 32 == 0, p <= 2^30; else
 * Q8D_EUNSUPPORTED.  m == 0 or p == 0: no-op.  Matrices are read once (with more than
 * eight f32 rows at most twice; what meets f32 elements below 2^-32 of the largest
 * of their 128 columns once more).  Nothing depends on the order in which threads
 * finish.  Waits inside are bounded (seconds); the sums that miss a copy are NaN
 * (these calls have no error word: NaN is the only sign).
 * ---------------------------------------------------------------------- */
int q8d_q4_matmul(const void* X, int x_dtype, long long ldx, const void* w_q4, int group,
                  const float* bias, const float* residual, long long ldr, float* Y, long long ldy,
                  int m, int n, int p, void* stream);

/* ------------------------------------------------------------------------
 * q8d_q4_gated - the gated projections of a feed-forward block in one kernel:
 *   H[i][r] = silu(sum_k X[i][k] Wg[r][k]) * sum_k X[i][k] Wu[r][k],
 *   silu(v) = v / (1 + exp(-v))
 * Wg, Wu: 4-bit matrices [p][n] of the same group.  Other arguments as for
 * q8d_q4_matmul.
 * ---------------------------------------------------------------------- */
int q8d_q4_gated(const void* X, int x_dtype, long long ldx, const void* wg_q4, const void* wu_q4,
                 int group, float* H, long long ldh, int m, int n, int p, void* stream);

/* Sets at which poll a wait inside these products gives up (1: without waiting;
 * 0: the default, 2^24), for every later call of the process and the graphs that
 * capture it.  On expiry the sums that miss a copy are NaN, the copies in flight
 * are waited for, and the CUDA context stays usable.  A small value is a way to
 * check that a caller's error handling sees such a call. */
int q8d_q4_set_wait_limit(unsigned polls);

/* ------------------------------------------------------------------------
 * Decode step graph ("IV.4: One command buffer per token", "One command
 * buffer": the whole step encoded once and submitted as one unit).
 * The step, per layer: RMSNorm -> q/k/v Q8_0 matvecs -> (q/k/v bias) ->
 * (per-head q/k RMSNorm) -> RoPE(q, k) -> KV append -> attention -> o
 * matvec -> residual add -> RMSNorm -> gate/up matvecs -> SiLU(gate)*up ->
 * down matvec -> residual add; then final RMSNorm -> lm_head -> argmax.
 * The token id and position are read from device memory at replay time,
 * the argmax is written back as the next token and the position advanced,
 * so consecutive launches decode consecutive tokens with no host work.
 * All pointers in the descriptors are device pointers owned by the caller
 * and must stay valid until q8d_step_destroy.  Weights, caches and RMSNorm
 * weights must be 16-byte aligned, the other f32 vectors 4-byte aligned
 * (Q8D_EALIGN otherwise).  head_dim in {64, 128}; n_heads % n_kv_heads ==
 * 0; n_heads/n_kv_heads <= 16 with an f32 cache, <= 12 with an f16 cache;
 * n_kv_heads at most the device's SM count (Q8D_EUNSUPPORTED otherwise).
 * ---------------------------------------------------------------------- */
typedef struct q8d_layer_desc {
  const void *wq, *wk, *wv, *wo, *wg, *wu, *wd; /* Q8_0: [H*hd][hidden], [Hk*hd][hidden] x2,
                                                   [hidden][H*hd], [ffn][hidden] x2,
                                                   [hidden][ffn]                          */
  const float *attn_norm, *ffn_norm;            /* f32 [hidden], 16-byte aligned          */
  const float *q_norm, *k_norm;                 /* f32 [head_dim] (qk_norm) or NULL       */
  const float *bq, *bk, *bv;                    /* f32 biases (qkv_bias) or NULL          */
  void *kcache, *vcache;                        /* [cap][Hk*hd] of kv_dtype               */
} q8d_layer_desc;

typedef struct q8d_step_desc {
  int hidden, n_layers, n_heads, n_kv_heads, head_dim, ffn, vocab;
  int qk_norm;  /* 1: Qwen3-style per-head RMSNorm of q and k after projection */
  int qkv_bias; /* 1: Qwen2-style bias add on q, k, v                          */
  int kv_dtype; /* Q8D_KV_F32 or Q8D_KV_F16                                    */
  int cap;      /* rows of every KV cache                                      */
  float rms_eps, rope_theta;
  const void* embed;      /* Q8_0 [vocab][hidden]                 */
  const float* out_norm;  /* f32 [hidden], 16-byte aligned        */
  const void* lm_head;    /* Q8_0 [vocab][hidden]                 */
  const q8d_layer_desc* layers; /* host array of n_layers (copied at create) */
  int* d_token;           /* device int: input token; receives the argmax     */
  int* d_pos;             /* device int: position of the input token; +1 after */
  int* d_err;             /* device int error word (OR-ed into)               */
  float* d_logits;        /* device f32 [vocab] or NULL (library-owned then)  */
} q8d_step_desc;

typedef struct q8d_step q8d_step;

/* Builds the step: allocates its activation workspace (the only allocation
 * the library makes), prepares per-step tables with kernels on `stream`,
 * captures the step into a CUDA graph and instantiates it.  Synchronises
 * `stream`. */
int q8d_step_create(const q8d_step_desc* desc, void* stream, q8d_step** out);

/* Enqueues one decode step (one graph launch) on `stream`. */
int q8d_step_launch(q8d_step* step, void* stream);

/* One decode step with its inputs and output in host memory, in one call:
 * copies h_token_pos[0] (token id) and h_token_pos[1] (position) to the
 * step's device token and position (one 8-byte copy when they are adjacent
 * in device memory, d_pos == d_token + 1), launches the step graph, and
 * copies the next token id to *h_next_token, all enqueued on `stream`
 * (asynchronous: read *h_next_token after synchronising the stream; pinned
 * host memory keeps the copies asynchronous).  Either pointer may be NULL
 * to skip that copy.  The same operation as the host copies around
 * q8d_step_launch ("IV.4: One command buffer per token": token and
 * position in, next token out), with one call per step instead of four. */
int q8d_step_launch_host(q8d_step* step, const int* h_token_pos, int* h_next_token, void* stream);

/* Copies the step's device error word into *err (synchronous; waits for
 * work already enqueued on `stream`, polling with a time limit of
 * timeout_ms milliseconds, <= 0 meaning 10 s).  Returns Q8D_ETIMEOUT if the
 * limit ran out. */
int q8d_step_status(q8d_step* step, void* stream, int timeout_ms, int* err);

/* Sets how many polls a grid-wide barrier wait inside the step kernel makes
 * before the step gives up (polls == 0 restores the default, 2^21 polls,
 * about a second).  On expiry the step sets Q8D_DERR_WAIT in the error
 * word, every CTA of the step leaves at its next barrier, the remaining
 * phases are skipped (the token and position are not advanced) and the
 * CUDA context stays usable.  The value is written in stream order on
 * `stream` and applies to later launches.  A small value is a way to check
 * that a caller's error handling sees an abandoned step. */
int q8d_step_set_wait_limit(q8d_step* step, unsigned polls, void* stream);

/* Number of kernel nodes one launch runs. */
int q8d_step_kernel_count(const q8d_step* step);

/* Device pointer of the step's logits buffer (f32 [vocab]). */
float* q8d_step_logits(q8d_step* step);

/* Releases the graph and the workspace (not the caller's buffers). */
void q8d_step_destroy(q8d_step* step);

#ifdef __cplusplus
}
#endif
#endif /* Q8D_H */
