// C-ABI entry points of the operators between the products of a layer and of
// the products with 4-bit weights: argument checks, then the kernels.
#include <cmath>

#include "q8d_args.cuh"
#include "q8d_layer.cuh"

namespace q8d {
namespace {

bool row_type(int t) { return t == Q8D_KV_F32 || t == Q8D_KV_F16; }
int row_align(int t) { return t == Q8D_KV_F32 ? 4 : 2; }  // (Q8_0 rows: 2)

// An operand's bytes: n of them from p on; rows of `row` bytes, `pitch` apart (0: in
// one piece).
struct Span {
  const void* p;
  size_t n;
  long long row = 0, pitch = 0;
};
// `rows` rows of n elements, ld apart (nothing without a pointer).
Span rows_span(const void* p, int dtype, long long rows, long long ld, long long n) {
  if (!p || rows <= 0) return {nullptr, 0};
  const long long row = kv_bytes(dtype, n), pitch = kv_bytes(dtype, ld);
  return {p, (size_t)(pitch * (rows - 1) + row), row, pitch};
}
// Whether two operands share a byte.  Rows of one pitch may be other columns of one
// buffer; those of different ones are counted whole, from the first one's start to
// the last one's end.
bool meets(const Span& a, const Span& b) {
  if (!overlap(a.p, a.n, b.p, b.n)) return false;
  if (!a.pitch || a.pitch != b.pitch) return true;
  const long long off = (long long)(reinterpret_cast<uintptr_t>(b.p) - reinterpret_cast<uintptr_t>(a.p));
  const long long at = (off % a.pitch + a.pitch) % a.pitch;  // where b's rows start between a's
  return at < a.row || at + b.row > a.pitch;
}

// Largest distance between rows: (2^31 - 1) rows of it stay below 2^63 bytes.
constexpr long long kMaxLd = 1LL << 29;

bool q4_shape(int p, int n, int group) {
  return p >= 0 && p <= 1 << 30 && n >= 32 && n <= kQ4MaxN && n % 32 == 0 && q4_group_known(group);
}

int q4_copy(const void* w, const void* rows, int dtype, long long ld, int p, int n, int group, bool pack,
            Q4CopyParams* P) {
  if (p < 0 || n <= 0) return Q8D_EINVAL;
  if (!q4_shape(p, n, group)) return Q8D_EUNSUPPORTED;
  if (!row_type(dtype) && !(pack && dtype == Q8D_KV_Q8_0)) return Q8D_EUNSUPPORTED;
  if (p == 0) return Q8D_OK;
  if (!w || !rows || ld < n || ld > kMaxLd) return Q8D_EINVAL;
  if (!aligned(w, 16) || !aligned(rows, row_align(dtype)) || (dtype == Q8D_KV_Q8_0 && ld % 32))
    return Q8D_EALIGN;
  if (meets({w, q8d_q4_matrix_bytes(p, n, group)}, rows_span(rows, dtype, p, ld, n))) return Q8D_EINVAL;
  *P = {const_cast<void*>(rows), dtype, ld, static_cast<uint8_t*>(const_cast<void*>(w)), p, n, group};
  return Q8D_OK;
}

int q4_product(const void* X, int x_dtype, long long ldx, const void* w0, const void* w1, int nmat, int group,
               const float* bias, const float* residual, long long ldr, float* Y, long long ldy, int m,
               int n, int p, void* stream) {
  if (m < 0 || n <= 0 || p < 0) return Q8D_EINVAL;
  if (m > kQ4MaxRows || !q4_shape(p, n, group)) return Q8D_EUNSUPPORTED;
  if (!row_type(x_dtype) && x_dtype != Q8D_KV_Q8_0) return Q8D_EUNSUPPORTED;
  if (m == 0 || p == 0) return Q8D_OK;
  if (!X || !w0 || (nmat == 2 && !w1) || !Y) return Q8D_EINVAL;
  if (ldx < n || ldx > kMaxLd || ldy < p || ldy > 1LL << 40 || (residual && (ldr < p || ldr > 1LL << 40)))
    return Q8D_EINVAL;
  if (!aligned(w0, 16) || !aligned(w1, 16) || !aligned(Y, 4) || !aligned(bias, 4) || !aligned(residual, 4))
    return Q8D_EALIGN;
  if (x_dtype == Q8D_KV_Q8_0 ? !aligned(X, 2) || ldx % 32
                             : !aligned(X, 16) || ldx % (x_dtype == Q8D_KV_F32 ? 4 : 8))
    return Q8D_EALIGN;
  const size_t wb = q8d_q4_matrix_bytes(p, n, group);
  const Span out = rows_span(Y, Q8D_KV_F32, m, ldy, p), res = rows_span(residual, Q8D_KV_F32, m, ldr, p);
  if (meets(out, rows_span(X, x_dtype, m, ldx, n)) || meets(out, {w0, wb}) || meets(out, {w1, w1 ? wb : 0}) ||
      meets(out, {bias, bias ? 4 * (size_t)p : 0}) || (meets(out, res) && !(residual == Y && ldr == ldy)))
    return Q8D_EINVAL;
  Q4Params P{};
  P.w[0] = static_cast<const uint8_t*>(w0);
  P.w[1] = static_cast<const uint8_t*>(w1);
  P.nmat = nmat;
  P.group = group;
  P.X = X;
  P.x_dtype = x_dtype;
  P.ldx = ldx;
  P.bias = bias;
  P.residual = residual;
  P.ldr = ldr;
  P.Y = Y;
  P.ldy = ldy;
  P.m = m;
  P.n = n;
  P.p = p;
  return q4_launch(P, static_cast<cudaStream_t>(stream));
}

}  // namespace
}  // namespace q8d

using namespace q8d;

extern "C" {

int q8d_rmsnorm_rows(const void* x, const void* residual, void* sum_out, int row_dtype, long long ldx,
                     long long ldr, long long lds, const float* weight, float eps, void* y, int y_dtype,
                     long long ldy, int rows, int n, void* stream) {
  if (rows < 0 || n <= 0 || !(eps >= 0.f) || std::isinf(eps)) return Q8D_EINVAL;
  if (!row_type(row_dtype) || (!row_type(y_dtype) && y_dtype != Q8D_KV_Q8_0)) return Q8D_EUNSUPPORTED;
  if (n > kNormMaxN || (y_dtype == Q8D_KV_Q8_0 && n % 32)) return Q8D_EUNSUPPORTED;
  if (rows == 0) return Q8D_OK;
  if (!x || !weight || !y) return Q8D_EINVAL;
  if (ldx < n || ldx > kMaxLd || ldy < n || ldy > kMaxLd || (residual && (ldr < n || ldr > kMaxLd)) ||
      (sum_out && (lds < n || lds > kMaxLd)))
    return Q8D_EINVAL;
  const int a = row_align(row_dtype);
  if (!aligned(x, a) || !aligned(residual, a) || !aligned(sum_out, a) || !aligned(weight, 4) ||
      !aligned(y, row_align(y_dtype)) || (y_dtype == Q8D_KV_Q8_0 && ldy % 32))
    return Q8D_EALIGN;
  const Span sx = rows_span(x, row_dtype, rows, ldx, n), sr = rows_span(residual, row_dtype, rows, ldr, n),
             ss = rows_span(sum_out, row_dtype, rows, lds, n), sy = rows_span(y, y_dtype, rows, ldy, n),
             sw{weight, 4 * (size_t)n};
  if (meets(sy, sx) || meets(sy, sr) || meets(sy, ss) || meets(sy, sw) || meets(ss, sw)) return Q8D_EINVAL;
  if ((meets(ss, sx) && !(sum_out == x && lds == ldx)) || (meets(ss, sr) && !(sum_out == residual && lds == ldr)))
    return Q8D_EINVAL;
  const NormParams P{x, residual, sum_out, row_dtype, ldx, ldr, lds, weight, eps, y, y_dtype, ldy, rows, n};
  return norm_launch(P, static_cast<cudaStream_t>(stream));
}

int q8d_rope_table(float* table, int max_pos, int rot_dim, double theta, int scaling, double factor,
                   double orig_ctx, double beta_fast, double beta_slow, double mscale, void* stream) {
  if (!table || max_pos <= 0 || rot_dim <= 0) return Q8D_EINVAL;
  if (rot_dim % 2 || rot_dim > 256) return Q8D_EUNSUPPORTED;
  if (scaling < Q8D_ROPE_PLAIN || scaling > Q8D_ROPE_YARN) return Q8D_EUNSUPPORTED;
  if (!(theta > 1.0) || !std::isfinite(theta) || !(factor > 0.0) || !std::isfinite(factor) ||
      !std::isfinite(mscale))
    return Q8D_EINVAL;
  if (scaling == Q8D_ROPE_NTK && rot_dim <= 2) return Q8D_EUNSUPPORTED;
  if (scaling == Q8D_ROPE_YARN &&
      (!(orig_ctx > 0.0) || !(beta_fast > 0.0) || !(beta_slow > 0.0) || !std::isfinite(orig_ctx) ||
       !std::isfinite(beta_fast) || !std::isfinite(beta_slow)))
    return Q8D_EINVAL;
  if (!aligned(table, 16)) return Q8D_EALIGN;
  return rope_table_launch(table, max_pos, rot_dim, theta, scaling, factor, orig_ctx, beta_fast, beta_slow,
                           mscale, static_cast<cudaStream_t>(stream));
}

int q8d_rope_append_rows(const q8d_rope_desc* d, const void* q, const void* k, const void* v, void* q_out,
                         void* kcache, void* vcache, int batch, int rows, const int* d_pos,
                         const int* d_rope_pos, const int* d_counts, int* d_err, void* stream) {
  if (!d || (!q && !k) || !q != !q_out || !k != !v || !k != !kcache || !k != !vcache || !d_pos)
    return Q8D_EINVAL;
  if (batch <= 0 || rows < 0 || d->head_dim <= 0 || d->max_pos <= 0 || !(d->eps >= 0.f) || std::isinf(d->eps))
    return Q8D_EINVAL;
  if (d->rot_dim < 0 || d->rot_dim > d->head_dim || (d->rot_dim && !d->table)) return Q8D_EINVAL;
  if ((q && d->n_heads <= 0) || (k && (d->n_kv_heads <= 0 || d->cap <= 0))) return Q8D_EINVAL;
  if (!d->bq != !d->bk || !d->bq != !d->bv || !d->q_norm != !d->k_norm) return Q8D_EINVAL;
  if (d->head_dim % 8 || d->head_dim > 256 || d->rot_dim % 2) return Q8D_EUNSUPPORTED;
  if (d->layout != Q8D_ROPE_HALF && d->layout != Q8D_ROPE_PAIRS) return Q8D_EUNSUPPORTED;
  if (!row_type(d->row_dtype) || (q && !row_type(d->q_dtype)) || (k && !kv_known(d->kv_dtype)))
    return Q8D_EUNSUPPORTED;
  if (k && kv_packed(d->kv_dtype) && d->head_dim % 32) return Q8D_EUNSUPPORTED;
  const long long qw = q ? (long long)d->n_heads * d->head_dim : 0, kw = k ? (long long)d->n_kv_heads * d->head_dim : 0;
  if (qw > 1 << 24 || kw > 1 << 24) return Q8D_EUNSUPPORTED;
  if ((q && (d->ldq < qw || d->ldq > kMaxLd || d->ldo < qw || d->ldo > kMaxLd)) ||
      (k && (d->ldkv < kw || d->ldkv > kMaxLd)))
    return Q8D_EINVAL;
  const long long need = k ? d->cap * kw : 0, stride = k ? d->cache_batch_stride : 0;
  if (stride < 0 || stride > (1LL << 60) / batch || (batch > 1 && stride < need)) return Q8D_EINVAL;
  if (k && kv_packed(d->kv_dtype) && stride % 32) return Q8D_EALIGN;
  if (k && (!aligned(kcache, 16) || !aligned(vcache, 16) || kv_bytes(d->kv_dtype, stride) % 16)) return Q8D_EALIGN;
  const int a = row_align(d->row_dtype);
  if (!aligned(q, a) || !aligned(k, a) || !aligned(v, a) || (q && !aligned(q_out, row_align(d->q_dtype))))
    return Q8D_EALIGN;
  const void* const words[] = {d->bq, d->bk, d->bv, d->q_norm, d->k_norm, d_pos, d_rope_pos, d_counts, d_err};
  for (const void* p : words)
    if (!aligned(p, 4)) return Q8D_EALIGN;
  if (d->rot_dim && !aligned(d->table, 16)) return Q8D_EALIGN;
  const long long all = (long long)batch * rows;
  if (all > 0x7fff0000LL) return Q8D_EUNSUPPORTED;  // (row numbers are 32 bits)
  if (rows == 0) return Q8D_OK;
  const Span sq = rows_span(q, d->row_dtype, all, d->ldq, qw), sk = rows_span(k, d->row_dtype, all, d->ldkv, kw),
             sv = rows_span(v, d->row_dtype, all, d->ldkv, kw),
             so = rows_span(q_out, q ? d->q_dtype : Q8D_KV_F32, all, d->ldo, qw);
  const size_t cb = k ? (size_t)(kv_bytes(d->kv_dtype, stride) * (batch - 1) + kv_bytes(d->kv_dtype, need)) : 0;
  const Span st{d->rot_dim ? d->table : nullptr, d->rot_dim ? 4 * (size_t)d->max_pos * d->rot_dim : 0};
  const Span out[] = {so, {kcache, cb}, {vcache, cb}}, in[] = {sq, sk, sv, st};
  const bool same = q == q_out && d->ldq == d->ldo && d->row_dtype == d->q_dtype;
  for (const Span& o : out)
    for (const Span& i : in)
      if (meets(o, i) && !(&o == &out[0] && &i == &in[0] && same)) return Q8D_EINVAL;  // (q turned in place)
  for (int x = 0; x < 3; ++x)
    for (int y = x + 1; y < 3; ++y)
      if (meets(out[x], out[y])) return Q8D_EINVAL;
  RopeRowsParams P{};
  P.d = *d;
  P.q = q;
  P.k = k;
  P.v = v;
  P.q_out = q_out;
  P.kc = static_cast<uint8_t*>(kcache);
  P.vc = static_cast<uint8_t*>(vcache);
  P.seq_bytes = k ? kv_bytes(d->kv_dtype, stride) : 0;
  P.batch = batch;
  P.rows = rows;
  P.d_pos = d_pos;
  P.d_rope_pos = d_rope_pos;
  P.d_counts = d_counts;
  P.d_err = d_err;
  return rope_rows_launch(P, static_cast<cudaStream_t>(stream));
}

size_t q8d_q4_matrix_bytes(int p, int n, int group) {
  if (p <= 0 || !q4_shape(p, n, group)) return 0;
  return (size_t)(q4_strips(p) * q4_tiles(n)) * q4_tile_bytes(group);
}

int q8d_q4_pack(const void* src, int src_dtype, long long ld, void* w_q4, int p, int n, int group, void* stream) {
  Q4CopyParams P{};
  const int rc = q4_copy(w_q4, src, src_dtype, ld, p, n, group, true, &P);
  if (rc || p == 0) return rc;
  return q4_pack_launch(P, static_cast<cudaStream_t>(stream));
}

int q8d_q4_unpack(const void* w_q4, void* dst, int dst_dtype, long long ld, int p, int n, int group,
                  void* stream) {
  Q4CopyParams P{};
  const int rc = q4_copy(w_q4, dst, dst_dtype, ld, p, n, group, false, &P);
  if (rc || p == 0) return rc;
  return q4_unpack_launch(P, static_cast<cudaStream_t>(stream));
}

int q8d_q4_matmul(const void* X, int x_dtype, long long ldx, const void* w_q4, int group, const float* bias,
                  const float* residual, long long ldr, float* Y, long long ldy, int m, int n, int p,
                  void* stream) {
  return q4_product(X, x_dtype, ldx, w_q4, nullptr, 1, group, bias, residual, ldr, Y, ldy, m, n, p, stream);
}

int q8d_q4_gated(const void* X, int x_dtype, long long ldx, const void* wg_q4, const void* wu_q4, int group,
                 float* H, long long ldh, int m, int n, int p, void* stream) {
  return q4_product(X, x_dtype, ldx, wg_q4, wu_q4, 2, group, nullptr, nullptr, 0, H, ldh, m, n, p, stream);
}

int q8d_q4_set_wait_limit(unsigned polls) {
  q4_set_wait_limit(polls);
  return Q8D_OK;
}

}  // extern "C"
