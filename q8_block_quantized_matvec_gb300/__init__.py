"""Python binding of libq8d, the GB300 Q8_0 decode hot path.

Argument marshalling only: every computation runs in the CUDA kernels of
libq8d.so (built in-tree by build.py for sm_103a).  Functions carry the C
entry points' names and arguments; tensors are torch tensors on the CUDA
device (or raw integer device addresses), `stream` defaults to torch's
current stream.  A non-zero status raises Q8DError.  If the library is
missing the import of any entry point fails loudly; there is no fallback.
"""
from __future__ import annotations

import ctypes as C
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libq8d.so")

Q8D_OK = 0
Q8D_EINVAL = -1
Q8D_EALIGN = -2
Q8D_EUNSUPPORTED = -3
Q8D_ERANGE = -4
Q8D_ECUDA = -5
Q8D_ETIMEOUT = -6
Q8D_ENOMEM = -7

Q8D_KV_F32 = 0
Q8D_KV_F16 = 1
Q8D_KV_Q8_0 = 2
Q8D_KV_Q4 = 4

Q8D_MAX_RUNS = 4

Q8D_ROPE_PLAIN = 0
Q8D_ROPE_LINEAR = 1
Q8D_ROPE_NTK = 2
Q8D_ROPE_YARN = 3
Q8D_ROPE_HALF = 0
Q8D_ROPE_PAIRS = 1

Q8D_DERR_POS_RANGE = 0x1
Q8D_DERR_LEN_RANGE = 0x2
Q8D_DERR_TOKEN_RANGE = 0x4
Q8D_DERR_WAIT = 0x8


class Q8DError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {strerror(status)} (status {status}, cuda {last_cuda_error()})")


class LayerDesc(C.Structure):
    _fields_ = [(nm, C.c_void_p) for nm in
                ("wq", "wk", "wv", "wo", "wg", "wu", "wd", "attn_norm", "ffn_norm", "q_norm",
                 "k_norm", "bq", "bk", "bv", "kcache", "vcache")]


class StepDesc(C.Structure):
    _fields_ = [("hidden", C.c_int), ("n_layers", C.c_int), ("n_heads", C.c_int),
                ("n_kv_heads", C.c_int), ("head_dim", C.c_int), ("ffn", C.c_int),
                ("vocab", C.c_int), ("qk_norm", C.c_int), ("qkv_bias", C.c_int),
                ("kv_dtype", C.c_int), ("cap", C.c_int), ("rms_eps", C.c_float),
                ("rope_theta", C.c_float), ("embed", C.c_void_p), ("out_norm", C.c_void_p),
                ("lm_head", C.c_void_p), ("layers", C.POINTER(LayerDesc)),
                ("d_token", C.c_void_p), ("d_pos", C.c_void_p), ("d_err", C.c_void_p),
                ("d_logits", C.c_void_p)]


class RopeDesc(C.Structure):
    _fields_ = [("n_heads", C.c_int), ("n_kv_heads", C.c_int), ("head_dim", C.c_int),
                ("rot_dim", C.c_int), ("layout", C.c_int), ("max_pos", C.c_int),
                ("row_dtype", C.c_int), ("q_dtype", C.c_int), ("kv_dtype", C.c_int),
                ("cap", C.c_int), ("eps", C.c_float), ("ldq", C.c_longlong),
                ("ldkv", C.c_longlong), ("ldo", C.c_longlong),
                ("cache_batch_stride", C.c_longlong), ("table", C.c_void_p), ("bq", C.c_void_p),
                ("bk", C.c_void_p), ("bv", C.c_void_p), ("q_norm", C.c_void_p),
                ("k_norm", C.c_void_p)]


_lib = None


def lib():
    """The loaded libq8d (ctypes CDLL) with argument types declared."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"libq8d.so is not built ({LIB_PATH}); run "
                              "q8_block_quantized_matvec_gb300.build.build()")
        L = C.CDLL(LIB_PATH)
        vp, i32, i64, f32, sz = C.c_void_p, C.c_int, C.c_longlong, C.c_float, C.c_size_t
        f64 = C.c_double
        L.q8d_version.restype = i32
        L.q8d_strerror.argtypes = [i32]
        L.q8d_strerror.restype = C.c_char_p
        L.q8d_last_cuda_error.restype = i32
        L.q8d_matvec.argtypes = [vp, vp, vp, i32, i32, vp]
        L.q8d_matvec.restype = i32
        L.q8d_matmul_small_m.argtypes = [vp, i32, vp, vp, i32, i32, i32, i32, vp]
        L.q8d_matmul_small_m.restype = i32
        L.q8d_matmul_small_m_workspace_bytes.argtypes = [i32, i32]
        L.q8d_matmul_small_m_workspace_bytes.restype = sz
        L.q8d_matmul_small_m_ws.argtypes = [vp, i32, vp, vp, i32, i32, i32, i32, vp, sz, vp]
        L.q8d_matmul_small_m_ws.restype = i32
        L.q8d_kv_append.argtypes = [vp, vp, vp, vp, i32, i32, i32, vp, vp, vp]
        L.q8d_kv_append.restype = i32
        L.q8d_kv_cache_bytes.argtypes = [i32, i32, i32]
        L.q8d_kv_cache_bytes.restype = sz
        L.q8d_kv_append_rows.argtypes = [vp, vp, i32, i32, vp, vp, i32, i32, i32, i32, i32, i64, vp,
                                         vp, vp, vp]
        L.q8d_kv_append_rows.restype = i32
        L.q8d_kv_read_rows.argtypes = [vp, vp, i32, vp, vp, i32, i32, i32, i32, i32, i32, i64, vp,
                                       vp, vp, vp]
        L.q8d_kv_read_rows.restype = i32
        L.q8d_gqa_workspace_bytes.argtypes = [i32, i32, i32, i32, i32]
        L.q8d_gqa_workspace_bytes.restype = sz
        L.q8d_gqa_decode_attn.argtypes = [vp, vp, vp, vp, vp, i32, vp, i32, i32, i32, i32, i32,
                                          i64, vp, f32, vp, sz, vp, vp]
        L.q8d_gqa_decode_attn.restype = i32
        L.q8d_gqa_decode_attn_window.argtypes = [vp, vp, vp, vp, vp, i32, vp, i32, i32, i32, i32,
                                                 i32, i64, vp, f32, vp, sz, vp, vp]
        L.q8d_gqa_decode_attn_window.restype = i32
        L.q8d_noalloc_scratch_bytes.argtypes = []
        L.q8d_noalloc_scratch_bytes.restype = sz
        L.q8d_gqa_decode_attn_noalloc.argtypes = [vp, vp, vp, vp, vp, i32, vp, i32, i32, i32, i32,
                                                  i32, i64, vp, f32, vp, vp]
        L.q8d_gqa_decode_attn_noalloc.restype = i32
        L.q8d_moe_workspace_bytes.argtypes = [i32, i32, i32, i32, i32]
        L.q8d_moe_workspace_bytes.restype = sz
        L.q8d_moe_ffn.argtypes = [vp, i32, vp, vp, vp, vp, vp, i32, vp, i32, i32, i32, i32, i32, i32,
                                  i32, vp, vp, vp, sz, vp, vp]
        L.q8d_moe_ffn.restype = i32
        L.q8d_moe_set_wait_limit.argtypes = [C.c_uint]
        L.q8d_moe_set_wait_limit.restype = i32
        L.q8d_rmsnorm_rows.argtypes = [vp, vp, vp, i32, i64, i64, i64, vp, f32, vp, i32, i64, i32,
                                       i32, vp]
        L.q8d_rmsnorm_rows.restype = i32
        L.q8d_rope_table.argtypes = [vp, i32, i32, f64, i32, f64, f64, f64, f64, f64, vp]
        L.q8d_rope_table.restype = i32
        L.q8d_rope_append_rows.argtypes = [C.POINTER(RopeDesc), vp, vp, vp, vp, vp, vp, i32, i32,
                                           vp, vp, vp, vp, vp]
        L.q8d_rope_append_rows.restype = i32
        L.q8d_q4_matrix_bytes.argtypes = [i32, i32, i32]
        L.q8d_q4_matrix_bytes.restype = sz
        L.q8d_q4_pack.argtypes = [vp, i32, i64, vp, i32, i32, i32, vp]
        L.q8d_q4_pack.restype = i32
        L.q8d_q4_unpack.argtypes = [vp, vp, i32, i64, i32, i32, i32, vp]
        L.q8d_q4_unpack.restype = i32
        L.q8d_q4_matmul.argtypes = [vp, i32, i64, vp, i32, vp, vp, i64, vp, i64, i32, i32, i32, vp]
        L.q8d_q4_matmul.restype = i32
        L.q8d_q4_gated.argtypes = [vp, i32, i64, vp, vp, i32, vp, i64, i32, i32, i32, vp]
        L.q8d_q4_gated.restype = i32
        L.q8d_q4_set_wait_limit.argtypes = [C.c_uint]
        L.q8d_q4_set_wait_limit.restype = i32
        L.q8d_step_create.argtypes = [C.POINTER(StepDesc), vp, C.POINTER(vp)]
        L.q8d_step_create.restype = i32
        L.q8d_step_launch.argtypes = [vp, vp]
        L.q8d_step_launch.restype = i32
        L.q8d_step_launch_host.argtypes = [vp, vp, vp, vp]
        L.q8d_step_launch_host.restype = i32
        L.q8d_step_status.argtypes = [vp, vp, i32, C.POINTER(i32)]
        L.q8d_step_status.restype = i32
        L.q8d_step_set_wait_limit.argtypes = [vp, C.c_uint, vp]
        L.q8d_step_set_wait_limit.restype = i32
        L.q8d_step_kernel_count.argtypes = [vp]
        L.q8d_step_kernel_count.restype = i32
        L.q8d_step_logits.argtypes = [vp]
        L.q8d_step_logits.restype = vp
        L.q8d_step_destroy.argtypes = [vp]
        L.q8d_step_destroy.restype = None
        _lib = L
    return _lib


def strerror(status: int) -> str:
    return lib().q8d_strerror(int(status)).decode()


def last_cuda_error() -> int:
    return lib().q8d_last_cuda_error()


def _ptr(t):
    if t is None or t.__class__ is int:
        return t
    try:
        return t.data_ptr()
    except AttributeError:
        if isinstance(t, int):
            return int(t)
        raise


_raw_stream = _device = None


def _find_stream() -> None:
    """Sets _raw_stream and _device: torch's current stream on the current
    device.  torch.cuda.current_stream builds a Stream object (3 us on the Arm
    host, more than a launch); its raw handle comes from the same place
    without one."""
    global _raw_stream, _device
    import torch
    torch.cuda.current_stream()  # (initialises CUDA)
    try:
        raw, device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
        raw(device())
    except AttributeError:
        raw, device = lambda _: torch.cuda.current_stream().cuda_stream, lambda: 0  # noqa: E731
    _raw_stream, _device = raw, device


def _stream(stream):
    if stream is None:
        if _raw_stream is None:
            _find_stream()
        return _raw_stream(_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(status: int, what: str) -> int:
    if status != Q8D_OK:
        raise Q8DError(status, what)
    return status


# ---- entry points (same names and argument order as include/q8d.h) --------

def q8d_matvec(x, w_q8, out, n: int, p: int, stream=None) -> int:
    return _check(lib().q8d_matvec(_ptr(x), _ptr(w_q8), _ptr(out), int(n), int(p),
                                   _stream(stream)), "q8d_matvec")


def q8d_matmul_small_m(X, ldx: int, w_q8, Y, ldy: int, m: int, n: int, p: int, stream=None) -> int:
    return _check(lib().q8d_matmul_small_m(_ptr(X), int(ldx), _ptr(w_q8), _ptr(Y), int(ldy), int(m),
                                           int(n), int(p), _stream(stream)), "q8d_matmul_small_m")


def q8d_matmul_small_m_workspace_bytes(m: int, n: int) -> int:
    return int(lib().q8d_matmul_small_m_workspace_bytes(int(m), int(n)))


def q8d_matmul_small_m_ws(X, ldx: int, w_q8, Y, ldy: int, m: int, n: int, p: int, workspace,
                          ws_bytes: int, stream=None) -> int:
    return _check(lib().q8d_matmul_small_m_ws(_ptr(X), int(ldx), _ptr(w_q8), _ptr(Y), int(ldy),
                                              int(m), int(n), int(p), _ptr(workspace),
                                              int(ws_bytes), _stream(stream)),
                  "q8d_matmul_small_m_ws")


def q8d_kv_append(k, v, kcache, vcache, kv_dtype: int, kv_width: int, cap: int, d_pos, d_err,
                  stream=None) -> int:
    return _check(lib().q8d_kv_append(_ptr(k), _ptr(v), _ptr(kcache), _ptr(vcache), int(kv_dtype),
                                      int(kv_width), int(cap), _ptr(d_pos), _ptr(d_err),
                                      _stream(stream)), "q8d_kv_append")


def q8d_kv_cache_bytes(kv_dtype: int, kv_width: int, cap: int) -> int:
    return int(lib().q8d_kv_cache_bytes(int(kv_dtype), int(kv_width), int(cap)))


def q8d_kv_append_rows(k, v, row_dtype: int, ld: int, kcache, vcache, kv_dtype: int, batch: int,
                       rows: int, kv_width: int, cap: int, cache_batch_stride: int, d_pos,
                       d_counts, d_err, stream=None) -> int:
    return _check(lib().q8d_kv_append_rows(
        _ptr(k), _ptr(v), int(row_dtype), int(ld), _ptr(kcache), _ptr(vcache), int(kv_dtype),
        int(batch), int(rows), int(kv_width), int(cap), int(cache_batch_stride), _ptr(d_pos),
        _ptr(d_counts), _ptr(d_err), _stream(stream)), "q8d_kv_append_rows")


def q8d_kv_read_rows(kcache, vcache, kv_dtype: int, k_out, v_out, row_dtype: int, ld: int,
                     batch: int, rows: int, kv_width: int, cap: int, cache_batch_stride: int,
                     d_pos, d_counts, d_err, stream=None) -> int:
    return _check(lib().q8d_kv_read_rows(
        _ptr(kcache), _ptr(vcache), int(kv_dtype), _ptr(k_out), _ptr(v_out), int(row_dtype),
        int(ld), int(batch), int(rows), int(kv_width), int(cap), int(cache_batch_stride),
        _ptr(d_pos), _ptr(d_counts), _ptr(d_err), _stream(stream)), "q8d_kv_read_rows")


def q8d_gqa_workspace_bytes(batch: int, n_heads: int, n_kv_heads: int, head_dim: int,
                            max_len: int) -> int:
    return int(lib().q8d_gqa_workspace_bytes(batch, n_heads, n_kv_heads, head_dim, max_len))


def q8d_gqa_decode_attn(q, k_new, v_new, kcache, vcache, kv_dtype: int, out, batch: int,
                        n_heads: int, n_kv_heads: int, head_dim: int, cap: int,
                        cache_batch_stride: int, d_lens, scale: float, workspace, ws_bytes: int,
                        d_err, stream=None) -> int:
    return _check(lib().q8d_gqa_decode_attn(
        _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(kcache), _ptr(vcache), int(kv_dtype), _ptr(out),
        int(batch), int(n_heads), int(n_kv_heads), int(head_dim), int(cap),
        int(cache_batch_stride), _ptr(d_lens), float(scale), _ptr(workspace), int(ws_bytes),
        _ptr(d_err), _stream(stream)), "q8d_gqa_decode_attn")


def q8d_gqa_decode_attn_window(q, k_new, v_new, kcache, vcache, kv_dtype: int, out, batch: int,
                               n_heads: int, n_kv_heads: int, head_dim: int, cap: int,
                               cache_batch_stride: int, d_runs, scale: float, workspace,
                               ws_bytes: int, d_err, stream=None) -> int:
    return _check(lib().q8d_gqa_decode_attn_window(
        _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(kcache), _ptr(vcache), int(kv_dtype), _ptr(out),
        int(batch), int(n_heads), int(n_kv_heads), int(head_dim), int(cap),
        int(cache_batch_stride), _ptr(d_runs), float(scale), _ptr(workspace), int(ws_bytes),
        _ptr(d_err), _stream(stream)), "q8d_gqa_decode_attn_window")


def q8d_noalloc_scratch_bytes() -> int:
    return int(lib().q8d_noalloc_scratch_bytes())


def q8d_gqa_decode_attn_noalloc(q, k_new, v_new, kcache, vcache, kv_dtype: int, out, batch: int,
                                n_heads: int, n_kv_heads: int, head_dim: int, cap: int,
                                cache_batch_stride: int, d_lens, scale: float, d_err,
                                stream=None) -> int:
    """q8d_gqa_decode_attn with the scratch in the library's fixed device
    array (for callers that cannot allocate device memory)."""
    return _check(lib().q8d_gqa_decode_attn_noalloc(
        _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(kcache), _ptr(vcache), int(kv_dtype), _ptr(out),
        int(batch), int(n_heads), int(n_kv_heads), int(head_dim), int(cap),
        int(cache_batch_stride), _ptr(d_lens), float(scale), _ptr(d_err), _stream(stream)),
        "q8d_gqa_decode_attn_noalloc")


def q8d_moe_workspace_bytes(m: int, hidden: int, ffn: int, n_experts: int, top_k: int) -> int:
    return int(lib().q8d_moe_workspace_bytes(int(m), int(hidden), int(ffn), int(n_experts),
                                             int(top_k)))


def q8d_moe_ffn(X, ldx: int, router, wg, wu, wd, residual, ldr: int, Y, ldy: int, m: int,
                hidden: int, ffn: int, n_experts: int, top_k: int, norm_topk: int, experts, weights,
                workspace, ws_bytes: int, d_err, stream=None) -> int:
    return _check(lib().q8d_moe_ffn(
        _ptr(X), int(ldx), _ptr(router), _ptr(wg), _ptr(wu), _ptr(wd), _ptr(residual), int(ldr),
        _ptr(Y), int(ldy), int(m), int(hidden), int(ffn), int(n_experts), int(top_k),
        int(norm_topk), _ptr(experts), _ptr(weights), _ptr(workspace), int(ws_bytes), _ptr(d_err),
        _stream(stream)), "q8d_moe_ffn")


def q8d_moe_set_wait_limit(polls: int) -> int:
    return _check(lib().q8d_moe_set_wait_limit(int(polls)), "q8d_moe_set_wait_limit")


# (numbers go to ctypes as they are: it takes whole numbers of any type and
# refuses others, and ten conversions cost a call 0.6 us)
def q8d_rmsnorm_rows(x, residual, sum_out, row_dtype: int, ldx: int, ldr: int, lds: int, weight,
                     eps: float, y, y_dtype: int, ldy: int, rows: int, n: int, stream=None) -> int:
    return _check(lib().q8d_rmsnorm_rows(
        _ptr(x), _ptr(residual), _ptr(sum_out), row_dtype, ldx, ldr, lds,
        _ptr(weight), eps, _ptr(y), y_dtype, ldy, rows, n,
        _stream(stream)), "q8d_rmsnorm_rows")


def q8d_rope_table(table, max_pos: int, rot_dim: int, theta: float, scaling: int, factor: float,
                   orig_ctx: float, beta_fast: float, beta_slow: float, mscale: float,
                   stream=None) -> int:
    return _check(lib().q8d_rope_table(_ptr(table), max_pos, rot_dim, theta,
                                       scaling, factor, orig_ctx,
                                       beta_fast, beta_slow, mscale,
                                       _stream(stream)), "q8d_rope_table")


def rope_desc(**fields) -> RopeDesc:
    """A RopeDesc from its fields' values; tensors among them stay alive with it."""
    desc = RopeDesc()
    for name, value in fields.items():
        if not hasattr(RopeDesc, name):
            raise TypeError(f"q8d_rope_desc has no field {name!r}")
        setattr(desc, name, _ptr(value) if hasattr(value, "data_ptr") else value)
    desc._tensors = fields
    return desc


def q8d_rope_append_rows(desc: RopeDesc, q, k, v, q_out, kcache, vcache, batch: int, rows: int,
                         d_pos, d_rope_pos, d_counts, d_err, stream=None) -> int:
    return _check(lib().q8d_rope_append_rows(
        desc, _ptr(q), _ptr(k), _ptr(v), _ptr(q_out), _ptr(kcache), _ptr(vcache), batch,
        rows, _ptr(d_pos), _ptr(d_rope_pos), _ptr(d_counts), _ptr(d_err), _stream(stream)),
        "q8d_rope_append_rows")


def q8d_q4_matrix_bytes(p: int, n: int, group: int) -> int:
    return int(lib().q8d_q4_matrix_bytes(int(p), int(n), int(group)))


def q8d_q4_pack(src, src_dtype: int, ld: int, w_q4, p: int, n: int, group: int, stream=None) -> int:
    return _check(lib().q8d_q4_pack(_ptr(src), src_dtype, ld, _ptr(w_q4), p, n,
                                    group, _stream(stream)), "q8d_q4_pack")


def q8d_q4_unpack(w_q4, dst, dst_dtype: int, ld: int, p: int, n: int, group: int,
                  stream=None) -> int:
    return _check(lib().q8d_q4_unpack(_ptr(w_q4), _ptr(dst), dst_dtype, ld, p,
                                      n, group, _stream(stream)), "q8d_q4_unpack")


def q8d_q4_matmul(X, x_dtype: int, ldx: int, w_q4, group: int, bias, residual, ldr: int, Y,
                  ldy: int, m: int, n: int, p: int, stream=None) -> int:
    return _check(lib().q8d_q4_matmul(
        _ptr(X), x_dtype, ldx, _ptr(w_q4), group, _ptr(bias), _ptr(residual),
        ldr, _ptr(Y), ldy, m, n, p, _stream(stream)), "q8d_q4_matmul")


def q8d_q4_gated(X, x_dtype: int, ldx: int, wg_q4, wu_q4, group: int, H, ldh: int, m: int, n: int,
                 p: int, stream=None) -> int:
    return _check(lib().q8d_q4_gated(
        _ptr(X), x_dtype, ldx, _ptr(wg_q4), _ptr(wu_q4), group, _ptr(H), ldh,
        m, n, p, _stream(stream)), "q8d_q4_gated")


def q8d_q4_set_wait_limit(polls: int) -> int:
    return _check(lib().q8d_q4_set_wait_limit(int(polls)), "q8d_q4_set_wait_limit")


class Step:
    """Owns a q8d_step (the captured decode-step graph)."""

    def __init__(self, desc: StepDesc, layers, stream=None):
        self._desc = desc
        self._layers = layers  # keep the ctypes array alive
        h = C.c_void_p()
        _check(lib().q8d_step_create(C.byref(desc), _stream(stream), C.byref(h)), "q8d_step_create")
        self.handle = h.value

    def launch(self, stream=None) -> int:
        return _check(lib().q8d_step_launch(self.handle, _stream(stream)), "q8d_step_launch")

    def launch_host(self, h_token_pos, h_next_token, stream=None) -> int:
        """q8d_step_launch_host: host int32 [token, position] in (or None),
        the next token id out to host int32 [1] (or None); both pinned CPU
        tensors, read the output after synchronising the stream."""
        return _check(lib().q8d_step_launch_host(self.handle, _ptr(h_token_pos), _ptr(h_next_token),
                                                 _stream(stream)), "q8d_step_launch_host")

    def status(self, stream=None, timeout_ms: int = 10000) -> int:
        err = C.c_int(0)
        _check(lib().q8d_step_status(self.handle, _stream(stream), int(timeout_ms), C.byref(err)),
               "q8d_step_status")
        return err.value

    def set_wait_limit(self, polls: int, stream=None) -> int:
        return _check(lib().q8d_step_set_wait_limit(self.handle, int(polls), _stream(stream)),
                      "q8d_step_set_wait_limit")

    def kernel_count(self) -> int:
        return lib().q8d_step_kernel_count(self.handle)

    def logits_ptr(self) -> int:
        return lib().q8d_step_logits(self.handle)

    def close(self):
        if self.handle:
            lib().q8d_step_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def q8d_step_create(desc: StepDesc, layers, stream=None) -> Step:
    return Step(desc, layers, stream)
