"""Plain numpy forms of the KV caches' rows for the tests: the quantizers in
f32 steps, the stored bytes of every cache type, and the values they stand
for in f64."""
import numpy as np

F32, F16, Q8_0, Q4 = 0, 1, 2, 4


def cache_bytes(kind, n):
    return {F32: 4 * n, F16: 2 * n, Q8_0: n // 32 * 34, Q4: n // 32 * 18}[kind]


def q8_blocks(x):
    """f32 [..., nb, 32] -> uint8 [..., nb, 34]."""
    one = np.float32(1)
    amax = np.abs(x).max(-1, keepdims=True)
    d = (amax / np.float32(127)).astype(np.float32)
    with np.errstate(divide="ignore"):
        inv = np.where(d != 0, one / d, np.float32(0)).astype(np.float32)
    r = (x * inv).astype(np.float32)
    q = np.trunc(r)
    q = q + np.sign(r) * (np.abs(r - q) >= 0.5)
    out = np.empty(x.shape[:-1] + (34,), np.uint8)
    out[..., :2] = np.ascontiguousarray(d.astype(np.float16)).view(np.uint8)
    out[..., 2:] = q.astype(np.int8).view(np.uint8)
    return out


def q4_blocks(x):
    """f32 [..., nb, 32] -> (quant bytes [..., nb, 16], f16 scales [..., nb])."""
    first = np.abs(x).argmax(-1)[..., None]
    d = np.take_along_axis(x, first, -1) / np.float32(-8)
    with np.errstate(divide="ignore", over="ignore"):
        inv = np.float32(1) / d
    inv = np.where(np.isfinite(inv), inv, np.float32(0)).astype(np.float32)
    t = ((x * inv).astype(np.float32) + np.float32(8.5)).astype(np.float32)
    n = np.clip(np.floor(t), 0, 15).astype(np.uint8)
    with np.errstate(over="ignore"):
        return n[..., :16] | n[..., 16:] << 4, d[..., 0].astype(np.float16)


def store(cache, kind, width, cap, row, x):
    """Stores f32 rows x [count, width] from cache row `row` on into one
    sequence's cache (uint8, flat)."""
    count = x.shape[0]
    if count == 0:
        return
    if kind == Q4:
        q, d = q4_blocks(x.reshape(count, -1, 32))
        cache[:cap * width // 2].reshape(cap, -1)[row:row + count] = q.reshape(count, -1)
        plane = cache[cap * width // 2:cap * width // 16 * 9].reshape(cap, -1)
        plane[row:row + count] = np.ascontiguousarray(d).view(np.uint8).reshape(count, -1)
        return
    if kind == Q8_0:
        new = q8_blocks(x.reshape(count, -1, 32)).reshape(count, -1)
    else:
        with np.errstate(over="ignore"):
            new = np.ascontiguousarray(x.astype(np.float16 if kind == F16 else np.float32))
        new = new.view(np.uint8).reshape(count, -1)
    cache[:cap * new.shape[1]].reshape(cap, -1)[row:row + count] = new


def values(cache, kind, width, cap):
    """f32 values [cap, width] of one sequence's cache (uint8, flat): exact,
    an 11-bit scale times an 8-bit quant at most."""
    n = cache_bytes(kind, cap * width)
    c = np.ascontiguousarray(cache[:n])
    if kind == F32:
        return c.view(np.float32).reshape(cap, width)
    if kind == F16:
        return c.view(np.float16).reshape(cap, width).astype(np.float32)
    if kind == Q8_0:
        b = c.reshape(cap, width // 32, 34)
        d = np.ascontiguousarray(b[..., :2]).view(np.float16).astype(np.float32)
        return (d * b[..., 2:].view(np.int8).astype(np.float32)).reshape(cap, width)
    q = c[:cap * width // 2].reshape(cap, width // 32, 16)
    d = c[cap * width // 2:].view(np.float16).reshape(cap, width // 32, 1).astype(np.float32)
    n4 = np.concatenate([q & 15, q >> 4], -1).astype(np.float32) - 8
    return (d * n4).reshape(cap, width)
