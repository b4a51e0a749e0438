"""Timed cases of the operators with which a dense decoder layer is put
together from this package's calls: root-mean-square norm with the residual's
addition (an f32, f16 or Q8_0 output), rotary positions with the rows' store
into the KV caches, products with 4-bit weights and group scales for a few
tokens, and the gated projections of a feed-forward block over such weights.

`run` computes a case in plain torch arithmetic (`own` false) or through this
package's entry points (`own` true).

A 4-bit matrix [p][n] holds n_j in 0..15 for every element and an f16 scale
for every group of 32, 64 or 128 neighbours of a row (the last one of a row
may be shorter), the value being scale * (n_j - 8).  Its quantizer is the
4-bit KV cache's: scale = the element of largest magnitude / -8 (the first of
them), n_j = floor(x / scale + 8.5) limited to 0..15, in f32 steps.  Eight-bit
rows are Q8_0 blocks: 34 bytes for 32 elements, an f16 scale first."""
import math

import torch

own = False

F32, F16, Q8_0, Q4 = 0, 1, 2, 4
CODE = {"f32": F32, "f16": F16, "q8_0": Q8_0, "q4": Q4}
TORCH = {"f32": torch.float32, "f16": torch.float16}
EPS = 1e-6
THETA = 1e6
YARN = {"factor": 4.0, "orig": 32768, "fast": 32.0, "slow": 1.0}
GOLDEN = 0.6180339887498949


# ---- cases -----------------------------------------------------------------

def listed():
    return [
        # one token's stream before a layer: latency
        _norm("norm_1x3584", 1, 3584, "f32", "f32", True),
        # a prompt's stream in half precision
        _norm("norm_prompt_4096x3584", 4096, 3584, "f16", "f16", True),
        # rows of an odd length, without a residual
        _norm("norm_odd_1000x2887", 1000, 2887, "f32", "f32", False),
        # a prompt's stream into 8 bits
        _norm("norm_q8_2048x4864", 2048, 4864, "f32", "q8_0", True),
        # one token of each of 64 sequences, biases on q, k and v, into f16 caches: a decode step
        _rope("rope_decode_64x1", 64, 1, 28, 4, 128, 128, "half", "none", "f32", "f16", 4096, True, False),
        # a prompt far out in a long context: YaRN, norms of the heads, a packed cache
        _rope("rope_prompt_4096_yarn", 1, 4096, 16, 8, 128, 128, "half", "yarn", "f32", "q8_0", 131072, False, True),
        # ragged prompts, half of each head rotated in neighbouring pairs, f16 rows into a 4-bit cache
        _rope("rope_ragged_8x1999", 8, 1999, 14, 2, 64, 32, "pairs", "linear", "f16", "q4", 2048, False, False),
        # q, k and v of one token, with their biases
        _q4("q4_qkv_1", 1, 3584, 4608, 32, "f32", True, False),
        # the vocabulary's logits of one token
        _q4("q4_vocab_1", 1, 896, 151936, 64, "f32", False, False),
        # sixteen tokens back into the stream
        _q4("q4_down_16", 16, 18944, 3584, 128, "f32", False, True),
        # one token through the gated projections
        _gated("gated_1", 1, 3584, 18944, 32, "f32"),
        # the norm's 8-bit rows of sixteen tokens through them
        _gated("norm_gated_q8_16", 16, 3584, 4736, 64, "norm"),
    ]


def _norm(name, rows, n, src, dst, residual):
    return {"name": name, "op": "norm", "rows": rows, "n": n, "src": src, "dst": dst, "residual": residual}


def _rope(name, batch, rows, heads, kv_heads, dim, rot, layout, scaling, src, cache, cap, bias, norm):
    """layout: which elements make a pair: "half" (i, i + rot / 2), "pairs" (2 i, 2 i + 1)."""
    return {"name": name, "op": "rope", "batch": batch, "rows": rows, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "rot": rot, "layout": layout, "scaling": scaling, "src": src, "cache": cache, "cap": cap, "bias": bias,
            "norm": norm}


def _q4(name, m, n, p, group, x, bias, residual):
    return {"name": name, "op": "q4", "m": m, "n": n, "p": p, "group": group, "x": x, "bias": bias, "residual": residual}


def _gated(name, m, n, p, group, x):
    """x: the type of the rows, or "norm": f32 rows go through the norm with a residual into Q8_0 rows first."""
    return {"name": name, "op": "gated", "m": m, "n": n, "p": p, "group": group, "x": x}


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "rope", "q4", "gated"])
    if op == "norm":
        dst = rng.choice(["f32", "f16", "q8_0"])
        n = 32 * _log(rng, 2, 512) if dst == "q8_0" or rng.random() < 0.5 else _log(rng, 33, 16384)
        rows = _log(rng, 1, max(1, min(16384, 9_000_000 // n)))
        c = _norm("", rows, n, rng.choice(["f32", "f16"]), dst, rng.random() < 0.7)
    elif op == "rope":
        kv_heads, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 7, 8])
        dim = rng.choice([64, 96, 128, 128, 256])
        batch = _log(rng, 1, 64)
        rows = _log(rng, 1, max(1, min(8192, 9_000_000 // (kv_heads * (group + 2) * dim * batch))))
        c = _rope("", batch, rows, kv_heads * group, kv_heads, dim, rng.choice([dim, dim, dim // 2, dim // 4]),
                  rng.choice(["half", "half", "pairs"]), rng.choice(["none", "linear", "ntk", "yarn"]),
                  rng.choice(["f32", "f32", "f16"]), rng.choice(["f32", "f16", "q8_0", "q4"]),
                  rows + rng.randrange(0, 3 * rows + 64), rng.random() < 0.4, rng.random() < 0.4)
    else:
        n = 32 * _log(rng, 4, 592)
        m = _log(rng, 1, 16)
        p = _log(rng, 16, max(16, min(65536, (60_000_000 if op == "gated" else 120_000_000) // n, 1_000_000_000 // (n * m))))
        group = rng.choice([32, 64, 128])
        if op == "gated":
            c = _gated("", m, n, p, group, rng.choice(["f32", "f32", "f16", "q8_0", "norm"]))
        else:
            c = _q4("", m, n, p, group, rng.choice(["f32", "f32", "f16", "q8_0"]), rng.random() < 0.4, rng.random() < 0.4)
    del c["name"]
    return c


def _counts(case):
    b, n = case["batch"], case["rows"]
    return [1 + int((n - 1) * (((i + 1) * GOLDEN) % 1.0)) for i in range(b - 1)] + [n] if n > 1 else [n] * b


def _starts(case):
    """First rows: the last sequence's ends the cache."""
    room, b = case["cap"] - case["rows"], case["batch"]
    return [int(room * (((i + 3) * GOLDEN) % 1.0)) for i in range(b - 1)] + [room]


def _stride(case):
    """Elements from one sequence's cache to the next's: whole lines of memory for every cache type."""
    return -(-case["cap"] * case["kv_heads"] * case["dim"] // 256) * 256


def _row_bytes(kind, n):
    return {"f32": 4 * n, "f16": 2 * n, "q8_0": n // 32 * 34, "q4": n // 32 * 18}[kind]


def _q4_bytes(p, n, group):
    return p * (n // 2 + 2 * -(-n // group))


def work(case):
    if case["op"] == "norm":
        e, n = {"f32": 4, "f16": 2}[case["src"]], case["n"]
        # x, the residual and their sum; the output; an 8-bit one is read back as f16
        moved = n * e * (3 if case["residual"] else 1) + _row_bytes(case["dst"], n)
        back = _row_bytes("q8_0", n) + 2 * n if case["dst"] == "q8_0" else 0
        return {"bytes": case["rows"] * (moved + back) + 4 * n, "flops": case["rows"] * n * 5}
    if case["op"] == "rope":
        rows, w, q = sum(_counts(case)), case["kv_heads"] * case["dim"], case["heads"] * case["dim"]
        e, packed = {"f32": 4, "f16": 2}[case["src"]], case["cache"] in ("q8_0", "q4")
        cached = 2 * _row_bytes(case["cache"], w)
        # the projection's rows; q as f32; the cache rows, packed ones read back as f32; the positions' angles
        each = e * (q + 2 * w) + 4 * q + cached + (cached + 8 * w if packed else 0) + 4 * case["rot"]
        return {"bytes": rows * each, "flops": rows * (q + w) * 3}
    m, n, p = case["m"], case["n"], case["p"]
    two = 2 if case["op"] == "gated" else 1
    x = _row_bytes("f32", n) * 3 + _row_bytes("q8_0", n) * 2 if case["x"] == "norm" else _row_bytes(case["x"], n)
    out = 4 * m * p * (2 if case.get("residual") else 1) + (4 * p if case.get("bias") else 0)
    return {"bytes": two * _q4_bytes(p, n, case["group"]) + m * x + out, "flops": two * 2 * m * n * p}


# ---- inputs ----------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    s = {"case": case}
    if case["op"] == "norm":
        _prepare_norm(s, gen, case["rows"], case["n"], case["src"], case["dst"], case["residual"])
    elif case["op"] == "rope":
        _prepare_rope(s, gen)
    else:
        m, n, p = case["m"], case["n"], case["p"]
        if case["x"] == "norm":
            _prepare_norm(s, gen, m, n, "f32", "q8_0", True)
        else:
            s["x"] = _rows_of(_normal(gen, (m, n)), case["x"])
        for name in ("wg", "wu") if case["op"] == "gated" else ("w",):
            w = _normal(gen, (p, n)) / math.sqrt(n)
            if own:
                s[name] = _packed(w, case["group"])
            else:
                s[name] = _quantized(w, case["group"])
            del w
        s["bias"] = 0.1 * _normal(gen, (p,)) if case.get("bias") else None
        s["residual"] = _normal(gen, (m, p)) if case.get("residual") else None
        s["y"] = torch.empty(m, p, device="cuda")
    if own:
        import q8_block_quantized_matvec_gb300 as q8d
        s["q8d"] = q8d
    return s


def _prepare_norm(s, gen, rows, n, src, dst, residual):
    s["x"] = _stream(gen, rows, n, src)
    s["r"] = _stream(gen, rows, n, src) if residual else None
    s["sum"] = torch.empty_like(s["x"]) if residual else None
    s["weight"] = 1 + 0.1 * _normal(gen, (n,))
    if dst == "q8_0":
        # rows of whole 16-byte lines; the values are read back as f16
        s["ld"] = -(-n // 256) * 256
        s["out"] = torch.zeros(rows + rows % 2, _row_bytes("q8_0", s["ld"]), dtype=torch.uint8, device="cuda")
        s["back"] = torch.empty(rows + rows % 2, s["ld"], dtype=torch.float16, device="cuda")
        s["zero"] = _ints([0])
    else:
        s["ld"] = n
        s["out"] = torch.empty(rows, n, dtype=TORCH[dst], device="cuda")


def _stream(gen, rows, n, kind):
    """Rows of a residual stream: normal values, a few columns ten times as large, rows of unequal size."""
    x = _normal(gen, (rows, n)) * torch.exp(_normal(gen, (rows, 1)))
    x[:, ::97] *= 10
    return x.clamp_(-6e4, 6e4).to(TORCH[kind])


def _prepare_rope(s, gen):
    c = s["case"]
    batch, rows, heads, kv_heads, dim, cap = (c[x] for x in ("batch", "rows", "heads", "kv_heads", "dim", "cap"))
    q, w = heads * dim, kv_heads * dim
    both = _normal(gen, (batch * rows, q + 2 * w)).to(TORCH[c["src"]])  # one projection's rows
    s["q"], s["k"], s["v"] = both[:, :q], both[:, q:q + w], both[:, q + w:]
    s["bias"] = [0.1 * _normal(gen, (x,)) for x in (q, w, w)] if c["bias"] else [None] * 3
    s["norms"] = [1 + 0.1 * _normal(gen, (dim,)) for _ in range(2)] if c["norm"] else [None] * 2
    s["q_out"] = torch.zeros(batch * rows, q, device="cuda")
    n = _row_bytes(c["cache"], _stride(c))
    if c["cache"] in TORCH:
        s["kc"], s["vc"] = (_normal(gen, (batch, _stride(c))).to(TORCH[c["cache"]]) for _ in range(2))
    else:
        s["kc"], s["vc"] = (torch.zeros(batch, n, dtype=torch.uint8, device="cuda") for _ in range(2))
        s["k_out"], s["v_out"] = (torch.zeros(batch, rows, w, device="cuda") for _ in range(2))
    s["pos"], s["count"], s["err"] = _ints(_starts(c)), _ints(_counts(c)), _ints([0])
    if own:
        import q8_block_quantized_matvec_gb300 as q8d
        s["table"] = torch.empty(cap, c["rot"], device="cuda")
        factor = 1.0 if c["scaling"] == "none" else YARN["factor"]
        q8d.q8d_rope_table(s["table"], cap, c["rot"], THETA,
                           {"none": q8d.Q8D_ROPE_PLAIN, "linear": q8d.Q8D_ROPE_LINEAR, "ntk": q8d.Q8D_ROPE_NTK,
                            "yarn": q8d.Q8D_ROPE_YARN}[c["scaling"]], factor, YARN["orig"], YARN["fast"], YARN["slow"],
                           _mscale(c))
        s["desc"] = q8d.rope_desc(n_heads=heads, n_kv_heads=kv_heads, head_dim=dim, rot_dim=c["rot"],
                                  layout=q8d.Q8D_ROPE_HALF if c["layout"] == "half" else q8d.Q8D_ROPE_PAIRS,
                                  max_pos=cap, table=s["table"], row_dtype=CODE[c["src"]], ldq=q + 2 * w, ldkv=q + 2 * w,
                                  bq=s["bias"][0], bk=s["bias"][1], bv=s["bias"][2], q_norm=s["norms"][0],
                                  k_norm=s["norms"][1], eps=EPS, q_dtype=F32, ldo=q, kv_dtype=CODE[c["cache"]], cap=cap,
                                  cache_batch_stride=_stride(c))


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _normal(gen, shape):
    return torch.randn(shape, generator=gen, device="cuda")


def _packed(w, group):
    import q8_block_quantized_matvec_gb300 as q8d
    p, n = w.shape
    out = torch.empty(q8d.q8d_q4_matrix_bytes(p, n, group), dtype=torch.uint8, device="cuda")
    q8d.q8d_q4_pack(w, F32, n, out, p, n, group)
    return out


def _rows_of(x, kind):
    """f32 rows in a type of rows: f32, f16 or the bytes of Q8_0 blocks."""
    return x.to(TORCH[kind]) if kind in TORCH else _q8_rows(x)


# ---- formats, in f32 steps -------------------------------------------------

def _q8_rows(x):
    """Q8_0 rows (bytes) of f32 rows."""
    b = x.unflatten(-1, (-1, 32))
    d = b.abs().amax(-1, keepdim=True)
    d = d / torch.full_like(d, 127)  # (a tensor's division by a number is a product with its inverse)
    r = b * torch.where(d > 0, 1 / d, torch.zeros_like(d))
    q = torch.trunc(r)
    q = (q + torch.sign(r) * ((r - q).abs() >= 0.5)).to(torch.int8)  # to nearest, halves away from zero
    return torch.cat([d.half().view(torch.uint8), q.view(torch.uint8)], -1).flatten(-2)


def _q8_values(b):
    """f32 values of Q8_0 rows (bytes)."""
    b = b.unflatten(-1, (-1, 34))
    return (b[..., :2].contiguous().view(torch.float16).float() * b[..., 2:].view(torch.int8).float()).flatten(-2)


def _q4_codes(g):
    """(n_j, f32 scales) of f32 groups [..., size]."""
    d = g.gather(-1, g.abs().argmax(-1, keepdim=True)) / -8
    inv = 1 / d
    inv = torch.where(torch.isfinite(inv), inv, torch.zeros_like(inv))
    return torch.floor(g * inv + 8.5).clamp(0, 15).to(torch.uint8), d


def _groups(w, group):
    """[p][n] as [p][groups][group], zeros behind the last element."""
    n = w.shape[1]
    return torch.nn.functional.pad(w, (0, -n % group)).unflatten(1, (-1, group))


def _quantized(w, group):
    """(bytes of two neighbours each [p][n / 2], f16 scales [p][groups]) of an f32 matrix."""
    q, d = _q4_codes(_groups(w, group))
    q = q.flatten(1)[:, :w.shape[1]]
    return q[:, 0::2] | q[:, 1::2] << 4, d[..., 0].half()


def _values(wq, group):
    """f32 [p][n] of a quantized matrix."""
    q, d = wq
    q = torch.stack([q & 15, q >> 4], -1).flatten(1).float() - 8
    return q * d.float().repeat_interleave(group, 1)[:, :q.shape[1]]


# ---- one pass --------------------------------------------------------------

def run(s):
    c = s["case"]
    if c["op"] == "norm":
        return _run_norm(s, c["rows"], c["n"], c["src"], c["dst"])
    if c["op"] == "rope":
        return _run_rope(s)
    return _run_product(s)


def _call_norm(s, rows, n, src, dst):
    s["q8d"].q8d_rmsnorm_rows(s["x"], s["r"], s["sum"], CODE[src], n, n, n, s["weight"], EPS, s["out"], CODE[dst], s["ld"],
                              rows, n)


def _normed(s):
    """(sum, f32 norm of it) in the operator's f32 steps."""
    h = s["x"].float()
    if s["r"] is not None:
        h = h + s["r"].float()
    mean = h.double().square().mean(-1, keepdim=True)
    return h, h * (1 / torch.sqrt(mean + EPS)).float() * s["weight"]


def _run_norm(s, rows, n, src, dst):
    if own:
        _call_norm(s, rows, n, src, dst)
        if dst != "q8_0":
            return {"y": s["out"], "sum": s["sum"]}
        # the 8-bit rows as f16 values: rows of a packed cache, the first half read as K's, the others as V's
        half = s["out"].shape[0] // 2
        s["q8d"].q8d_kv_read_rows(s["out"][:half], s["out"][half:], Q8_0, s["back"][:half], s["back"][half:], F16, s["ld"], 1,
                                  half, s["ld"], half, 0, s["zero"], None, None)
        return {"y": s["back"][:rows, :n], "sum": s["sum"]}
    h, y = _normed(s)
    y = _q8_values(_q8_rows(y)).half() if dst == "q8_0" else y.to(TORCH[dst])
    return {"y": y, "sum": h.to(TORCH[src]) if s["r"] is not None else None}


def _mscale(c):
    """What YaRN multiplies the rotation with."""
    return 0.1 * math.log(YARN["factor"]) + 1 if c["scaling"] == "yarn" else 1.0


def _frequencies(c):
    """f64 angle of each pair for one position."""
    i = torch.arange(c["rot"] // 2, device="cuda", dtype=torch.float64)
    if c["scaling"] == "ntk":
        base = THETA * YARN["factor"] ** (c["rot"] / (c["rot"] - 2))
        return base ** (-2 * i / c["rot"])
    f = THETA ** (-2 * i / c["rot"])
    if c["scaling"] == "linear":
        return f / YARN["factor"]
    if c["scaling"] == "yarn":
        at = lambda turns: c["rot"] * math.log(YARN["orig"] / (turns * 2 * math.pi)) / (2 * math.log(THETA))  # noqa: E731
        low, high = max(math.floor(at(YARN["fast"])), 0), min(math.ceil(at(YARN["slow"])), c["rot"] - 1)
        ramp = ((i - low) / max(high - low, 0.001)).clamp(0, 1)
        return f / YARN["factor"] * ramp + f * (1 - ramp)
    return f


def _rotated(c, x, cos, sin):
    """Heads [..., heads, dim] turned by the angles of cos, sin [..., 1, rot / 2]; single rounded steps in x's type."""
    r = c["rot"]
    a, b = (x[..., :r // 2], x[..., r // 2:r]) if c["layout"] == "half" else (x[..., 0:r:2], x[..., 1:r:2])
    a, b = a * cos - b * sin, a * sin + b * cos
    turned = torch.cat([a, b], -1) if c["layout"] == "half" else torch.stack([a, b], -1).flatten(-2)
    return torch.cat([turned, x[..., r:]], -1)


def _run_rope(s):
    c = s["case"]
    batch, rows, heads, kv_heads, dim, cap = (c[x] for x in ("batch", "rows", "heads", "kv_heads", "dim", "cap"))
    w = kv_heads * dim
    if own:
        q8d = s["q8d"]
        q8d.q8d_rope_append_rows(s["desc"], s["q"], s["k"], s["v"], s["q_out"], s["kc"], s["vc"], batch, rows, s["pos"], None,
                                 s["count"], s["err"])
        if c["cache"] in TORCH:
            return {"q": s["q_out"], "k": s["kc"], "v": s["vc"]}
        q8d.q8d_kv_read_rows(s["kc"], s["vc"], CODE[c["cache"]], s["k_out"], s["v_out"], F32, w, batch, rows, w, cap,
                             _stride(c), s["pos"], s["count"], s["err"])
        return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"]}
    step = torch.arange(rows, device="cuda")
    at = s["pos"].long()[:, None] + step  # [batch][rows]
    live = (step < s["count"][:, None])[..., None]
    angle = at.double()[..., None] * _frequencies(c)
    cos, sin = ((f(angle) * _mscale(c)).float()[:, :, None] for f in (torch.cos, torch.sin))
    q, k, v = (x.float() if b is None else x.float() + b for x, b in zip((s["q"], s["k"], s["v"]), s["bias"]))
    q, k = q.view(batch, rows, heads, dim), k.view(batch, rows, kv_heads, dim)
    if c["norm"]:
        q, k = (x * (1 / torch.sqrt(x.double().square().mean(-1, keepdim=True) + EPS)).float() * g
                for x, g in zip((q, k), s["norms"]))
    q, k = (_rotated(c, x, cos, sin).flatten(2) for x in (q, k))
    q_out = s["q_out"].view(batch, rows, -1)
    q_out.copy_(torch.where(live, q, q_out))
    kv = {"k": k, "v": v.view(batch, rows, w)}
    if c["cache"] in TORCH:
        seq = torch.arange(batch, device="cuda")[:, None]
        planes = {x: s[x + "c"][:, :cap * w].view(batch, cap, w) for x in kv}
        at = at.clamp(max=cap - 1)
        at = torch.where(live[..., 0], at, at[:, :1])  # (dead rows write the first row's value again)
        new = {x: torch.where(live, y.to(TORCH[c["cache"]]), y[:, :1].to(TORCH[c["cache"]])) for x, y in kv.items()}
        planes["k"][seq, at], planes["v"][seq, at] = new["k"], new["v"]
        return {"q": s["q_out"], "k": s["kc"], "v": s["vc"]}
    new = {x: _cached(y, c["cache"]) for x, y in kv.items()}
    for x in new:
        s[x + "_out"].copy_(torch.where(live, new[x], s[x + "_out"]))
    return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"]}


def _cached(x, kind):
    """f32 values of f32 rows after their store in a packed cache."""
    if kind == "q8_0":
        return _q8_values(_q8_rows(x))
    q, d = _q4_codes(x.unflatten(-1, (-1, 32)))
    return ((q.float() - 8) * d.half().float()).flatten(-2)


def _run_product(s):
    c = s["case"]
    m, n, p, group = (c[x] for x in ("m", "n", "p", "group"))
    if own:
        q8d = s["q8d"]
        x, kind, ld = s["x"], c["x"], n
        if kind == "norm":
            _call_norm(s, m, n, "f32", "q8_0")
            x, kind, ld = s["out"], "q8_0", s["ld"]
        if c["op"] == "gated":
            q8d.q8d_q4_gated(x, CODE[kind], ld, s["wg"], s["wu"], group, s["y"], p, m, n, p)
        else:
            q8d.q8d_q4_matmul(x, CODE[kind], ld, s["w"], group, s["bias"], s["residual"], p, s["y"], p, m, n, p)
        return {"y": s["y"], "sum": s.get("sum")}
    if c["x"] == "norm":
        h, x = _normed(s)
        x = _q8_values(_q8_rows(x))
    else:
        h, x = None, _q8_values(s["x"]) if c["x"] == "q8_0" else s["x"].float()
    if c["op"] == "gated":
        g, u = torch.matmul(x, _values(s["wg"], group).T), torch.matmul(x, _values(s["wu"], group).T)
        y = g / (1 + torch.exp(-g)) * u
    else:
        y = torch.matmul(x, _values(s["w"], group).T)
        if s["bias"] is not None:
            y = y + s["bias"]
        if s["residual"] is not None:
            y = y + s["residual"]
    return {"y": y, "sum": h}


# ---- the definition in 64 bits ---------------------------------------------

def exact(case, seed):
    global own
    mode, own = own, False  # (the inputs alone)
    try:
        s = prepare(case, seed)
    finally:
        own = mode
    if case["op"] == "norm":
        h, y = _exact_norm(s, case["dst"] == "q8_0")
        return {"y": y, "sum": h if case["residual"] else None}
    if case["op"] == "rope":
        return _exact_rope(case, s)
    if case["x"] == "norm":
        h, x = _exact_norm(s, True)
    else:
        h, x = None, _exact_q8(s["x"]) if case["x"] == "q8_0" else s["x"].double()
    if case["op"] == "gated":
        g = x @ _exact_q4(s["wg"], case["group"]).T
        return {"y": torch.nn.functional.silu(g) * (x @ _exact_q4(s["wu"], case["group"]).T), "sum": h}
    y = x @ _exact_q4(s["w"], case["group"]).T
    for more in (s["bias"], s["residual"]):
        y = y if more is None else y + more.double()
    return {"y": y, "sum": h}


def _round32(v):
    return v.float().double()


def _exact_q8(rows):
    """f64 values of Q8_0 rows (bytes)."""
    b = rows.view(rows.shape[0], -1, 34).int()
    scale = (b[:, :, 0] + 256 * b[:, :, 1]).to(torch.int16).view(torch.float16).double()
    quants = b[:, :, 2:]
    return ((quants - 256 * (quants > 127).int()).double() * scale[:, :, None]).reshape(rows.shape[0], -1)


def _exact_q4(wq, group):
    """f64 [p][n] of a quantized matrix."""
    q, d = wq
    p, n = q.shape[0], 2 * q.shape[1]
    out = torch.empty(p, n, dtype=torch.float64, device="cuda")
    out[:, 0::2] = (q % 16).double() - 8
    out[:, 1::2] = (q // 16).double() - 8
    at = torch.arange(n, device="cuda") // group
    return out.mul_(d.double()[:, at])


def _exact_store(x, kind):
    """What a packed type keeps of f64 rows of f32 values.  The quantizers' steps are 32-bit ones by definition: each is done
    in 64 bits and rounded."""
    v = x.reshape(x.shape[0], -1, 32)
    if kind == "q8_0":  # scale = largest / 127, halves away from zero
        d = _round32(v.abs().max(2, keepdim=True).values / 127)
        r = torch.where(d > 0, _round32(v * _round32(1 / d)), 0.0)
        return (torch.sign(r) * torch.floor(r.abs() + 0.5) * d.half().double()).view(x.shape)
    largest = v.abs() == v.abs().max(2, keepdim=True).values
    first = torch.where(largest, torch.arange(32, device="cuda"), 32).min(2, keepdim=True).values
    d = v.gather(2, first) / -8
    r = torch.where(_round32(1 / d).isfinite(), _round32(v * _round32(1 / d)), 0.0)
    return ((torch.floor(_round32(r + 8.5)).clamp(0, 15) - 8) * d.half().double()).view(x.shape)


def _exact_norm(s, eight):
    """(sum, norm); into 8 bits the norm's steps are 32-bit ones by definition, but for the mean."""
    step = _round32 if eight else (lambda v: v)
    h = s["x"].double()
    if s["r"] is not None:
        h = h + s["r"].double()
    true = h
    h = step(h)
    scale = step(torch.rsqrt(torch.sum(h * h, 1, keepdim=True) / h.shape[1] + EPS))
    y = step(step(h * scale) * s["weight"].double())
    return true, _exact_store(y, "q8_0") if eight else y


def _exact_rope(c, s):
    batch, rows, dim, cap = (c[x] for x in ("batch", "rows", "dim", "cap"))
    packed = c["cache"] not in TORCH
    step = _round32 if packed else (lambda v: v)
    r = c["rot"]
    out = {"q": s["q_out"].double().clone().view(batch, rows, -1)}
    w = c["kv_heads"] * dim
    for x in ("k", "v"):
        out[x] = (s[x + "_out"] if packed else s[x + "c"]).double().clone()
    for b, (first, n) in enumerate(zip(_starts(c), _counts(c))):
        pos = torch.arange(first, first + n, device="cuda", dtype=torch.float64)
        turn = torch.outer(pos, _frequencies(c))
        turn = torch.polar(torch.full_like(turn, _mscale(c)), turn)[:, None]  # [n][1][rot / 2]
        for i, x in enumerate(("q", "k", "v")):
            st = step if x != "q" else (lambda v: v)
            h = s[x][b * rows:b * rows + n].double()
            if s["bias"][i] is not None:
                h = st(h + s["bias"][i].double())
            if x != "v":
                h = h.reshape(n, -1, dim)
                if c["norm"]:
                    inv = st(torch.rsqrt((h * h).sum(2, keepdim=True) / dim + EPS))
                    h = st(st(h * inv) * s["norms"][i].double())
                if c["layout"] == "half":
                    a, e = h[..., :r // 2], h[..., r // 2:r]
                else:
                    a, e = h[..., :r].unflatten(2, (r // 2, 2)).unbind(3)
                re, im = st(turn.real), st(turn.imag)
                a, e = st(st(a * re) - st(e * im)), st(st(a * im) + st(e * re))
                t = torch.cat([a, e], 2) if c["layout"] == "half" else torch.stack([a, e], 3).flatten(2)
                h = torch.cat([t, h[..., r:]], 2).flatten(1)
            if x == "q":
                out[x][b, :n] = h
            elif packed:
                out[x][b, :n] = _exact_store(h, c["cache"])
            else:
                out[x][b, first * w:(first + n) * w] = h.flatten()
    out["q"] = out["q"].view(batch * rows, -1)
    return out
