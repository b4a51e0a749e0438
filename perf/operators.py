"""Timed cases of three operators of a decode layer: the 4-bit KV cache's row
store and read-back, the decode attention over that cache, and a
mixture-of-experts feed-forward layer over Q8_0 experts for a few tokens.

`run` computes a case in plain torch arithmetic (`own` false) or through this
package's entry points (`own` true).

The 4-bit cache of one sequence is two planes, quants then scales: row t's
kv_width/32 blocks of 16 bytes at byte t * kv_width/2, its f16 scales at byte
cap * kv_width/2 + t * kv_width/16.  Byte i of a block holds element i in its
low half and element i + 16 in its high half, the value being
scale * (nibble - 8).  Every sequence's cache starts at a multiple of 256
elements."""
import math

import torch

own = False

F32, F16, Q8_0, Q4 = 0, 1, 2, 4
KV = {"f32": F32, "f16": F16, "q8_0": Q8_0, "q4": Q4}
TORCH = {"f32": torch.float32, "f16": torch.float16}
GOLDEN = 0.6180339887498949


# ---- cases -----------------------------------------------------------------

def listed():
    return [
        # one token of each of 64 sequences stored and read back: a decode step's write
        _kv("kv_decode_64x1", "q4", "f32", "f32", 64, 1, 1024, 4096, 0),
        # a prompt stored from the fused q|k|v projection's output (rows of 4608 values)
        _kv("kv_prompt_4096", "q4", "f32", "f16", 1, 4096, 512, 8192, 4608),
        # prompts of unequal lengths into a packed Q8_0 cache, in half precision
        _kv("kv_prompts_ragged_q8", "q8_0", "f16", "f16", 8, 2047, 1024, 4096, 0),
        # a long cache read back, as before attention over a whole prompt
        _kv("kv_read_long", "q4", "", "f16", 1, 131071, 512, 131072, 0),
        # one sequence at a short context: the latency of a decode step's attention
        _attn("attn_7b_ctx2048", 1, 28, 4, 128, 2048, False),
        # a serving batch whose contexts are unequal
        _attn("attn_7b_batch8_ragged32k", 8, 28, 4, 128, 32768, True),
        # many sequences, two query heads per KV head
        _attn("attn_16_8_batch32_ragged8k", 32, 16, 8, 128, 8192, True),
        # one long context of odd length, head_dim 64
        _attn("attn_14_2_long", 1, 14, 2, 64, 131071, False),
        # one token through a small layer: latency
        _moe("moe_1_small", 1, 1024, 512, 32, 4, True, True),
        # one token through an ordinary layer
        _moe("moe_1", 1, 2048, 1024, 64, 8, True, True),
        # a few tokens, expert rows that are not whole 16-byte lines
        _moe("moe_8_odd", 8, 3584, 1184, 64, 6, False, False),
        # a serving batch: nearly every expert is asked
        _moe("moe_64", 64, 2048, 768, 128, 8, True, True),
    ]


def _kv(name, cache, src, dst, batch, rows, width, cap, ld):
    """src: type of the rows stored ("" reads only); ld: values from one source row to the next (0: rows side by side)."""
    return {"name": name, "op": "kv", "cache": cache, "src": src, "dst": dst, "batch": batch, "rows": rows, "width": width,
            "cap": cap, "ld": ld}


def _attn(name, batch, heads, kv_heads, dim, cap, ragged):
    return {"name": name, "op": "attn", "batch": batch, "heads": heads, "kv_heads": kv_heads, "dim": dim, "cap": cap,
            "ragged": ragged}


def _moe(name, tokens, hidden, ffn, experts, top, norm, residual):
    return {"name": name, "op": "moe", "tokens": tokens, "hidden": hidden, "ffn": ffn, "experts": experts, "top": top,
            "norm": norm, "residual": residual}


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["kv", "attn", "moe"])
    if op == "kv":
        cache = rng.choice(["q4", "q4", "q8_0", "f16", "f32"])
        width = 32 * _log(rng, 2, 64)
        batch = _log(rng, 1, 64)
        rows = _log(rng, 1, max(1, min(32768, 16_000_000 // (width * batch))))
        cap = rows + rng.randrange(0, rows + 64)
        c = _kv("", cache, rng.choice(["f32", "f32", "f16", ""]), rng.choice(["f32", "f16"]), batch, rows, width, cap,
                rng.choice([0, 0, 3 * width + 32 * rng.randrange(0, 8)]))
    elif op == "attn":
        kv_heads, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 12, 16])
        dim = rng.choice([64, 128])
        batch = _log(rng, 1, 64)
        cap = _log(rng, 1, min(131072, 60_000_000 // (kv_heads * dim * batch)))
        c = _attn("", batch, kv_heads * group, kv_heads, dim, cap, rng.random() < 0.7)
    else:
        experts = rng.choice([4, 8, 16, 32, 60, 64, 128])
        hidden, ffn = 32 * _log(rng, 16, 112), 32 * _log(rng, 4, 48)
        tokens = _log(rng, 1, 64)
        c = _moe("", tokens, hidden, ffn, experts, rng.randrange(1, min(8, experts) + 1), rng.random() < 0.6,
                 rng.random() < 0.6)
    del c["name"]
    return c


def _spread(n, lo, hi):
    """n whole numbers spread unevenly over [lo, hi], the last of them hi."""
    return [lo + int((hi - lo) * (((i + 1) * GOLDEN) % 1.0)) for i in range(n - 1)] + [hi]


def _lens(case):
    return _spread(case["batch"], 1, case["cap"]) if case["ragged"] else [case["cap"]] * case["batch"]


def _counts(case):
    return _spread(case["batch"], 1, case["rows"]) if case["batch"] > 1 and case["rows"] > 1 else [case["rows"]] * case["batch"]


def _starts(case):
    room = case["cap"] - case["rows"]
    return [int(room * (((i + 3) * GOLDEN) % 1.0)) for i in range(case["batch"])]


def _stride(case):
    """Elements from one sequence's cache to the next's: whole lines of memory for every cache type."""
    width = case["width"] if case["op"] == "kv" else case["kv_heads"] * case["dim"]
    return -(-case["cap"] * width // 256) * 256


def _row_bytes(cache, width):
    return {"f32": 4 * width, "f16": 2 * width, "q8_0": width // 32 * 34, "q4": width // 32 * 18}[cache]


def work(case):
    if case["op"] == "kv":
        n, w = sum(_counts(case)), case["width"]
        cached, out = n * _row_bytes(case["cache"], w), n * w * (4 if case["dst"] == "f32" else 2)
        src = n * w * {"f32": 4, "f16": 2, "": 0}[case["src"]]
        # stored: the source is read and the cache row written; read back: the cache row is read and the values written
        return {"bytes": 2 * (src + (cached if src else 0) + cached + out), "flops": 2 * n * w * (6 if src else 2)}
    if case["op"] == "attn":
        n, h = sum(_lens(case)), case["heads"] * case["dim"]
        return {"bytes": 2 * n * _row_bytes("q4", case["kv_heads"] * case["dim"]) + 8 * case["batch"] * h, "flops": 4 * n * h}
    m, hid, ffn, e, k = (case[x] for x in ("tokens", "hidden", "ffn", "experts", "top"))
    asked = e * (1.0 - (1.0 - k / e) ** m)  # experts that m independent tokens ask for
    return {"bytes": asked * 3 * ffn * (hid // 32) * 34 + 4 * e * hid + 4 * m * hid * (3 if case["residual"] else 2) + 8 * m * k,
            "flops": 6 * m * k * ffn * hid + 2 * m * e * hid}


# ---- inputs ----------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    s = {"case": case}
    if case["op"] == "kv":
        batch, rows, width, cap = (case[x] for x in ("batch", "rows", "width", "cap"))
        s["pos"], s["count"] = _ints(_starts(case)), _ints(_counts(case))
        s["err"] = _ints([0])
        for x in ("k", "v"):
            s[x + "cache"] = _filled(gen, case["cache"], batch, cap, width, _stride(case))
            s[x + "_out"] = torch.zeros(batch, rows, width, dtype=TORCH[case["dst"]], device="cuda")
        if case["src"]:
            ld = case["ld"] or width
            if case["ld"]:  # k and v are the last columns of one projection's rows
                both = _normal(gen, (batch * rows, ld)).to(TORCH[case["src"]])
                s["k"], s["v"] = both[:, ld - 2 * width:ld - width], both[:, ld - width:]
            else:
                s["k"] = _normal(gen, (batch * rows, width)).to(TORCH[case["src"]])
                s["v"] = _normal(gen, (batch * rows, width)).to(TORCH[case["src"]])
            s["ld"] = ld
    elif case["op"] == "attn":
        batch, heads, kv_heads, dim, cap = (case[x] for x in ("batch", "heads", "kv_heads", "dim", "cap"))
        s["q"] = _normal(gen, (batch, heads * dim))
        s["kcache"] = _filled(gen, "q4", batch, cap, kv_heads * dim, _stride(case))
        s["vcache"] = _filled(gen, "q4", batch, cap, kv_heads * dim, _stride(case))
        s["lens"], s["err"] = _ints(_lens(case)), _ints([0])
        s["out"] = torch.empty(batch, heads * dim, device="cuda")
    else:
        m, hid, ffn, e, k = (case[x] for x in ("tokens", "hidden", "ffn", "experts", "top"))
        s["x"] = _normal(gen, (m, hid))  # a layer's RMS-normalised activations
        s["router"] = _normal(gen, (e, hid)) / math.sqrt(hid) * 2
        s["wg"], s["wu"], s["wd"] = _q8(gen, e, ffn, hid), _q8(gen, e, ffn, hid), _q8(gen, e, hid, ffn)
        s["res"] = _normal(gen, (m, hid)) if case["residual"] else None
        s["y"] = torch.empty(m, hid, device="cuda")
        s["experts"] = torch.empty(m, k, dtype=torch.int32, device="cuda")
        s["weights"] = torch.empty(m, k, device="cuda")
        s["err"] = _ints([0])
    if own:
        import q8_block_quantized_matvec_gb300 as q8d
        s["q8d"] = q8d
        if case["op"] == "attn":
            n = q8d.q8d_gqa_workspace_bytes(case["batch"], case["heads"], case["kv_heads"], case["dim"], case["cap"])
        elif case["op"] == "moe":
            n = q8d.q8d_moe_workspace_bytes(m, hid, ffn, e, k)
        else:
            n = 0
        s["ws"], s["ws_bytes"] = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda"), n
    return s


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _normal(gen, shape):
    return torch.randn(shape, generator=gen, device="cuda")


def _filled(gen, cache, batch, cap, width, stride):
    """Caches [batch][stride elements] of normally distributed rows."""
    if cache in TORCH:
        return _normal(gen, (batch, stride)).to(TORCH[cache])
    blocks = width // 32
    c = torch.zeros(batch, _row_bytes(cache, stride), dtype=torch.uint8, device="cuda")
    # the scales that blocks of 32 normal values get, and quants of about their spread
    planes = _planes(c, cache, cap, width)
    if cache == "q8_0":
        rows = torch.randint(-100, 101, (batch, cap, blocks, 34), generator=gen, device="cuda", dtype=torch.int8).view(torch.uint8)
        rows[..., :2] = (_top(gen, batch, cap, blocks) / 127).half().unsqueeze(-1).view(torch.uint8)
        planes[0].copy_(rows.flatten(2))
        return c
    planes[0].copy_(torch.randint(0, 256, planes[0].shape, generator=gen, device="cuda", dtype=torch.uint8))
    sign = torch.randint(0, 2, (batch, cap, blocks), generator=gen, device="cuda") * 2 - 1
    planes[1].copy_((_top(gen, batch, cap, blocks) * sign / 8).half().view(torch.uint8))
    return c


def _top(gen, *shape):
    """The largest magnitude of a block of 32 normal values, near enough."""
    return (2.07 + 0.4 * _normal(gen, shape)).clamp_(1.2, 4.5)


def _q8(gen, e, p, n):
    """e matrices [p][n] of Q8_0 blocks whose products with unit activations have unit size."""
    w = torch.randint(-127, 128, (e, p, n // 32, 34), generator=gen, device="cuda", dtype=torch.int8).view(torch.uint8)
    scale = (0.5 + torch.rand((e, p, n // 32), generator=gen, device="cuda")) / (73 * math.sqrt(n))
    w[..., :2] = scale.half().unsqueeze(-1).view(torch.uint8)
    return w


# ---- one pass --------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if op == "kv":
        return _run_kv(s)
    if op == "attn":
        return _run_attn(s)
    return _run_moe(s)


def _run_kv(s):
    c = s["case"]
    batch, rows, width, cap = c["batch"], c["rows"], c["width"], c["cap"]
    if own:
        q8d = s["q8d"]
        if c["src"]:
            q8d.q8d_kv_append_rows(s["k"], s["v"], KV[c["src"]], s["ld"], s["kcache"], s["vcache"], KV[c["cache"]], batch, rows,
                                   width, cap, _stride(c), s["pos"], s["count"], s["err"])
        q8d.q8d_kv_read_rows(s["kcache"], s["vcache"], KV[c["cache"]], s["k_out"], s["v_out"], KV[c["dst"]], width, batch, rows,
                             width, cap, _stride(c), s["pos"], s["count"], s["err"])
        return {"k": s["k_out"], "v": s["v_out"]}
    step = torch.arange(rows, device="cuda")
    at = s["pos"].long()[:, None] + step  # [batch][rows] cache rows
    live = (step < s["count"][:, None])[..., None]
    seq = torch.arange(batch, device="cuda")[:, None]
    for x in ("k", "v"):
        planes = _planes(s[x + "cache"], c["cache"], cap, width)
        if c["src"]:
            new = _encode(s[x].float().view(batch, rows, width), c["cache"])
            for plane, rows_new in zip(planes, new):
                plane[seq, at] = torch.where(live, rows_new, plane[seq, at])
        got = _decode([plane[seq, at] for plane in planes], c["cache"])
        out = s[x + "_out"]
        out.copy_(torch.where(live, got.to(out.dtype), out))
    return {"k": s["k_out"], "v": s["v_out"]}


def _planes(cache, kind, cap, width):
    """Views [batch][cap][...] of what the caches [batch][...] keep for each row."""
    if kind == "q4":
        n = cap * width // 2
        return [cache[:, :n].unflatten(1, (cap, width // 2)), cache[:, n:n + n // 8].unflatten(1, (cap, width // 16))]
    row = width if kind in TORCH else _row_bytes(kind, width)
    return [cache[:, :cap * row].unflatten(1, (cap, row))]


def _encode(x, kind):
    """f32 rows [..., width] as the planes' rows."""
    if kind in TORCH:
        return [x.to(TORCH[kind])]
    b = x.unflatten(-1, (-1, 32))
    if kind == "q8_0":
        d = b.abs().amax(-1, keepdim=True)
        d = d / torch.full_like(d, 127)  # (a tensor's division by a number is a product with its inverse)
        r = b * torch.where(d > 0, 1 / d, torch.zeros_like(d))
        q = torch.trunc(r)
        q = (q + torch.sign(r) * ((r - q).abs() >= 0.5)).to(torch.int8)  # to nearest, halves away from zero
        return [torch.cat([d.half().view(torch.uint8), q.view(torch.uint8)], -1).flatten(-2)]
    # the element of largest magnitude (the first of them) becomes nibble 0
    d = b.gather(-1, b.abs().argmax(-1, keepdim=True)) / -8
    inv = 1 / d
    inv = torch.where(torch.isfinite(inv), inv, torch.zeros_like(inv))
    q = torch.floor(b * inv + 8.5).clamp(0, 15).to(torch.uint8)
    return [(q[..., :16] | q[..., 16:] << 4).flatten(-2), d.half().view(torch.uint8).flatten(-2)]


def _decode(planes, kind):
    """The f32 values of the planes' rows."""
    if kind in TORCH:
        return planes[0].float()
    if kind == "q8_0":
        b = planes[0].unflatten(-1, (-1, 34))
        return (b[..., :2].contiguous().view(torch.float16).float() * b[..., 2:].view(torch.int8).float()).flatten(-2)
    q = planes[0].unflatten(-1, (-1, 16))
    q = torch.cat([q & 15, q >> 4], -1).float() - 8
    return (planes[1].contiguous().view(torch.float16).float()[..., None] * q).flatten(-2)


def _run_attn(s):
    c = s["case"]
    batch, heads, kv_heads, dim, cap = (c[x] for x in ("batch", "heads", "kv_heads", "dim", "cap"))
    if own:
        s["q8d"].q8d_gqa_decode_attn(s["q"], None, None, s["kcache"], s["vcache"], Q4, s["out"], batch, heads, kv_heads, dim, cap,
                                     _stride(c), s["lens"], 1 / math.sqrt(dim), s["ws"], s["ws_bytes"], s["err"])
        return s["out"]
    width = kv_heads * dim
    k, v = (_decode(_planes(s[x], "q4", cap, width), "q4").view(batch, cap, kv_heads, dim).transpose(1, 2)
            for x in ("kcache", "vcache"))
    q = s["q"].view(batch, kv_heads, heads // kv_heads, dim)
    p = torch.matmul(q, k.transpose(2, 3)) * (1 / math.sqrt(dim))
    p = p.masked_fill((torch.arange(cap, device="cuda") >= s["lens"][:, None])[:, None, None], -math.inf)
    p = torch.exp(p - p.amax(-1, keepdim=True))
    return (torch.matmul(p, v) / p.sum(-1, keepdim=True)).reshape(batch, heads * dim)


def _run_moe(s):
    c = s["case"]
    m, hid, ffn, e, k = (c[x] for x in ("tokens", "hidden", "ffn", "experts", "top"))
    if own:
        s["q8d"].q8d_moe_ffn(s["x"], hid, s["router"], s["wg"], s["wu"], s["wd"], s["res"], hid, s["y"], hid, m, hid, ffn, e, k,
                             int(c["norm"]), s["experts"], s["weights"], s["ws"], s["ws_bytes"], s["err"])
        return {"y": s["y"], "experts": s["experts"], "weights": s["weights"]}
    x = s["x"]
    # the choice in 64 bits: experts next to one another in rank may be near
    p = torch.matmul(x.double(), s["router"].double().T)
    p = torch.exp(p - p.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    w, at = torch.sort(p, dim=-1, descending=True, stable=True)
    w, at = w[:, :k], at[:, :k]
    if c["norm"]:
        w = w / w.sum(-1, keepdim=True)
    w = w.float()
    if m * k < e:  # the chosen experts' matrices, one copy for each (token, expert)
        of = at.flatten()
        xs = x.repeat_interleave(k, 0)[..., None]
        g, u = torch.bmm(_matrices(s["wg"][of]), xs), torch.bmm(_matrices(s["wu"][of]), xs)
        y = torch.bmm(_matrices(s["wd"][of]), g / (1 + torch.exp(-g)) * u)
        y = (y.view(m, k, hid) * w[..., None]).sum(1)
    else:  # every expert on every token
        g, u = torch.matmul(_matrices(s["wg"]), x.T), torch.matmul(_matrices(s["wu"]), x.T)
        y = torch.matmul(_matrices(s["wd"]), g / (1 + torch.exp(-g)) * u)  # [expert][hidden][token]
        share = torch.zeros(m, e, device="cuda").scatter_(1, at, w)
        y = (y * share.T[:, None]).sum(0).T.contiguous()
    if s["res"] is not None:
        y = y + s["res"]
    return {"y": y, "experts": at.int(), "weights": w}


def _matrices(w):
    """f32 values of Q8_0 matrices [..., p, n/32, 34]."""
    return (w[..., :2].contiguous().view(torch.float16).float() * w[..., 2:].view(torch.int8).float()).flatten(-2)


# ---- the definition in 64 bits ---------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "kv":
        return {x: _exact_kv(case, s, x) for x in ("k", "v")}
    if case["op"] == "attn":
        return _exact_attn(case, s)
    return _exact_moe(case, s)


def _exact_q4(cache, width, cap, rows):
    """Rows of one sequence's 4-bit cache as f64 [rows][width]."""
    quants = cache[:cap * width // 2].view(cap, width // 32, 16)[rows].int()
    scales = cache[cap * width // 2:cap * width // 16 * 9].view(torch.float16).view(cap, width // 32, 1)[rows].double()
    return (torch.cat([quants % 16, quants // 16], 2).double() - 8).mul_(scales).view(-1, width)


def _exact_q8(block_bytes):
    scale = block_bytes[..., 0].int() + 256 * block_bytes[..., 1].int()
    scale = scale.to(torch.int16).view(torch.float16).double()
    return block_bytes[..., 2:].view(torch.int8).double() * scale[..., None]


def _round32(v):
    return v.float().double()


def _exact_kv(case, s, x):
    kind, width, cap, rows = case["cache"], case["width"], case["cap"], case["rows"]
    out = s[x + "_out"].double()
    for b, (first, n) in enumerate(zip(_starts(case), _counts(case))):
        at = slice(first, first + n)
        if not case["src"]:
            cache = s[x + "cache"][b]
            if kind == "q4":
                out[b, :n] = _exact_q4(cache, width, cap, at)
            elif kind == "q8_0":
                out[b, :n] = _exact_q8(cache[:cap * width // 32 * 34].view(cap, width // 32, 34)[at]).view(n, width)
            else:
                out[b, :n] = cache[:cap * width].view(cap, width)[at].double()
            continue
        v = s[x][b * rows:b * rows + n].double().reshape(n, width // 32, 32)
        # the quantizers' steps are 32-bit ones by definition: each is done in 64 bits and rounded
        if kind == "q8_0":  # scale = largest / 127, halves away from zero
            d = _round32(v.abs().max(2, keepdim=True).values / 127)
            r = torch.where(d > 0, _round32(v * _round32(1 / d)), 0.0)
            v = torch.sign(r) * torch.floor(r.abs() + 0.5) * d.half().double()
        elif kind == "q4":
            largest = v.abs() == v.abs().max(2, keepdim=True).values
            first = torch.where(largest, torch.arange(32, device="cuda"), 32).min(2, keepdim=True).values
            d = v.gather(2, first) / -8
            r = torch.where(_round32(1 / d).isfinite(), _round32(v * _round32(1 / d)), 0.0)
            v = (torch.floor(_round32(r + 8.5)).clamp(0, 15) - 8) * d.half().double()
        elif kind == "f16":
            v = v.half().double()
        out[b, :n] = v.view(n, width)
    return out


def _exact_attn(case, s):
    heads, kv_heads, dim, cap = (case[x] for x in ("heads", "kv_heads", "dim", "cap"))
    out = torch.empty(case["batch"], kv_heads, heads // kv_heads, dim, dtype=torch.float64, device="cuda")
    q = s["q"].double().view(out.shape)
    for b, n in enumerate(_lens(case)):
        k, v = (_exact_q4(s[x][b], kv_heads * dim, cap, slice(0, n)).view(n, kv_heads, dim) for x in ("kcache", "vcache"))
        for g in range(kv_heads):
            p = torch.softmax(q[b, g] @ k[:, g].T / math.sqrt(dim), -1)
            out[b, g] = p @ v[:, g]
    return out.view(case["batch"], heads * dim)


def _exact_moe(case, s):
    k = case["top"]
    y = s["res"].double() if case["residual"] else torch.zeros_like(s["x"], dtype=torch.float64)
    logits = s["x"].double() @ s["router"].double().T
    chosen = torch.argsort(logits, dim=1, descending=True, stable=True)[:, :k]
    weights = torch.softmax(logits, 1).gather(1, chosen)
    if case["norm"]:
        weights = weights / weights.sum(1, keepdim=True)
    for e in torch.unique(chosen).tolist():
        t, j = (chosen == e).nonzero(as_tuple=True)
        wg, wu, wd = (_exact_q8(s[w][e]).flatten(1) for w in ("wg", "wu", "wd"))
        x = s["x"][t].double()
        h = torch.nn.functional.silu(x @ wg.T) * (x @ wu.T)
        y.index_add_(0, t, (h @ wd.T) * weights[t, j][:, None])
    return {"y": y, "experts": chosen.int(), "weights": weights}
