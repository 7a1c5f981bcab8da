"""Measured cases of the serving operators: the product in 8-bit floating point with a scale for
each block of 128 (and the quantizer that feeds it), and the quantized key/value cache.

``run`` computes each operator in its plain form (elementary torch operations in 32 bits) or, with
``own`` set, by the library's entry points. ``exact`` gives the same outputs from the definitions
in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
E4M3_MAX = 448.0
TINY = 2.0 ** -126


# ------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------

def listed():
    return [
        # one token's activations in front of a projection of the 2048 x 6144 layer: latency
        dict(name="quantize_token", op="quantize", rows=1, cols=6144, block_rows=1, dtype="bf16"),
        # the activations of a long prompt
        dict(name="quantize_prompt", op="quantize", rows=16384, cols=6144, block_rows=1, dtype="bf16"),
        # a weight in 128 x 128 blocks, its last blocks ragged both ways
        dict(name="quantize_weight", op="quantize", rows=2047, cols=6100, block_rows=128, dtype="fp32"),
        # one token through the 2048 x 6144 layer: reading the weight is all there is to it
        dict(name="matmul_token", op="matmul", m=1, n=2048, k=6144, out="bf16"),
        # a decode batch
        dict(name="matmul_batch", op="matmul", m=64, n=6144, k=2048, out="bf16"),
        # sizes that divide nothing
        dict(name="matmul_ragged", op="matmul", m=777, n=1500, k=2900, out="fp32"),
        # a long prompt through the 2048 x 6144 layer
        dict(name="matmul_prompt", op="matmul", m=16384, n=2048, k=6144, out="bf16"),
        # one new token of each of 64 sequences, K and V views of a fused projection
        dict(name="append_tokens", op="append", tokens=64, heads=8, head_dim=128, format="int8",
             group=0, dtype="bf16", fused=True, skipped=0.0, slots=16384),
        # a padded batch of prompts, heads of 96
        dict(name="append_padded", op="append", tokens=1000, heads=3, head_dim=96, format="e4m3",
             group=0, dtype="fp16", fused=False, skipped=0.3, slots=4096),
        # a prompt's chunk at 4 bits, two groups a head
        dict(name="append_prompt", op="append", tokens=8192, heads=8, head_dim=128, format="int4",
             group=64, dtype="bf16", fused=True, skipped=0.0, slots=32768),
        # a short prefix read back
        dict(name="read_short", op="read", tokens=500, heads=8, head_dim=128, format="int4",
             group=64, dtype="bf16", skipped=0.0, slots=16384),
        # a long prefix read back
        dict(name="read_long", op="read", tokens=131072, heads=8, head_dim=128, format="int8",
             group=0, dtype="bf16", skipped=0.0, slots=139264),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


MAX_QUANT = 16384 * 6144
MAX_MNK = 16384 * 2048 * 6144
MAX_READ = 131072 * 8 * 128


def draw(rng):
    op = rng.choice(["quantize", "matmul", "matmul", "append", "read"])
    if op == "quantize":
        cols = _log(rng, 1, 8192)
        rows = _log(rng, 1, 16384)
        rows = min(rows, MAX_QUANT // cols)
        dtype = rng.choice(["bf16", "fp16", "fp32"])
        if dtype == "fp32":
            rows = max(1, rows // 2)
        return dict(op=op, rows=rows, cols=cols, block_rows=rng.choice([1, 1, 128]), dtype=dtype)
    if op == "matmul":
        n, k = _log(rng, 32, 8192), _log(rng, 32, 8192)
        m = max(1, min(_log(rng, 1, 16384), MAX_MNK // (n * k)))
        out = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        if out == "fp32":
            m = max(1, min(m, 16384 * 2048 // (2 * n)))
        return dict(op=op, m=m, n=n, k=k, out=out)
    heads = rng.choice([1, 2, 3, 4, 8, 16])
    dim = rng.choice([32, 64, 80, 96, 112, 128, 192, 256])
    group = rng.choice([0] + [g for g in (16, 32, 64, 128) if g < dim and dim % g == 0])
    fmt = rng.choice(["int4", "int8", "e4m3"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    skipped = rng.choice([0.0, 0.0, 0.25])
    if op == "append":
        tokens = min(_log(rng, 1, 8192), 8192 * 1024 // (heads * dim))
        if dtype == "fp32":
            tokens = max(1, tokens // 2)
        return dict(op=op, tokens=tokens, heads=heads, head_dim=dim, format=fmt, group=group,
                    dtype=dtype, fused=rng.random() < 0.5, skipped=skipped,
                    slots=tokens + _log(rng, 1, 16384))
    tokens = min(_log(rng, 1, 131072), MAX_READ // (heads * dim))
    if dtype == "fp32":
        tokens = max(1, tokens // 2)
    return dict(op=op, tokens=tokens, heads=heads, head_dim=dim, format=fmt, group=group,
                dtype=dtype, skipped=skipped, slots=tokens + _log(rng, 1, 8192))


# ------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _activations(rows, cols, g):
    """Gaussian rows with a few channels much larger than the rest, as the inputs of a
    projection have them."""
    ch = torch.exp(0.5 * torch.randn(cols, generator=g, device=DEV))
    ch = torch.where(torch.rand(cols, generator=g, device=DEV) < 0.01, 20.0 * ch, ch)
    return torch.randn(rows, cols, generator=g, device=DEV) * ch


def _weights(rows, cols, g):
    w = 0.02 * torch.randn(rows, cols, generator=g, device=DEV)
    return torch.where(torch.rand(rows, cols, generator=g, device=DEV) < 0.001, 10.0 * w, w)


def _pitched(codes):
    """The codes in rows that start on 16-byte boundaries, as the quantizer lays them out."""
    rows, cols = codes.shape
    buf = torch.zeros(rows, -(-cols // 16) * 16, dtype=torch.uint8, device=DEV)
    buf[:, :cols] = codes.view(torch.uint8)
    return buf.view(torch.float8_e4m3fn)[:, :cols]


def _groups(case):
    return 1 if not case["group"] else case["head_dim"] // case["group"]


def _row_bytes(case):
    return case["head_dim"] // 2 if case["format"] == "int4" else case["head_dim"]


def _slots(case, g):
    """Distinct slots out of shuffled pages of 16, some of them skipped (a padded batch)."""
    n, t = case["slots"], case["tokens"]
    pages = torch.randperm(n // 16 + 1, generator=g, device=DEV)
    s = (pages[:, None] * 16 + torch.arange(16, device=DEV)[None, :]).reshape(-1)
    s = s[s < n][:t]
    skip = torch.rand(t, generator=g, device=DEV) < case["skipped"]
    return torch.where(skip, torch.full_like(s, -1), s).to(torch.int64).contiguous()


def _cache(case, g, filled):
    """Codes, scales and zero-points for K and V. One slot more than the cache has is kept behind
    its end: the plain form sends the tokens that are skipped there."""
    n, h, gr = case["slots"] + 1, case["heads"], _groups(case)
    c = {}
    for p in ("k", "v"):
        codes = torch.zeros(n, h, _row_bytes(case), dtype=torch.uint8, device=DEV)
        scales = torch.ones(n, h, gr, device=DEV)
        zeros = torch.zeros(n, h, gr, dtype=torch.uint8, device=DEV)
        if filled:
            if case["format"] == "e4m3":
                x = 100.0 * torch.randn(codes.shape, generator=g, device=DEV, dtype=torch.float16)
                codes = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                scales = (torch.rand(n, h, gr, generator=g, device=DEV) + 0.5) / 448.0
            else:
                maxq = 15 if case["format"] == "int4" else 255
                codes = torch.randint(0, 256, codes.shape, generator=g, device=DEV,
                                      dtype=torch.uint8)
                scales = (torch.rand(n, h, gr, generator=g, device=DEV) + 0.5) * (6.0 / maxq)
                zeros = torch.randint(maxq // 4, maxq - maxq // 4, zeros.shape, generator=g,
                                      device=DEV, dtype=torch.uint8)
        c["codes_" + p], c["scales_" + p], c["zeros_" + p] = codes, scales, zeros
    c["claims"] = torch.zeros(n, dtype=torch.int32, device=DEV)
    return c


def prepare(case, seed):
    g = _gen(seed)
    st = {"case": case}
    if case["op"] == "quantize":
        make = _activations if case["block_rows"] == 1 else _weights
        st["x"] = make(case["rows"], case["cols"], g).to(DTYPES[case["dtype"]])
    elif case["op"] == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        a, sa = _plain_quantize(_activations(m, k, g), 1)
        b, sb = _plain_quantize(_weights(n, k, g), 128)
        st.update(a=_pitched(a), sa=sa, b=_pitched(b), sb=sb)
    else:
        t, h, d = case["tokens"], case["heads"], case["head_dim"]
        dt = DTYPES[case["dtype"]]
        st["slots"] = _slots(case, g)
        st["cache"] = _cache(case, g, case["op"] == "read")
        st["out_k"] = torch.zeros(t, h, d, dtype=dt, device=DEV)
        st["out_v"] = torch.zeros(t, h, d, dtype=dt, device=DEV)
        if case["op"] == "append":
            if case["fused"]:
                # one projection's output: 2 query heads a key head, then K, then V
                qkv = _activations(t, 4 * h * d, g).to(dt).view(t, 4 * h, d)
                st["k"], st["v"] = qkv[:, 2 * h:3 * h], qkv[:, 3 * h:]
            else:
                st["k"] = _activations(t, h * d, g).to(dt).view(t, h, d)
                st["v"] = _activations(t, h * d, g).to(dt).view(t, h, d)
    return st


# ------------------------------------------------------------------------------------------
# plain forms
# ------------------------------------------------------------------------------------------

def _scale_of(amax):
    # a tensor as the divisor: a division by a number is done as a product with its reciprocal
    return torch.clamp_min(amax / torch.full_like(amax, E4M3_MAX), TINY)


def _to_e4m3(x, scale):
    """The codes of x under a scale: the nearest values of the format to x times the scale's 32-bit
    reciprocal. That product is exact in 64 bits, and there is one rounding: a second one would
    decide wrongly next to a border between two codes."""
    v = x.double() * torch.reciprocal(scale).double()
    step = torch.ldexp(torch.ones_like(v), ((v.float().view(torch.int32) >> 23) & 255).clamp_min(121) - 130)
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _plain_quantize(x, block_rows):
    rows, cols = x.shape
    br, bc = -(-rows // block_rows), -(-cols // 128)
    x = x.float()
    pad = torch.zeros(br * block_rows, bc * 128, device=x.device)
    pad[:rows, :cols] = x
    t = pad.view(br, block_rows, bc, 128)
    scale = _scale_of(t.abs().amax(dim=(1, 3)))
    q = _to_e4m3(t, scale[:, None, :, None])
    return q.view(br * block_rows, bc * 128)[:rows, :cols], scale


def _dequantize(codes, scales, block_rows):
    rows, cols = codes.shape
    s = scales.repeat_interleave(block_rows, 0)[:rows].repeat_interleave(128, 1)[:, :cols]
    return codes.float() * s


def _plain_matmul(a, sa, b, sb, dtype):
    return torch.matmul(_dequantize(a, sa, 1), _dequantize(b, sb, 128).t()).to(dtype)


def _plain_write(x, slots, case, codes, scales, zeros):
    t, h, d = x.shape
    gr = _groups(case)
    x = x.float().reshape(t, h, gr, d // gr)
    if case["format"] == "e4m3":
        s = _scale_of(x.abs().amax(-1))
        row = _to_e4m3(x, s[..., None]).view(torch.uint8).reshape(t, h, d)
        z = torch.zeros_like(s)
    else:
        maxq = 15.0 if case["format"] == "int4" else 255.0
        mn, mx = x.amin(-1).clamp_max(0.0), x.amax(-1).clamp_min(0.0)
        flat = mn == mx
        mn, mx = torch.where(flat, -1.0, mn), torch.where(flat, 1.0, mx)
        s = torch.clamp_min((mx - mn) / torch.full_like(mx, maxq), TINY)
        # next to a border between two whole numbers 32 bits would decide by their own rounding
        z = torch.round(-mn.double() * maxq / (mx.double() - mn.double()))
        v = x.double() * torch.reciprocal(s).double()[..., None] + z.double()[..., None]
        c = torch.round(v).clamp(0.0, maxq).to(torch.uint8).reshape(t, h, d)
        row = c[..., 0::2] | (c[..., 1::2] << 4) if case["format"] == "int4" else c
    at = torch.where(slots < 0, codes.shape[0] - 1, slots)
    codes[at], scales[at], zeros[at] = row, s, z.to(torch.uint8)


def _plain_read(slots, case, codes, scales, zeros, out):
    t, h, d = out.shape
    gr = _groups(case)
    at = torch.where(slots < 0, codes.shape[0] - 1, slots)
    row, s = codes[at], scales[at]
    if case["format"] == "e4m3":
        v = row.view(torch.float8_e4m3fn).float().view(t, h, gr, d // gr) * s[..., None]
    else:
        if case["format"] == "int4":
            row = torch.stack((row & 15, row >> 4), -1)
        v = row.reshape(t, h, gr, d // gr).float() - zeros[at].float()[..., None]
        v = v * s[..., None]
    out.copy_(torch.where((slots < 0)[:, None, None], out, v.reshape(t, h, d).to(out.dtype)))


# ------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------

def _formats():
    import post_weight_quantization_06_b200 as g
    return {"int4": g.GPTQ_CACHE_INT4, "int8": g.GPTQ_CACHE_INT8, "e4m3": g.GPTQ_CACHE_E4M3}


def _own_planes(c, n):
    return [c[f][:n] for f in ("codes_k", "scales_k", "zeros_k", "codes_v", "scales_v", "zeros_v")]


def run(st):
    case = st["case"]
    op = case["op"]
    if own:
        import post_weight_quantization_06_b200 as g
    if op == "quantize":
        if own:
            codes, scales = g.fp8_quantize(st["x"], block_rows=case["block_rows"])
        else:
            codes, scales = _plain_quantize(st["x"], case["block_rows"])
        return {"codes": codes, "scales": scales}
    if op == "matmul":
        dt = DTYPES[case["out"]]
        if own:
            return g.fp8_matmul(st["a"], st["sa"], st["b"], st["sb"], out_dtype=dt)
        return _plain_matmul(st["a"], st["sa"], st["b"], st["sb"], dt)
    c, slots, n = st["cache"], st["slots"], case["slots"]
    if own:
        if "planes" not in st:  # the views a program with such a cache holds
            st["planes"], st["format"] = _own_planes(c, n), _formats()[case["format"]]
            st["claims"] = c["claims"][:n]
        if op == "append":
            g.gptq_cache_write(st["k"], st["v"], slots, st["format"], case["group"],
                               *st["planes"], st["claims"])
        g.gptq_cache_read(slots, st["format"], case["group"], *st["planes"], st["out_k"],
                          st["out_v"])
    else:
        for p in ("k", "v"):
            planes = c["codes_" + p], c["scales_" + p], c["zeros_" + p]
            if op == "append":
                _plain_write(st[p], slots, case, *planes)
            _plain_read(slots, case, *planes, st["out_" + p])
    out = {"k": st["out_k"], "v": st["out_v"]}
    if op == "append":
        out.update(scales_k=c["scales_k"][:n], scales_v=c["scales_v"][:n])
    return out


def work(case):
    if case["op"] == "quantize":
        e = case["rows"] * case["cols"]
        blocks = -(-case["rows"] // case["block_rows"]) * -(-case["cols"] // 128)
        return {"bytes": e * (BYTES[case["dtype"]] + 1) + 4 * blocks, "flops": 3 * e}
    if case["op"] == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        kb = -(-k // 128)
        return {"bytes": (m + n) * k + 4 * kb * (m + -(-n // 128)) + m * n * BYTES[case["out"]],
                "flops": 2 * m * n * k}
    rows = 2 * case["tokens"] * case["heads"]
    live = rows * (1.0 - case["skipped"])
    meta = _groups(case) * (4 if case["format"] == "e4m3" else 5)
    stored = live * (_row_bytes(case) + meta)
    values = live * case["head_dim"]
    wide = values * BYTES[case["dtype"]]
    slots = 8 * case["tokens"]
    if case["op"] == "read":
        return {"bytes": stored + wide + slots, "flops": 2 * values}
    # written from the wide values, and read back
    return {"bytes": 2 * (stored + wide + slots), "flops": 6 * values}


# ------------------------------------------------------------------------------------------
# 64 bits
# ------------------------------------------------------------------------------------------

def _nearest_e4m3(v):
    """The nearest value of the format (3 stored mantissa bits, exponents -6 to 8), ties to even."""
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), torch.clamp_min(e - 1, -6) - 3)
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def _exact_blocks(x, rows_of, cols_of):
    """max |x| of each rows_of x cols_of block, by index."""
    r, c = x.shape
    i = torch.arange(r, device=x.device) // rows_of
    j = torch.arange(c, device=x.device) // cols_of
    top = torch.zeros(int(i[-1]) + 1, c, dtype=torch.float64, device=x.device)
    top = top.index_reduce(0, i, x.abs(), "amax")
    out = torch.zeros(top.shape[0], int(j[-1]) + 1, dtype=torch.float64, device=x.device)
    return out.index_reduce(1, j, top, "amax"), i, j


def _held(scale):
    """What multiplies the values to be coded: by the definition a scale is held in 32 bits, and
    its reciprocal too. Values on a border between two codes go by these."""
    return (1.0 / scale.float().double()).float().double()


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "quantize":
        x = st["x"].double()
        top, i, j = _exact_blocks(x, case["block_rows"], 128)
        scale = (top / 448.0).clamp_min(TINY)
        return {"codes": _nearest_e4m3(x * _held(scale)[i][:, j]), "scales": scale}
    if case["op"] == "matmul":
        a, b = st["a"].double(), st["b"].double()
        y = torch.zeros(case["m"], case["n"], dtype=torch.float64, device=DEV)
        cols = torch.arange(case["n"], device=DEV) // 128
        for kb in range(st["sa"].shape[1]):
            part = a[:, 128 * kb:128 * kb + 128] @ b[:, 128 * kb:128 * kb + 128].t()
            y += part * st["sa"][:, kb].double()[:, None] * st["sb"][cols, kb].double()[None, :]
        return y
    t, h, d = case["tokens"], case["heads"], case["head_dim"]
    gr, n, slots = _groups(case), case["slots"], st["slots"]
    bits = {"int4": 4, "int8": 8, "e4m3": None}[case["format"]]
    live = slots >= 0
    out = {}
    for p in ("k", "v"):
        full = torch.zeros(t, h, d, dtype=torch.float64, device=DEV)
        if case["op"] == "append":
            x = st[p].double()[live].reshape(-1, h, gr, d // gr)
            if bits is None:
                s = (x.abs().amax(-1, keepdim=True) / 448.0).clamp_min(TINY)
                y = _nearest_e4m3(x * _held(s)) * s
            else:
                top = 2 ** bits - 1
                lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
                lo, hi = torch.minimum(lo, 0 * lo), torch.maximum(hi, 0 * hi)
                zero = (lo == 0) & (hi == 0)
                lo, hi = lo - zero.double(), hi + zero.double()
                s = ((hi - lo) / top).clamp_min(TINY)
                z = torch.round(-lo * top / (hi - lo))
                y = (torch.round(x * _held(s) + z).clamp(0, top) - z) * s
            scales = st["cache"]["scales_" + p][:n].double()
            scales[slots[live]] = s[..., 0]
            out["scales_" + p] = scales
        else:
            raw = st["cache"]["codes_" + p][slots[live]]
            s = st["cache"]["scales_" + p][slots[live]].double()[..., None]
            if bits is None:
                q = raw.view(torch.float8_e4m3fn).double()
            else:
                q = raw.double()
                if bits == 4:
                    high = torch.floor(q / 16)
                    q = torch.stack((q - 16 * high, high), -1)
            q = q.reshape(-1, h, gr, d // gr)
            if bits is not None:
                q = q - st["cache"]["zeros_" + p][slots[live]].double()[..., None]
            y = q * s
        full[live] = y.reshape(-1, h, d)
        out[p] = full
    return out
