"""Cases for measuring the operators around products in microscaled 4-bit floating point (MXFP4) and
the norm that feeds them and the 8-bit product.

A case's "op" is one of

  norm      root-mean-square norm of tokens, with the residual's addition (or without): h = x + r in
            the tokens' type, v = h w / sqrt(mean h^2 + eps).  "out" says what the values are left in:
            "same" (the tokens' type), "int8" (rows of 8-bit integers with a step each) or "mxfp4";
            what is held in 8 or 4 bits is read back as the values it stands for;
  quantise  rows to MXFP4 (weights times their smoothing scales, tokens divided by them, or as they
            are) and back to the values that the codes stand for;
  product   y = x w^T (+ bias) from MXFP4 codes that are there already;
  linear    the same from floating tokens: each is divided by the smoothing scales (if any),
            quantised to MXFP4, then multiplied.

MXFP4 rows: blocks of 32 columns share a scale 2^(b - 127) with one byte b (255: NaN); an element is a
sign bit and one of 0, 0.5, 1, 1.5, 2, 3, 4, 6 by the three bits below it.  Codes are uint8 [rows]
[16 a block], column 2 j in the low half of byte j; scales are uint8 [blocks / 4, rounded up][rows,
rounded up to 4][4]: byte c of (q, r) is that of block 4 q + c of row r.  Columns past the last
are zeros.  b = max(0, 127 + floor(log2 max |v|) - 2) of the block's values v, an element is the value
nearest to |v| / scale, the one with an even code on ties, 6 above it.
"""
import math

import torch

own = False

FP = {"fp16": torch.float16, "bf16": torch.bfloat16}


# ---------------------------------------------------------------------------------- cases
def listed():
    return [
        # between two layers of a decode step, one user: latency
        {"name": "norm-1", "op": "norm", "tokens": 1, "in": 4096, "out": "same", "residual": True,
         "weight": "same", "dtype": "fp16"},
        # before an 8-bit projection, sequences decoding together, an odd number of them
        {"name": "norm-int8-33", "op": "norm", "tokens": 33, "in": 5120, "out": "int8", "residual": True,
         "weight": "fp32", "dtype": "bf16"},
        # a prompt's first norm (no residual yet), before an MXFP4 projection, a ragged width
        {"name": "norm-mxfp4-2047", "op": "norm", "tokens": 2047, "in": 5000, "out": "mxfp4",
         "residual": False, "weight": "same", "dtype": "fp16"},
        # a batch of prompts, wide layers, the search's scales folded into an fp32 weight
        {"name": "norm-mxfp4-16384", "op": "norm", "tokens": 16384, "in": 8192, "out": "mxfp4",
         "residual": True, "weight": "fp32", "dtype": "bf16"},
        # tokens of a decode batch into an MLP down-projection
        {"name": "quantise-333", "op": "quantise", "rows": 333, "in": 13824, "fold": "divide",
         "dtype": "bf16"},
        # the largest layer's weights under their smoothing scales
        {"name": "quantise-28672", "op": "quantise", "rows": 28672, "in": 8192, "fold": "multiply",
         "dtype": "fp16"},
        # sixteen sequences decoding together, codes made by the norm before
        {"name": "product-16", "op": "product", "tokens": 16, "out": 11008, "in": 4096, "dtype": "bf16",
         "bias": False},
        # an odd number of tokens in flight, a wide input
        {"name": "product-333", "op": "product", "tokens": 333, "out": 5120, "in": 13824,
         "dtype": "bf16", "bias": False},
        # the largest layer: a batch of prompts through a 28672 x 8192 projection
        {"name": "product-8192", "op": "product", "tokens": 8192, "out": 28672, "in": 8192,
         "dtype": "bf16", "bias": True},
        # one token through a square projection, smoothing scales not folded: decode latency
        {"name": "linear-1", "op": "linear", "tokens": 1, "out": 4096, "in": 4096, "dtype": "fp16",
         "smooth": True, "bias": False},
        # a few dozen sequences through an MLP up-projection
        {"name": "linear-50", "op": "linear", "tokens": 50, "out": 11008, "in": 4096, "dtype": "bf16",
         "smooth": False, "bias": True},
        # a prompt through the same, quantisation included
        {"name": "linear-4096", "op": "linear", "tokens": 4096, "out": 11008, "in": 4096,
         "dtype": "fp16", "smooth": True, "bias": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "quantise", "product", "product", "linear"])
    dtype = rng.choice(["fp16", "bf16"])
    if op == "norm":
        while True:
            t, k = _log(rng, 1, 16384), _log(rng, 64, 16384)
            if t * k <= 16384 * 8192 // 2:
                break
        return {"op": op, "tokens": t, "in": k, "out": rng.choice(["same", "int8", "mxfp4"]),
                "residual": rng.random() < 0.7, "weight": rng.choice(["same", "fp32"]), "dtype": dtype}
    if op == "quantise":
        while True:
            r, k = _log(rng, 1, 28672), _log(rng, 64, 16384)
            if r * k <= 28672 * 8192 // 2:
                break
        return {"op": op, "rows": r, "in": k, "fold": rng.choice(["none", "divide", "multiply"]),
                "dtype": dtype}
    while True:
        t, m, k = _log(rng, 1, 8192), _log(rng, 256, 28672), _log(rng, 256, 16384)
        if t * m * k <= 8192 * 28672 * 8192 // 2:
            break
    c = {"op": op, "tokens": t, "out": m, "in": k, "dtype": dtype, "bias": rng.random() < 0.5}
    if op == "linear":
        c["smooth"] = rng.random() < 0.5
    return c


# --------------------------------------------------------------------------------- inputs
EPS = 1e-6


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = FP[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    st = {"case": case}
    k = case["in"]
    if case["op"] == "norm":
        x = normal(case["tokens"], k)
        x[:, ::97] *= 20  # a few channels stand out
        st["x"] = x.to(dt)
        st["r"] = (4 * normal(case["tokens"], k)).to(dt) if case["residual"] else None
        w = 1 + 0.2 * normal(k)
        st["w"] = w.to(dt) if case["weight"] == "same" else w
        return st
    if case["op"] == "quantise":
        a = normal(case["rows"], k)
        if case["fold"] == "multiply":
            a.mul_(0.02)
        else:
            a[:, ::97] *= 20
        st["a"] = a.to(dt)
        st["s"] = None if case["fold"] == "none" else torch.exp(0.5 * normal(k))
        return st
    t, m = case["tokens"], case["out"]
    x = normal(t, k)
    x[:, ::97] *= 20
    st["s"] = None
    if case["op"] == "linear":
        st["x"] = x.to(dt)
        if case["smooth"]:
            st["s"] = (x.abs().mean(0) + 1e-3) ** 0.5
    else:
        st["xc"], st["xs"] = _quantise(x)
    w = 0.02 * normal(m, k)
    st["wc"], st["ws"] = _quantise(w)
    st["bias"] = normal(m).to(dt) if case["bias"] else None
    return st


# ------------------------------------------------------------------------ the plain forms
VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _pow2(byte):
    """fp32 2^(byte - 127) of bytes 0 .. 254, from its bits."""
    return torch.where(byte == 0, 1 << 22, byte.int() << 23).int().view(torch.float32)


def _blocks(v):
    """fp32 rows as blocks of 32, zeros past the last column: [rows][blocks][32]."""
    return torch.nn.functional.pad(v, (0, -v.shape[1] % 32)).unflatten(1, (-1, 32))


def _elements(v):
    """What the elements of fp32 rows stand for, without the scale, and the scale's byte."""
    b = _blocks(v)
    top = b.abs().amax(-1)
    byte = (torch.frexp(top)[1].to(torch.int32) + (127 - 3)).clamp(min=0)  # 2^(e - 1) <= top < 2^e
    byte = torch.where(top == 0, 0, byte)
    a = b.abs() * _pow2(254 - byte)[..., None]  # over the scale: a power of two, exact
    q = torch.where(a < 2, torch.round(a * 2) / 2,
                    torch.where(a < 4, torch.round(a), (torch.round(a / 2) * 2).clamp(max=6)))
    return q.copysign(b), byte


def _quantise(v):
    """Codes and scales, as described above, of fp32 rows."""
    q, byte = _elements(v)
    a = q.abs()
    code = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code = (code + 8 * torch.signbit(q).to(torch.uint8)).flatten(1)
    codes = code[:, 0::2] | (code[:, 1::2] << 4)
    rows, nb = byte.shape
    byte = torch.nn.functional.pad(byte, (0, -nb % 4, 0, -rows % 4)).to(torch.uint8)
    return codes.contiguous(), byte.unflatten(1, (-1, 4)).transpose(0, 1).contiguous()


def _values(codes, scales):
    """fp32 rows of codes and scales."""
    table = torch.tensor(VALUES + tuple(-x for x in VALUES), device=codes.device)
    v = torch.stack((table[(codes & 15).int()], table[(codes >> 4).int()]), -1)
    v = v.flatten(1).unflatten(1, (-1, 32))
    byte = scales.transpose(0, 1).flatten(1)[:v.shape[0], :v.shape[1]]
    return (v * _pow2(byte)[..., None]).flatten(1)


def _as_held(v):
    """fp32 rows as their MXFP4 elements stand for."""
    q, byte = _elements(v)
    return (q * _pow2(byte)[..., None]).flatten(1)[:, :v.shape[1]]


def run(st):
    c = st["case"]
    if own:
        return _run_own(st, c)
    dt = FP[c["dtype"]]
    if c["op"] == "norm":
        h = st["x"] if st["r"] is None else (st["x"].float() + st["r"].float()).to(dt)
        if c["out"] == "same":
            f = h.float()
            y = (f * torch.rsqrt(f.square().mean(1, keepdim=True) + EPS) * st["w"].float()).to(dt)
            return {"h": h, "y": y}
        # in 64 bits and rounded to 32: values next to a border between two codes
        f = h.double()
        v = (f * st["w"].double() / (f.square().mean(1, keepdim=True) + EPS).sqrt()).float()
        if c["out"] == "mxfp4":
            return {"h": h, "y": _as_held(v).to(dt)}
        # (divisors are tensors: torch turns a division by a Python number into a product)
        step = v.abs().amax(1, keepdim=True)
        step = step / torch.full_like(step, 127)
        step = torch.where(step == 0, 1.0, step)
        return {"h": h, "y": (torch.round(v / step) * step).to(dt)}
    if c["op"] == "quantise":
        v = st["a"].float()
        if st["s"] is not None:
            v = v * st["s"] if c["fold"] == "multiply" else v / st["s"]
        return _as_held(v).to(dt)
    if c["op"] == "linear":
        x = _as_held(st["x"].float() if st["s"] is None else st["x"].float() / st["s"])
    else:
        x = _values(st["xc"], st["xs"])
    y = x @ _values(st["wc"], st["ws"])[:, :x.shape[1]].t()
    if st["bias"] is not None:
        y = y + st["bias"].float()
    return y.to(dt)


def _run_own(st, c):
    import weight_only_quantization_act_amd as awq

    dt = FP[c["dtype"]]
    if c["op"] == "norm":
        x, w, r, k = st["x"], st["w"], st["r"], c["in"]
        if c["out"] == "same":
            y, h = awq.awq_rmsnorm(x, w, EPS, residual=r)
        elif c["out"] == "int8":
            codes, steps, h = awq.awq_rmsnorm_int8(x, w, EPS, residual=r)
            y = awq.awq_int8_dequantize(codes, steps, k, dtype=dt)
        else:
            codes, scales, h = awq.awq_rmsnorm_mxfp4(x, w, EPS, residual=r)
            y = awq.awq_mxfp4_dequantize(codes, scales, k, dtype=dt)
        return {"h": h, "y": y}
    if c["op"] == "quantise":
        codes, scales = awq.awq_mxfp4_quantize(
            st["a"], st["s"], fold="multiply" if c["fold"] == "multiply" else "divide")
        return awq.awq_mxfp4_dequantize(codes, scales, c["in"], dtype=dt)
    if c["op"] == "product":
        return awq.awq_mxfp4_matmul(st["xc"], st["xs"], st["wc"], st["ws"], dtype=dt, bias=st["bias"])
    return awq.awq_mxfp4_linear(st["x"], st["wc"], st["ws"], s=st["s"], bias=st["bias"])


# ------------------------------------------------------------------------ work and 64 bits
def work(case):
    k = case["in"]
    nb = (k + 31) // 32
    if case["op"] == "norm":
        t = case["tokens"]
        held = {"same": 0, "int8": t * (k + 4), "mxfp4": t * nb * 17}[case["out"]]
        w = k * (2 if case["weight"] == "same" else 4)
        # tokens (and residual in, sum out), what is held written and read, values out
        return {"bytes": t * k * (6 if case["residual"] else 2) + w + 2 * held + 2 * t * k, "flops": 0}
    if case["op"] == "quantise":
        r = case["rows"]
        return {"bytes": 4 * r * k + 2 * r * nb * 17 + (0 if case["fold"] == "none" else 4 * k), "flops": 0}
    t, m = case["tokens"], case["out"]
    x = t * k * 2 if case["op"] == "linear" else t * nb * 17
    extra = (4 * k if case.get("smooth") else 0) + (2 * m if case["bias"] else 0)
    return {"bytes": x + m * nb * 17 + 2 * t * m + extra, "flops": 2 * t * m * k}


def _round32(v):
    """A 64-bit value as the fp32 operation that gives it rounds it."""
    return v.float().double()


def _power64(x):
    """fp64 2^x of whole numbers x, from its bits."""
    return ((x.long() + 1023) << 52).view(torch.float64)


def _held64(v):
    """What the rows' MXFP4 elements stand for, each value looked up between the borders."""
    f = torch.float64
    rows, k = v.shape
    nb = (k + 31) // 32
    out = torch.zeros((rows, nb * 32), dtype=f, device=v.device)
    out[:, :k] = v
    b = out.view(rows, nb, 32)
    top = b.abs().max(-1, keepdim=True).values
    x = torch.floor(torch.log2(torch.where(top == 0, 1.0, top)))
    x = x + (_power64(x + 1) <= top).to(f) - (_power64(x) > top).to(f)  # the logarithm is rounded
    unit = _power64((x - 2).clamp(min=-127))
    a = (b.abs() / unit).contiguous()
    borders = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=f, device=v.device)
    at = torch.searchsorted(borders, a)  # borders below a: a tie stays below it
    tie = (a == torch.nn.functional.pad(borders, (0, 1))[at]) & (at < 7)
    at = at + (tie & (at % 2 == 1)).long()  # ... unless the upper one is even
    vals = torch.tensor(VALUES, dtype=f, device=v.device)[at]
    return (torch.where(b < 0, -vals, vals) * unit).view(rows, -1)[:, :k]


def _read64(codes, scales, rows, k):
    """fp64 rows of stored codes, each element computed from its bits."""
    col = torch.arange(k, device=codes.device)
    code = (codes[:rows, col // 2].int() >> (4 * (col % 2)).int()) & 15
    e, m = (code >> 1) & 3, (code & 1).double()
    mag = torch.where(e == 0, m * 0.5, (1 + 0.5 * m) * _power64(e - 1))
    byte = scales[col // 128, :rows, (col // 32) % 4].t()
    return torch.where(code >= 8, -mag, mag) * _power64(byte.long() - 127)


def exact(case, seed):
    st = prepare(case, seed)
    f = torch.float64
    k = case["in"]
    if case["op"] == "norm":
        h = st["x"].to(f)
        if st["r"] is not None:
            h = (h + st["r"].to(f)).to(FP[case["dtype"]]).to(f)  # the sum is kept in the tokens' type
        v = h / torch.sqrt((h * h).sum(1, keepdim=True) / k + EPS) * st["w"].to(f)
        if case["out"] == "same":
            return {"h": h, "y": v}
        # codes are defined on values of 32 bits
        v = _round32(v)
        if case["out"] == "mxfp4":
            return {"h": h, "y": _held64(v)}
        step = _round32(v.abs().amax(1, keepdim=True) / 127)
        step = step + (step == 0)
        return {"h": h, "y": torch.round(_round32(v / step)) * step}
    if case["op"] in ("quantise", "linear"):
        x = st["a" if case["op"] == "quantise" else "x"].to(f)
        if st["s"] is not None:
            s = st["s"].to(f)
            x = _round32(x * s if case.get("fold") == "multiply" else x / s)
        x = _held64(x)
        if case["op"] == "quantise":
            return x
    else:
        x = _read64(st["xc"], st["xs"], case["tokens"], k)
    m = case["out"]
    y = torch.empty((x.shape[0], m), dtype=f, device="cuda")
    for a in range(0, m, 4096):
        n = min(4096, m - a)
        y[:, a:a + n] = x @ _read64(st["wc"][a:a + n], st["ws"][:, a:a + n], n, k).t()
    return y if st["bias"] is None else y + st["bias"].to(f)
