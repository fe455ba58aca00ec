"""The microscaled 4-bit operators: what is measured of them, and their plain forms.

A microscaled tensor holds E2M1 values (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their
negatives) under a scale for each block of a row:

  e8m0  blocks of 32, the scale a power of two;
  e4m3  blocks of 16, an E4M3 scale, and a power of two for the whole row.

Operators: quantisation (of activations, of a SwiGLU's two halves), the way
back to bf16, the product of quantised activations with quantised weights, and
that product grouped by expert over ragged rows.
"""
import math

import torch

own = False

E8M0, E4M3 = "e8m0", "e4m3"
BLOCK = {E8M0: 32, E4M3: 16}


# ---------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one decoded token's hidden state to 4 bits and back: the call's latency
        dict(name="roundtrip-1x4096", op="roundtrip", fmt=E4M3, m=1, k=4096),
        # what 4-bit activations cost a layer, judged over a long batch of calibration rows
        dict(name="roundtrip-8192x14336", op="roundtrip", fmt=E8M0, m=8192, k=14336),
        # the MLP's inner activations from the gate and up halves, an odd number of rows
        dict(name="swiglu-4099x8192", op="swiglu", fmt=E4M3, m=4099, k=8192),
        # a layer's weights back to bf16, the largest projection
        dict(name="dequant-27648x5120", op="dequant", fmt=E4M3, m=27648, k=5120),
        # the same for a small layer with ragged sizes
        dict(name="dequant-1000x2080", op="dequant", fmt=E8M0, m=1000, k=2080),
        # one decoded token through an attention projection
        dict(name="linear-1-4096x4096", op="linear", fmt=E4M3, m=1, n=4096, k=4096, out="f32"),
        # a small decoding batch through a gate projection
        dict(name="linear-24-14336x4096", op="linear", fmt=E8M0, m=24, n=14336, k=4096, out="bf16"),
        # a short prompt, an odd length, through the longest sums
        dict(name="linear-333-5120x27648", op="linear", fmt=E4M3, m=333, n=5120, k=27648, out="bf16"),
        # a long prompt through a gate projection
        dict(name="linear-8192-14336x4096", op="linear", fmt=E4M3, m=8192, n=14336, k=4096, out="bf16"),
        # one quantised input into the q, k and v projections, side by side in one output
        dict(name="shared-qkv-2048", op="shared", fmt=E4M3, m=2048, n=4096, n2=1024, k=4096, out="bf16"),
        # a decoding batch over many small experts, most of them with a few rows
        dict(name="experts-64x2048x2048-t16", op="grouped", fmt=E4M3, m=16, top=8, experts=64,
             n=2048, k=2048, skew=0.5, out="f32"),
        # a prompt over few large experts, crowded and empty ones among them
        dict(name="experts-16x4096x4096-t4100", op="grouped", fmt=E8M0, m=4100, top=2, experts=16,
             n=4096, k=4096, skew=2.0, out="bf16"),
    ]


def _log(rng, lo, hi, step=1):
    return max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step)


def draw(rng):
    op = rng.choice(["roundtrip", "swiglu", "dequant", "linear", "linear", "shared", "grouped", "grouped"])
    fmt = rng.choice([E8M0, E4M3])
    out = rng.choice(["f32", "bf16"])
    if op in ("roundtrip", "swiglu", "dequant"):
        k = _log(rng, 1024, 14336, 32)
        return dict(op=op, fmt=fmt, m=_log(rng, 1, (1 << 26) // k), k=k)
    if op == "linear":
        n, k = _log(rng, 1000, 14336), _log(rng, 1024, 14336, 32)
        return dict(op=op, fmt=fmt, m=_log(rng, 1, 4096), n=n, k=k, out=out)
    if op == "shared":
        return dict(op=op, fmt=fmt, m=_log(rng, 1, 4096), n=_log(rng, 1024, 5120, 8), n2=_log(rng, 256, 1024, 8),
                    k=_log(rng, 1024, 5120, 32), out=out)
    experts = rng.choice([4, 8, 13, 16, 32, 64])
    return dict(op=op, fmt=fmt, m=_log(rng, 1, 2048), top=rng.choice([1, 2, 4]), experts=experts,
                n=_log(rng, 512, 2048), k=_log(rng, 512, 2048, 32), skew=round(rng.uniform(0.0, 2.0), 2), out=out)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _activations(rows, k, g):
    """N(0, 1) by a lognormal scale for each channel, five channels much larger."""
    c = torch.exp(torch.randn(k, generator=g, device="cuda"))
    c[torch.randperm(k, generator=g, device="cuda")[:5]] *= 32.0
    return (torch.randn(rows, k, generator=g, device="cuda") * c).to(torch.bfloat16)


def _weights(rows, k, g):
    """N(0, 0.02), one in a thousand ten times larger."""
    w = torch.randn(rows, k, generator=g, device="cuda") * 0.02
    w.view(-1)[torch.randint(rows * k, (rows * k // 1000 + 1,), generator=g, device="cuda")] *= 10.0
    return w.to(torch.bfloat16)


def _packed(rows, k, fmt, groups, g):
    """Quantised weights as a program keeps them: groups of rows / groups rows each."""
    w = _weights(rows, k, g).float()
    start = torch.arange(groups + 1, device="cuda") * (rows // groups)
    codes, scales, row_scale = [], [], []
    for r in range(0, rows, 8192):  # in parts: the elementwise forms hold several copies
        v, s, p = _quantized(w[r:r + 8192], fmt)
        code = torch.searchsorted(_magnitudes(w.device), v.abs()).to(torch.uint8) | (v < 0).to(torch.uint8) * 8
        codes.append(code[:, 0::2] | code[:, 1::2] << 4)
        scales.append(s)
        row_scale.append(p)
    s = torch.cat(scales)
    if fmt == E8M0:
        bytes_ = (torch.log2(s.double()).round() + 127).to(torch.uint8)
    else:
        bytes_ = s.to(torch.float8_e4m3fn).view(torch.uint8)
    return dict(codes=torch.cat(codes), scales=_tiled(bytes_, start), row_scale=torch.cat(row_scale) if fmt == E4M3 else None,
                start=start, groups=groups, fmt=fmt)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, fmt, m, k = case["op"], case["fmt"], case["m"], case["k"]
    st = dict(case)
    if op == "dequant":
        st["w"] = _packed(m, k, fmt, 1, g)
    elif op == "roundtrip":
        st["x"] = _activations(m, k, g)
    elif op == "swiglu":
        st["x"] = torch.cat([_activations(m, k, g), _activations(m, k, g)], 1)
    elif op in ("linear", "shared"):
        st["x"] = _activations(m, k, g)
        st["w"] = [_packed(n, k, fmt, 1, g) for n in ([case["n"]] if op == "linear" else [case["n"], case["n2"], case["n2"]])]
    else:
        e, top, n = case["experts"], case["top"], case["n"]
        st["x"] = _activations(m, k, g)
        st["w"] = _packed(e * n, k, fmt, e, g)
        # a router's choice: scores with a skew over the experts, the best `top` of each token
        bias = torch.randn(e, generator=g, device="cuda") * case["skew"]
        pick = (torch.randn(m, e, generator=g, device="cuda") + bias).topk(top, dim=1).indices.reshape(-1)
        order = torch.sort(pick, stable=True).indices
        st["rows"] = (order // top).to(torch.int32)
        counts = torch.bincount(pick, minlength=e)
        st["offsets"] = torch.cat([torch.zeros(1, device="cuda", dtype=torch.int64), counts.cumsum(0)]).to(torch.int32)
        st["most"] = int(counts.max())  # the plain form's padding
    st["dtype"] = torch.float32 if case.get("out") == "f32" else torch.bfloat16
    return st


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _magnitudes(device):
    return torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=device)


def _power_of_two(p):
    """2^p as fp32, -126 <= p <= 127."""
    return ((p + 127) << 23).view(torch.float32)


def _round_e2m1(q):
    """The nearest E2M1 value, ties to the even code, 6 at most."""
    a = q.abs().clamp(max=6.0)
    step = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0))
    return torch.copysign(torch.round(a / step) * step, q)


def _quantized(x, fmt):
    """fp32 rows -> (E2M1 values, block scales, row scales)."""
    r, k = x.shape
    b = x.view(r, k // BLOCK[fmt], BLOCK[fmt])
    if fmt == E8M0:
        # the block's exponent less E2M1's largest
        byte = ((b.abs().amax(-1).view(torch.int32) >> 23) - 2).clamp(0, 254)
        s = torch.where(byte > 0, (byte << 23).view(torch.float32), 2.0 ** -127)
        inverse = _power_of_two((127 - byte).clamp(min=-126))
        # 2^-127's fellow: byte 254 has the inverse 2^-127, in two factors
        v = _round_e2m1(torch.where(byte == 254, 0.5, 1.0)[..., None] * (b * inverse[..., None]))
        return v.view(r, k), s, None
    top = x.abs().amax(1)
    bits = top.view(torch.int32)
    # the smallest power of two under which the row's largest scale stays within E4M3's 448: 2688 = 6 * 448 = 1.3125 * 2^11
    p = ((bits >> 23) - 138 + ((bits & 0x7FFFFF) > 0x280000)).clamp(min=-126)
    p = torch.where(top > 0, p, 0)
    b = b * _power_of_two(-p)[:, None, None]
    s = (b.abs().amax(-1) / 6.0).to(torch.float8_e4m3fn).float()
    v = _round_e2m1(torch.where(s[..., None] > 0, b / s[..., None], 0.0))
    return v.view(r, k), s, _power_of_two(p)


def _values(v, s, p):
    r, k = v.shape
    x = (v.view(r, s.shape[1], -1) * s[..., None]).view(r, k)
    return x if p is None else x * p[:, None]


def _place(rows, start):
    """Where a row's scales lie: (tile of 128 rows, row of 32, column of 4).  Each group starts a tile of its own:
    group e, whose first row is o, at tile o // 128 + e."""
    r = torch.arange(rows, device=start.device)
    e = torch.searchsorted(start, r, right=True) - 1
    local = r - start[e]
    return start[e] // 128 + e + local // 128, local % 32, local % 128 // 32


def _tiled(bytes_, start):
    """[rows, blocks] scale bytes -> tiles of 128 rows by 4 blocks, 512 bytes each: row i's four bytes at
    (i % 32) * 16 + i // 32 * 4."""
    rows, nb = bytes_.shape
    words = (nb + 3) // 4
    padded = torch.zeros(rows, words * 4, dtype=torch.uint8, device=bytes_.device)
    padded[:, :nb] = bytes_
    t = torch.zeros(rows // 128 + len(start) - 1, words, 32, 4, 4, dtype=torch.uint8, device=bytes_.device)
    tile, lane, col = _place(rows, start)
    t[tile, :, lane, col] = padded.view(rows, words, 4)
    return t.view(-1)


def _unpacked(w):
    """A packed tensor's values, fp32."""
    rows, k = w["codes"].shape[0], w["codes"].shape[1] * 2
    code = torch.stack([w["codes"] & 15, w["codes"] >> 4], -1).view(rows, k).long()
    m = _magnitudes(code.device)
    nb = k // BLOCK[w["fmt"]]
    words = (nb + 3) // 4
    tile, lane, col = _place(rows, w["start"])
    bytes_ = w["scales"].view(-1, words, 32, 4, 4)[tile, :, lane, col].reshape(rows, words * 4)[:, :nb].contiguous()
    if w["fmt"] == E8M0:
        s = torch.where(bytes_ > 0, (bytes_.int() << 23).view(torch.float32), 2.0 ** -127)
    else:
        s = bytes_.view(torch.float8_e4m3fn).float()
    return _values(torch.cat([m, -m])[code], s, w["row_scale"])


def _silu_product(x):
    a, b = x.float().chunk(2, 1)
    return a / (1.0 + torch.exp(-a)) * b


def _plain(st):
    op, fmt = st["op"], st["fmt"]
    if op == "dequant":
        return _unpacked(st["w"]).to(torch.bfloat16)
    if op == "roundtrip":
        return _values(*_quantized(st["x"].float(), fmt)).to(torch.bfloat16)
    if op == "swiglu":
        return _values(*_quantized(_silu_product(st["x"]), fmt)).to(torch.bfloat16)
    if op in ("linear", "shared"):
        x = _values(*_quantized(st["x"].float(), fmt))
        return torch.cat([x @ _unpacked(w).t() for w in st["w"]], 1).to(st["dtype"])
    # grouped: each expert's rows padded to the longest, then one batched product
    e, n, k = st["experts"], st["n"], st["k"]
    x = _values(*_quantized(st["x"][st["rows"].long()].float(), fmt))
    off = st["offsets"].long()
    r = torch.arange(x.shape[0], device=x.device)
    group = torch.searchsorted(off, r, right=True) - 1
    at = r - off[group]
    padded = torch.zeros(e, st["most"], k, device=x.device)
    padded[group, at] = x
    y = torch.bmm(padded, _unpacked(st["w"]).view(e, n, k).transpose(1, 2))
    return y[group, at].to(st["dtype"])


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------
def _tensor(bb, w):
    return bb.MxTensor(w["codes"], w["scales"], w["row_scale"], bb.MX_E8M0 if w["fmt"] == E8M0 else bb.MX_E4M3, groups=w["groups"])


def _calls(st):
    from activation_aware_codebook_b200 import binding as bb
    op, fmt = st["op"], bb.MX_E8M0 if st["fmt"] == E8M0 else bb.MX_E4M3
    if op == "dequant":
        return bb.mx_dequant(_tensor(bb, st["w"]))
    if op in ("roundtrip", "swiglu"):
        return bb.mx_dequant(bb.mx_quantize(st["x"], fmt, swiglu=op == "swiglu"))
    if op == "linear":
        return bb.mx_linear(st["x"], _tensor(bb, st["w"][0]), out_dtype=st["dtype"])
    if op == "shared":
        x = bb.mx_quantize(st["x"], fmt)
        widths = [w["codes"].shape[0] for w in st["w"]]
        y = torch.empty(st["m"], sum(widths), dtype=st["dtype"], device=st["x"].device)
        for w, part in zip(st["w"], y.split(widths, 1)):
            bb.mx_linear(x, _tensor(bb, w), out=part)
        return y
    return bb.mx_linear(st["x"], _tensor(bb, st["w"]), rows=st["rows"], offsets=st["offsets"], out_dtype=st["dtype"])


def run(state):
    return _calls(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    op, m, k = case["op"], case["m"], case["k"]
    held = 0.5 + 1.0 / BLOCK[case["fmt"]]  # bytes of a quantised value
    size = 4 if case.get("out") == "f32" else 2
    if op == "dequant":
        return {"bytes": m * k * (held + 2), "flops": 0}
    if op == "roundtrip":
        return {"bytes": m * k * 4, "flops": 0}
    if op == "swiglu":
        return {"bytes": m * k * 6, "flops": 0}
    if op in ("linear", "shared"):
        n = case["n"] + 2 * case.get("n2", 0)
        return {"bytes": m * k * 2 + n * k * held + m * n * size, "flops": 2.0 * m * n * k}
    r, e = m * case["top"], case["experts"]
    # experts that get rows, as if every token chose its `top` evenly
    busy = e * (1 - (1 - case["top"] / e) ** m)
    return {"bytes": m * k * 2 + busy * case["n"] * k * held + r * case["n"] * size, "flops": 2.0 * r * case["n"] * k}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_rows(x, fmt):
    """fp64 rows to the values that their quantised form stands for: each step by comparing with the format's borders."""
    r, k = x.shape
    b = x.reshape(r, -1, BLOCK[fmt])
    most = b.abs().amax(2, keepdim=True)
    if fmt == E8M0:
        e = torch.frexp(most).exponent - 1 - 2  # frexp's mantissa lies in [0.5, 1)
        s = torch.ldexp(torch.ones_like(most), torch.where(most > 0, e, -127).clamp(-127, 127))
    else:
        row = x.abs().amax(1)[:, None, None]
        f = torch.frexp(row / 2688.0)
        p = torch.where(f.mantissa > 0.5, f.exponent, f.exponent - 1)
        g = torch.ldexp(torch.ones_like(row), torch.where(row > 0, p, 0).clamp(min=-126))
        t = most / (6.0 * g)
        step = torch.ldexp(torch.ones_like(t), (torch.frexp(t).exponent - 1).clamp(min=-6) - 3)
        s = torch.round(t / step) * step * g
    borders = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64, device=x.device)
    levels = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device=x.device)
    q = torch.where(s > 0, b.abs() / s, 0.0)
    below, upto = torch.bucketize(q, borders), torch.bucketize(q, borders, right=True)
    code = torch.where(below == upto, below, below + below % 2)  # on a border: the even one of the two
    return (levels[code] * s * torch.sign(b)).reshape(r, k)


def _exact_weights(w):
    """fp64 values of a packed tensor, a row's scale found from its place in the tiles."""
    rows, half = w["codes"].shape
    block = BLOCK[w["fmt"]]
    words = -(-(2 * half // block) // 4)
    levels = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device=w["codes"].device)
    v = torch.empty(rows, 2 * half, dtype=torch.float64, device=w["codes"].device)
    for odd in (0, 1):
        c = (w["codes"].int() >> 4 * odd) & 15
        v[:, odd::2] = levels[c & 7] * (1.0 - 2.0 * (c >> 3))
    per = rows // w["groups"]
    r = torch.arange(rows, device=v.device)
    e, i = r // per, r % per
    base = ((e * per) // 128 + e + i // 128) * words * 512 + i % 32 * 16 + i % 128 // 32 * 4
    j = torch.arange(2 * half // block, device=v.device)
    byte = w["scales"][base[:, None] + j // 4 * 512 + j % 4].double()
    if w["fmt"] == E8M0:
        s = torch.exp2(byte - 127)
    else:
        e8, m8 = torch.div(byte, 8, rounding_mode="floor"), byte % 8
        s = torch.where(e8 > 0, (8 + m8) * torch.exp2(e8 - 10), m8 * torch.exp2(torch.full_like(e8, -9.0)))
        s = s * w["row_scale"].double()[:, None]
    return v * s.repeat_interleave(block, 1)


def exact(case, seed):
    st = prepare(case, seed)
    op, fmt = case["op"], case["fmt"]
    if op == "dequant":
        return _exact_weights(st["w"])
    x = st["x"].double()
    if op == "roundtrip":
        return _exact_rows(x, fmt)
    if op == "swiglu":
        a, b = x[:, :case["k"]], x[:, case["k"]:]
        return _exact_rows(a * torch.sigmoid(a) * b, fmt)
    if op in ("linear", "shared"):
        x = _exact_rows(x, fmt)
        return torch.cat([x @ _exact_weights(w).t() for w in st["w"]], 1)
    x = _exact_rows(x[st["rows"].long()], fmt)
    y = torch.empty(x.shape[0], case["n"], dtype=torch.float64, device=x.device)
    w = _exact_weights(st["w"])
    off = st["offsets"].tolist()
    for e in range(case["experts"]):
        y[off[e]:off[e + 1]] = x[off[e]:off[e + 1]] @ w[e * case["n"]:(e + 1) * case["n"]].t()
    return y
