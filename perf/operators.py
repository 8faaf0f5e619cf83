"""Measured cases of the 4-bit (MXFP4) operators, with their plain forms.

The operators: quantisation to microscaled 4-bit floats and back, the product
of two such matrices, a training step of a layer built on them, the thin
product of a few float rows with 4-bit weights, and a mixture-of-experts layer
for a few tokens with 4-bit experts.

The format (one matrix of R rows and K columns, blocks of 32 along a row):
  codes   uint8 (R, Kp/2), Kp = K rounded up to 128: value k of a row in byte
          k // 2, even k in the low four bits; sign, then the index into
          0, 0.5, 1, 1.5, 2, 3, 4, 6; zeros beyond K
  scales  uint8 (Kp/128, Rp, 4), Rp = R rounded up to 32: the scale of block b
          of row r at [b // 4, r, b % 4], 2^(s - 127); zeros in the padding

With `own` false, run() computes the plain forms with elementary torch
operations in 32 bits; with `own` true it calls the framework.
"""
import math

import torch

own = False

DEV = "cuda:0"
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
BYTES = {"fp32": 4, "bf16": 2, "fp16": 2}
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # The activations of a few decoded tokens, on their way into a 4-bit product.
        {"name": "quantize 16x4096 bf16", "op": "quantize", "rows": 16, "cols": 4096, "type": "bf16", "both": False},
        # A weight matrix of odd size, needed along both axes (forward and backward).
        {"name": "quantize 8191x16388 fp32 both", "op": "quantize", "rows": 8191, "cols": 16388, "type": "fp32",
         "both": True},
        # The products of this repository's own benchmark: the smallest, the usual one, ...
        {"name": "product 256^3", "op": "product", "m": 256, "n": 256, "k": 256, "type": "fp32"},
        {"name": "product 4096^3", "op": "product", "m": 4096, "n": 4096, "k": 4096, "type": "fp32"},
        # ... an odd one: a ragged batch of tokens, no size a multiple of a tile ...
        {"name": "product 1111x4097x2050", "op": "product", "m": 1111, "n": 4097, "k": 2050, "type": "bf16"},
        # ... and the largest.
        {"name": "product 16384^3", "op": "product", "m": 16384, "n": 16384, "k": 16384, "type": "bf16"},
        # A layer's forward and backward pass on a short ragged batch, and on a full one.
        {"name": "train 333x1000x1536", "op": "train", "m": 333, "n": 1000, "k": 1536, "type": "bf16"},
        {"name": "train 8192x4096x4096", "op": "train", "m": 8192, "n": 4096, "k": 4096, "type": "bf16"},
        # One decoded token through a 4-bit layer, and a batch of 13 through an odd one.
        {"name": "linear 1x4096x4096", "op": "linear", "m": 1, "n": 4096, "k": 4096, "type": "bf16"},
        {"name": "linear 13x5001x16384", "op": "linear", "m": 13, "n": 5001, "k": 16384, "type": "fp32"},
        # One token through an expert layer, and a decode batch that reaches most of the experts.
        {"name": "experts 1 of 64x2048x768", "op": "experts", "tokens": 1, "experts": 64, "top": 8, "hidden": 2048,
         "inner": 768, "type": "bf16", "norm": True},
        {"name": "experts 48 of 128x4096x1536", "op": "experts", "tokens": 48, "experts": 128, "top": 8,
         "hidden": 4096, "inner": 1536, "type": "bf16", "norm": True},
    ]


def _size(rng, lo, hi):
    """A size of [lo, hi], spread over the logarithm; every other one odd or ragged as it comes, the rest a multiple of 32."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5 and v > 64:
        v = v // 32 * 32
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["quantize", "product", "train", "linear", "experts"])
    ty = rng.choice(["fp32", "bf16", "fp16"])
    if op == "quantize":
        return {"op": op, "rows": _size(rng, 1, 8191), "cols": _size(rng, 32, 16388), "type": ty,
                "both": rng.random() < 0.5}
    if op == "product":
        return {"op": op, "m": _size(rng, 1, 8192), "n": _size(rng, 16, 8192), "k": _size(rng, 32, 16384), "type": ty}
    if op == "train":
        return {"op": op, "m": _size(rng, 32, 8192), "n": _size(rng, 64, 4096), "k": _size(rng, 64, 4096), "type": ty}
    if op == "linear":
        return {"op": op, "m": _size(rng, 1, 64), "n": _size(rng, 64, 16384), "k": _size(rng, 64, 16384), "type": ty}
    experts = rng.choice([8, 16, 60, 64, 128])
    return {"op": op, "tokens": _size(rng, 1, 48), "experts": experts, "top": rng.randint(1, 8),
            "hidden": _size(rng, 256, 4096), "inner": _size(rng, 64, 1536), "type": ty, "norm": rng.random() < 0.7}


# ---- inputs -----------------------------------------------------------------------------------------------------

def _normal(gen, rows, cols, std, ty):
    return (torch.randn(rows, cols, generator=gen, device=DEV) * std).to(TYPES[ty])


def _activations(gen, rows, cols, ty):
    """Activations: normal values, with a few channels that are far larger than the rest, as layers have them."""
    x = torch.randn(rows, cols, generator=gen, device=DEV)
    big = torch.rand(cols, generator=gen, device=DEV) < 0.01
    return (x * torch.where(big, 12.0, 1.0)).to(TYPES[ty])


def _weights(gen, rows, cols):
    """4-bit weights (codes, scales) of a layer with `cols` inputs."""
    return _pack(*_codes(torch.randn(rows, cols, generator=gen, device=DEV) / math.sqrt(cols)))


def _inputs(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op = case["op"]
    if op == "quantize":
        return {"x": _activations(gen, case["rows"], case["cols"], case["type"])}
    if op == "product":
        a = _pack(*_codes(_activations(gen, case["m"], case["k"], "fp32")))
        return {"a": a, "b": _weights(gen, case["n"], case["k"])}
    if op == "train":
        m, n, k, ty = case["m"], case["n"], case["k"], case["type"]
        return {"x": _activations(gen, m, k, ty), "w": _normal(gen, n, k, 1.0 / math.sqrt(k), ty),
                "dy": _normal(gen, m, n, 0.01, ty)}
    if op == "linear":
        return {"x": _activations(gen, case["m"], case["k"], case["type"]), "w": _weights(gen, case["n"], case["k"])}
    e, h, f = case["experts"], case["hidden"], case["inner"]
    up = _stack([_codes(torch.randn(2 * f, h, generator=gen, device=DEV) / math.sqrt(h)) for _ in range(e)])
    down = _stack([_codes(torch.randn(h, f, generator=gen, device=DEV) / math.sqrt(f)) for _ in range(e)])
    return {"x": _normal(gen, case["tokens"], h, 1.0, case["type"]),
            "router": _normal(gen, e, h, 1.0 / math.sqrt(h), case["type"]), "up": up, "down": down}


def prepare(case, seed):
    state = {"case": case, **_inputs(case, seed)}
    if own:
        import fp32_sgemm_f32_amd as sg

        shapes = {"product": lambda c: {"a": (c["m"], c["k"]), "b": (c["n"], c["k"])},
                  "linear": lambda c: {"w": (c["n"], c["k"])},
                  "experts": lambda c: {"up": (c["experts"] * 2 * c["inner"], c["hidden"]),
                                        "down": (c["experts"] * c["hidden"], c["inner"])}}
        for name, shape in shapes.get(case["op"], lambda c: {})(case).items():
            state[name] = sg.Mx4(*state[name], *shape)
    return state


# ---- the plain forms --------------------------------------------------------------------------------------------

def _blocks(x):
    """x (R, K) in 32 bits as (R, Kp/32, 32), zeros beyond K."""
    r, k = x.shape
    kp = (k + 127) // 128 * 128
    x = torch.nn.functional.pad(x.float(), (0, kp - k))
    return x.view(r, kp // 32, 32)


def _power(s):
    """2^s in 32 bits for whole s of [-127, 127], exactly (a rounded power would move values off their ties)."""
    return torch.where(s > -127, ((s.int() + 127) << 23).view(torch.float32), 2.0 ** -127)


def _codes(x):
    """Codes 0..15 (R, Kp/32, 32) and scale bytes (R, Kp/32): the scale is 2^(floor(log2 max |x|) - 2), the
    values are rounded to the nearest level, ties to the even code, and held at 6 above it."""
    b = _blocks(x)
    a = b.abs()
    top = a.amax(-1)
    s = torch.where(top > 0, torch.frexp(top)[1] - 3, -127).clamp(min=-127)
    y = a * _power(-s).unsqueeze(-1)
    c = torch.zeros_like(y, dtype=torch.uint8)
    for i, edge in enumerate((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)):
        c += (y > edge) if i % 2 == 0 else (y >= edge)
    c += torch.signbit(b).to(torch.uint8) * 8
    return c, (s + 127).to(torch.uint8)


def _pack(c, s):
    r, nb, _ = c.shape
    c = c.view(r, nb * 16, 2)
    codes = c[..., 0] | (c[..., 1] << 4)
    scales = torch.zeros(nb // 4, (r + 31) // 32 * 32, 4, dtype=torch.uint8, device=c.device)
    scales[:, :r] = s.view(r, nb // 4, 4).transpose(0, 1)
    return codes, scales


def _stack(parts):
    """The matrices of all experts as one, row after row."""
    codes = torch.cat([_pack(c, s)[0] for c, s in parts])
    rows = codes.shape[0]
    s = torch.cat([s for _, s in parts])
    scales = torch.zeros(s.shape[1] // 4, (rows + 31) // 32 * 32, 4, dtype=torch.uint8, device=s.device)
    scales[:, :rows] = s.view(rows, -1, 4).transpose(0, 1)
    return codes, scales


def _values(q, k, rows=slice(None)):
    """The values (R, K), in 32 bits, that codes and scales stand for."""
    codes, scales = q
    codes = codes[rows]
    r, half = codes.shape
    level = torch.tensor(LEVELS + tuple(-v for v in LEVELS), device=codes.device)
    v = torch.stack((level[(codes & 15).long()], level[(codes >> 4).long()]), -1).view(r, half // 16, 32)
    s = scales[:, :q[0].shape[0]][:, rows].transpose(0, 1).reshape(r, half // 16)
    return (v * _power(s.int() - 127).unsqueeze(-1)).view(r, 2 * half)[:, :k]


def _rounded(x):
    """x as the 4-bit format holds it, in 32 bits."""
    return _values(_pack(*_codes(x)), x.shape[1])


def _chosen(x, router, top, norm):
    """Experts (T, top), best first and the lower index first on ties, and their weights. The logits are held in
    64 bits: a choice between two experts must not hang on the order of a sum."""
    logits = x.double() @ router.double().t()
    best, idx = torch.sort(logits, dim=1, descending=True, stable=True)
    p = torch.exp((best[:, :top] - best[:, :1]).float())
    total = p.sum(1) if norm else torch.exp((logits - best[:, :1]).float()).sum(1)
    return idx[:, :top], p / total.unsqueeze(1)


def _experts(state, c):
    x = state["x"].float()
    idx, p = _chosen(state["x"], state["router"], c["top"], c["norm"])
    h, f = c["hidden"], c["inner"]
    y = torch.zeros_like(x)
    for e in torch.unique(idx).tolist():
        t, j = (idx == e).nonzero(as_tuple=True)
        z = x[t] @ _values(state["up"], h, slice(e * 2 * f, (e + 1) * 2 * f)).t()
        g, u = z[:, :f], z[:, f:]
        act = g / (1.0 + torch.exp(-g)) * u
        y[t] += p[t, j].unsqueeze(1) * (act @ _values(state["down"], f, slice(e * h, (e + 1) * h)).t())
    return y.to(TYPES[c["type"]])


def run(state):
    c = state["case"]
    op = c["op"]
    if own:
        import fp32_sgemm_f32_amd as sg

        out = TYPES[c["type"]]
        if op == "quantize":
            if c["both"]:
                q, qt = sg.mx4_quantize_both(state["x"])
                return sg.mx4_dequantize(q, dtype=out), sg.mx4_dequantize(qt, dtype=out)
            return sg.mx4_dequantize(sg.mx4_quantize(state["x"]), dtype=out)
        if op == "product":
            return sg.mx4_gemm(state["a"], state["b"], dtype=out)
        if op == "train":
            y, saved = sg.mx4_train_forward(state["x"], state["w"])
            dx, dw = sg.mx4_train_backward(state["dy"], saved)
            return y, dx, dw
        if op == "linear":
            return sg.mx4_linear(state["x"], state["w"])
        return sg.mx4_moe(state["x"], state["router"], state["up"], state["down"], c["top"], norm=c["norm"])
    ty = TYPES[c["type"]]
    if op == "quantize":
        if c["both"]:
            return _rounded(state["x"]).to(ty), _rounded(state["x"].t()).to(ty)
        return _rounded(state["x"]).to(ty)
    if op == "product":
        return (_values(state["a"], c["k"]) @ _values(state["b"], c["k"]).t()).to(ty)
    if op == "train":
        x, w, dy = state["x"], state["w"], state["dy"]
        y = _rounded(x) @ _rounded(w).t()
        dx = _rounded(dy) @ _rounded(w.t()).t()
        dw = _rounded(dy.t()) @ _rounded(x.t()).t()
        return y.to(ty), dx.to(ty), dw          # the weights' gradient stays in 32 bits
    if op == "linear":
        return (state["x"].float() @ _values(state["w"], c["k"]).t()).to(ty)
    return _experts(state, c)


# ---- the definition in 64 bits ----------------------------------------------------------------------------------

def _power64(e):
    """2^e for whole e of [-160, 160], from a table: a computed power may be a last bit off."""
    table = torch.tensor([math.ldexp(1.0, i) for i in range(-160, 161)], dtype=torch.float64, device=DEV)
    return table[e.long() + 160]


def _decode64(q, k, first=0, rows=None):
    codes, scales = q
    rows = codes.shape[0] if rows is None else rows
    c = codes[first:first + rows].to(torch.int16)
    both = torch.empty(rows, 2 * c.shape[1], dtype=torch.int16, device=DEV)
    both[:, 0::2], both[:, 1::2] = c % 16, c // 16
    e, m = both % 8 // 2, both % 2              # value: m/2 where e = 0, else (1 + m/2) 2^(e-1)
    v = torch.where(e == 0, m * 0.5, (1 + m * 0.5) * _power64(e - 1)).double()
    v = torch.where(both >= 8, -v, v)
    s = _power64(scales[:, first:first + rows].long() - 127)       # (Kp/128, rows, 4)
    return (v * s.permute(1, 0, 2).reshape(rows, -1).repeat_interleave(32, dim=1))[:, :k]


def _round64(x):
    """x in 64 bits, each block of 32 along a row divided by its scale, rounded to a multiple of the step at
    its size (half of even steps to the even one), held at 6, and multiplied back."""
    r, k = x.shape
    v = torch.zeros(r, (k + 31) // 32 * 32, dtype=torch.float64, device=DEV)
    v[:, :k] = x.double()
    v = v.view(r, -1, 32)
    top = v.abs().max(dim=2, keepdim=True).values
    ex = torch.floor(torch.log2(torch.where(top > 0, top, 1.0)))
    ex = ex - (_power64(ex) > top).double() + (_power64(ex + 1) <= top).double()
    scale = _power64(torch.clamp(ex - 2, min=-127.0))
    y = v / scale
    step = torch.where(y.abs() < 2, 0.5, torch.where(y.abs() < 4, 1.0, 2.0)).double()
    y = torch.clamp(torch.round(y / step) * step, -6.0, 6.0)
    return torch.where(top > 0, y * scale, 0.0).view(r, -1)[:, :k]


def exact(case, seed):
    c, d = case, _inputs(case, seed)
    op = c["op"]
    if op == "quantize":
        return (_round64(d["x"]), _round64(d["x"].t())) if c["both"] else _round64(d["x"])
    if op == "product":
        return _decode64(d["a"], c["k"]) @ _decode64(d["b"], c["k"]).t()
    if op == "train":
        x, w, dy = d["x"], d["w"], d["dy"]
        return (_round64(x) @ _round64(w).t(), _round64(dy) @ _round64(w.t()).t(), _round64(dy.t()) @ _round64(x.t()).t())
    if op == "linear":
        return d["x"].double() @ _decode64(d["w"], c["k"]).t()
    h, f = c["hidden"], c["inner"]
    x = d["x"].double()
    y = torch.zeros_like(x)
    logits = torch.stack([(x * row).sum(1) for row in d["router"].double()], 1)
    for t in range(x.shape[0]):
        row = logits[t].tolist()
        picked = sorted(range(len(row)), key=lambda e: (-row[e], e))[:c["top"]]
        total = sum(math.exp(row[e] - row[picked[0]]) for e in (picked if c["norm"] else range(len(row))))
        logits[t] = float("-inf")
        for e in picked:
            logits[t, e] = math.exp(row[e] - row[picked[0]]) / total
    for e in range(c["experts"]):
        t = torch.nonzero(logits[:, e] > float("-inf")).flatten()
        if not len(t):
            continue
        z = x[t] @ _decode64(d["up"], h, e * 2 * f, 2 * f).t()
        g, u = z.split(f, dim=1)
        y[t] += logits[t, e, None] * ((g * torch.sigmoid(g) * u) @ _decode64(d["down"], f, e * h, h).t())
    return y


# ---- what a pass cannot do without ------------------------------------------------------------------------------

def _packed(rows, cols):
    return rows * ((cols + 31) // 32) * 17


def work(case):
    c, op, b = case, case["op"], BYTES[case["type"]]
    if op == "quantize":
        r, k = c["rows"], c["cols"]
        ways = [_packed(r, k)] + ([_packed(k, r)] if c["both"] else [])
        # the values read once; each packed form written, read back and written as the values it stands for
        return {"bytes": r * k * b + sum(2 * p + r * k * b for p in ways), "flops": 3 * r * k * len(ways)}
    if op == "product":
        m, n, k = c["m"], c["n"], c["k"]
        return {"bytes": _packed(m, k) + _packed(n, k) + m * n * b, "flops": 2 * m * n * k}
    if op == "train":
        m, n, k = c["m"], c["n"], c["k"]
        return {"bytes": b * 2 * (m * k + m * n) + b * n * k + 4 * n * k, "flops": 6 * m * n * k}
    if op == "linear":
        m, n, k = c["m"], c["n"], c["k"]
        return {"bytes": _packed(n, k) + b * m * (n + k), "flops": 2 * m * n * k}
    t, e, k, h, f = c["tokens"], c["experts"], c["top"], c["hidden"], c["inner"]
    reached = e * (1.0 - (1.0 - k / e) ** t)    # experts that at least one token chooses, on average
    return {"bytes": int(reached * (_packed(2 * f, h) + _packed(h, f))) + b * (e * h + 2 * t * h),
            "flops": 2 * t * (e * h + 3 * k * f * h)}
