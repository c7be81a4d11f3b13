"""Cases and plain forms of a packed encoder layer's linear steps in 16 and 32 bits, and of
what its training adds, on the flat [num_tokens, channels] buffer:

  matmul          act(a b^T + bias) + residual for a [m, k] and b [n, k], either one stored
                  transposed; act is none, relu, gelu or geglu (the product's first half,
                  through gelu, times its second); also the product before act;
  activation_bwd  the gradient before act and the bias's, from the gradient after it;
  layernorm_bwd   the gradients of LayerNorm in its input, weight and bias;
  dropout         x kept with probability 1 - p and divided by it, plus a residual; what is
                  kept follows from (seed, offset) and the element's index alone;
  rope            rotary positions with several axes, from views of one buffer of q, k and v.

The widths are those of the repository's workloads: 12 heads x 64 = 768 (q, k and v
together 2304, feed-forward 1152), 16 x 64 = 1024 and 8 x 64 = 512; the token counts are a
contrastive batch (32299), the long documents (169151), the graph batch (90487), one
first-token row per sequence (320) and single rows.
"""

import math

import torch

own = False

IO = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-5
MOST_TOKENS = 169151
LARGEST_PRODUCT = MOST_TOKENS * 1024 * 1024


def listed():
    return [
        # One query's first token through q, k and v: a launch and the weight.
        {"name": "matmul 1 x 2304 x 768", "op": "matmul", "m": 1, "n": 2304, "k": 768,
         "io": "bf16", "out": "bf16", "turn": "none", "bias": True, "act": "none",
         "residual": False, "pre": False},
        # The contrastive batch into the feed-forward, training (what goes into geglu is kept).
        {"name": "matmul 32299 x 2304 x 768 geglu", "op": "matmul", "m": 32299, "n": 2304,
         "k": 768, "io": "bf16", "out": "bf16", "turn": "none", "bias": True, "act": "geglu",
         "residual": False, "pre": True},
        # The attention output's projection on the long documents, with the residual stream.
        {"name": "matmul 169151 x 1024 x 1024 residual", "op": "matmul", "m": MOST_TOKENS,
         "n": 1024, "k": 1024, "io": "bf16", "out": "bf16", "turn": "none", "bias": True,
         "act": "none", "residual": True, "pre": False},
        # The gradient of the q, k and v weight: a sum over the batch's tokens.
        {"name": "matmul 2304 x 768 x 32299 weight gradient", "op": "matmul", "m": 2304,
         "n": 768, "k": 32299, "io": "bf16", "out": "fp32", "turn": "both", "bias": False,
         "act": "none", "residual": False, "pre": False},
        # Back through the feed-forward of the contrastive batch.
        {"name": "activation_bwd 32299 x 1152 geglu", "op": "activation_bwd", "rows": 32299,
         "cols": 1152, "io": "bf16", "act": "geglu"},
        # A small odd batch of an fp32 model.
        {"name": "activation_bwd 1001 x 333 gelu fp32", "op": "activation_bwd", "rows": 1001,
         "cols": 333, "io": "fp32", "act": "gelu"},
        # Training on the contrastive batch, with the residual stream's gradient.
        {"name": "layernorm_bwd 32299 x 768", "op": "layernorm_bwd", "rows": 32299, "cols": 768,
         "io": "bf16", "residual": True},
        # One first-token row per sequence of an fp32 model.
        {"name": "layernorm_bwd 320 x 500 fp32", "op": "layernorm_bwd", "rows": 320, "cols": 500,
         "io": "fp32", "residual": False},
        # A block's output joins the residual stream of the long documents.
        {"name": "dropout 169151 x 1024 residual", "op": "dropout", "rows": MOST_TOKENS,
         "cols": 1024, "io": "bf16", "residual": True, "p": 0.1},
        # The read-out's input, a row per sequence.
        {"name": "dropout 320 x 768", "op": "dropout", "rows": 320, "cols": 768, "io": "bf16",
         "residual": False, "p": 0.25},
        # Images as long as the long documents: rows and columns, each with its own angles.
        {"name": "rope 169151 x 16 x 64 two axes", "op": "rope", "rows": MOST_TOKENS,
         "heads": 16, "dim": 64, "io": "bf16", "sections": "16+16", "per_axis": True,
         "inverse": False},
        # A few short clips in fp32: time, height and width.
        {"name": "rope 1001 x 8 x 64 three axes fp32", "op": "rope", "rows": 1001, "heads": 8,
         "dim": 64, "io": "fp32", "sections": "8+12+12", "per_axis": False, "inverse": False},
    ]


def _spread(rng, low, high):
    return min(high, max(low, round(math.exp(rng.uniform(math.log(low), math.log(high))))))


def _width(rng):
    width = _spread(rng, 64, 2304)
    return max(64, width // 64 * 64) if rng.random() < 0.5 else width


def draw(rng):
    op = rng.choice(["matmul", "matmul", "matmul", "activation_bwd", "layernorm_bwd", "dropout",
                     "rope"])
    io = rng.choice(["bf16", "bf16", "fp32"])
    if op == "matmul":
        tokens, wide, deep = _spread(rng, 1, MOST_TOKENS), _width(rng), _width(rng)
        most = LARGEST_PRODUCT if io == "bf16" else LARGEST_PRODUCT // 8
        case = {"op": op, "io": io, "bias": False, "act": "none", "residual": False,
                "pre": False}
        turn = rng.choice(["none", "none", "b", "both"])
        if turn == "both":                                      # a weight's gradient
            most = min(most, 32299 * 2304 * 768)
            while tokens * wide * deep > most:
                tokens = tokens * 3 // 4
            return {**case, "m": wide, "n": deep, "k": tokens, "turn": turn, "out": "fp32",
                    "residual": rng.random() < 0.5}
        while tokens * wide * deep > most:
            tokens = tokens * 3 // 4
        case.update(m=tokens, n=wide, k=deep, turn=turn, out=io)
        if turn == "b":                                         # the input's gradient
            case["residual"] = rng.random() < 0.3
            return case
        act = rng.choice(["none", "none", "relu", "gelu", "geglu"])
        if act == "geglu":
            case["n"] = wide // 2 * 2
        case.update(act=act, bias=rng.random() < 0.7, residual=rng.random() < 0.4,
                    pre=act != "none" and rng.random() < 0.5)
        if io == "bf16" and rng.random() < 0.2:
            case["out"] = "fp32"
        return case
    rows = _spread(rng, 1, MOST_TOKENS)
    if op == "rope":
        dim = rng.choice([32, 40, 64, 64, 72, 128])
        heads = rng.choice([2, 8, 12, 16])
        axes = rng.choice([1, 2, 3])
        cuts = sorted(rng.randrange(1, dim // 2) for _ in range(axes - 1))
        ends = [0] + cuts + [dim // 2]
        while rows * heads * dim > (MOST_TOKENS * 1024 if io == "bf16" else MOST_TOKENS * 512):
            rows = rows * 3 // 4
        return {"op": op, "rows": rows, "heads": heads, "dim": dim, "io": io,
                "sections": "+".join(str(b - a) for a, b in zip(ends, ends[1:])),
                "per_axis": rng.random() < 0.5, "inverse": rng.random() < 0.5}
    cols = _width(rng)
    most = {"activation_bwd": 32299 * 1152, "layernorm_bwd": 32299 * 768,
            "dropout": MOST_TOKENS * 1024}[op]
    while rows * cols * (1 if io == "bf16" else 2) > most:
        rows = max(1, rows * 3 // 4)
    case = {"op": op, "rows": rows, "cols": cols, "io": io}
    if op == "activation_bwd":
        case["act"] = rng.choice(["none", "relu", "gelu", "geglu"])
        return case
    case["residual"] = rng.random() < 0.5
    if op == "dropout":
        case["p"] = rng.choice([0.0, 0.1, 0.25, 0.5, 0.9])
    return case


# ---------------------------------------------------------------- plain forms

def _gelu(z):
    return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))


def _gelu_slope(z):
    return (0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
            + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi))


def _activated(z, act):
    if act == "relu":
        return torch.clamp(z, min=0)
    if act == "gelu":
        return _gelu(z)
    if act == "geglu":
        gate, up = z.chunk(2, dim=1)
        return _gelu(gate) * up
    return z


def _plain_matmul(s):
    a = s["a"].float().t() if s["turn"] == "both" else s["a"].float()
    b = s["b"].float() if s["turn"] == "none" else s["b"].float().t()
    z = torch.matmul(a, b.t())
    if s["bias"] is not None:
        z = z + s["bias"].float()
    y = _activated(z, s["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    dtype = s["out"].dtype
    return [y.to(dtype)] + ([z.to(dtype)] if s["pre"] is not None else [])


def _plain_activation_bwd(s):
    dy = s["dy"].float()
    if s["act"] == "none":
        return [dy.sum(dim=0)]
    z = s["pre"].float()
    if s["act"] == "geglu":
        gate, up = z.chunk(2, dim=1)
        dz = torch.cat([dy * up * _gelu_slope(gate), dy * _gelu(gate)], dim=1)
    elif s["act"] == "gelu":
        dz = dy * _gelu_slope(z)
    else:
        dz = torch.where(z > 0, dy, torch.zeros_like(dy))
    return [dz.to(s["dy"].dtype), dz.sum(dim=0)]


def _plain_layernorm_bwd(s):
    h, dy = s["h"].float(), s["dy"].float()
    off = h - h.mean(dim=1, keepdim=True)
    rstd = torch.rsqrt(off.square().mean(dim=1, keepdim=True) + EPS)
    n = off * rstd
    g = dy * s["weight"].float()
    dx = rstd * (g - g.mean(dim=1, keepdim=True) - n * (g * n).mean(dim=1, keepdim=True))
    if s["dresidual"] is not None:
        dx = dx + s["dresidual"].float()
    return [dx.to(s["h"].dtype), (dy * n).sum(dim=0), dy.sum(dim=0)]


def _random_words(seed, offset, count, device):
    """Philox4x32-10 (Salmon et al., Parallel random numbers: as easy as 1, 2, 3, 2011): key
    `seed`, counters (block, offset) for blocks 0, 1, ..; the first `count` 32-bit words."""
    low = 0xFFFFFFFF
    block = torch.arange(-(-count // 4), dtype=torch.int64, device=device)
    c0, c1 = block & low, block >> 32
    c2 = torch.full_like(block, offset & low)
    c3 = torch.full_like(block, (offset >> 32) & low)
    k0, k1 = seed & low, (seed >> 32) & low
    for _ in range(10):
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57       # the 64-bit products, modulo 2^64
        c0, c1, c2, c3 = (((p1 >> 32) & low) ^ c1 ^ k0, p1 & low,
                          ((p0 >> 32) & low) ^ c3 ^ k1, p0 & low)
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    return torch.stack([c0, c1, c2, c3], dim=1).flatten()[:count]


def _plain_dropout(s):
    x, p = s["x"], s["p"]
    words = _random_words(s["seed"], s["offset"], x.numel(), x.device).view(x.shape)
    y = torch.where(words >= math.ceil(p * 2 ** 32), x.float() * (1 / (1 - p)),
                    torch.zeros((), device=x.device))
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return [y.to(x.dtype)]


def _plain_rope(s):
    half = s["q"].shape[2] // 2
    turns = []
    for axis, size in enumerate(s["sections"]):
        start = sum(s["sections"][:axis])
        i = torch.arange(size, dtype=torch.float64, device=s["q"].device)
        power = -i / size if s["per_axis"] else -(i + start) / half
        turns.append(s["positions"][axis].double()[:, None] * s["theta"] ** power)
    angle = torch.cat(turns, dim=1)[:, None, :] * (-1 if s["inverse"] else 1)
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    out = []
    for x in (s["q"], s["k"]):
        x1, x2 = x[..., :half].float(), x[..., half:].float()
        out.append(torch.cat([x1 * cos - x2 * sin, x2 * cos + x1 * sin], dim=2).to(x.dtype))
    return out


# ---------------------------------------------------------------- the framework's calls

def _own_matmul(s):
    import padding_free_packed_gb300 as pe
    y = pe.pe_matmul(s["a"], s["b"], bias=s["bias"], activation=s["act"],
                     residual=s["residual"], out=s["out"], pre=s["pre"],
                     a_transposed=s["turn"] == "both", b_transposed=s["turn"] != "none")
    return [y] if s["pre"] is None else [y, s["pre"]]


def _own_activation_bwd(s):
    import padding_free_packed_gb300 as pe
    dz, dbias = pe.pe_activation_bwd(s["dy"], s["pre"], s["act"])
    return [dbias] if s["act"] == "none" else [dz, dbias]


def _own_layernorm_bwd(s):
    import padding_free_packed_gb300 as pe
    return list(pe.pe_layernorm_bwd(s["dy"], s["h"], s["weight"], EPS,
                                    dresidual=s["dresidual"]))


def _own_dropout(s):
    import padding_free_packed_gb300 as pe
    return [pe.pe_dropout(s["x"], s["p"], s["seed"], s["offset"], residual=s["residual"])]


def _own_rope(s):
    import padding_free_packed_gb300 as pe
    return list(pe.pe_rope_axes(s["q"], s["k"], s["positions"], s["sections"], s["theta"],
                                per_axis=s["per_axis"], inverse=s["inverse"]))


PLAIN = {"matmul": _plain_matmul, "activation_bwd": _plain_activation_bwd,
         "layernorm_bwd": _plain_layernorm_bwd, "dropout": _plain_dropout, "rope": _plain_rope}
OWN = {"matmul": _own_matmul, "activation_bwd": _own_activation_bwd,
       "layernorm_bwd": _own_layernorm_bwd, "dropout": _own_dropout, "rope": _own_rope}


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 6151 + 29)
    op, io = case["op"], IO[case["io"]]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    def activations(rows, cols):
        # Channels of very different size, as in trained encoders.
        return normal(rows, cols) * torch.exp(0.8 * normal(cols))

    def stored(x, turned):
        """The matrix as a program keeps it: rows that start at multiples of 16 bytes."""
        x = x.t() if turned else x
        store = torch.empty(x.shape[0], -(-x.shape[1] // 8) * 8, dtype=io, device="cuda")
        return store[:, :x.shape[1]].copy_(x)

    s = {"op": op}
    if op == "matmul":
        m, n, k, turn = case["m"], case["n"], case["k"], case["turn"]
        out = IO[case["out"]]
        wide = n // 2 if case["act"] == "geglu" else n
        s.update(turn=turn, act=case["act"], out=torch.empty(m, wide, dtype=out, device="cuda"))
        if turn == "both":                          # an output gradient and activations
            s["a"] = stored(normal(m, k) * 0.1, True)
            s["b"] = stored(activations(k, n).t(), True)
        else:
            s["a"] = stored(activations(m, k) if turn == "none" else normal(m, k) * 0.1, False)
            s["b"] = stored(normal(n, k) / math.sqrt(k), turn == "b")
        s["bias"] = (0.2 * normal(n)).to(out) if case["bias"] else None
        s["residual"] = activations(m, wide).to(out) if case["residual"] else None
        s["pre"] = torch.empty(m, n, dtype=out, device="cuda") if case["pre"] else None
        return s
    rows = case["rows"]
    if op == "rope":
        heads, dim = case["heads"], case["dim"]
        sections = tuple(int(x) for x in case["sections"].split("+"))
        qkv = normal(rows, 3, heads, dim).to(io)
        # The last axes are an image's rows and columns, the first one counts frames or tokens.
        most = [8192, 256, 256][:len(sections)] if len(sections) != 2 else [256, 256]
        positions = torch.stack([torch.randint(0, top, (rows,), generator=gen, device="cuda",
                                               dtype=torch.int32) for top in most])
        s.update(q=qkv[:, 0], k=qkv[:, 1], positions=positions, sections=sections,
                 theta=10000.0, per_axis=case["per_axis"], inverse=case["inverse"])
        return s
    cols = case["cols"]
    if op == "dropout":
        s.update(x=activations(rows, cols).to(io), p=case["p"], offset=int(seed) % 1000,
                 seed=(int(seed) * 0x9E3779B97F4A7C15 + 0x1234567) % 2 ** 63,
                 residual=activations(rows, cols).to(io) if case["residual"] else None)
        return s
    s["dy"] = (normal(rows, cols) * 0.1).to(io)
    if op == "activation_bwd":
        wide = 2 * cols if case["act"] == "geglu" else cols
        s.update(act=case["act"], pre=None)
        if case["act"] != "none":
            s["pre"] = (1.5 * normal(rows, wide)).to(io)
        return s
    s.update(h=activations(rows, cols).to(io), weight=(1.0 + 0.2 * normal(cols)).to(io),
             dresidual=(normal(rows, cols) * 0.1).to(io) if case["residual"] else None)
    return s


def run(state):
    return (OWN if own else PLAIN)[state["op"]](state)


def work(case):
    op, size = case["op"], 2 if case["io"] == "bf16" else 4
    if op == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        out = 2 if case["out"] == "bf16" else 4
        wide = n // 2 if case["act"] == "geglu" else n
        moved = size * (m * k + n * k) + out * m * wide * (2 if case["residual"] else 1)
        moved += out * m * n if case["pre"] else 0
        return {"bytes": moved + (out * n if case["bias"] else 0), "flops": 2 * m * n * k}
    if op == "rope":
        each = 2 * case["rows"] * case["heads"] * case["dim"]
        axes = case["sections"].count("+") + 1
        return {"bytes": 2 * size * each + 4 * axes * case["rows"], "flops": 3 * each}
    rows, cols = case["rows"], case["cols"]
    each = rows * cols
    if op == "activation_bwd":
        wide = 2 if case["act"] == "geglu" else 1
        if case["act"] == "none":
            return {"bytes": size * each + 4 * cols, "flops": each}
        return {"bytes": size * each * (1 + 2 * wide) + 4 * cols * wide, "flops": 20 * each}
    if op == "layernorm_bwd":
        return {"bytes": size * each * (4 if case["residual"] else 3) + (size + 8) * cols,
                "flops": 14 * each}
    return {"bytes": size * each * (3 if case["residual"] else 2), "flops": 2 * each}


# ---------------------------------------------------------------- from the definitions, in 64 bits

def _upper(z):
    """The normal distribution function."""
    return 0.5 * torch.special.erfc(-z / math.sqrt(2.0))


def _high_half(x, factor):
    """The upper 32 bits of x * factor for 32-bit numbers, by halves of 16 bits."""
    x0, x1 = x & 0xFFFF, x >> 16
    f0, f1 = factor & 0xFFFF, factor >> 16
    middle = x1 * f0 + ((x0 * f0) >> 16)
    return x1 * f1 + (middle >> 16) + ((x0 * f1 + (middle & 0xFFFF)) >> 16)


def _exact_kept(count, seed, offset, p):
    """Which elements Philox4x32-10 keeps, in pieces."""
    kept = torch.empty(-(-count // 4), 4, dtype=torch.bool, device="cuda")
    for start in range(0, kept.shape[0], 1 << 24):
        n = min(1 << 24, kept.shape[0] - start)
        block = torch.arange(start, start + n, device="cuda")
        words = [block % 2 ** 32, block // 2 ** 32, torch.tensor(offset % 2 ** 32, device="cuda"),
                 torch.tensor(offset // 2 ** 32, device="cuda")]
        key = [seed % 2 ** 32, seed // 2 ** 32]
        for _ in range(10):
            a, b, c, d = words
            words = [_high_half(c, 0xCD9E8D57) ^ b ^ key[0], (c * 0xCD9E8D57) % 2 ** 32,
                     _high_half(a, 0xD2511F53) ^ d ^ key[1], (a * 0xD2511F53) % 2 ** 32]
            key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
        for j, w in enumerate(words):
            kept[start:start + n, j] = w >= p * 2 ** 32
    return kept.flatten()[:count]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "matmul":
        a, b = s["a"].double(), s["b"].double()
        z = torch.einsum({"none": "mk,nk->mn", "b": "mk,kn->mn", "both": "km,kn->mn"}[s["turn"]],
                         a, b)
        if case["bias"]:
            z += s["bias"].double()[None, :]
        half = case["n"] // 2
        y = {"none": lambda: z.clone(), "relu": lambda: torch.where(z > 0, z, 0.0),
             "gelu": lambda: z * _upper(z),
             "geglu": lambda: z[:, :half] * _upper(z[:, :half]) * z[:, half:]}[case["act"]]()
        if case["residual"]:
            y += s["residual"].double()
        return [y, z] if case["pre"] else [y]
    if op == "rope":
        half = case["dim"] // 2
        angle = torch.empty(case["rows"], half, dtype=torch.float64, device="cuda")
        pair = 0
        for axis, size in enumerate(s["sections"]):
            for j in range(size):
                share = j / size if case["per_axis"] else pair / half
                angle[:, pair] = s["positions"][axis].double() / math.pow(s["theta"], share)
                pair += 1
        turned = torch.polar(torch.ones_like(angle), -angle if case["inverse"] else angle)
        out = []
        for x in (s["q"], s["k"]):
            z = torch.complex(x[..., :half].double(), x[..., half:].double()) * turned[:, None]
            out.append(torch.cat([z.real, z.imag], dim=2))
        return out
    if op == "dropout":
        x = s["x"].double()
        kept = _exact_kept(x.numel(), s["seed"], s["offset"], s["p"]).view(x.shape)
        y = torch.where(kept, x / (1.0 - s["p"]), 0.0)
        return [y + s["residual"].double() if case["residual"] else y]
    dy = s["dy"].double()
    if op == "activation_bwd":
        if case["act"] == "none":
            return [torch.einsum("rc->c", dy)]
        z = s["pre"].double()

        def slope(t):
            return _upper(t) + t * torch.exp(-t * t / 2) / math.sqrt(2 * math.pi)

        if case["act"] == "geglu":
            gate, up = z[:, :case["cols"]], z[:, case["cols"]:]
            dz = torch.empty_like(z)
            dz[:, :case["cols"]] = dy * up * slope(gate)
            dz[:, case["cols"]:] = dy * gate * _upper(gate)
        else:
            dz = dy * slope(z) if case["act"] == "gelu" else dy * (z > 0).double()
        return [dz, torch.einsum("rc->c", dz)]
    h = s["h"].double()
    c = case["cols"]
    off = h - (h.sum(dim=1) / c)[:, None]
    inverse = 1.0 / torch.sqrt((off * off).sum(dim=1) / c + EPS)
    g = s["weight"].double() * dy
    along = (g * off).sum(dim=1) * inverse ** 3 / c
    dx = inverse[:, None] * (g - (g.sum(dim=1) / c)[:, None]) - along[:, None] * off
    if s["dresidual"] is not None:
        dx = dx + s["dresidual"].double()
    return [dx, torch.einsum("rc,rc,r->c", dy, off, inverse), dy.sum(dim=0)]
