"""Cases and plain forms of the 8-bit layer operators on the packed token buffer.

A packed encoder layer in 8-bit floating point is a chain of four operators on
the flat [num_tokens, channels] buffer:

  rmsnorm      h = x (+ residual), y = h / rms(h) * weight, y in 8 bits with one
               fp32 scale for each row's block of 128 channels;
  rmsnorm_bwd  the gradients of that norm in x (and residual) and in the weight;
  quantize     a matrix in 8 bits with a scale for each 1 x 128 or 128 x 128
               block, as it is and (or) transposed;
  matmul       out[m, n] = sum over blocks c of 128 along k of
               a_scale[c, m] * b_scale[c, n / 128] * sum_(k in c) a[m, k] b[n, k].

The widths are those of the repository's workloads: 12 heads x 64 = 768 (q, k
and v together 2304, feed-forward 1152), 16 x 64 = 1024 and 8 x 64 = 512; the
token counts are a contrastive batch (32299), the long documents (169151), the
graph batch (90487), one first-token row per sequence (320) and single rows.
"""

import math

import numpy as np
import torch

own = False

LARGEST = {"e4m3": 448.0, "e5m2": 57344.0}
SMALLEST_AMAX = 2.0 ** -117       # keeps a block's scale and its reciprocal normal numbers
FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
IO = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-5
MOST_TOKENS = 169151


def listed():
    return [
        # One query's first token between two layers: a launch, hardly any data.
        {"name": "rmsnorm 1 x 768", "op": "rmsnorm", "rows": 1, "cols": 768, "io": "bf16",
         "fp8": "e4m3", "residual": True},
        # The contrastive batch between attention and feed-forward.
        {"name": "rmsnorm 32299 x 768", "op": "rmsnorm", "rows": 32299, "cols": 768,
         "io": "bf16", "fp8": "e4m3", "residual": True},
        # The graph batch's fp32 activations, first norm of the stack; ragged width.
        {"name": "rmsnorm 90487 x 500 fp32", "op": "rmsnorm", "rows": 90487, "cols": 500,
         "io": "fp32", "fp8": "e4m3", "residual": False},
        # Training on the contrastive batch, with the residual stream's gradient.
        {"name": "rmsnorm_bwd 32299 x 768", "op": "rmsnorm_bwd", "rows": 32299, "cols": 768,
         "io": "bf16", "residual": True},
        # A small odd batch of an fp32 model.
        {"name": "rmsnorm_bwd 1001 x 333 fp32", "op": "rmsnorm_bwd", "rows": 1001, "cols": 333,
         "io": "fp32", "residual": False},
        # A weight after an optimizer step, for the forward and the input gradient.
        {"name": "quantize weight 2304 x 768", "op": "quantize", "rows": 2304, "cols": 768,
         "io": "bf16", "fp8": "e4m3", "block_rows": 128, "plain": True, "transposed": True},
        # An output gradient, for the input gradient and for the weight's.
        {"name": "quantize gradient 32299 x 2304", "op": "quantize", "rows": 32299, "cols": 2304,
         "io": "bf16", "fp8": "e5m2", "block_rows": 1, "plain": True, "transposed": True},
        # One query's first token through q, k and v.
        {"name": "matmul 1 x 2304 x 768", "op": "matmul", "m": 1, "n": 2304, "k": 768,
         "a": "e4m3", "out": "bf16"},
        # The first token of every sequence through a ragged read-out head.
        {"name": "matmul 320 x 1001 x 1140", "op": "matmul", "m": 320, "n": 1001, "k": 1140,
         "a": "e4m3", "out": "fp32"},
        # q, k and v of the contrastive batch.
        {"name": "matmul 32299 x 2304 x 768", "op": "matmul", "m": 32299, "n": 2304, "k": 768,
         "a": "e4m3", "out": "bf16"},
        # The attention output's projection on the long documents.
        {"name": "matmul 169151 x 1024 x 1024", "op": "matmul", "m": 169151, "n": 1024, "k": 1024,
         "a": "e4m3", "out": "bf16"},
        # The gradient of the q, k and v weight: a sum over the batch's tokens.
        {"name": "matmul 2304 x 768 x 32299", "op": "matmul", "m": 2304, "n": 768, "k": 32299,
         "a": "e5m2", "out": "fp32"},
    ]


def _spread(rng, low, high):
    return min(high, max(low, round(math.exp(rng.uniform(math.log(low), math.log(high))))))


def draw(rng):
    op = rng.choice(["rmsnorm", "rmsnorm_bwd", "quantize", "matmul", "matmul"])
    if op == "matmul":
        case = {"op": op, "a": rng.choice(["e4m3", "e5m2"]), "out": rng.choice(["bf16", "fp32"])}
        tokens = _spread(rng, 1, MOST_TOKENS)
        wide, deep = (_spread(rng, 64, 2304) for _ in range(2))
        if rng.random() < 0.7:                      # tokens through a weight, the widths ragged or not
            if rng.random() < 0.5:
                wide, deep = max(64, wide // 64 * 64), max(64, deep // 64 * 64)
            while tokens * wide * deep > MOST_TOKENS * 1024 * 1024:
                tokens = tokens * 3 // 4
            return {**case, "m": tokens, "n": wide, "k": deep}
        while tokens * wide * deep > 32299 * 2304 * 768:
            tokens = tokens * 3 // 4
        return {**case, "m": wide, "n": deep, "k": tokens}      # a weight's gradient
    rows, cols = _spread(rng, 1, MOST_TOKENS), _spread(rng, 64, 2304)
    if rng.random() < 0.5:
        cols = max(64, cols // 64 * 64)
    while rows * cols > 32299 * 2304:
        rows = rows * 3 // 4
    case = {"op": op, "rows": rows, "cols": cols, "io": rng.choice(["bf16", "fp32"])}
    if op != "quantize":
        case["residual"] = rng.random() < 0.5
    if op != "rmsnorm_bwd":
        case["fp8"] = rng.choice(["e4m3", "e5m2"])
    if op == "quantize":
        which = rng.choice([(True, False), (False, True), (True, True)])
        case.update(block_rows=rng.choice([1, 128]), plain=which[0], transposed=which[1])
    return case


# ---------------------------------------------------------------- plain forms

def _blocks(n):
    return -(-n // 128)


def _padded(rows, cols, fp8, device):
    """An 8-bit matrix whose rows start at multiples of 16 bytes."""
    return torch.empty(rows, -(-cols // 16) * 16, dtype=fp8, device=device)[:, :cols]


def _quantized(x, fp8, block_rows):
    """x [R, C] fp32 -> (8-bit values [R, C], scales [blocks of C, R or blocks of R])."""
    r, c = x.shape
    rb, cb = -(-r // block_rows), _blocks(c)
    p = torch.nn.functional.pad(x, (0, cb * 128 - c, 0, rb * block_rows - r))
    p = p.view(rb, block_rows, cb, 128)
    amax = p.abs().amax(dim=(1, 3)).clamp(min=SMALLEST_AMAX)
    q = p * (LARGEST[fp8] / amax)[:, None, :, None]
    q = q.view(rb * block_rows, cb * 128)[:r, :c].to(FP8[fp8])
    return q, (amax / LARGEST[fp8]).t().contiguous()


def _summed(x, residual):
    h = x.float()
    return h if residual is None else (h + residual.float()).to(x.dtype).float()


def _plain_rmsnorm(s):
    h = _summed(s["x"], s["residual"])
    y = h * torch.rsqrt(h.square().mean(dim=1, keepdim=True) + EPS) * s["weight"].float()
    q, scales = _quantized(y, s["fp8"], 1)
    return [q, scales] + ([] if s["residual"] is None else [h.to(s["x"].dtype)])


def _plain_rmsnorm_bwd(s):
    h, dy = s["h"].float(), s["dy"].float()
    rstd = torch.rsqrt(h.square().mean(dim=1, keepdim=True) + EPS)
    n = h * rstd
    g = dy * s["weight"].float()
    dx = rstd * (g - n * (g * n).mean(dim=1, keepdim=True))
    if s["dresidual"] is not None:
        dx = dx + s["dresidual"].float()
    return [dx.to(s["h"].dtype), (dy * n).sum(dim=0)]


def _plain_quantize(s):
    x, out = s["x"].float(), []
    if s["plain"]:
        out += list(_quantized(x, s["fp8"], s["block_rows"]))
    if s["transposed"]:
        out += list(_quantized(x.t(), s["fp8"], s["block_rows"]))
    return out


def _plain_matmul(s):
    (m, k), n = s["a"].shape, s["b"].shape[0]
    a = s["a"].float() * s["a_scales"].t().repeat_interleave(128, dim=1)[:, :k]
    rows = s["b_scales"].repeat_interleave(128, dim=0)[:k]
    b = s["b"].float() * rows.t().repeat_interleave(128, dim=0)[:n]
    return [torch.matmul(a, b.t()).to(s["out"].dtype)]


# ---------------------------------------------------------------- the framework's calls

def _own_rmsnorm(s):
    import padding_free_packed_gb300 as pe
    return list(pe.pe_rmsnorm_fp8(s["x"], s["weight"], EPS, residual=s["residual"],
                                  dtype=FP8[s["fp8"]], out=s["q"]))


def _own_rmsnorm_bwd(s):
    import padding_free_packed_gb300 as pe
    return list(pe.pe_rmsnorm_bwd(s["dy"], s["h"], s["weight"], EPS, dresidual=s["dresidual"]))


def _own_quantize(s):
    import padding_free_packed_gb300 as pe
    return list(pe.pe_quantize_fp8(s["x"], s["block_rows"], dtype=FP8[s["fp8"]],
                                   plain=s["plain"], transposed=s["transposed"]))


def _own_matmul(s):
    import padding_free_packed_gb300 as pe
    return [pe.pe_matmul_fp8(s["a"], s["a_scales"], s["b"], s["b_scales"], out=s["out"])]


PLAIN = {"rmsnorm": _plain_rmsnorm, "rmsnorm_bwd": _plain_rmsnorm_bwd,
         "quantize": _plain_quantize, "matmul": _plain_matmul}
OWN = {"rmsnorm": _own_rmsnorm, "rmsnorm_bwd": _own_rmsnorm_bwd,
       "quantize": _own_quantize, "matmul": _own_matmul}


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 13)
    op = case["op"]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    def activations(rows, cols):
        # Channels of very different size, as in trained encoders.
        return normal(rows, cols) * torch.exp(0.8 * normal(cols))

    s = {"op": op}
    if op == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        a, a_scales = _quantized(activations(m, k), case["a"], 1)
        b, b_scales = _quantized(normal(n, k) / math.sqrt(k), "e4m3", 128)
        s["a"] = _padded(m, k, a.dtype, "cuda").copy_(a)
        s["b"] = _padded(n, k, b.dtype, "cuda").copy_(b)
        s.update(a_scales=a_scales, b_scales=b_scales,
                 out=torch.empty(m, n, dtype=IO[case["out"]], device="cuda"))
        return s
    rows, cols, io = case["rows"], case["cols"], IO[case["io"]]
    if op == "quantize":
        s.update(x=activations(rows, cols).to(io), fp8=case["fp8"], block_rows=case["block_rows"],
                 plain=case["plain"], transposed=case["transposed"])
        return s
    s["weight"] = (1.0 + 0.2 * normal(cols)).to(io)
    if op == "rmsnorm":
        s.update(x=activations(rows, cols).to(io), fp8=case["fp8"],
                 residual=activations(rows, cols).to(io) if case["residual"] else None,
                 q=_padded(rows, cols, FP8[case["fp8"]], "cuda"))
    else:
        s.update(h=activations(rows, cols).to(io), dy=(normal(rows, cols) * 0.1).to(io),
                 dresidual=(normal(rows, cols) * 0.1).to(io) if case["residual"] else None)
    return s


def run(state):
    return (OWN if own else PLAIN)[state["op"]](state)


def work(case):
    op = case["op"]
    if op == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        size = 2 if case["out"] == "bf16" else 4
        scales = 4 * _blocks(k) * (m + _blocks(n))
        return {"bytes": m * k + n * k + m * n * size + scales, "flops": 2 * m * n * k}
    rows, cols, size = case["rows"], case["cols"], 2 if case["io"] == "bf16" else 4
    each = rows * cols
    if op == "rmsnorm":
        moved = size * (3 if case["residual"] else 1) + 1
        return {"bytes": each * moved + 4 * rows * _blocks(cols) + size * cols, "flops": 7 * each}
    if op == "rmsnorm_bwd":
        moved = size * (4 if case["residual"] else 3)
        return {"bytes": each * moved + (size + 4) * cols, "flops": 11 * each}
    ways = int(case["plain"]) + int(case["transposed"])
    scales = 0
    for wanted, r, c in ((case["plain"], rows, cols), (case["transposed"], cols, rows)):
        scales += 4 * _blocks(c) * -(-r // case["block_rows"]) if wanted else 0
    return {"bytes": each * (size + ways) + scales, "flops": 3 * each * ways}


# ---------------------------------------------------------------- from the definitions, in 64 bits

def _nearest_fp8(v, fp8):
    """The 8-bit number nearest to each value (ties to even), from the formats' definition."""
    mantissa, lowest = {"e4m3": (3, -6), "e5m2": (2, -14)}[fp8]
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (e - 1).clamp(min=lowest) - mantissa)
    return (torch.round(v / step) * step).clamp(-LARGEST[fp8], LARGEST[fp8])


def _exact_blocks(v, fp8, block_rows):
    rows, cols = v.shape
    tall = torch.arange(rows, device=v.device) // block_rows
    largest = torch.stack([part.abs().amax(dim=1) for part in v.split(128, dim=1)])
    if block_rows > 1:
        empty = torch.zeros(largest.shape[0], -(-rows // block_rows), dtype=v.dtype,
                            device=v.device)
        largest = empty.index_reduce(1, tall, largest, "amax")
    scales = largest.clamp(min=SMALLEST_AMAX) / LARGEST[fp8]
    wide = torch.arange(cols, device=v.device) // 128
    return _nearest_fp8(v / scales.t()[tall][:, wide], fp8), scales


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "matmul":
        total = torch.zeros(case["m"], case["n"], dtype=torch.float64, device="cuda")
        b_block = torch.arange(case["n"], device="cuda") // 128
        for c in range(0, case["k"], 128):
            a = s["a"][:, c:c + 128].double() * s["a_scales"][c // 128].double()[:, None]
            b = s["b"][:, c:c + 128].double() * s["b_scales"][c // 128].double()[b_block][:, None]
            total.addmm_(a, b.T)
        return [total]
    if op == "quantize":
        v, out = s["x"].double(), []
        if case["plain"]:
            out.extend(_exact_blocks(v, case["fp8"], case["block_rows"]))
        if case["transposed"]:
            out.extend(_exact_blocks(v.T, case["fp8"], case["block_rows"]))
        return out
    w = s["weight"].double()
    if op == "rmsnorm":
        h = s["x"].double()
        if s["residual"] is not None:
            h = (h + s["residual"].double()).to(s["x"].dtype).double()
        rms = torch.sqrt((h * h).sum(dim=1) / case["cols"] + EPS)
        q, scales = _exact_blocks(h / rms[:, None] * w, case["fp8"], 1)
        return [q, scales] + ([h] if case["residual"] else [])
    h, dy = s["h"].double(), s["dy"].double()
    inverse = 1.0 / torch.sqrt((h * h).sum(dim=1) / case["cols"] + EPS)
    along = (w * dy * h).sum(dim=1) * inverse ** 3 / case["cols"]
    dx = inverse[:, None] * w * dy - along[:, None] * h
    if s["dresidual"] is not None:
        dx = dx + s["dresidual"].double()
    return [dx, torch.einsum("rc,rc,r->c", dy, h, inverse)]
