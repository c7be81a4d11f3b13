"""64-bit references of the layer-tail backward calls and bounds on what fp32 arithmetic may
lose. U is half a step of fp32 relative to the value; a sum of `depth` additions in a row is
off by at most depth * U times the sum of magnitudes."""

import math

import torch

U = 2.0 ** -24
TINY = 2.0 ** -126


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def rounded(bound, want, dtype):
    """`bound` on the unrounded result, plus the rounding to `dtype`."""
    return bound + half_step(dtype) * (want.abs() + bound) + 1e-38


def assert_within(got, want, bound, what):
    got, want = got.double(), want.double()
    assert got.shape == want.shape, what
    over = (got - want).abs() - bound
    assert not bool(torch.isnan(over).any()), f"{what}: NaN"
    worst = float(over.max()) if over.numel() else 0.0
    assert worst <= 0, f"{what}: {worst:.3e} beyond the bound"


# ---------------------------------------------------------------- activations

def phi(z):
    return 0.5 * torch.special.erfc(-z / math.sqrt(2.0))


def bell(z):
    return torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)


def phi_error(z, dtype):
    """Relative error of the normal distribution function and its density as the kernels
    form them. bf16: the polynomial's 1.2e-6 and four roundings; the exponent z^2 / 2 log2 e
    carries three roundings, each U of its size. fp32: CUDA's normcdff (5 ulp) and expf
    (2 ulp) of an argument with two roundings."""
    own = 1.3e-6 + 12 * U if dtype == torch.bfloat16 else 12 * U
    return own + 3 * U * z * z


def activation(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return z * phi(z)
    if act == "geglu":
        gate, up = z.chunk(2, dim=1)
        return gate * phi(gate) * up
    return z


def activation_bwd(dy, z, act, dtype):
    """dz and its bound before rounding, for 64-bit dy and z."""
    if act == "none":
        return dy, torch.zeros_like(dy)
    if act == "relu":
        return dy * (z > 0), torch.zeros_like(dy)

    def slope(t):
        # The exponential is zero below 2^-126, the smallest normal number: phi, at most
        # half of it there, and the density, 0.4 of it, lose no more than that.
        e = phi_error(t, dtype) + 4 * U
        lost = TINY * (1 + t.abs())
        return phi(t) + t * bell(t), e * (phi(t) + (t * bell(t)).abs()) + lost

    if act == "gelu":
        s, e = slope(z)
        return dy * s, dy.abs() * (e + 2 * U * s.abs())
    gate, up = z.chunk(2, dim=1)
    s, e = slope(gate)
    value = gate * phi(gate)
    lost = dy.abs() * TINY * (1 + gate.abs())                # as above
    return (torch.cat([dy * up * s, dy * value], dim=1),
            torch.cat([(dy * up).abs() * (e + 4 * U * s.abs()),
                       (dy * value).abs() * (phi_error(gate, dtype) + 4 * U) + lost], dim=1))


# ---------------------------------------------------------------- LayerNorm

def layernorm_bwd(dy, h, w, eps, dres):
    """(dx, bound), (dweight, terms, term bounds), dbias for 64-bit inputs."""
    c = h.shape[1]
    mean = h.mean(dim=1, keepdim=True)
    d = h - mean
    rstd = 1 / torch.sqrt((d * d).mean(dim=1, keepdim=True) + eps)
    n, g = d * rstd, dy * w
    mg, mgn = g.mean(dim=1, keepdim=True), (g * n).mean(dim=1, keepdim=True)
    dx = rstd * (g - mg - n * mgn)
    # A row's sums: at most 16 channels a thread, 5 steps in a warp, 32 warps; a few roundings.
    e = 64 * U
    size = h.abs().mean(dim=1, keepdim=True) * rstd          # the mean's error, in deviations
    dn = e * (size + n.abs() + 1)
    er = e * (2 + 2 * size)
    agn, ag = (g * n).abs().mean(dim=1, keepdim=True), g.abs().mean(dim=1, keepdim=True)
    bound = rstd * ((g.abs() + ag) * (e + er) + 3 * n.abs() * agn * (e + er) + dn * agn +
                    n.abs() * (g.abs() * dn).mean(dim=1, keepdim=True))
    if dres is not None:
        dx = dx + dres
        bound = bound + 2 * U * dres.abs()
    bound = bound + 2 * U * dx.abs()
    term, term_bound = dy * n, dy.abs() * (dn + n.abs() * er)
    del c
    return (dx, bound), (term.sum(0), term.abs().sum(0), term_bound.sum(0)), dy.sum(0)


# ---------------------------------------------------------------- dropout

def philox_words(block, seed, offset):
    """The four words of one block, in Python's integers."""
    low = 2 ** 32 - 1
    c = [block & low, block >> 32, offset & low, (offset >> 32) & low]
    k = [seed & low, seed >> 32]
    for _ in range(10):
        p0, p1 = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(p1 >> 32) ^ c[1] ^ k[0], p1 & low, (p0 >> 32) ^ c[3] ^ k[1], p0 & low]
        k = [(k[0] + 0x9E3779B9) & low, (k[1] + 0xBB67AE85) & low]
    return c


def kept(count, seed, offset, p):
    """Which of `count` elements stay, as a bool tensor on the CPU."""
    limit = math.ceil(p * 2 ** 32)
    out = []
    for block in range(-(-count // 4)):
        out += [w >= limit for w in philox_words(block, seed, offset)]
    return torch.tensor(out[:count], dtype=torch.bool)


# ---------------------------------------------------------------- rotary positions

def rope_angles(positions, sections, theta, per_axis):
    cols, pair, half = [], 0, sum(sections)
    for axis, size in enumerate(sections):
        for j in range(size):
            power = j / size if per_axis else pair / half
            cols.append(positions[axis].double() * theta ** -power)
            pair += 1
    return torch.stack(cols, dim=1)


def rope(x, angles):
    """(turned, bound) for 64-bit x [N, H, D] and angles [N, D / 2]. A cosine or sine is off
    by 2 U from its own rounding, pi / 4 U from its argument's and less than U from the angle
    (2^-33 turns, and 2^-52 of the turns that a far position makes, at most 2^31 / 6); two
    products and a sum follow."""
    half = x.shape[2] // 2
    c, s = torch.cos(angles)[:, None], torch.sin(angles)[:, None]
    x1, x2 = x[..., :half], x[..., half:]
    out = torch.cat([x1 * c - x2 * s, x2 * c + x1 * s], dim=2)
    size = x1.abs() + x2.abs()
    return out, 8 * U * torch.cat([size, size], dim=2)
