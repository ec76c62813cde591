"""Plain 64-bit implementations of the training operators, for their tests
(numpy and torch on the CPU; no library code)."""
import math

import numpy as np
import torch

# Half the distance between neighbours, relative: what one rounding costs
# (2^-p for p significant bits: 53, 24, 8, 11).
UNIT = {torch.float64: 2.0 ** -53, torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8,
        torch.float16: 2.0 ** -11}


def assert_rounded(got, ref, dtype, what, sums=1e-5, terms=0.0):
    """got is ref computed in fp32 (fp64) and rounded once to dtype: each element
    within one rounding, beside `sums` of the largest magnitude for the arithmetic
    (1e-5 / 1e-11, the accuracy stated for sums over rows of this length).
    `terms`: the size of what is subtracted where ref is a difference.
    binary16 spaces its subnormals by 2^-24, half of which is added."""
    got = got.detach().cpu().double()
    ref = ref.detach().cpu().double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    if not ref.numel():
        return
    assert torch.isfinite(ref).all(), what
    assert torch.isfinite(got).all(), what
    if dtype == torch.float64:
        sums = 1e-11
    tol = 1.001 * UNIT[dtype] * ref.abs() + sums * max(ref.abs().max().item(), terms)
    if dtype == torch.float16:
        tol = tol + 2.0 ** -25
    off = ((got - ref).abs() - tol).max().item()
    assert off <= 0, f"{what}: beyond the tolerance by {off:.3e} (largest {ref.abs().max():.3e})"


def parse(irreps):
    return [(int(t.split("x")[0]), int(t.split("x")[1][:-1])) for t in irreps.split("+")]


def per_component(v, irreps):
    """A value per irrep and channel at each element of a row."""
    out, at = [], 0
    for m, l in parse(irreps):
        out.append(v[..., at:at + m].repeat(*([1] * (v.dim() - 1)), 2 * l + 1))
        at += m
    return torch.cat(out, -1)


def norm(x, weight, irreps, eps):
    out, at = [], 0
    for m, l in parse(irreps):
        d = m * (2 * l + 1)
        p = x[:, at:at + d]
        out.append(p / torch.sqrt((p * p).sum(1, keepdim=True) / d + eps))
        at += d
    y = torch.cat(out, 1)
    return y if weight is None else y * per_component(weight, irreps)


def norm_grad_terms(x, g, weight, irreps, eps):
    """The size of the two terms whose difference is a gradient through norm():
    r weight g and its mean's part.  They cancel in an irrep of one element."""
    if not x.numel():
        return 0.0
    x = x.detach()
    g = g if weight is None else g * per_component(weight.detach(), irreps)
    return (g.abs() * row_scale(x, irreps, eps)).max().item()


def row_scale(x, irreps, eps):
    """1 / sqrt(mean square + eps) of its irrep at each element."""
    out, at = [], 0
    for m, l in parse(irreps):
        d = m * (2 * l + 1)
        p = x[:, at:at + d]
        out.append(((p * p).sum(1, keepdim=True) / d + eps).rsqrt().expand_as(p))
        at += d
    return torch.cat(out, 1)


def residual(x, b, weight, gate, scale, irreps, eps):
    t = norm(b, weight, irreps, eps)
    if scale is not None:
        t = t * per_component(scale, irreps)
    if gate is not None:
        t = t * per_component(torch.sigmoid(gate), irreps)
    return t if x is None else x + t


def embed_grad(index, g, v, scale):
    out = torch.zeros(v, g.shape[1], dtype=torch.float64)
    for i, row in zip(index.tolist(), g.double()):
        if 0 <= i < v:
            out[i] += row
    return out * scale


# ----------------------------------------------------------- 8-bit states --

def mix32(h):
    h = h & 0xFFFFFFFF
    h = (h ^ (h >> 16)) * 0x85EBCA6B & 0xFFFFFFFF
    h = (h ^ (h >> 13)) * 0xC2B2AE35 & 0xFFFFFFFF
    return h ^ (h >> 16)


def noise(seed, step, tensor, numel):
    """The two 16-bit random numbers of each element, as fractions in (0, 1)."""
    key = mix32(mix32(mix32(seed) ^ (seed >> 32)) + step)
    key = mix32(mix32(key + tensor))
    h = [mix32(k ^ key) for k in range(numel)]
    um = np.array([(x >> 16) + 0.5 for x in h]) / 65536
    uv = np.array([(x & 0xFFFF) + 0.5 for x in h]) / 65536
    return um, uv


def grid(ebits):
    """The magnitudes of the 2^(ebits+3) codes under a power of two of 1."""
    v = [f for f in range(8)]
    for e in range(1, 2 ** ebits):
        v += [(8 + f) * 2.0 ** (e - 1) for f in range(8)]
    return np.array(v, dtype=np.float64) * 2.0 ** (-(2 ** ebits) - 2)


def code_value(codes, exps, ebits):
    """What 8-bit states stand for."""
    codes = np.asarray(codes).astype(np.int64).reshape(-1, 256)
    scale = 2.0 ** (np.asarray(exps).astype(np.float64)[:, None] - 128)
    n = 2 ** (ebits + 3)
    return (np.where(codes >= n, -1.0, 1.0) * grid(ebits)[codes % n] * scale).reshape(-1)


def encode(x, ebits, u):
    """Codes and exponent bytes of x (a multiple of 256 values): the neighbour
    below, or above where the distance to the one below exceeds 1 - u steps."""
    x = np.asarray(x, dtype=np.float64).reshape(-1, 256)
    u = np.asarray(u).reshape(-1, 256)
    top = np.abs(x).max(1)
    e = np.clip(np.where(top > 0, np.frexp(top)[1], -80), -80, 126)
    g = np.append(grid(ebits), 1.0)  # past the last code: the next power of two
    y = np.abs(x) / 2.0 ** e[:, None]
    lo = np.searchsorted(g, y, side="right") - 1
    lo = np.minimum(lo, len(g) - 2)
    frac = (y - g[lo]) / (g[lo + 1] - g[lo])
    c = np.minimum(lo + (frac + u >= 1), len(g) - 2)
    if ebits == 5:
        c = np.where(x > 0, np.maximum(c, 1), c)
    else:
        c = c + np.where(np.signbit(x), 128, 0)
    return c.astype(np.uint8).reshape(-1), (e + 128).astype(np.uint8)


def adamw(p, g, m, v, lr, b1, b2, eps, wd, t):
    """One step in the precision of the arrays."""
    f = p.dtype.type
    m = m * f(b1) + g * f(1 - b1)
    v = v * f(b2) + (g * g) * f(1 - b2)
    p64, m64, v64 = (a.astype(np.float64) for a in (p, m, v))
    step = (m64 / (1 - b1 ** t)) / (np.sqrt(v64 / (1 - b2 ** t)) + eps)
    return p64 * (1 - lr * wd) - lr * step, m, v


def pad256(a):
    return np.concatenate([a, np.zeros(-len(a) % 256, dtype=a.dtype)])


assert math.isclose(code_value([127] + [0] * 255, [128], 4)[0], 15 / 16)
