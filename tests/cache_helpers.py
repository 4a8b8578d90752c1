"""Shared by the tests of the rotation and of the 8-bit cache: the definitions in 64 bits.

One rounding to bf16 is half a step (ops_helpers.BF16), one to E4M3 half a step of 2^-3 relative (2^-4), at least half of the
smallest step 2^-9 (in units of the head's power of two)."""
import math

import torch

D = 128


def turn(x, cos, sin, layout):
    """x [tokens, heads, 128] with its first 2 x cos.shape[1] values rotated; cos, sin [tokens, pairs]."""
    r = 2 * cos.shape[1]
    cos, sin = cos[:, None], sin[:, None]
    y = x.clone()
    if layout == "half":
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y[..., :r // 2], y[..., r // 2:r] = a * cos - b * sin, a * sin + b * cos
    else:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y[..., 0:r:2], y[..., 1:r:2] = a * cos - b * sin, a * sin + b * cos
    return y


def cos_sin(positions, frequencies, amplitude=1.0):
    if frequencies is None:
        return None, None
    # (the product is rounded to 53 bits: its fraction of a turn is good to 2^-30 even at 2^20 turns)
    angle = positions.double()[:, None] * frequencies.double()[None]
    return amplitude * angle.cos(), amplitude * angle.sin()


def rotary(x, w, positions, frequencies, layout="half", eps=1e-6, amplitude=1.0):
    """(y, slop): the definition, and the size of what its fp32 arithmetic rounds: a value's own magnitude and its
    partner's."""
    x = x.double()
    if w is not None:
        x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * w.double()
    if frequencies is None:
        return x, x.abs()
    cos, sin = cos_sin(positions, frequencies, amplitude)
    one = torch.full_like(cos, abs(amplitude))
    size = turn(x.abs(), one, -one, layout)  # |a| + |b|, and their difference
    size = torch.maximum(size.abs(), turn(x.abs(), one, one, layout).abs())
    return turn(x, cos, sin, layout), size


def rotary_grad(gy, x, w, positions, frequencies, layout="half", eps=1e-6, amplitude=1.0):
    """(gx, gw, slop of gx, sum of |terms| of gw)."""
    u, usize = gy.double(), gy.double().abs()
    if frequencies is not None:
        cos, sin = cos_sin(positions, frequencies, amplitude)
        one = torch.full_like(cos, abs(amplitude))
        usize = torch.maximum(turn(u.abs(), one, -one, layout).abs(), turn(u.abs(), one, one, layout).abs())
        u = turn(u, cos, -sin, layout)
    if w is None:
        return u, None, usize, None
    x, w = x.double(), w.double()
    rstd = 1 / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
    n = x * rstd
    gx = rstd * (u * w - n * (u * w * n).mean(-1, keepdim=True))
    size = rstd * (usize * w.abs() + n.abs() * (usize * w.abs() * n.abs()).mean(-1, keepdim=True))
    return gx, (u * n).sum((0, 1)), size, (usize * n.abs()).sum((0, 1))


def power(e):
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32).double()


def exponents(x):
    """Of heads [..., 128] (64 bits, finite): the least e with amax <= 448 x 2^e, in [-51, 51]; 0 for zeros."""
    amax = x.abs().amax(-1)
    m, e = torch.frexp(amax)
    return torch.where(amax > 0, (e - 9 + (m > 0.875).int()).clamp(-51, 51), torch.zeros_like(e))


def e4m3(y):
    """The nearest E4M3 value, ties to even, saturating (64 bits)."""
    step = power(torch.frexp(y.abs().clamp(min=2.0 ** -6))[1] - 4)
    return (torch.round(y / step) * step).clamp(-448, 448)


def held(x):
    """What the cache stands for after x was written (64 bits in and out)."""
    p = power(exponents(x))[..., None]
    return e4m3(x / p) * p


def random_cache(rows, hkv, seed=0, spread=3, nan=False, device="cuda"):
    """A cache of random codes (all but NaN, unless asked for) and powers of two."""
    from comm_overlap_gb300 import torch_ops as ops
    g = torch.Generator().manual_seed(seed)
    parts = []
    for _ in range(2):
        c = torch.randint(0, 254, (rows, hkv, D), generator=g)
        c = c + (c >= 127).int()
        c = torch.where((c & 127) > 0x60, c - 0x20, c)  # fewer of the very large
        if nan:
            c = torch.where(torch.rand(c.shape, generator=g) < 0.2, torch.full_like(c, 127), c)
        parts.append(c.to(torch.uint8).to(device).view(torch.float8_e4m3fn))
    for _ in range(2):
        parts.append((torch.randint(-spread, spread + 1, (hkv, rows), generator=g) + 127 - 4).to(torch.uint8).to(device))
    return ops.QuantizedCache(*parts)


def values(cache, name, rows):
    """What the cache holds at rows (a list or tensor), [len(rows), heads, 128] in 64 bits."""
    rows = torch.as_tensor(rows, device=cache.k.device).long()
    codes, e = (cache.k, cache.k_exp) if name == "k" else (cache.v, cache.v_exp)
    return codes.view(torch.uint8)[rows].view(torch.float8_e4m3fn).to(torch.float32).double() * power(e[:, rows].t().int() - 127)[..., None]


SQRT_D = math.sqrt(D)
