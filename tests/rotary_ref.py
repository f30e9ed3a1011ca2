"""The rotation of heads and the norm before it in 64 bits, from the formulas."""
import math

import torch

D = 128


def frequencies(rot_dim, base=10000.0, scaling=None, factor=1.0, original=4096.0, low=1.0, high=None):
    """Radians a token of each pair, in Python floats."""
    high = high if high is not None else (32.0 if scaling == "yarn" else 4.0)
    if scaling == "ntk":
        base = base * factor ** (rot_dim / (rot_dim - 2))
    out = []
    for i in range(rot_dim // 2):
        theta = base ** (-2 * i / rot_dim)
        if scaling == "linear":
            theta /= factor
        if scaling in ("yarn", "banded"):
            if scaling == "yarn":
                edge = [rot_dim * math.log(original / (n * 2 * math.pi)) / (2 * math.log(base)) for n in (high, low)]
                first, last = max(math.floor(edge[0]), 0), min(math.ceil(edge[1]), rot_dim - 1)
                keep = 1 - (i - first) / max(last - first, 1e-3)
            else:
                keep = (original * theta / (2 * math.pi) - low) / (high - low)
            keep = min(max(keep, 0.0), 1.0)
            theta = theta / factor * (1 - keep) + theta * keep
        out.append(theta)
    return out


def rotated(x, positions, theta, interleaved, amplitude=1.0, weight=None, eps=1e-6):
    """(out, slack): the rows x [T, H, 128] normed and rotated in 64 bits, and
    A (|a| + |b|) of each element's pair (|y| where nothing is rotated): what errors of
    the fp32 arithmetic are proportional to."""
    y = x.double()
    if weight is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * weight.double()
    if theta is None:
        return y, y.abs()
    r = 2 * len(theta)
    # the angle modulo a turn, in exact whole numbers: positions may be far
    turns = [int(t / (2 * math.pi) * 2 ** 64) for t in theta]
    angle = torch.tensor([[p * f % 2 ** 64 / 2 ** 64 * 2 * math.pi for f in turns] for p in positions.tolist()],
                         dtype=torch.float64, device=x.device).view(-1, 1, r // 2)
    c, s = amplitude * torch.cos(angle), amplitude * torch.sin(angle)
    i = torch.arange(r // 2, device=x.device)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + r // 2)
    a, b = y[..., ia], y[..., ib]
    out, slack = y.clone(), y.abs()
    out[..., ia], out[..., ib] = a * c - b * s, b * c + a * s
    slack[..., ia] = slack[..., ib] = abs(amplitude) * (a.abs() + b.abs())
    return out, slack


def bound(out, slack):
    """A result is rounded to bf16 (half a step: 2^-8 relative). In fp32 before that: the
    sum of squares of 128 terms in 11 levels and its root (11 + 3 roundings of 2^-24),
    two products for the norm; the angle as a signed 32-bit fraction of a turn rounded to
    24 bits (2 pi 2^-26), sincospif (2 units of 2^-24), the amplitude, a product and an
    fma: in all below 32 roundings of 2^-24 of |a| + |b|."""
    return 2 ** -8 * (out.abs() + 2 ** -19 * slack) + 2 ** -19 * slack
