"""How far an FP8 value may lie from the exact one it stands for, in units of its scale."""
import torch

# mantissa bits, exponent of the smallest normal, largest value
FORMATS = {torch.float8_e4m3fn: (3, -6, 448.0), torch.float8_e5m2: (2, -14, 57344.0)}


def room(q, rel, f8):
    """Bound of |value - q| for a value rounded to nearest from one within `rel` of q (binary64, any sign): half a
    step of the binade that q is in, and the error itself; above the format's largest value, the distance to it."""
    bits, lowest, top = FORMATS[f8]
    a = q.abs()
    e = torch.frexp(a * (1 + rel))[1] - 1  # a * (1 + rel) in [2^e, 2^(e + 1))
    half = torch.ldexp(torch.ones_like(a), e.clamp(min=lowest) - bits - 1)
    return torch.maximum(half, a - top) + rel * a
