"""The gated feed-forward products and their gradients in binary64, with bounds on how far the
kernels may be from them.

Sums.  The tensor core adds 16 products at a time to a binary32 sum and truncates: 17 numbers are
aligned to the largest and each is cut by half a step 2^-23 of the running sum's magnitude on
average, which grows to A = sum |a||b| and is half of that on average.  A run of 2048 terms is 128
such additions: 128 * 17 / 4 * 2^-23 * A = 2^-13.9 * A; runs (of a part of it each) are added with
half a step each, fewer than 64 of them here: SUM = 2^-13.8.
The logistic function is within 6.2 * 2^-24, products and sums of a few rounded factors within
16 * 2^-24 of the magnitudes that go in: FEW = 2^-20.
"""
import torch

SUM, FEW = 2.0**-13.8, 2.0**-20
F64 = torch.float64
EPS = {torch.bfloat16: 2.0**-8, torch.float16: 2.0**-11}  # half a step: torch.finfo(t).eps / 2
TINY = {torch.bfloat16: 2.0**-134, torch.float16: 2.0**-25}  # half the smallest subnormal


def d(t):
    return t.to(F64)


def product(a, b):
    """a @ b.T, and the bound of its error."""
    return d(a) @ d(b).t(), SUM * (d(a).abs() @ d(b).abs().t())


def gated(x, w_gate, w_up):
    """g, u, p = silu(g) * u and their bounds before rounding."""
    (g, eg), (u, eu) = product(x, w_gate), product(x, w_up)
    s = torch.sigmoid(g)
    p = g * s * u
    # |d silu / dg| <= 1.1; the rest from the factors' roundings
    ep = 1.1 * eg * (u.abs() + eu) + (g * s).abs() * eu + FEW * p.abs()
    return (g, eg), (u, eu), (p, ep)


def slopes(dp, g, u, eg=0.0, eu=0.0):
    """dg and du, and their bounds before rounding.  |silu''| <= 0.5, |silu'| <= 1.1."""
    s = torch.sigmoid(g)
    ds = s * (1 + g * (1 - s))
    dg, du = d(dp) * u * ds, d(dp) * g * s
    mag = s * (1 + g.abs())  # what 1 - s and the sum cancel in
    a = d(dp).abs()
    return (dg, a * (u.abs() * 0.5 * eg + 1.1 * eu + 0.5 * eg * eu + FEW * u.abs() * mag)), (du, a * (1.1 * eg) + FEW * du.abs())


def gradients(dp, x, w_gate, w_up, g, u, eg=0.0, eu=0.0):
    """{name: (value, bound before rounding)} of dx, dw_gate and dw_up: dg and du are rounded once, to x's type."""
    t = x.dtype
    (dg, e1), (du, e2) = slopes(dp, g, u, eg, eu)
    e1, e2 = e1 + EPS[t] * (dg.abs() + e1) + TINY[t], e2 + EPS[t] * (du.abs() + e2) + TINY[t]
    a1, a2, wg, wu, xx = dg.abs() + e1, du.abs() + e2, d(w_gate), d(w_up), d(x)
    out = {"dx": (dg @ wg + du @ wu, e1 @ wg.abs() + e2 @ wu.abs() + SUM * (a1 @ wg.abs() + a2 @ wu.abs()))}
    out["dw_gate"] = dg.t() @ xx, e1.t() @ xx.abs() + SUM * (a1.t() @ xx.abs())
    out["dw_up"] = du.t() @ xx, e2.t() @ xx.abs() + SUM * (a2.t() @ xx.abs())
    return out


def check(name, got, want, bound):
    """A rounded result against the value and the bound of what was rounded."""
    t = got.dtype
    step = EPS[t] if t in EPS else 2.0**-24
    limit = bound + step * (want.abs() + bound) + TINY.get(t, 2.0**-150)
    off = (d(got) - want).abs()
    worst = float((off - limit).max()) if off.numel() else 0.0
    assert torch.isfinite(d(got)).all() and worst <= 0, f"{name}: {worst} over the bound, {float(off.max())} off"


def inputs(rows, width, hidden, dtype, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, sigma=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * sigma).to(dtype)

    return (normal(rows, width), normal(hidden, width, sigma=width**-0.5), normal(hidden, width, sigma=width**-0.5),
            normal(rows, hidden, sigma=0.05))


def tiles(n):
    return -(-n // 128)


def codes(v, block, fp8=torch.float8_e4m3fn):
    """Codes and scales of float32 rows as the library's block rules give them (finite values)."""
    rows, cols = v.shape
    top, emax = (448.0, 8) if fp8 == torch.float8_e4m3fn else (57344.0, 15)
    t = torch.nn.functional.pad(v, (0, -cols % block)).view(rows, -1, block)
    amax = t.abs().amax(2, keepdim=True)
    if block == 128:
        scale, mul = amax / top, torch.where(amax > 0, top / amax, 0.0)
        return (t * mul).clamp(-top, top).view(rows, -1)[:, :cols].to(fp8), scale[..., 0]
    e = (torch.frexp(amax.clamp(min=2.0**-126))[1] - 1 - emax).clamp(min=-127)
    c = torch.ldexp(t, -e).clamp(-top, top).view(rows, -1)[:, :cols].to(fp8)
    return c, (e[..., 0] + 127).to(torch.uint8)


def close_codes(name, got, scales, value, bound, block, fp8=torch.float8_e4m3fn):
    """FP8 codes with their scales against a value and the bound of its error: the stored scale within what the
    bound allows, every code at most half a step (plus that error) from the value that it stands for."""
    rows, cols = value.shape
    top = 448.0 if fp8 == torch.float8_e4m3fn else 57344.0
    half, least = (2.0**-4, 2.0**-10) if fp8 == torch.float8_e4m3fn else (2.0**-3, 2.0**-17)  # relative, of subnormals
    t = torch.nn.functional.pad(value, (0, -cols % block)).view(rows, -1, block)
    amax = t.abs().amax(2)
    off = torch.nn.functional.pad(bound, (0, -cols % block)).view(rows, -1, block).amax(2)
    if block == 128:
        s = d(scales.view(rows, -1))
        assert ((s * top - amax).abs() <= off + 2.0**-23 * (amax + off)).all(), name
    else:
        e = scales.view(torch.uint8).view(rows, -1).to(F64) - 127
        s = torch.exp2(e)
        emax = 8 if fp8 == torch.float8_e4m3fn else 15
        low, high = (amax - off).clamp(min=0), amax + off  # floor(log2) of something in between
        assert (torch.exp2(e + emax) <= high).all() or float(amax.min()) == 0.0, name
        assert (torch.exp2(e + emax + 1) > low).all(), name
    s = s.repeat_interleave(block, 1)[:, :cols]
    v = d(got.view(fp8).float()) * s
    top_v = top * s  # mx: what is above saturates
    want = torch.minimum(torch.maximum(value, -top_v), top_v)
    limit = bound + (half + 2.0**-20) * (want.abs() + bound) + least * s * (1 + 2.0**-20)
    worst = float(((v - want).abs() - limit).max())
    assert worst <= 0, f"{name}: {worst} over the bound"
