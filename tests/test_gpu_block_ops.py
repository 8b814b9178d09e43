"""GPU tests of the block operators with 8-bit outputs and checkpoints:
rmsnorm_residual_fp8 / rmsnorm_residual_backward, swiglu_fp8 / swiglu_backward.

Two kinds of comparison.  What is a rounding of values that the test can form
itself (the stream h, the checkpoints, the codes of the norm given its rstd)
has to be equal bit for bit: to the library's own blockwise cast or to the
oracle.  What contains a sum, a square root or an exponential is compared with
a plain implementation in 64 bits, within bounds counted in roundings of
binary32 (EPS = 2^-24) plus the rounding of the output type:

* a sum of n positive terms in binary32 whose longest chain of additions is D
  long is within D * EPS of itself, relative; a signed one within D * EPS of
  the sum of magnitudes;
* exp(-g) through a base-2 exponential is within (|g| + 8) EPS, relative.
"""
import numpy as np
import pytest
import torch

import oracle as O

import mixed_precision_numerics_gb300 as M  # noqa: E402

pytestmark = pytest.mark.gpu
EPS = 2.0**-24
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
OUT_EPS = {torch.float32: 2.0**-24, torch.float16: 2.0**-11, torch.bfloat16: 2.0**-8}  # half a step, relative, and some
OUT_TINY = {torch.float32: 2.0**-140, torch.float16: 2.0**-24, torch.bfloat16: 2.0**-130}
FP8 = {M.MP_E4M3: (O.E4M3, torch.float8_e4m3fn, 448.0, 2.0**-4, 2.0**-10),
       M.MP_E5M2: (O.E5M2, torch.float8_e5m2, 57344.0, 2.0**-3, 2.0**-17)}
SENTINEL = 0xA5
# longest chain of additions in a row's sum: at most 64 elements a thread, a warp's 5, the warps' 5, and the mean
ROW_CHAIN = 64 + 5 + 5 + 2


@pytest.fixture(autouse=True)
def _gpu(cuda_ok):
    yield


def normal(seed, *shape, sigma=1.0, dtype=torch.float32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * sigma).to(dtype)


class Guarded:
    """An output between two bands that must stay as they are."""

    def __init__(self, shape, dtype=torch.uint8, band=2048):
        n = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
        self.raw = torch.full((band + n + band,), SENTINEL, dtype=torch.uint8, device="cuda")
        self.t = self.raw[band:band + n].view(dtype).view(shape)
        self.band = band

    def check(self):
        assert bool((self.raw[:self.band] == SENTINEL).all()) and bool((self.raw[-self.band:] == SENTINEL).all())


def tiles(cols):
    return -(-cols // 128)


def bits(t):
    return t.contiguous().view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


def assert_bits(a, b, what):
    a, b = bits(a), bits(b)
    assert torch.equal(a, b), f"{what}: {int((a != b).sum())} of {a.numel()} differ"


def scale_outputs(rows, cols, block):
    if block == 32:
        return Guarded((rows, cols // 32))
    return Guarded((rows, tiles(cols)), torch.float32)


def oracle_cast(v, fp8, block):
    """The oracle's codes and scales of a float32 tensor."""
    x = v.cpu().numpy()
    if block == 128:
        return O.fp8_quantize_blockwise(x, O.F32, 1, 128, FP8[fp8][0])
    c, s, _ = O.mx_quantize(x, O.F32, FP8[fp8][0], want_dequant=False)
    return c, s


def dequantise(codes, scales):
    cols = codes.shape[-1]
    return codes.view(torch.float8_e4m3fn).double() * scales.double().repeat_interleave(128, -1)[..., :cols]


# ---- forward norm ----------------------------------------------------------------------


def norm(x, w, *, residual=None, eps=1e-5, fp8=M.MP_E4M3, block=128, save=True, want_h=True):
    rows, cols = x.shape
    o = dict(y=Guarded((rows, cols)), y_scales=scale_outputs(rows, cols, block), rstd=Guarded((rows,), torch.float32))
    if want_h:
        o["h"] = Guarded((rows, cols), x.dtype)
    if save:
        o["ckpt"], o["ckpt_scales"] = Guarded((rows, cols)), Guarded((rows, tiles(cols)), torch.float32)
    t = {k: v.t for k, v in o.items()}
    M.rmsnorm_residual_fp8(x, w, t["y"], t["y_scales"], residual=residual, h=t.get("h"), rstd=t["rstd"],
                           ckpt=t.get("ckpt"), ckpt_scales=t.get("ckpt_scales"), eps=eps, fp8_dtype=fp8,
                           scale_block=block)
    torch.cuda.synchronize()
    for v in o.values():
        v.check()
    return t


def check_norm(x, w, residual, o, eps, fp8, block):
    h = x if residual is None else (x.float() + residual.float()).to(x.dtype)
    if "h" in o:
        assert_bits(o["h"], h, "h")
    if "ckpt" in o:
        c, s = torch.empty_like(o["ckpt"]), torch.empty_like(o["ckpt_scales"])
        M.fp8_quantize_blockwise(h.contiguous(), c, s)
        assert_bits(o["ckpt"], c, "checkpoint codes")
        assert_bits(o["ckpt_scales"], s, "checkpoint scales")
    want = 1.0 / torch.sqrt(h.double().square().mean(1) + eps)
    # the root halves the sum's relative error; its own operations add a few roundings
    assert bool(((o["rstd"].double() - want).abs() <= (ROW_CHAIN / 2 + 4) * EPS * want).all())
    v = (h.float() * o["rstd"][:, None]) * w.float()  # given rstd, each value is two roundings
    rc, rs = oracle_cast(v, fp8, block)
    np.testing.assert_array_equal(o["y_scales"].cpu().numpy().view(rs.dtype), rs)
    np.testing.assert_array_equal(o["y"].cpu().numpy(), rc)


SHAPES = [(1, 32), (1, 4096), (3, 96), (33, 128), (5, 160), (17, 256), (2, 544), (7, 1056), (129, 512), (4, 2080),
          (3, 5120), (2, 8224), (2, 16384), (1, 12320)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("block", [128, 32])
def test_norm_forward(shape, dtype, block):
    rows, cols = shape
    dt = TYPES[dtype]
    x, r = normal(rows + cols, rows, cols, dtype=dt), normal(2, rows, cols, sigma=3.0, dtype=dt)
    r[:, :: 37] *= 20.0
    w = 1.0 + normal(3, cols, sigma=0.2)
    fp8 = M.MP_E5M2 if rows % 2 else M.MP_E4M3
    o = norm(x, w, residual=r, fp8=fp8, block=block)
    check_norm(x, w, r, o, 1e-5, fp8, block)


@pytest.mark.parametrize("cols", [16, 48, 1040, 4112, 14352])
def test_norm_rows_that_end_inside_a_tile(cols):
    x, w = normal(5, 9, cols, dtype=torch.bfloat16), normal(6, cols).to(torch.bfloat16)
    o = norm(x, w)
    check_norm(x, w, None, o, 1e-5, M.MP_E4M3, 128)


@pytest.mark.parametrize("wt", TYPES)
@pytest.mark.parametrize("dtype", TYPES)
def test_norm_weight_types_and_optional_outputs(dtype, wt):
    x, w = normal(7, 21, 384, dtype=TYPES[dtype]), normal(8, 384).to(TYPES[wt])
    o = norm(x, w, residual=x, save=False, want_h=False, eps=1e-2)
    check_norm(x, w, x, o, 1e-2, M.MP_E4M3, 128)
    y, ys = torch.empty(21, 384, dtype=torch.uint8, device="cuda"), torch.empty(21, 3, device="cuda")
    M.rmsnorm_residual_fp8(x, w, y, ys, residual=x, eps=1e-2)
    assert_bits(y, o["y"], "codes without rstd")


@pytest.mark.parametrize("cols", [272, 512, 576, 1040, 2064, 4096, 5120, 8208, 16384])
@pytest.mark.parametrize("dtype", TYPES)
def test_a_row_does_not_depend_on_the_number_of_rows(dtype, cols):
    """Layouts that are chosen by the number of rows give the same bits, forward and for dx."""
    rows, few = 2800 if cols < 4096 else 1900, 5
    x, dy = normal(50, rows, cols, dtype=TYPES[dtype]), normal(51, rows, cols, dtype=TYPES[dtype])
    w = (1.0 + normal(52, cols, sigma=0.3)).to(TYPES[dtype])
    a = norm(x, w, residual=dy)
    da, _ = norm_backward(dy, w, a["rstd"], ckpt=a["ckpt"], scales=a["ckpt_scales"], dh=x)
    for part in (slice(0, few), slice(rows - few, rows)):
        xs, dys = x[part].clone(), dy[part].clone()
        b = norm(xs, w, residual=dys)
        for k in ("h", "rstd", "y", "y_scales", "ckpt", "ckpt_scales"):
            assert_bits(a[k][part], b[k], k)
        db, _ = norm_backward(dys, w, b["rstd"], ckpt=b["ckpt"], scales=b["ckpt_scales"], dh=xs)
        assert_bits(da[part], db, "dx")


@pytest.mark.parametrize("cols", [272, 384, 528, 640, 768, 896, 1152, 1280, 1408, 1664, 1792, 1920, 2048])
@pytest.mark.parametrize("dtype", TYPES)
def test_norm_of_rows_of_whole_tiles(dtype, cols):
    """Rows that share a CTA, and numbers of them that end inside one."""
    for rows in (1, 2, 3, 5, 163):
        for block in (128, 32) if cols % 32 == 0 else (128,):
            test_norm_forward((rows, cols), dtype, block)


def test_norm_writes_the_stream_over_its_input():
    x, r = normal(9, 13, 1040, dtype=torch.bfloat16), normal(10, 13, 1040, dtype=torch.bfloat16)
    w = normal(11, 1040)
    o = norm(x, w, residual=r)
    for in_place in ("x", "residual"):
        a, b = x.clone(), r.clone()
        y, ys = torch.empty_like(o["y"]), torch.empty_like(o["y_scales"])
        M.rmsnorm_residual_fp8(a, w, y, ys, residual=b, h=a if in_place == "x" else b)
        assert_bits(a if in_place == "x" else b, o["h"], "h")
        assert_bits(y, o["y"], "codes")


@pytest.mark.parametrize("block", [128, 32])
@pytest.mark.parametrize("dtype", TYPES)
def test_norm_of_infinities_nans_and_zeros(dtype, block):
    """A row with a NaN or an infinity has no finite norm; the other rows keep theirs."""
    dt = TYPES[dtype]
    x = normal(12, 12, 640, dtype=dt)
    x[1, 5], x[2, 130], x[3, 639], x[4] = float("nan"), float("inf"), float("-inf"), 0.0
    x[5, ::2] = -0.0
    x[6, :128] = 0.0
    x[7, 0] = -float("nan")
    w = normal(13, 640)
    w[3], w[200] = 0.0, -0.0
    o = norm(x, w, block=block)
    check_rows = [0, 4, 5, 6, 8, 9, 10, 11]
    sub = {k: v[check_rows].contiguous() for k, v in o.items()}
    check_norm(x[check_rows].contiguous(), w, None, sub, 1e-5, M.MP_E4M3, block)
    c, s = torch.empty_like(o["ckpt"]), torch.empty_like(o["ckpt_scales"])
    M.fp8_quantize_blockwise(x, c, s)  # the checkpoint holds non-finite tiles as the cast does
    assert_bits(o["ckpt"], c, "checkpoint codes")
    assert_bits(o["ckpt_scales"], s, "checkpoint scales")
    rstd = o["rstd"].cpu()
    assert torch.isnan(rstd[[1, 7]]).all() and (rstd[[2, 3]] == 0).all()
    v = ((x.float() * o["rstd"][:, None]) * w).cpu()
    for r in (1, 2, 3, 7):
        rc, rs = oracle_cast(v[r:r + 1], M.MP_E4M3, block)
        np.testing.assert_array_equal(o["y_scales"][r:r + 1].cpu().numpy().view(np.uint8),
                                      np.ascontiguousarray(rs).view(np.uint8))
        # a NaN that arithmetic makes has no defined sign
        np.testing.assert_array_equal(o["y"][r:r + 1].cpu().numpy() & 0x7F, rc & 0x7F)


def test_norm_of_zero_rows_without_eps_is_nan():
    x = torch.zeros(2, 256, dtype=torch.bfloat16, device="cuda")
    o = norm(x, torch.ones(256, device="cuda"), eps=0.0)
    assert bool(torch.isinf(o["rstd"]).all()) and bool((o["y"] & 0x7F == 0x7F).all())
    o = norm(x, torch.ones(256, device="cuda"))
    assert not o["y"].any() and not o["y_scales"].any() and not o["ckpt"].any()


def test_tiles_below_the_multipliers_range_become_zeros():
    """448 / amax overflows for an amax below 448 / FLT_MAX: the tile's codes are zeros, none of them NaN."""
    x = torch.zeros(1, 384, dtype=torch.float32, device="cuda")
    x[0, :4] = torch.tensor([1e-37, -1e-37, 0.0, 5e-38])
    x[0, 128:132] = torch.tensor([2e-36, -2e-36, 0.0, 1e-36])
    x[0, 256] = 1.0
    o = norm(x, torch.ones(384, device="cuda"))
    assert not (o["ckpt"][0, :128] & 0x7F).any()  # the sign of each element stays
    d = dequantise(o["ckpt"], o["ckpt_scales"])[0, 128:132].cpu()
    want = torch.tensor([2e-36, -2e-36, 0.0, 1e-36], dtype=torch.float64)
    assert ((d - want).abs() <= 2.0**-4 * want.abs() + 2.0**-149 * 448).all()


def test_norm_long_rows_count():
    """More rows than one wave of CTAs, of each row layout."""
    for rows, cols in ((70_001, 32), (9_001, 144), (2_003, 1040)):
        x, w = normal(14, rows, cols, dtype=torch.bfloat16), normal(15, cols)
        o = norm(x, w)
        check_norm(x, w, None, o, 1e-5, M.MP_E4M3, 128)


# ---- backward norm ----------------------------------------------------------------------


def norm_backward(dy, w, rstd, *, h=None, ckpt=None, scales=None, dh=None, dw_type=torch.float32, in_place=None):
    rows, cols = dy.shape
    dx, dw = Guarded((rows, cols), dy.dtype), Guarded((cols,), dw_type)
    ws = Guarded((M.rmsnorm_workspace_size(rows, cols),))
    out = dx.t if in_place is None else in_place
    M.rmsnorm_residual_backward(dy, w, rstd, out, dw.t, ws.t, h=h, ckpt=ckpt, ckpt_scales=scales, dh=dh)
    torch.cuda.synchronize()
    for b in (dx, dw, ws):
        b.check()
    return out, dw.t


def check_norm_backward(dy, w, rstd, v, dh, dx, dw):
    rows, cols = dy.shape
    d, r = dy.double(), rstd.double()[:, None]
    xh, g = v.double() * r, dy.double() * w.double()
    c, c_abs = (g * xh).mean(1, keepdim=True), (g * xh).abs().mean(1, keepdim=True)
    e = 0.0 if dh is None else dh.double()
    want = r * (g - xh * c) + e
    room = EPS * (8 * (r * g.abs() + (r * xh * c).abs() + abs(e)) + (ROW_CHAIN + 4) * (r * xh).abs() * c_abs)
    room = room + OUT_EPS[dx.dtype] * want.abs() + OUT_TINY[dx.dtype]
    off = (dx.double() - want).abs()
    assert bool((off <= room).all()), f"dx off by {float((off / room).max()):.2f} of the bound"
    want, mag = (d * xh).sum(0), (d * xh).abs().sum(0)
    # rows of one CTA in turn, then at most 608 partial sums in 16 chains, and the joins of both
    chain = -(-rows // min(max(rows // 32, 1), 608)) + 32 + 608 // 16 + 16 + 4
    room = chain * EPS * mag + OUT_EPS[dw.dtype] * want.abs() + OUT_TINY[dw.dtype]
    off = (dw.double() - want).abs()
    assert bool((off <= room).all()), f"dweight off by {float((off / room).max()):.2f} of the bound"


BWD_SHAPES = [(1, 16), (1, 4096), (2, 48), (65, 128), (33, 240), (301, 512), (40, 1040), (700, 2064), (9, 5120),
              (3, 8208), (5, 16384), (2, 12304), (5000, 32)]


@pytest.mark.parametrize("shape", BWD_SHAPES)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("saved", [True, False])
def test_norm_backward(shape, dtype, saved):
    rows, cols = shape
    dt = TYPES[dtype]
    h, dy = normal(20, rows, cols, sigma=2.0, dtype=dt), normal(21, rows, cols, sigma=0.1, dtype=dt)
    dh = normal(22, rows, cols, sigma=0.1, dtype=dt)
    w = (1.0 + normal(23, cols, sigma=0.3)).to(dt)
    o = norm(h, w)
    if saved:
        v = dequantise(o["ckpt"], o["ckpt_scales"])
        dx, dw = norm_backward(dy, w, o["rstd"], ckpt=o["ckpt"], scales=o["ckpt_scales"], dh=dh)
    else:
        v = h
        dx, dw = norm_backward(dy, w, o["rstd"], h=h, dh=dh)
    check_norm_backward(dy, w, o["rstd"], v, dh, dx, dw)


@pytest.mark.parametrize("shape", [(100_003, 32), (20_011, 208), (9001, 512), (6007, 1040), (3001, 4096), (330, 16384)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("saved", [True, False])
def test_norm_backward_of_many_rounds(shape, dtype, saved):
    """So many rows that every stage of a team's rings is filled several times."""
    test_norm_backward(shape, dtype, saved)


@pytest.mark.parametrize("dw_type", TYPES)
@pytest.mark.parametrize("wt", TYPES)
def test_norm_backward_weight_types_without_stream_gradient(wt, dw_type):
    h, dy = normal(24, 50, 208, dtype=torch.float16), normal(25, 50, 208, sigma=0.5, dtype=torch.float16)
    w = normal(26, 208).to(TYPES[wt])
    rstd = norm(h, w)["rstd"]
    dx, dw = norm_backward(dy, w, rstd, h=h, dw_type=TYPES[dw_type])
    check_norm_backward(dy, w, rstd, h, None, dx, dw)


@pytest.mark.parametrize("cols", [96, 1040])
def test_norm_backward_in_place_and_repeatable(cols):
    h, dy, dh = (normal(27 + i, 65, cols, dtype=torch.bfloat16) for i in range(3))
    w = normal(31, cols)
    rstd = norm(h, w)["rstd"]
    dx, dw = norm_backward(dy, w, rstd, h=h, dh=dh)
    for which in range(3):
        t = [dy.clone(), dh.clone(), h.clone()]
        got, gw = norm_backward(t[0], w, rstd, h=t[2], dh=t[1], in_place=t[which])
        assert_bits(got, dx, "dx")
        assert_bits(gw, dw, "dweight")


def test_norm_backward_against_differences():
    """The gradient of sum(dy * norm(h) * w) + sum(dh * h) by central differences in 64 bits."""
    rows, cols, eps, step = 3, 80, 1e-3, 1e-5
    x, dy, dh = normal(40, rows, cols), normal(41, rows, cols), normal(42, rows, cols)
    w = 1.0 + normal(43, cols, sigma=0.5)
    rstd = norm(x, w, eps=eps)["rstd"]
    dx, dw = norm_backward(dy, w, rstd, h=x, dh=dh)

    def loss(a, b):
        return (dy.double() * a * torch.rsqrt(a.square().mean(1, keepdim=True) + eps) * b + dh.double() * a).sum()

    a, b = x.double(), w.double()
    for r, c in ((0, 0), (1, 17), (2, 79), (0, 40)):
        d = torch.zeros_like(a)
        d[r, c] = step
        want = float(loss(a + d, b) - loss(a - d, b)) / (2 * step)
        assert abs(float(dx[r, c]) - want) <= 1e-5 * (1 + abs(want))  # binary32 sums; the differences are good to 1e-9
    for c in (0, 17, 79):
        d = torch.zeros_like(b)
        d[c] = step
        want = float(loss(a, b + d) - loss(a, b - d)) / (2 * step)
        assert abs(float(dw[c]) - want) <= 1e-5 * (1 + abs(want))


@pytest.mark.parametrize("cols", [528, 640, 768, 1152, 1280, 1536, 1552, 2064, 4096, 4112])
@pytest.mark.parametrize("dtype", TYPES)
def test_norm_backward_of_pairs_of_rows(dtype, cols):
    """Rows that come to a team two at a time, and the lengths next to that rule; a last row alone."""
    for rows in (1, 2, 3, 303, 304, 305, 1217):
        for saved in (True, False):
            test_norm_backward((rows, cols), dtype, saved)


@pytest.mark.parametrize("cols", [256, 1040, 5120])
@pytest.mark.parametrize("bad", [0, 7, 8, 610])
def test_norm_backward_keeps_a_nonfinite_row_to_itself(cols, bad):
    rows = 611
    h, dy = normal(46, rows, cols, dtype=torch.bfloat16), normal(47, rows, cols, dtype=torch.bfloat16)
    w = torch.ones(cols, device="cuda")
    rstd = norm(h, w)["rstd"]
    want, _ = norm_backward(dy, w, rstd, h=h)
    want = want.clone()
    dy[bad, 3] = float("inf")
    dx, dw = norm_backward(dy, w, rstd, h=h)
    keep = torch.arange(rows, device="cuda") != bad
    assert_bits(dx[keep], want[keep], "dx of the other rows")
    assert not bool(torch.isfinite(dx[bad]).any())
    assert bool(torch.isfinite(dw).sum() == cols - 1)


def test_no_wait_gave_up():
    assert M.mp_wait_failures() == 0


def test_norm_backward_of_no_rows_and_of_nonfinite_rows():
    dw = torch.full((64,), 7.0, dtype=torch.bfloat16, device="cuda")
    e = torch.empty(0, 64, device="cuda")
    M.rmsnorm_residual_backward(e, torch.ones(64, device="cuda"), torch.empty(0, device="cuda"), e, dw,
                                torch.empty(0, dtype=torch.uint8, device="cuda"), h=e)
    assert not dw.any()
    h, dy = normal(44, 6, 256), normal(45, 6, 256)
    h[2, 3] = float("nan")
    w = torch.ones(256, device="cuda")
    rstd = norm(h, w)["rstd"]
    dx, dw = norm_backward(dy, w, rstd, h=h)
    keep = [0, 1, 3, 4, 5]
    assert bool(torch.isnan(dx[2]).all()) and bool(torch.isfinite(dx[keep]).all())
    assert bool(torch.isnan(dw).all())  # the row's rstd is NaN, so every column's sum is


# ---- SwiGLU -----------------------------------------------------------------------------


def halves(seed, rows, cols, dtype, sigma=2.0):
    t = normal(seed, rows, 2 * cols, sigma=sigma, dtype=dtype)
    return t[:, :cols], t[:, cols:]


def swiglu(g, u, *, fp8=M.MP_E4M3, block=128, save=True):
    rows, cols = g.shape
    o = dict(y=Guarded((rows, cols)), y_scales=scale_outputs(rows, cols, block))
    if save:
        o["ckpt"], o["ckpt_scales"] = Guarded((2, rows, cols)), Guarded((2, rows, tiles(cols)), torch.float32)
    t = {k: v.t for k, v in o.items()}
    M.swiglu_fp8(g, u, t["y"], t["y_scales"], ckpt=t.get("ckpt"), ckpt_scales=t.get("ckpt_scales"), fp8_dtype=fp8,
                 scale_block=block)
    torch.cuda.synchronize()
    for v in o.values():
        v.check()
    return t


def check_swiglu(g, u, o, fp8, block):
    rows, cols = g.shape
    if "ckpt" in o:
        for k, t in enumerate((g, u)):
            c = torch.empty(rows, cols, dtype=torch.uint8, device="cuda")
            s = torch.empty(rows, tiles(cols), device="cuda")
            M.fp8_quantize_blockwise(t.contiguous(), c, s)
            assert_bits(o["ckpt"][k], c, "checkpoint codes")
            assert_bits(o["ckpt_scales"][k], s, "checkpoint scales")
    _, f8, top, half, sub = FP8[fp8]
    p = g.double() * torch.special.expit(g.double()) * u.double()
    pad = torch.nn.functional.pad(p, (0, -cols % block)).view(rows, -1, block)
    amax = pad.abs().amax(2)
    # the exponential, the sum below it, the division and two products
    rel = (g.double().abs().max() + 16) * EPS
    if block == 128:
        s = o["y_scales"].double()
        assert bool(((s * top - amax).abs() <= (rel + 2 * EPS) * amax + top * 2.0**-149).all())
    else:
        e = o["y_scales"].to(torch.int32) - 127
        s = torch.ldexp(torch.ones_like(amax), e)
        emax = 8 if fp8 == M.MP_E4M3 else 15
        lo, hi = ((torch.frexp(amax * f)[1] - 1 - emax).clamp(min=-127) for f in (1 - rel, 1 + rel))
        assert bool(((e >= lo) & (e <= hi)).all())
    s = s.repeat_interleave(block, 1)[:, :cols]
    y = o["y"].view(f8).double() * s
    # half a step of the format; a 1x32 block's maximum may lie above the largest code and saturate
    near = (half * (1 + 8 * half) * p.abs()).clamp_min(0) + sub * s + rel * p.abs()
    if block == 32:
        near = torch.maximum(near, p.abs() - top * s)
    off = (y - p).abs()
    assert bool((off <= near).all()), f"y off by {float((off / near).max()):.2f} of the bound"


@pytest.mark.parametrize("shape", [(1, 32), (1, 14336), (3, 96), (37, 160), (129, 1056), (301, 1440), (2, 40_000)])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("block", [128, 32])
def test_swiglu_forward(shape, dtype, block):
    rows, cols = shape
    g, u = halves(50 + rows, rows, cols, TYPES[dtype])
    fp8 = M.MP_E5M2 if cols % 3 else M.MP_E4M3
    o = swiglu(g, u, fp8=fp8, block=block)
    check_swiglu(g, u, o, fp8, block)


@pytest.mark.parametrize("cols", [16, 48, 1456, 2064])
def test_swiglu_dense_rows_that_end_inside_a_tile(cols):
    g, u = (normal(60 + i, 7, cols, dtype=torch.bfloat16) for i in range(2))
    o = swiglu(g, u)
    check_swiglu(g, u, o, M.MP_E4M3, 128)
    y = swiglu(g, u, save=False)
    assert_bits(y["y"], o["y"], "codes without a checkpoint")


def test_swiglu_of_infinities_nans_and_extremes():
    g, u = (normal(62 + i, 8, 256) for i in range(2))
    ok = swiglu(g, u)
    g[1, 3], g[2, 130], u[3, 7], g[4, 0] = float("nan"), float("inf"), float("-inf"), float("-inf")
    g[5, 0], u[5, 0] = float("inf"), 0.0
    o = swiglu(g, u)
    # only the tiles that hold one differ from the finite run
    bad = [(1, 0), (2, 1), (3, 0), (4, 0), (5, 0)]
    for r in range(8):
        for t in range(2):
            if (r, t) not in bad:
                assert_bits(o["y"][r, 128 * t:128 * t + 128], ok["y"][r, 128 * t:128 * t + 128], "codes")
    s = o["y_scales"].cpu()
    assert torch.isnan(s[1, 0]) and torch.isinf(s[2, 1]) and torch.isinf(s[3, 0])
    assert torch.isnan(s[4, 0]) and torch.isnan(s[5, 0])  # -inf * s(-inf) and inf * 0 have no value
    assert int(o["y"][1, 3]) & 0x7F == 0x7F and int(o["y"][2, 130]) & 0x7F == 0x7F
    # gates far below zero give zeros, far above the identity
    g = torch.full((1, 128), -200.0, device="cuda")
    u = torch.ones(1, 128, device="cuda")
    assert not (swiglu(g, u)["y"] & 0x7F).any()
    o = swiglu(-g, u)
    assert bool((o["y"].view(torch.float8_e4m3fn).float() == 448.0).all()) and float(o["y_scales"]) == np.float32(200 / 448)


def swiglu_backward(dp, **kw):
    rows, cols = dp.shape
    d = Guarded((rows, 2 * cols), dp.dtype)
    dg, du = d.t[:, :cols], d.t[:, cols:]
    M.swiglu_backward(dp, dg, du, **kw)
    torch.cuda.synchronize()
    d.check()
    return dg, du


def check_swiglu_backward(dp, g, u, dg, du):
    d, g, u = dp.double(), g.double(), u.double()
    s = torch.special.expit(g)
    rel = (g.abs() + 20) * EPS
    want = d * g * s
    room = (rel + OUT_EPS[du.dtype]) * want.abs() + OUT_TINY[du.dtype]
    assert bool(((du.double() - want).abs() <= room).all())
    want = d * u * (s + g * s * (1 - s))
    room = rel * (d * u).abs() * s * (1 + 2 * g.abs()) + OUT_EPS[dg.dtype] * want.abs() + OUT_TINY[dg.dtype]
    off = (dg.double() - want).abs()
    assert bool((off <= room).all()), f"dgate off by {float((off / room).max()):.2f} of the bound"


@pytest.mark.parametrize("shape", [(1, 16), (1, 14336), (3, 48), (37, 160), (301, 1456), (1000, 144)])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("saved", [True, False])
def test_swiglu_backward(shape, dtype, saved):
    rows, cols = shape
    dt = TYPES[dtype]
    g, u = halves(70 + rows, rows, cols, dt)
    dp = normal(71, rows, cols, sigma=0.3, dtype=dt)
    if saved:
        o = swiglu(g, u)
        g, u = dequantise(o["ckpt"], o["ckpt_scales"])
        dg, du = swiglu_backward(dp, ckpt=o["ckpt"], ckpt_scales=o["ckpt_scales"])
    else:
        dg, du = swiglu_backward(dp, gate=g, up=u)
    check_swiglu_backward(dp, g, u, dg, du)


def test_swiglu_backward_in_place():
    g, u = halves(73, 19, 272, torch.bfloat16)
    dp = normal(74, 19, 272, dtype=torch.bfloat16)
    dg, du = swiglu_backward(dp, gate=g, up=u)
    M.swiglu_backward(dp, g, u, gate=g, up=u)
    assert_bits(g, dg, "dgate")
    assert_bits(u, du, "dup")


def test_swiglu_backward_against_differences():
    g, u, dp = (normal(75 + i, 2, 32, sigma=2.0) for i in range(3))
    dg, du = swiglu_backward(dp, gate=g, up=u)
    step = 1e-5

    def value(a, b):
        return a * torch.special.expit(a) * b

    a, b = g.double(), u.double()
    for got, want in ((dg, (value(a + step, b) - value(a - step, b)) / (2 * step)),
                      (du, (value(a, b + step) - value(a, b - step)) / (2 * step))):
        want = want * dp.double()
        assert bool(((got.double() - want).abs() <= 1e-5 * (1 + want.abs())).all())


# ---- how they are called -----------------------------------------------------------------


def test_calls_on_another_stream_and_in_a_graph():
    x, w = normal(80, 64, 1024, dtype=torch.bfloat16), normal(81, 1024)
    ref = norm(x, w)
    y, ys = torch.zeros_like(ref["y"]), torch.zeros_like(ref["y_scales"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    M.rmsnorm_residual_fp8(x, w, y, ys, stream=side)
    side.synchronize()
    assert_bits(y, ref["y"], "codes")
    dy, dx, dw = normal(82, 64, 1024, dtype=torch.bfloat16), torch.empty_like(x), torch.empty(1024, device="cuda")
    ws = M.new_rmsnorm_workspace(64, 1024)
    g, u = halves(83, 64, 512, torch.bfloat16)
    p, ps = torch.empty(64, 512, dtype=torch.uint8, device="cuda"), torch.empty(64, 4, device="cuda")
    dg, du = torch.empty(2, 64, 512, dtype=torch.bfloat16, device="cuda")
    dp = normal(84, 64, 512, dtype=torch.bfloat16)

    def calls():
        M.rmsnorm_residual_fp8(x, w, y, ys, rstd=ref["rstd"])
        M.rmsnorm_residual_backward(dy, w, ref["rstd"], dx, dw, ws, h=x)
        M.swiglu_fp8(g, u, p, ps)
        M.swiglu_backward(dp, dg, du, gate=g, up=u)

    calls()
    torch.cuda.synchronize()
    want = [t.clone() for t in (y, ys, dx, dw, p, ps, dg, du)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for t in (y, ys, dx, dw, p, ps, dg, du):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip((y, ys, dx, dw, p, ps, dg, du), want):
        assert_bits(a, b, "replayed output")


def test_offsets_beyond_32_bits():
    """A tensor of more than 2^32 elements: its last rows are what a call on them alone gives."""
    rows, cols, tail = 2**18 + 37, 16384, 40
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    x[-tail:] = normal(95, tail, cols, dtype=torch.bfloat16)
    last, w = x[-tail:].clone(), normal(96, cols)
    y = torch.empty(rows, cols, dtype=torch.uint8, device="cuda")
    ys, cs = (torch.empty(rows, 128, device="cuda") for _ in range(2))
    ckpt, rstd = torch.empty_like(y), torch.empty(rows, device="cuda")
    M.rmsnorm_residual_fp8(x, w, y, ys, rstd=rstd, ckpt=ckpt, ckpt_scales=cs)
    o = norm(last, w)
    for got, key in ((y, "y"), (ys, "y_scales"), (rstd, "rstd"), (ckpt, "ckpt"), (cs, "ckpt_scales")):
        assert_bits(got[-tail:], o[key], key)
    assert not (y[:-tail] & 0x7F).any()  # zeros, signed as their weights
    del y, ys
    dx, dw = torch.empty_like(x), torch.empty(cols, device="cuda")
    M.rmsnorm_residual_backward(x, w, rstd, dx, dw, M.new_rmsnorm_workspace(rows, cols), ckpt=ckpt, ckpt_scales=cs)
    want, want_w = norm_backward(last, w, o["rstd"], ckpt=o["ckpt"], scales=o["ckpt_scales"])
    assert_bits(dx[-tail:], want, "dx")
    # other rows add zeros, in other chains of additions
    mag = (last.double() * dequantise(o["ckpt"], o["ckpt_scales"]) * o["rstd"].double()[:, None]).abs().sum(0)
    assert bool(((dw.double() - want_w.double()).abs() <= 2 * (tail + 64) * EPS * mag).all())
    del ckpt, cs, rstd
    half = cols // 2
    g, u = x[:, :half], x[:, half:]
    y, ys = torch.empty(rows, half, dtype=torch.uint8, device="cuda"), torch.empty(rows, 64, device="cuda")
    ckpt, cs = torch.empty(2, rows, half, dtype=torch.uint8, device="cuda"), torch.empty(2, rows, 64, device="cuda")
    M.swiglu_fp8(g, u, y, ys, ckpt=ckpt, ckpt_scales=cs)
    o = swiglu(last[:, :half], last[:, half:])
    assert_bits(y[-tail:], o["y"], "codes")
    assert_bits(ckpt[:, -tail:], o["ckpt"], "checkpoint codes")
    assert_bits(cs[:, -tail:], o["ckpt_scales"], "checkpoint scales")
    dp = torch.zeros(rows, half, dtype=torch.bfloat16, device="cuda")
    dp[-tail:] = last[:, half:]
    M.swiglu_backward(dp, dx[:, :half], dx[:, half:], ckpt=ckpt, ckpt_scales=cs)
    dg, du = swiglu_backward(dp[-tail:].clone(), ckpt=o["ckpt"], ckpt_scales=o["ckpt_scales"])
    assert_bits(dx[-tail:, :half], dg, "dgate")
    assert_bits(dx[-tail:, half:], du, "dup")
    assert not dx[:-tail].any()


def odd(t):
    """The tensor in a buffer that starts 16 bytes past a multiple of 32."""
    n, es = t.numel(), t.element_size()
    buf = torch.empty(n * es + 64, dtype=torch.uint8, device="cuda")
    at = (16 - buf.data_ptr()) % 32
    v = buf[at:at + n * es].view(t.dtype).view(t.shape)
    v.copy_(t)
    assert v.data_ptr() % 32 == 16
    return v


@pytest.mark.parametrize("shape", [(9, 48), (70, 1040)])
def test_pointers_aligned_to_16_bytes_only(shape):
    rows, cols = shape
    x, r, dy, dh = (odd(normal(100 + k, rows, cols, dtype=torch.bfloat16)) for k in range(4))
    w = odd(normal(104, cols, dtype=torch.bfloat16))
    ref = norm(x.clone(), w.clone(), residual=r.clone())
    o = {k: odd(torch.zeros_like(v)) for k, v in ref.items()}
    M.rmsnorm_residual_fp8(x, w, o["y"], o["y_scales"], residual=r, h=o["h"], rstd=o["rstd"], ckpt=o["ckpt"],
                           ckpt_scales=o["ckpt_scales"])
    for k in ref:
        assert_bits(o[k], ref[k], k)
    dx, dw = odd(torch.zeros_like(x)), odd(torch.zeros(cols, device="cuda"))
    ws = odd(M.new_rmsnorm_workspace(rows, cols))
    want = norm_backward(dy, w, ref["rstd"], ckpt=ref["ckpt"], scales=ref["ckpt_scales"], dh=dh)
    M.rmsnorm_residual_backward(dy, w, o["rstd"], dx, dw, ws, ckpt=o["ckpt"], ckpt_scales=o["ckpt_scales"], dh=dh)
    assert_bits(dx, want[0], "dx")
    assert_bits(dw, want[1], "dweight")
    ref = swiglu(x.clone(), r.clone())
    o = {k: odd(torch.zeros_like(v)) for k, v in ref.items()}
    M.swiglu_fp8(x, r, o["y"], o["y_scales"], ckpt=o["ckpt"], ckpt_scales=o["ckpt_scales"])
    for k in ref:
        assert_bits(o[k], ref[k], k)
    want = swiglu_backward(dy, ckpt=ref["ckpt"], ckpt_scales=ref["ckpt_scales"])
    dg, du = odd(torch.zeros_like(x)), odd(torch.zeros_like(x))
    M.swiglu_backward(dy, dg, du, ckpt=o["ckpt"], ckpt_scales=o["ckpt_scales"])
    assert_bits(dg, want[0], "dgate")
    assert_bits(du, want[1], "dup")


def test_calls_on_two_streams_at_once():
    """Calls with their own buffers may run together: nothing of one waits for the other."""
    rows, cols = 3000, 2048
    x, dy, w = normal(110, rows, cols, dtype=torch.bfloat16), normal(111, rows, cols, dtype=torch.bfloat16), normal(112, cols)
    rstd = norm(x, w)["rstd"]
    want = norm_backward(dy, w, rstd, h=x)
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in range(2)]
    outs = [(torch.empty_like(x), torch.empty(cols, device="cuda"), M.new_rmsnorm_workspace(rows, cols)) for _ in sides]
    torch.cuda.synchronize()
    for _ in range(20):
        for side, (dx, dw, ws) in zip(sides, outs):
            M.rmsnorm_residual_backward(dy, w, rstd, dx, dw, ws, h=x, stream=side)
    torch.cuda.synchronize()
    for dx, dw, _ in outs:
        assert_bits(dx, want[0], "dx")
        assert_bits(dw, want[1], "dweight")
    assert M.mp_wait_failures() == 0


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_every_nan_written_in_16_bits_is_the_canonical_one(dtype):
    dt = TYPES[dtype]
    x, r = normal(97, 2, 128, dtype=dt), normal(98, 2, 128, dtype=dt)
    x[0, 3], x[1, 5], r[1, 5] = -float("nan"), float("inf"), float("-inf")
    w = torch.ones(128, device="cuda")
    o = norm(x, w, residual=r)
    assert int(bits(o["h"])[0, 3]) == 0x7FFF and int(bits(o["h"])[1, 5]) == 0x7FFF
    dx, _ = norm_backward(x, w, o["rstd"], h=o["h"])
    assert bool((bits(dx) == 0x7FFF).all())
    dg, du = swiglu_backward(x, gate=o["h"], up=r)
    assert int(bits(dg)[0, 3]) == 0x7FFF and int(bits(du)[1, 5]) == 0x7FFF


def test_python_marshalling_gives_what_the_native_one_does():
    """A raw pointer among the arguments is left to the Python marshalling: same call, same results."""
    rows, cols = 33, 272
    x, r, dy, dh = (normal(120 + k, rows, cols, dtype=torch.float16) for k in range(4))
    w = normal(124, cols)
    ref = norm(x, w, residual=r, fp8=M.MP_E5M2)
    o = {k: torch.zeros_like(v) for k, v in ref.items()}
    n0 = M.mp_launch_count()
    M.rmsnorm_residual_fp8(x, w, o["y"].data_ptr(), o["y_scales"], residual=r, h=o["h"], rstd=o["rstd"], ckpt=o["ckpt"],
                           ckpt_scales=o["ckpt_scales"], fp8_dtype=M.MP_E5M2, stream=torch.cuda.current_stream())
    assert M.mp_launch_count() == n0 + 1
    for k in ref:
        assert_bits(o[k], ref[k], k)
    want = norm_backward(dy, w, ref["rstd"], ckpt=ref["ckpt"], scales=ref["ckpt_scales"], dh=dh)
    dx, dw = torch.zeros_like(x), torch.zeros(cols, device="cuda")
    ws = M.new_rmsnorm_workspace(rows, cols)
    M.rmsnorm_residual_backward(dy, w, o["rstd"].data_ptr(), dx, dw, ws, ckpt=o["ckpt"], ckpt_scales=o["ckpt_scales"], dh=dh,
                                stream=torch.cuda.current_stream().cuda_stream)
    assert_bits(dx, want[0], "dx")
    assert_bits(dw, want[1], "dweight")
    ref = swiglu(x, r)
    o = {k: torch.zeros_like(v) for k, v in ref.items()}
    M.swiglu_fp8(x, r, o["y"].data_ptr(), o["y_scales"], ckpt=o["ckpt"], ckpt_scales=o["ckpt_scales"])
    for k in ref:
        assert_bits(o[k], ref[k], k)
    want = swiglu_backward(dy, ckpt=ref["ckpt"], ckpt_scales=ref["ckpt_scales"])
    dg, du = torch.zeros_like(x), torch.zeros_like(x)
    M.swiglu_backward(dy, dg, du, ckpt=o["ckpt"].data_ptr(), ckpt_scales=o["ckpt_scales"])
    assert_bits(dg, want[0], "dgate")
    assert_bits(du, want[1], "dup")


def test_arguments_keep_their_reference_counts():
    import sys

    x, w = normal(130, 4, 256), normal(131, 256)
    y, ys = torch.empty(4, 256, dtype=torch.uint8, device="cuda"), torch.empty(4, 2, device="cuda")
    side = torch.cuda.Stream()
    held = (x, w, y, ys, side, torch.float32)
    before = [sys.getrefcount(t) for t in held]
    for _ in range(100):
        M.rmsnorm_residual_fp8(x, w, y, ys, stream=side)
        M.swiglu_fp8(x, x, y, ys)
        M.swiglu_backward(x, x, x, gate=x, up=x)
        with pytest.raises(ValueError):
            M.rmsnorm_residual_fp8(x, w, y, ys[:2])
    torch.cuda.synchronize()
    assert [sys.getrefcount(t) for t in held] == before


def test_refusals_launch_nothing():
    x, w = normal(90, 4, 256, dtype=torch.bfloat16), normal(91, 256)
    y, ys, rstd = torch.empty(4, 256, dtype=torch.uint8, device="cuda"), torch.empty(4, 2, device="cuda"), torch.empty(4, device="cuda")
    ws, dw = M.new_rmsnorm_workspace(4, 256), torch.empty(256, device="cuda")
    cs = torch.empty(4, 2, device="cuda")
    torch.cuda.synchronize()
    n0 = M.mp_launch_count()

    def status(fn, *a, **k):
        with pytest.raises(M.MpError) as e:
            fn(*a, **k)
        return e.value.status

    f, b = M.rmsnorm_residual_fp8, M.rmsnorm_residual_backward
    assert status(f, x, w, y, ys, fp8_dtype=M.MP_E2M1) == M.MP_EINVAL
    assert status(f, x, w, y, ys, scale_block=64) == M.MP_EINVAL
    assert status(f, x, w, y, ys, eps=-1.0) == M.MP_EINVAL
    assert status(f, x, w, y, ys, eps=float("nan")) == M.MP_EINVAL
    assert status(f, x, w, y, ys, ckpt=y) == M.MP_EINVAL
    assert status(f, x[:, :24].contiguous(), w, y, ys) == M.MP_ESHAPE
    wide = torch.empty(1, 16400, dtype=torch.bfloat16, device="cuda")
    assert status(f, wide, wide[0], torch.empty(16400, dtype=torch.uint8, device="cuda"),
                  torch.empty(129, device="cuda")) == M.MP_ESHAPE
    assert status(f, x[:, :48].contiguous(), w, y, ys, scale_block=32) == M.MP_ESHAPE
    assert status(f, x, w, y.view(-1)[1:], ys) == M.MP_EALIGN
    assert status(b, x, w, rstd, x, dw, ws) == M.MP_EINVAL
    assert status(b, x, w, rstd, x, dw, ws, h=x, ckpt=y, ckpt_scales=cs) == M.MP_EINVAL
    assert status(b, x, w, rstd, x, dw, ws[:16], h=x) == M.MP_EWORKSPACE
    assert status(M.swiglu_fp8, x, x, y, ys, fp8_dtype=M.MP_F16) == M.MP_EINVAL
    assert status(M.swiglu_fp8, x[:, :24], x[:, 24:48], y, ys) == M.MP_ESHAPE
    assert status(M.swiglu_fp8, x[:, 4:132], x[:, 4:132], y, ys) == M.MP_EALIGN
    assert status(M.swiglu_backward, x, x, x) == M.MP_EINVAL
    for call in (lambda: f(x.cpu(), w, y, ys), lambda: f(x, w, y, ys[:2]), lambda: f(x, w, y, ys, residual=x.half()),
                 lambda: f(x, w, y[:3], ys), lambda: f(x, w[:128], y, ys), lambda: f(x.t(), w, y, ys),
                 lambda: f(x, w, y, ys, rstd=rstd.double()), lambda: b(x, w, rstd, x.float(), dw, ws, h=x),
                 lambda: M.swiglu_fp8(x, x[:2], y, ys), lambda: M.swiglu_fp8(x[:, :128], x.clone()[:, :128].contiguous(), y, ys),
                 lambda: M.swiglu_fp8(x, x, y, ys, ckpt=y, ckpt_scales=cs),
                 lambda: M.swiglu_backward(x, x.half(), x, gate=x, up=x), lambda: M.swiglu_backward(x, x, x, gate=x)):
        with pytest.raises(ValueError):
            call()
    # nothing to do: nothing launched
    e = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    f(e, w, y, ys)
    M.swiglu_fp8(e, e, y, ys)
    M.swiglu_backward(e, e, e, gate=e, up=e)
    assert M.mp_launch_count() == n0
