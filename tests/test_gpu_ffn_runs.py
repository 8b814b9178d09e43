"""How many terms of a contraction the tensor core adds up by itself, seen in the results.

An instruction adds 16 products to a binary32 sum.  Here the first product is 1 and every other one 0.8984375 * 2^-27,
so the 16 of an instruction come to 0.8984375 steps of a sum in [1, 2), each product to less than one: however an
instruction aligns and rounds, it changes such a sum by the right amount with an error of less than one step, 2^-23.
The sums of runs that do not hold the first product have 7 bits and a number of products below 2^16: they are exact.
So a run of T terms that holds the first product is off by less than T / 16 steps, and the sums of the runs, added with
correct rounding, by half a step each: STEPS(T) = T / 16 + (joins) / 2.

Where one scale stands for 512 terms a run, the first run's loss of up to 32 steps is what may be seen; runs four
times as long lose 0.898 * 128 = 115 if sums are truncated, which is past the bound."""
import pytest
import torch

from . import ffn_util as U

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16
STEP = 2.0**-23
A, B = 2.0**-13, 0.8984375 * 2.0**-14  # A * B is the small product; exact in both types


@pytest.fixture
def M(cuda_ok):
    import mixed_precision_numerics_gb300

    return mixed_precision_numerics_gb300


def rows_of(rows, cols, small, dtype):
    t = torch.full((rows, cols), small, dtype=dtype, device="cuda")
    t[:, 0] = 1.0
    return t


# (rows, width): up to 64 rows, or 128 of weights of 2^23 elements, one tile of 128 hidden elements is shared by
# eight parts of the contraction; else one pair of CTAs has all of it
@pytest.mark.parametrize("out", [128, 32])
@pytest.mark.parametrize("rows,width", [(1, 2**14), (20, 2**14), (64, 2**14), (128, 2**14), (300, 2**14),
                                        (1, 2**17), (20, 2**17), (64, 2**17), (128, 2**17)])
def test_scales_of_32_bits_have_runs_of_512_terms(M, rows, width, out):
    hidden = 128
    x, w = rows_of(rows, width, A, BF16), rows_of(hidden, width, B, BF16)
    scales = torch.empty(2, rows, 1, device="cuda")
    ckpt = torch.empty(2, rows, hidden, dtype=torch.uint8, device="cuda")
    p = torch.empty(rows, hidden, dtype=BF16 if out == 16 else torch.uint8, device="cuda")
    ps = {16: None, 128: torch.empty(rows, 1, device="cuda"), 32: torch.empty(rows, 4, dtype=torch.uint8, device="cuda")}[out]
    M.linear_swiglu(x, w, w, p, p_scales=ps, ckpt=ckpt, ckpt_scales=scales, scale_block=32 if out == 32 else 128)
    g = 1.0 + (width - 1) * A * B
    joins = width / 512 / 8 + 8 if width > 2**14 else width / 512 + 8  # parts of a part's runs, and parts
    off = (32 + joins / 2) * STEP
    # the scale is the largest value / 448, rounded
    assert ((scales.double() * 448 - g).abs() <= off + g * 2.0**-24).all(), float((scales.double() * 448 - g).abs().max() / STEP)
    if out == 128:  # |d silu / dg| <= 1.1
        s = torch.sigmoid(torch.tensor(g, dtype=torch.float64))
        want = float(g * s * g)
        limit = float(1.1 * g + g * s + 2 * off) * off + U.FEW * want
        assert ((ps.double() * 448 - want).abs() <= limit).all()


MIDDLE = 1.0 + 2.0**-11  # between two FP16 numbers


def last_product(products):
    """The last product so that all of them come to a little more than MIDDLE."""
    t = torch.tensor(MIDDLE + 2.1e-5 - (1.0 + (products - 2) * A * B), dtype=F16)
    above = 1.0 + (products - 2) * A * B + float(t) - MIDDLE
    # more than a run of 2048 terms loses, 128 steps, with 72 joins; less than the 230 that one of 4096 would
    assert 164 * STEP < above < 0.8984375 * 256 * STEP
    return float(t)


@pytest.mark.parametrize("rows", [1, 20, 64, 128])
def test_results_of_16_bits_have_runs_of_2048_terms(M, rows):
    """gate, rounded to FP16, is on the right side of the middle between two numbers."""
    width, hidden = 2**18, 128
    x, w = rows_of(rows, width, A, F16), rows_of(hidden, width, B, F16)
    x[:, -1], w[:, -1] = 1.0, last_product(width)
    p, gate, up = (torch.empty(rows, hidden, dtype=F16, device="cuda") for _ in range(3))
    M.linear_swiglu(x, w, w, p, gate=gate, up=up)
    assert (gate == 1.0 + 2.0**-10).all() and (up == gate).all()


@pytest.mark.parametrize("rows", [1, 20, 64])
def test_dx_of_few_rows_has_runs_of_2048_terms(M, rows):
    """gate 0 and up 2 make dg = dp and du = 0."""
    width, hidden = 16, 2**18
    dp, gate = rows_of(rows, hidden, A, F16), torch.zeros(rows, hidden, dtype=F16, device="cuda")
    dp[:, -1] = 1.0
    w = torch.full((hidden, width), B, dtype=F16, device="cuda")
    w[0], w[-1] = 1.0, last_product(hidden)
    dx, x = torch.empty(rows, width, dtype=F16, device="cuda"), torch.zeros(rows, width, dtype=F16, device="cuda")
    M.linear_swiglu_backward(dp, x, w, w, dx, None, None, M.new_linear_swiglu_workspace(rows, width, hidden), gate=gate,
                             up=torch.full_like(gate, 2.0))
    assert (dx == 1.0 + 2.0**-10).all()
