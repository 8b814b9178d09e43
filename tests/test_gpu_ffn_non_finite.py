"""Infinities and NaN among the values of g and u, in every form of the forward call's results: where they are, what
stands for them is the rule of the other block operators; everything else keeps its bits."""
import pytest
import torch

from . import ffn_util as U

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
INF, NAN = float("inf"), float("nan")
WIDTH, HIDDEN = 320, 448
BAD = {5: ("gate", INF), 70: ("gate", -INF), 71: ("up", NAN), 200: ("up", INF), 310: ("gate", NAN)}


@pytest.fixture
def M(cuda_ok):
    import mixed_precision_numerics_gb300

    return mixed_precision_numerics_gb300


def copies(rows, dtype):
    """x without zeros and one weight a hidden element, so that g and u are columns of x; the same with the bad ones."""
    gen = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.randn(rows, WIDTH, generator=gen, device="cuda").to(dtype)
    x[x == 0] = 1.0
    pick = torch.randint(0, WIDTH, (2, HIDDEN), generator=gen, device="cuda")
    w = torch.zeros(2, HIDDEN, WIDTH, dtype=dtype, device="cuda")
    for k in range(2):
        w[k, torch.arange(HIDDEN, device="cuda"), pick[k]] = 1.0
    bad = w.clone()
    for h, (which, v) in BAD.items():
        k = ("gate", "up").index(which)
        bad[k, h, pick[k, h]] = v
    g, u = x[:, pick[0]], x[:, pick[1]]
    for h, (which, v) in BAD.items():
        (g if which == "gate" else u)[:, h] *= v
    return x, w, bad, g, u


def forward(M, x, w, fp8=None, block=128, save=None):
    rows = x.shape[0]
    r = {"p": torch.full((rows, HIDDEN), 7, dtype=torch.uint8 if fp8 else x.dtype, device="cuda")}
    if fp8:
        r["p_scales"] = (torch.full((rows, U.tiles(HIDDEN)), 3.0, device="cuda") if block == 128 else
                         torch.full((rows, HIDDEN // 32), 9, dtype=torch.uint8, device="cuda"))
    if save == 16:
        r["gate"], r["up"] = (torch.full((rows, HIDDEN), 3.0, dtype=x.dtype, device="cuda") for _ in range(2))
    elif save == 8:
        r["ckpt"] = torch.full((2, rows, HIDDEN), 7, dtype=torch.uint8, device="cuda")
        r["ckpt_scales"] = torch.full((2, rows, U.tiles(HIDDEN)), 3.0, device="cuda")
    kw = {k: v for k, v in r.items() if k != "p"}
    M.linear_swiglu(x, w[0], w[1], r["p"], **kw, fp8_dtype=M.MP_E5M2 if fp8 == E5M2 else M.MP_E4M3, scale_block=block)
    return r


def check_codes(name, value, codes, scales, clean_codes, clean_scales, block):
    """value: what the codes stand for, with infinities and NaN; clean_*: the same call's without them."""
    rows = value.shape[0]
    pad = -HIDDEN % block
    t = torch.nn.functional.pad(value, (0, pad)).view(rows, -1, block)
    nan, inf = t.isnan().any(2), t.isinf().any(2)
    hit = nan | inf
    assert hit.any() and not hit.all()
    if block == 128:
        assert scales[nan].isnan().all(), name
        assert (scales[inf & ~nan] == INF).all(), name
    else:
        assert (scales[hit] == 0xFF).all(), name
    assert torch.equal(scales[~hit], clean_scales[~hit]), name
    within = hit.repeat_interleave(block, 1)[:, :HIDDEN]
    assert torch.equal(codes[~within], clean_codes[~within]), name
    if block == 32:
        assert (codes[within] == 0).all(), name
        return
    finite = torch.isfinite(value)
    assert (codes[within & ~finite] & 0x7F == 0x7F).all() and (codes[within & finite] & 0x7F == 0).all(), name
    signed = within & ~value.isnan()
    assert ((codes[signed] >= 0x80) == (value[signed] < 0)).all(), name


# up to 64 rows and more are different kernels
@pytest.mark.parametrize("rows", [3, 40, 100, 2000])
@pytest.mark.parametrize("fp8,block", [(E4M3, 128), (E5M2, 128), (E4M3, 32), (E5M2, 32)])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_8_bit_products(M, dtype, fp8, block, rows):
    x, w, bad, g, u = copies(rows, dtype)
    clean, r = forward(M, x, w, fp8, block, 8), forward(M, x, bad, fp8, block, 8)
    p = U.d(g) * torch.sigmoid(U.d(g)) * U.d(u)
    check_codes("p", p, r["p"], r["p_scales"], clean["p"], clean["p_scales"], block)
    for k, v in enumerate((g, u)):
        check_codes("ckpt", U.d(v), r["ckpt"][k], r["ckpt_scales"][k], clean["ckpt"][k], clean["ckpt_scales"][k], 128)
    kept = forward(M, x, bad, fp8, block, 16)
    assert torch.equal(kept["p"], r["p"]) and torch.equal(kept["p_scales"].view(torch.uint8), r["p_scales"].view(torch.uint8))
    for name, v in (("gate", g), ("up", u)):
        assert torch.equal(kept[name].nan_to_num(9.0, 8.0, 7.0), v.nan_to_num(9.0, 8.0, 7.0))


@pytest.mark.parametrize("rows", [3, 40, 100, 2000])
@pytest.mark.parametrize("save", [None, 8, 16])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_16_bit_products(M, dtype, save, rows):
    x, w, bad, g, u = copies(rows, dtype)
    clean, r = forward(M, x, w, save=save), forward(M, x, bad, save=save)
    p = U.d(g) * torch.sigmoid(U.d(g)) * U.d(u)
    finite = torch.isfinite(p)
    assert torch.equal(r["p"][finite], clean["p"][finite])
    assert torch.equal(r["p"].isnan(), p.isnan())
    assert torch.equal(r["p"] == INF, p == INF) and torch.equal(r["p"] == -INF, p == -INF)
    assert (r["p"].view(torch.int16)[p.isnan()] == 0x7FFF).all()
    if save == 16:
        for name, v in (("gate", g), ("up", u)):
            assert torch.equal(r[name].nan_to_num(9.0, 8.0, 7.0), v.nan_to_num(9.0, 8.0, 7.0))
    elif save == 8:
        for k, v in enumerate((g, u)):
            check_codes("ckpt", U.d(v), r["ckpt"][k], r["ckpt_scales"][k], clean["ckpt"][k], clean["ckpt_scales"][k], 128)


@pytest.mark.parametrize("rows", [40, 300])
def test_gradients_beyond_fp16(M, rows):
    """dg and du are operands of 16 bits: beyond FP16's range they are infinite, and so are the gradients that they
    go into, although their products with small weights are not; a step's check sees it."""
    width, hidden = 32, 48
    x = torch.full((rows, width), 2.0**-12, dtype=F16, device="cuda")
    w = torch.full((hidden, width), 2.0**-12, dtype=F16, device="cuda")
    dp = torch.full((rows, hidden), 1.0, dtype=F16, device="cuda")
    dp[7] = 40000.0
    gate, up = torch.full_like(dp, 8.0), torch.full_like(dp, 8.0)
    dx, dw = torch.empty_like(x), torch.empty(2, hidden, width, dtype=F16, device="cuda")
    M.linear_swiglu_backward(dp, x, w, w, dx, dw[0], dw[1], M.new_linear_swiglu_workspace(rows, width, hidden), gate=gate, up=up)
    assert dx[7].isinf().all() and torch.isfinite(torch.cat([dx[:7], dx[8:]])).all() and dw.isinf().all()
