"""The gated feed-forward products and their gradients against binary64."""
import pytest
import torch

from . import ffn_util as U

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16
SIZES = [(1, 16, 16), (1, 4096, 512), (3, 64, 128), (17, 80, 144), (37, 1040, 272), (64, 512, 1456), (129, 48, 400),
         (256, 256, 688), (257, 5120, 96), (301, 1040, 1456), (513, 592, 16), (4113, 32, 48),
         (2, 8192, 160), (16, 1552, 4112), (33, 272, 128), (100, 4096, 528), (128, 2064, 256),
         (100, 4096, 2064), (128, 8192, 1040)]


@pytest.fixture
def M(cuda_ok):
    import mixed_precision_numerics_gb300

    return mixed_precision_numerics_gb300


def empty(*shape, dtype):
    return torch.full(shape, 3.0, dtype=dtype, device="cuda")


def run_forward(M, x, wg, wu, out, save, ld_extra=0, fp8=None):
    rows, hidden = x.shape[0], wg.shape[0]
    r = {}
    if out == 16:
        r["p"] = empty(rows, hidden, dtype=x.dtype)
    else:
        r["p"] = torch.full((rows, hidden), 7, dtype=torch.uint8, device="cuda")
        r["p_scales"] = (empty(rows, U.tiles(hidden), dtype=torch.float32) if out == 128 else
                         torch.full((rows, hidden // 32), 9, dtype=torch.uint8, device="cuda"))
    if save == 16:
        both = empty(rows, 2 * hidden + ld_extra, dtype=x.dtype)
        r["gate"], r["up"] = both[:, :hidden], both[:, hidden:2 * hidden]
    elif save == 8:
        r["ckpt"] = torch.full((2, rows, hidden), 7, dtype=torch.uint8, device="cuda")
        r["ckpt_scales"] = empty(2, rows, U.tiles(hidden), dtype=torch.float32)
    M.linear_swiglu(x, wg, wu, r["p"], p_scales=r.get("p_scales"), gate=r.get("gate"), up=r.get("up"),
                    ckpt=r.get("ckpt"), ckpt_scales=r.get("ckpt_scales"), fp8_dtype=M.MP_E4M3 if fp8 is None else fp8,
                    scale_block=32 if out == 32 else 128)
    return r


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("rows,width,hidden", SIZES)
def test_forward(M, rows, width, hidden, dtype):
    x, wg, wu, _ = U.inputs(rows, width, hidden, dtype)
    (g, eg), (u, eu), (p, ep) = U.gated(x, wg, wu)
    r = run_forward(M, x, wg, wu, 16, 16, ld_extra=24)
    U.check("gate", r["gate"], g, eg)
    U.check("up", r["up"], u, eu)
    U.check("p", r["p"], p, ep)
    alone = run_forward(M, x, wg, wu, 16, 0)
    assert torch.equal(alone["p"], r["p"])


@pytest.mark.parametrize("out,fp8", [(128, "e4m3"), (128, "e5m2"), (32, "e4m3"), (32, "e5m2")])
@pytest.mark.parametrize("save", [0, 8, 16])
@pytest.mark.parametrize("rows,width,hidden", [(1, 48, 32), (37, 1040, 288), (301, 528, 1440), (130, 2048, 160), (97, 4096, 2080)])
def test_forward_in_8_bits(M, rows, width, hidden, out, fp8, save):
    x, wg, wu, _ = U.inputs(rows, width, hidden, BF16, seed=3)
    (g, eg), (u, eu), (p, ep) = U.gated(x, wg, wu)
    t = torch.float8_e4m3fn if fp8 == "e4m3" else torch.float8_e5m2
    r = run_forward(M, x, wg, wu, out, save, fp8=M.MP_E4M3 if fp8 == "e4m3" else M.MP_E5M2)
    U.close_codes("p", r["p"], r["p_scales"], p, ep, out, t)
    if save == 8:
        for k, (v, e) in enumerate(((g, eg), (u, eu))):
            U.close_codes(f"ckpt {k}", r["ckpt"][k], r["ckpt_scales"][k], v, e, 128)
    elif save == 16:
        U.check("gate", r["gate"], g, eg)
        U.check("up", r["up"], u, eu)


def test_codes_follow_the_rules_of_the_other_block_operators(M):
    """Where gate and up are exact in binary32 and in BF16, the bytes are those of swiglu_fp8 and its checkpoint."""
    rows, hidden = 70, 304
    gen = torch.Generator(device="cuda").manual_seed(5)
    # one non-zero weight a row of each matrix: gate and up are copies of columns of x
    x = torch.randn(rows, 320, generator=gen, device="cuda").to(BF16)
    x[3] = 0.0
    pick = torch.randint(0, 320, (2, hidden), generator=gen, device="cuda")
    w = torch.zeros(2, hidden, 320, dtype=BF16, device="cuda")
    for k in range(2):
        w[k, torch.arange(hidden, device="cuda"), pick[k]] = 1.0
    r = run_forward(M, x, w[0], w[1], 128, 8)
    gate, up = x[:, pick[0]].contiguous(), x[:, pick[1]].contiguous()
    y, ys = torch.empty_like(r["p"]), torch.empty_like(r["p_scales"])
    ck, cs = torch.empty_like(r["ckpt"]), torch.empty_like(r["ckpt_scales"])
    M.swiglu_fp8(gate, up, y, ys, ckpt=ck, ckpt_scales=cs)
    assert torch.equal(ck, r["ckpt"]) and torch.equal(cs, r["ckpt_scales"])
    # swiglu_fp8 takes s of BF16 values within (1.25 |g| + 6) * 2^-24: 17 * 2^-24 to |g| = 4.5, here 6.2 * 2^-24
    assert ((ys - r["p_scales"]).abs() <= 28 * 2.0**-24 * ys).all()
    a, b = y.view(torch.float8_e4m3fn).float(), r["p"].view(torch.float8_e4m3fn).float()
    assert ((a - b).abs() <= torch.maximum(a.abs(), b.abs()) / 8 + 2.0**-9).all() and (a != b).float().mean() < 1e-3


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("save", ["16", "8", "again"])
@pytest.mark.parametrize("rows,width,hidden", SIZES)
def test_backward(M, rows, width, hidden, save, dtype):
    x, wg, wu, dp = U.inputs(rows, width, hidden, dtype, seed=1)
    (g, eg), (u, eu), _ = U.gated(x, wg, wu)
    saved = {}
    if save == "16":
        both = torch.empty(rows, 2 * hidden, dtype=dtype, device="cuda")
        both[:, :hidden], both[:, hidden:] = g.to(dtype), u.to(dtype)
        saved = {"gate": both[:, :hidden], "up": both[:, hidden:]}
        g, u, eg, eu = U.d(saved["gate"]), U.d(saved["up"]), 0.0, 0.0
    elif save == "8":
        pairs = [U.codes(v.float(), 128) for v in (g, u)]
        saved = {"ckpt": torch.stack([c.view(torch.uint8) for c, _ in pairs]), "ckpt_scales": torch.stack([s for _, s in pairs])}
        g, u = (U.d(c.float()) * U.d(s).repeat_interleave(128, 1)[:, :hidden] for c, s in pairs)
        eg, eu = 2.0**-24 * g.abs(), 2.0**-24 * u.abs()
    out = {"dx": empty(rows, width, dtype=dtype), "dw_gate": empty(hidden, width, dtype=dtype),
           "dw_up": empty(hidden, width, dtype=dtype)}
    ws = M.new_linear_swiglu_workspace(rows, width, hidden)
    ws.fill_(0x7F)
    M.linear_swiglu_backward(dp, x, wg, wu, out["dx"], out["dw_gate"], out["dw_up"], ws, **saved)
    for name, (v, e) in U.gradients(dp, x, wg, wu, g, u, eg, eu).items():
        U.check(name, out[name], v, e)
    # each gradient alone has the same bits
    dx = torch.empty_like(out["dx"])
    M.linear_swiglu_backward(dp, x, wg, wu, dx, None, None, ws, **saved)
    dw = torch.empty(2, hidden, width, dtype=dtype, device="cuda")
    M.linear_swiglu_backward(dp, x, wg, wu, None, dw[0], dw[1], ws, **saved)
    assert torch.equal(dx, out["dx"]) and torch.equal(dw[0], out["dw_gate"]) and torch.equal(dw[1], out["dw_up"])


def test_gradients_against_differences(M):
    """The loss sum(p * dp) around the inputs: central differences of the 64-bit forward definition."""
    rows, width, hidden = 5, 32, 48
    x, wg, wu, dp = U.inputs(rows, width, hidden, F16, seed=2)
    out = [torch.empty_like(x), torch.empty_like(wg), torch.empty_like(wu)]
    M.linear_swiglu_backward(dp, x, wg, wu, *out, M.new_linear_swiglu_workspace(rows, width, hidden))

    def loss(x, wg, wu):
        g = x @ wg.t()
        return (g * torch.sigmoid(g) * (x @ wu.t()) * U.d(dp)).sum()

    leaves = [U.d(v) for v in (x, wg, wu)]
    gen = torch.Generator(device="cuda").manual_seed(4)
    bounds = U.gradients(dp, x, wg, wu, leaves[0] @ leaves[1].t(), leaves[0] @ leaves[2].t(),
                         U.gated(x, wg, wu)[0][1], U.gated(x, wg, wu)[1][1])
    for k, name in enumerate(("dx", "dw_gate", "dw_up")):
        way = torch.randn(leaves[k].shape, generator=gen, device="cuda", dtype=torch.float64)
        h = 1e-4  # the error of the difference is of order h^2 = 1e-8
        up, down = list(leaves), list(leaves)
        up[k], down[k] = leaves[k] + h * way, leaves[k] - h * way
        slope = float((loss(*up) - loss(*down)) / (2 * h))
        got = float((U.d(out[k]) * way).sum())
        v, e = bounds[name]
        limit = float(((e + U.EPS[F16] * v.abs() + U.TINY[F16]) * way.abs()).sum()) + 1e-5
        assert abs(got - slope) <= limit, name


@pytest.mark.parametrize("rows", [40, 100, 300])
def test_non_finite_rows_stay_to_themselves(M, rows):
    width, hidden = 64, 144
    x, wg, wu, dp = U.inputs(rows, width, hidden, BF16)
    clean = run_forward(M, x, wg, wu, 128, 8)
    x[7, 3], x[20, 5] = float("nan"), float("inf")
    r = run_forward(M, x, wg, wu, 128, 8)
    rest = torch.tensor([i for i in range(rows) if i not in (7, 20)], device="cuda")
    for k in ("p", "p_scales"):
        assert torch.equal(r[k][rest], clean[k][rest])
    for k in ("ckpt", "ckpt_scales"):
        assert torch.equal(r[k][:, rest], clean[k][:, rest])
    assert r["p_scales"][7].isnan().all() and r["ckpt_scales"][:, 7].isnan().all()
    assert (r["ckpt"][:, 7] & 0x7F == 0x7F).all()
    assert r["ckpt_scales"][:, 20].isinf().all()  # columns past the end have no part in it
    assert (r["ckpt"][:, 20] & 0x7F == 0x7F).all()


@pytest.mark.parametrize("rows,width,hidden", [(0, 32, 48), (5, 32, 0), (0, 0, 0)])
def test_nothing_to_do(M, rows, width, hidden):
    x, wg = torch.empty(rows, width, dtype=BF16, device="cuda"), torch.empty(hidden, width, dtype=BF16, device="cuda")
    p = torch.empty(rows, hidden, dtype=BF16, device="cuda")
    M.linear_swiglu(x, wg, wg, p)
    dx, dw = torch.ones(rows, width, dtype=BF16, device="cuda"), torch.ones(2, hidden, width, dtype=BF16, device="cuda")
    M.linear_swiglu_backward(p, x, wg, wg, dx, dw[0], dw[1], None)
    assert (dx == 0).all() and (dw == 0).all()


def test_only_the_outputs_are_written(M):
    rows, width, hidden = 45, 80, 176
    x, wg, wu, dp = U.inputs(rows, width, hidden, BF16)

    def band(*shape, dtype):
        n = torch.empty(shape, dtype=dtype).numel() * torch.empty(0, dtype=dtype).element_size()
        raw = torch.full((n + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
        return raw, raw[4096:4096 + n].view(dtype).view(shape)

    outs = {"p": band(rows, hidden, dtype=torch.uint8), "p_scales": band(rows, U.tiles(hidden), dtype=torch.float32),
            "ckpt": band(2, rows, hidden, dtype=torch.uint8), "ckpt_scales": band(2, rows, U.tiles(hidden), dtype=torch.float32)}
    M.linear_swiglu(x, wg, wu, *[outs.pop("p")[1]], **{k: v[1] for k, v in outs.items()})
    ws_raw, ws = band(M.linear_swiglu_workspace_size(rows, width, hidden), dtype=torch.uint8)
    grads = {"dx": band(rows, width, dtype=BF16), "dw_gate": band(hidden, width, dtype=BF16), "dw_up": band(hidden, width, dtype=BF16)}
    wide_raw, wide = band(rows, 2 * hidden + 16, dtype=BF16)
    wide[:, hidden:hidden + 16] = 5.0
    p_raw, p = band(rows, hidden, dtype=BF16)
    M.linear_swiglu(x, wg, wu, p, gate=wide[:, :hidden], up=wide[:, hidden + 16:])
    assert (wide[:, hidden:hidden + 16] == 5.0).all()
    M.linear_swiglu_backward(dp, x, wg, wu, *[g[1] for g in grads.values()], ws, gate=wide[:, :hidden], up=wide[:, hidden + 16:])
    M.linear_swiglu_backward(dp, x, wg, wu, *[g[1] for g in grads.values()], ws)
    for raw in [v[0] for v in outs.values()] + [v[0] for v in grads.values()] + [ws_raw, wide_raw, p_raw]:
        assert (raw[:4096] == 0xA5).all() and (raw[-4096:] == 0xA5).all()


@pytest.mark.parametrize("rows", [40, 300])
def test_non_finite_gradients(M, rows):
    """A row of dp with a NaN: its row of dx, and what its hidden elements give the weights; nothing else."""
    width, hidden = 272, 400
    x, wg, wu, dp = U.inputs(rows, width, hidden, BF16, seed=11)
    dp[9, 33] = float("nan")
    dx, dw = torch.empty_like(x), torch.empty(2, hidden, width, dtype=BF16, device="cuda")
    M.linear_swiglu_backward(dp, x, wg, wu, dx, dw[0], dw[1], M.new_linear_swiglu_workspace(rows, width, hidden))
    assert dx[9].isnan().all() and torch.isfinite(torch.cat([dx[:9], dx[10:]])).all()
    assert dw[:, 33].isnan().all() and torch.isfinite(torch.cat([dw[:, :33], dw[:, 34:]], 1)).all()


def test_the_calls_allocate_nothing(M):
    sizes = [(5, 512, 288), (300, 512, 288), (200, 1040, 2064)]
    made = [(U.inputs(*s, BF16), [torch.empty(s[0], s[2], dtype=BF16, device="cuda"), torch.empty(s[0], s[1], dtype=BF16, device="cuda"),
                                  torch.empty(2, s[2], s[1], dtype=BF16, device="cuda"), M.new_linear_swiglu_workspace(*s)]) for s in sizes]
    norm = torch.empty(1, device="cuda")
    lists = [M.make_grad_array([o[2]]) for _, o in made]
    spaces = [M.new_grad_norm_workspace(a) for a in lists]

    def run():
        for (v, o), a, w in zip(made, lists, spaces):
            M.linear_swiglu(*v[:3], o[0])
            M.linear_swiglu_backward(v[3], *v[:3], o[1], o[2][0], o[2][1], o[3])
            M.mp_grad_norm(a, norm, w)
            M.mp_grad_clip(a, norm, 1.0)
        torch.cuda.synchronize()

    run()  # the kernels are loaded
    free, held = torch.cuda.mem_get_info()[0], torch.cuda.memory_stats()["allocation.all.allocated"]
    for _ in range(3):
        run()
    assert free - torch.cuda.mem_get_info()[0] < 2 << 20 and torch.cuda.memory_stats()["allocation.all.allocated"] == held


def test_captured_and_on_two_streams(M):
    """A forward and backward pass captured once and replayed on new inputs, and two streams at a time."""
    rows, width, hidden = 150, 272, 400
    a, b = U.inputs(rows, width, hidden, BF16, seed=6), U.inputs(rows, width, hidden, BF16, seed=7)

    def buffers():
        return [torch.empty(rows, hidden, dtype=BF16, device="cuda"), torch.empty(rows, width, dtype=BF16, device="cuda"),
                torch.empty(hidden, width, dtype=BF16, device="cuda"), torch.empty(hidden, width, dtype=BF16, device="cuda"),
                M.new_linear_swiglu_workspace(rows, width, hidden)]

    def step(x, wg, wu, dp, out):
        M.linear_swiglu(x, wg, wu, out[0])
        M.linear_swiglu_backward(dp, x, wg, wu, out[1], out[2], out[3], out[4])

    want = {}
    for k, v in (("a", a), ("b", b)):
        out = buffers()
        step(*v, out)
        want[k] = [t.clone() for t in out[:4]]
    torch.cuda.synchronize()
    held, out = [t.clone() for t in a], buffers()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(*held, out)
    for k, v in (("b", b), ("a", a), ("b", b)):
        for t, n in zip(held, v):
            t.copy_(n)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out[:4], want[k]))
    streams, outs = [torch.cuda.Stream(), torch.cuda.Stream()], [buffers(), buffers()]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, v, o in zip(streams, (a, b), outs):
            with torch.cuda.stream(s):
                step(*v, o)
    torch.cuda.synchronize()
    for k, o in zip("ab", outs):
        assert all(torch.equal(p, q) for p, q in zip(o[:4], want[k]))
    assert M.mp_wait_failures() == 0


def sampled(n, seed):
    """Places on both sides of tile edges, the ends, and some others."""
    gen = torch.Generator().manual_seed(seed)
    edges = [i for e in range(0, n, max(256, n // 12 // 256 * 256)) for i in (e - 1, e, e + 127, e + 128) if 0 <= i < n]
    return torch.tensor(sorted({*edges, n - 1, *torch.randint(0, n, (24,), generator=gen).tolist()}), device="cuda")


def test_many_tiles_for_every_pair(M):
    """More tiles than pairs of CTAs, ragged at every edge: sampled rows and columns of every result."""
    rows, width, hidden = 4100, 2064, 5520
    x, wg, wu, dp = U.inputs(rows, width, hidden, BF16, seed=8)
    r = run_forward(M, x, wg, wu, 128, 16)
    at = sampled(rows, 1)
    (g, eg), (u, eu), (p, ep) = U.gated(x[at], wg, wu)
    U.check("gate", r["gate"][at], g, eg)
    U.check("up", r["up"][at], u, eu)
    U.close_codes("p", r["p"][at], r["p_scales"][at], p, ep, 128)
    dx, dw = empty(rows, width, dtype=BF16), empty(2, hidden, width, dtype=BF16)
    M.linear_swiglu_backward(dp, x, wg, wu, dx, dw[0], dw[1], M.new_linear_swiglu_workspace(rows, width, hidden),
                             gate=r["gate"], up=r["up"])
    v, e = U.gradients(dp[at], x[at], wg, wu, U.d(r["gate"][at]), U.d(r["up"][at]))["dx"]
    U.check("dx", dx[at], v, e)
    cut = sampled(hidden, 2)
    out = U.gradients(dp[:, cut], x, wg[cut], wu[cut], U.d(r["gate"][:, cut]), U.d(r["up"][:, cut]))
    U.check("dw_gate", dw[0][cut], *out["dw_gate"])
    U.check("dw_up", dw[1][cut], *out["dw_up"])


@pytest.mark.parametrize("out,save", [(16, 16), (128, 8)])
def test_more_than_2_to_31_elements(M, out, save):
    width, hidden = 64, 14336
    rows = 2**31 // hidden + 700
    x, wg, wu, _ = U.inputs(rows, width, hidden, F16, seed=9)
    at = torch.tensor([0, 1, 255, 256, 2**31 // hidden - 1, 2**31 // hidden, 2**31 // hidden + 1, rows - 257, rows - 1], device="cuda")
    (g, eg), (u, eu), (p, ep) = U.gated(x[at], wg, wu)
    r = run_forward(M, x, wg, wu, out, save)
    if out == 16:
        U.check("p", r["p"][at], p, ep)
        U.check("gate", r["gate"][at], g, eg)
        U.check("up", r["up"][at], u, eu)
        del r["p"]
    else:
        U.close_codes("p", r["p"][at], r["p_scales"][at], p, ep, 128)
        for k, (v, e) in enumerate(((g, eg), (u, eu))):
            U.close_codes(f"ckpt {k}", r["ckpt"][k][at], r["ckpt_scales"][k][at], v, e, 128)
    dp = torch.randn(rows, 1, device="cuda").to(F16).expand(rows, hidden).contiguous()
    dx = empty(rows, width, dtype=F16)
    ws = M.new_linear_swiglu_workspace(rows, width, hidden)
    saved = {k: r[k] for k in ("gate", "up", "ckpt", "ckpt_scales") if k in r}
    M.linear_swiglu_backward(dp, x, wg, wu, dx, None, None, ws, **saved)
    if save == 16:
        g, u, eg, eu = U.d(r["gate"][at]), U.d(r["up"][at]), 0.0, 0.0
    else:
        g, u = (U.d(r["ckpt"][k][at].view(torch.float8_e4m3fn).float()) * U.d(r["ckpt_scales"][k][at]).repeat_interleave(128, 1)
                for k in (0, 1))
        eg, eu = 2.0**-24 * g.abs(), 2.0**-24 * u.abs()
    U.check("dx", dx[at], *U.gradients(dp[at], x[at], wg, wu, g, u, eg, eu)["dx"])
