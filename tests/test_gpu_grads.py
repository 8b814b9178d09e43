"""The global gradient norm and clipping against binary64.

The norm: a thread adds at most 64 squares and joins two partial sums in binary32, all positive, each rounding
at most 2^-24 relative: 66 of them, halved by the root, and the result's own rounding: 34.1 * 2^-24."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
HALF = {F32: 2.0**-24, F16: 2.0**-11, BF16: 2.0**-8}
LEAST = {F32: 2.0**-150, F16: 2.0**-25, BF16: 2.0**-134}
NORM = 34.1 * 2.0**-24


@pytest.fixture
def M(cuda_ok):
    import mixed_precision_numerics_gb300

    return mixed_precision_numerics_gb300


def tensors(sizes, dtype, sigma=1e-2, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    pick = dtype if isinstance(dtype, (list, tuple)) else [dtype]
    return [(torch.randn(n, generator=gen, device="cuda") * sigma).to(pick[i % len(pick)]) for i, n in enumerate(sizes)]


def norm_of(M, grads, **kw):
    norm = torch.full((1,), -7.0, device="cuda")
    M.mp_grad_norm(grads, norm, M.new_grad_norm_workspace(grads), **kw)
    return norm


def exact(grads):
    return math.sqrt(sum(float(g.double().square().sum()) for g in grads))


def check_clipped(grads, outs, norm, max_norm):
    c = min(1.0, max_norm / (float(norm) + 1e-6))
    for g, o in zip(grads, outs):
        want = g.double() * c
        # the factor and the binary32 product are rounded, then the result to its type
        limit = want.abs() * (3 * 2.0**-24 + HALF[o.dtype] * (1 + 2.0**-22)) + LEAST[o.dtype] + 2.0**-149
        assert ((o.double() - want).abs() <= limit).all()


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("sizes", [[1], [7, 0, 8], [16384], [16383, 16385, 3], [1 << 20, 100, 65537], [40] * 31 + [5000001],
                                   [33] * 700, [100001] * 40])
def test_norm_and_clip(M, sizes, dtype):
    grads = tensors(sizes, dtype)
    norm = norm_of(M, grads)
    want = exact(grads)
    assert abs(float(norm) - want) <= NORM * want
    for max_norm in (0.5 * want, 2 * want):
        outs = [torch.full_like(g, 9.0) for g in grads]
        M.mp_grad_clip(grads, norm, max_norm, out=outs)
        check_clipped(grads, outs, norm, max_norm)
        mine = [g.clone() for g in grads]
        M.mp_grad_clip(mine, norm, max_norm)
        assert all(torch.equal(a, b) for a, b in zip(mine, outs))
        assert max_norm < want or all(torch.equal(a, b) for a, b in zip(mine, grads))


@pytest.mark.parametrize("out", [F32, F16, BF16])
def test_mixed_types(M, out):
    grads = tensors([1000, 17, 30001, 8, 16385], [F32, BF16, F16], seed=1)
    norm = norm_of(M, grads)
    assert abs(float(norm) - exact(grads)) <= NORM * exact(grads)
    outs = [torch.empty(g.numel(), dtype=out, device="cuda") for g in grads]
    arr = M.make_grad_array(grads, outs)
    M.mp_grad_clip(arr, norm, 0.125)
    check_clipped(grads, outs, norm, 0.125)


@pytest.mark.parametrize("dtype,sigma", [(F32, 1e25), (F32, 1e-30), (F32, 1e-42), (F32, 1e18), (BF16, 1e30), (BF16, 1e-35), (F16, 1e-7)])
def test_squares_out_of_range(M, dtype, sigma):
    grads = tensors([70001, 64, 5], dtype, sigma=sigma)
    grads.append(torch.zeros(40000, dtype=dtype, device="cuda"))
    norm, want = norm_of(M, grads), exact(grads)
    assert abs(float(norm) - want) <= NORM * want + 2.0**-150


def test_a_large_and_many_small(M):
    g = torch.full((1 << 20,), 1e-20, device="cuda")
    g[12345] = 1e20
    assert abs(float(norm_of(M, [g])) - exact([g])) <= NORM * 1e20
    g[12345] = 0.0
    assert abs(float(norm_of(M, [g])) - exact([g])) <= NORM * exact([g])


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan")])
def test_non_finite(M, dtype, value):
    grads = tensors([20000, 300], dtype)
    grads[1][17] = value
    norm = norm_of(M, grads)
    assert math.isnan(float(norm)) if value != value else float(norm) == math.inf
    M.mp_grad_clip(grads, norm, 1.0)
    assert all(g.isnan().all() for g in grads)  # every part of the model sees a bad step


def test_loss_scale_and_empty_lists(M):
    grads = tensors([5000, 12], F16)
    state = M.new_scaler_state(1024.0)
    norm, plain = norm_of(M, grads, loss_scale=state[:4].view(F32)), norm_of(M, grads)
    assert float(norm) * 1024 == float(plain)
    assert float(norm_of(M, [])) == 0.0 and float(norm_of(M, [grads[0][:0]])) == 0.0
    M.mp_grad_clip([], norm, 1.0)


def test_same_norm_as_the_optimizer_step(M):
    """One list of 16-bit gradients through both: within both bounds of each other."""
    grads = tensors([50000, 1234], BF16, sigma=1.0)
    masters = [torch.zeros(g.numel(), device="cuda") for g in grads]
    params = [M.Param(w, torch.zeros_like(w), torch.zeros_like(w), g, torch.empty_like(g)) for w, g in zip(masters, grads)]
    state = M.new_scaler_state(256.0)
    ws = torch.empty(M.mp_adamw_workspace_size(params), dtype=torch.uint8, device="cuda")
    M.mp_adamw_check(params, M.AdamwHparams(1e-3, 0.9, 0.999, 1e-8, 0.0, 1.0), state, workspace=ws)
    norm = norm_of(M, grads, loss_scale=state[:4].view(F32))
    theirs = M.read_scaler_state(state).grad_norm
    assert abs(float(norm) - theirs) <= (34.1 + 38) * 2.0**-24 * theirs


def test_repeats_and_leaves_its_workspace_ready(M):
    grads = tensors([300007, 5, 90001], [F32, BF16])
    ws, norm = M.new_grad_norm_workspace(grads), torch.empty(1, device="cuda")
    got = []
    for _ in range(5):
        M.mp_grad_norm(grads, norm, ws)
        got.append(norm.clone())
    assert all(torch.equal(g, got[0]) for g in got)
    graph = torch.cuda.CUDAGraph()
    arr = M.make_grad_array(grads)
    with torch.cuda.graph(graph):
        M.mp_grad_norm(arr, norm, ws)
        M.mp_grad_clip(arr, norm, 0.01)
    first = [g.clone() for g in grads]
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(norm, got[0])
    check_clipped(first, grads, norm, 0.01)
    graph.replay()
    torch.cuda.synchronize()
    assert abs(float(norm) - 0.01) <= 1e-2 * 0.01


def test_guard_bands(M):
    raw = torch.full((8192 + 2 * 16391,), 0x3C, dtype=torch.uint8, device="cuda")
    g = raw[4096:4096 + 2 * 16391].view(F16)
    out_raw = torch.full((8192 + 4 * 16391,), 0x5A, dtype=torch.uint8, device="cuda")
    out = out_raw[4096:4096 + 4 * 16391].view(F32)
    norm = norm_of(M, [g])
    M.mp_grad_clip([g], norm, 1.0, out=[out])
    assert (out_raw[:4096] == 0x5A).all() and (out_raw[-4096:] == 0x5A).all()
    check_clipped([g], [out], norm, 1.0)
    M.mp_grad_clip([g], norm, 1.0)
    assert (raw[:4096] == 0x3C).all() and (raw[-4096:] == 0x3C).all()


def test_more_than_2_to_31_elements(M):
    n = 2**31 + 100003
    g = torch.empty(n, dtype=F16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(1)
    parts = g.split(1 << 28)
    for p in parts:
        p.copy_(torch.randn(p.numel(), generator=gen, device="cuda", dtype=F16) * 1e-2)
    want = math.sqrt(sum(float(p.double().square().sum()) for p in parts))
    norm = norm_of(M, [g])
    assert abs(float(norm) - want) <= NORM * want
    ends = torch.cat([torch.arange(0, 70000), torch.arange(2**31 - 70000, n)]).cuda()
    first = g[ends]
    M.mp_grad_clip([g], norm, 0.5 * want)
    check_clipped([first], [g[ends]], norm, 0.5 * want)
