"""Training steps of a gated feed-forward block through all of its calls: forward and backward on two micro-batches,
gradients accumulated in FP32, one norm over two parameter groups, clipping into the 16-bit gradients that the
optimizer step reads; eager, captured, and with an overflow."""
import math

import pytest
import torch

from . import ffn_util as U

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
ROWS, WIDTH, HIDDEN, SCALE = 200, 272, 400, 256.0


@pytest.fixture
def M(cuda_ok):
    import mixed_precision_numerics_gb300

    return mixed_precision_numerics_gb300


class Step:
    """Two groups: the gate and up weights, which decay, and a vector of gains on x, which does not."""

    def __init__(self, M, seed):
        self.M = M
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.master = [torch.randn(2 * HIDDEN, WIDTH, generator=gen, device="cuda") * WIDTH**-0.5, torch.ones(WIDTH, device="cuda")]
        self.work = [m.to(BF16) for m in self.master]
        self.x = [torch.randn(ROWS, WIDTH, generator=gen, device="cuda").to(BF16) for _ in range(2)]
        self.dp = [(torch.randn(ROWS, HIDDEN, generator=gen, device="cuda") * 0.01 * SCALE).to(BF16) for _ in range(2)]
        self.sums = [torch.zeros_like(m) for m in self.master]  # FP32
        self.grads = [torch.zeros_like(w) for w in self.work]
        self.groups = []
        for m, w, g, decay in zip(self.master, self.work, self.grads, (0.1, 0.0)):
            p = M.Param(m, torch.zeros_like(m), torch.zeros_like(m), g, w)
            self.groups.append((M.make_param_array([p]), p, M.AdamwHparams(1e-2, 0.9, 0.95, 1e-8, decay, 0.0), M.new_scaler_state(SCALE)))
        self.lists = M.make_grad_array(self.sums, self.grads)
        self.norm, self.norm_ws = torch.zeros(1, device="cuda"), M.new_grad_norm_workspace(self.lists)
        self.ws = M.new_linear_swiglu_workspace(ROWS, WIDTH, HIDDEN)
        f = dict(device="cuda", dtype=BF16)
        self.p, self.dxn = torch.empty(ROWS, HIDDEN, **f), torch.empty(ROWS, WIDTH, **f)
        self.dw, self.xn = torch.empty(2 * HIDDEN, WIDTH, **f), torch.empty(ROWS, WIDTH, **f)
        self.kept = torch.empty(2, ROWS, HIDDEN, dtype=torch.uint8, device="cuda")
        self.scales = torch.empty(2, ROWS, U.tiles(HIDDEN), device="cuda")
        self.seen = []

    def run(self, watch=False):
        M, (w, gain) = self.M, self.work
        for s in self.sums:
            s.zero_()
        for x, dp in zip(self.x, self.dp):
            torch.mul(x, gain, out=self.xn)
            M.linear_swiglu(self.xn, w[:HIDDEN], w[HIDDEN:], self.p, ckpt=self.kept, ckpt_scales=self.scales)
            M.linear_swiglu_backward(dp, self.xn, w[:HIDDEN], w[HIDDEN:], self.dxn, self.dw[:HIDDEN], self.dw[HIDDEN:], self.ws,
                                     ckpt=self.kept, ckpt_scales=self.scales)
            if watch:
                self.seen.append([t.clone() for t in (self.xn, self.p, self.dxn, self.dw, self.kept, self.scales)])
            self.sums[0] += self.dw
            self.sums[1] += (self.dxn.float() * x.float()).sum(0)
        M.mp_grad_norm(self.lists, self.norm, self.norm_ws, loss_scale=self.groups[0][3][:4].view(F32))
        M.mp_grad_clip(self.lists, self.norm, 0.05)
        for arr, _, hp, state in self.groups:
            M.mp_adamw_step(arr, hp, state, M.MP_BF16, M.MP_BF16)
            M.loss_scale_update(state, M.ScalerCfg(2.0, 0.5, 1000, 1))

    def state(self):
        return [t.clone() for t in (*self.master, *self.work, self.norm)]


def test_a_step_against_64_bits(M):
    s = Step(M, 1)
    before, w0 = [m.double() for m in s.master], s.work[0].clone()
    s.run(watch=True)
    for (xn, p, dxn, dw, kept, scales), x, dp in zip(s.seen, s.x, s.dp):
        (g, eg), (u, eu), (want, ep) = U.gated(xn, w0[:HIDDEN], w0[HIDDEN:])
        U.check("p", p, want, ep)
        for k, (v, e) in enumerate(((g, eg), (u, eu))):
            U.close_codes(f"ckpt {k}", kept[k], scales[k], v, e, 128)
        g, u = (U.d(kept[k].view(torch.float8_e4m3fn).float()) * U.d(scales[k]).repeat_interleave(128, 1)[:, :HIDDEN] for k in (0, 1))
        bounds = U.gradients(dp, xn, w0[:HIDDEN], w0[HIDDEN:], g, u, 2.0**-24 * g.abs(), 2.0**-24 * u.abs())
        for name, got in (("dx", dxn), ("dw_gate", dw[:HIDDEN]), ("dw_up", dw[HIDDEN:])):
            U.check(name, got, *bounds[name])
    want = math.sqrt(sum(float(t.double().square().sum()) for t in s.sums)) / SCALE
    assert abs(float(s.norm) - want) <= 34.1 * 2.0**-24 * want and want > 0.05  # clipping is active
    c = 0.05 / (want + 1e-6)
    for total, g in zip(s.sums, s.grads):
        exact = total.double() * c
        assert ((g.double() - exact).abs() <= exact.abs() * (2.0**-8 + 40 * 2.0**-24) + 2.0**-133).all()
    for m0, m, g, decay in zip(before, s.master, s.grads, (0.1, 0.0)):
        # the first step: m / (1 - b1) and v / (1 - b2) are g and g^2
        g = g.double() / SCALE
        exact = m0 * (1 - 1e-2 * decay) - 1e-2 * g / (g.abs() + 1e-8)
        assert ((m.double() - exact).abs() <= 2.0**-20 * (m0.abs() + 1e-2)).all()


def test_captured_steps_are_the_eager_ones(M):
    eager, graphed = Step(M, 2), Step(M, 2)
    for _ in range(4):
        eager.run()
    graphed.run()  # a first step outside of the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        graphed.run()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(eager.state(), graphed.state()))
    assert M.mp_wait_failures() == 0


def test_an_overflow_in_one_group_skips_both(M):
    s = Step(M, 3)
    s.run()
    before, moments = s.state(), [p.exp_avg.clone() for _, p, _, _ in s.groups]
    s.dp[1][5, 7] = float("inf")
    s.run()
    assert not math.isfinite(float(s.norm))
    assert all(torch.equal(a, b) for a, b in zip(before[:4], s.state()[:4]))
    assert all(torch.equal(a, p.exp_avg) for a, (_, p, _, _) in zip(moments, s.groups))
    for _, _, _, state in s.groups:
        r = M.read_scaler_state(state)
        assert (r.step, r.skipped, r.scale) == (1, 1, SCALE / 2)
