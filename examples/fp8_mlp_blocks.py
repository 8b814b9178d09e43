"""A stack of feed-forward blocks trained with this library's precision machinery.

    python examples/fp8_mlp_blocks.py [--steps 200] [--tokens 2048] [--blocks 4]

Each block adds the branch of the block before it to the residual stream and
norms the sum straight to FP8 (rmsnorm_residual_fp8), multiplies it by the gate
and up weights and forms the gated product of both straight to FP8 in one call
(linear_swiglu), and multiplies that by the down weights.  What the backward pass
reads of the stream, the gate and the up values are the 8-bit checkpoints that the
two calls write on the way; rmsnorm_residual_backward and linear_swiglu_backward
take them as they are.  The gradients of all blocks are clipped by one norm
(mp_grad_norm, mp_grad_clip), and the update is mp_adamw_step on FP32 masters under
a dynamic loss scale: one call for the matrices, one for the norms' weights, which
do not decay.

The products of linear_swiglu are of 16-bit operands, so its input is the FP8
norm dequantised to BF16; the down projection is torch's.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mixed_precision_numerics_gb300 as M  # noqa: E402

BF16 = torch.bfloat16


def tiles(n: int) -> int:
    return -(-n // 128)


def dequantise(codes, scales):
    cols = codes.shape[-1]
    return (codes.view(torch.float8_e4m3fn).float() * scales.repeat_interleave(128, -1)[..., :cols]).to(BF16)


def empty(*shape, dtype):
    return torch.empty(*shape, dtype=dtype, device="cuda")


class Weight:
    """An FP32 master with its moments, its BF16 working copy and its gradient."""

    def __init__(self, value):
        self.work, self.grad = value.to(BF16), torch.zeros_like(value, dtype=BF16)
        self.param = M.Param(value, torch.zeros_like(value), torch.zeros_like(value), self.grad, self.work)


class Block:
    """Buffers are made once: no call of a step allocates for the library's part."""

    def __init__(self, tokens: int, width: int, hidden: int, gen):
        def weight(rows, cols):
            return Weight(torch.randn(rows, cols, generator=gen, device="cuda") * cols**-0.5)

        self.norm, self.gate_up, self.down = Weight(torch.ones(width, device="cuda")), weight(2 * hidden, width), weight(width, hidden)
        self.hidden, u8, f32 = hidden, torch.uint8, torch.float32
        self.h, self.rstd = empty(tokens, width, dtype=BF16), empty(tokens, dtype=f32)
        self.y, self.y_scales = empty(tokens, width, dtype=u8), empty(tokens, tiles(width), dtype=f32)
        self.h_saved, self.h_scales = torch.empty_like(self.y), torch.empty_like(self.y_scales)
        self.p, self.p_scales = empty(tokens, hidden, dtype=u8), empty(tokens, tiles(hidden), dtype=f32)
        self.gu_saved, self.gu_scales = empty(2, tokens, hidden, dtype=u8), empty(2, tokens, tiles(hidden), dtype=f32)
        self.dy, self.dx = empty(tokens, width, dtype=BF16), empty(tokens, width, dtype=BF16)
        self.workspace = M.new_rmsnorm_workspace(tokens, width)
        self.products = M.new_linear_swiglu_workspace(tokens, width, hidden)

    def halves(self, gate_up):
        return gate_up[:self.hidden], gate_up[self.hidden:]

    def forward(self, branch, stream):
        """(the block's branch, the stream it is to be added to)"""
        M.rmsnorm_residual_fp8(branch, self.norm.work, self.y, self.y_scales, residual=stream, h=self.h, rstd=self.rstd,
                               ckpt=self.h_saved, ckpt_scales=self.h_scales)
        M.linear_swiglu(dequantise(self.y, self.y_scales), *self.halves(self.gate_up.work), self.p, p_scales=self.p_scales,
                        ckpt=self.gu_saved, ckpt_scales=self.gu_scales)
        return dequantise(self.p, self.p_scales) @ self.down.work.t(), self.h

    def backward(self, d_branch, d_stream):
        """Gradient of the branch and of the stream that came in (one tensor: they were added)."""
        torch.matmul(d_branch.t(), dequantise(self.p, self.p_scales), out=self.down.grad)
        dp = d_branch @ self.down.work
        M.linear_swiglu_backward(dp, dequantise(self.y, self.y_scales), *self.halves(self.gate_up.work), self.dy,
                                 *self.halves(self.gate_up.grad), self.products, ckpt=self.gu_saved, ckpt_scales=self.gu_scales)
        M.rmsnorm_residual_backward(self.dy, self.norm.work, self.rstd, self.dx, self.norm.grad, self.workspace,
                                    ckpt=self.h_saved, ckpt_scales=self.h_scales, dh=d_stream)
        return self.dx


def train(steps: int = 200, tokens: int = 2048, blocks: int = 4, width: int = 256, hidden: int = 688, seed: int = 0,
          log=print) -> list[float]:
    gen = torch.Generator(device="cuda").manual_seed(seed)
    stack = [Block(tokens, width, hidden, gen) for _ in range(blocks)]
    matrices, norms = [w for b in stack for w in (b.gate_up, b.down)], [b.norm for b in stack]
    groups = [([w.param for w in matrices], M.AdamwHparams(2e-3, 0.9, 0.95, 1e-8, 0.01, 0.0), M.new_scaler_state(1024.0)),
              ([w.param for w in norms], M.AdamwHparams(2e-3, 0.9, 0.95, 1e-8, 0.0, 0.0), M.new_scaler_state(1024.0))]
    grads = M.make_grad_array([w.grad for w in matrices + norms])
    norm, norm_workspace = empty(1, dtype=torch.float32), M.new_grad_norm_workspace(grads)
    mix = torch.randn(width, width, generator=gen, device="cuda") * width**-0.5
    cfg = M.ScalerCfg(2.0, 0.5, 100, 1)
    # the loss scale, on the device: a norm that is not finite makes every gradient NaN, so both groups see the
    # same bad steps and their scales stay the same
    scale = groups[0][2][:4].view(torch.float32)
    losses = []
    for step in range(steps):
        x = torch.randn(tokens, width, generator=gen, device="cuda")
        target = torch.tanh(x @ mix) + x
        branch, stream = x.to(BF16), None
        for b in stack:
            branch, stream = b.forward(branch, stream)
        off = (branch.float() + stream.float()) - target
        losses.append(off.square().mean())
        d = (off * (2.0 / off.numel() * scale)).to(BF16)
        d_branch, d_stream = d, d
        for b in reversed(stack):
            d_branch = d_stream = b.backward(d_branch, d_stream)
        M.mp_grad_norm(grads, norm, norm_workspace, loss_scale=scale)
        M.mp_grad_clip(grads, norm, 1.0)
        for params, hp, state in groups:
            M.mp_adamw_step(params, hp, state)
            M.loss_scale_update(state, cfg)
        if log and (step % 20 == 0 or step == steps - 1):
            log(f"step {step:4d}  loss {float(losses[-1]):.4f}")
    s = M.read_scaler_state(groups[0][2])
    if log:
        saved = sum(t.nbytes for b in stack for t in (b.h_saved, b.h_scales, b.gu_saved, b.gu_scales))
        kept = sum(2 * tokens * (width + 2 * hidden) for _ in stack)
        log(f"{s.step} steps, {s.skipped} skipped, loss scale {s.scale:g}; saved for the backward pass: "
            f"{saved / 2**20:.1f} MiB in 8 bits, {kept / 2**20:.1f} MiB in 16")
    return [float(v) for v in losses]


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--blocks", type=int, default=4)
    a = ap.parse_args()
    train(a.steps, a.tokens, a.blocks)
