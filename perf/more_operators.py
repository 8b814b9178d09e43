"""The cases on which the gated feed-forward products and the global gradient
norm are measured: both projections of a gated feed-forward block with the
SwiGLU product formed on them, its backward pass, and the norm of a list of
gradients with their clipping.

``run`` computes a case either in its plain form (elementary torch operations
in binary32, sums of squares in binary64) or, with ``own`` set, through the
library's entry points.  Hidden sizes 4096 and 5120, the feed-forward size
14336, the width 12288 and 8192 tokens are those of this repository's
workloads, 2048 tokens of 256 and 688 those of its example; the others are
generic.
"""
import torch

own = False

TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
FP8_MAX, FP8_EMAX = 448.0, 8  # E4M3
MOST = 8192 * 4096 * 14336  # rows * width * hidden of the largest products
MOST_GRADS = 4 * (2 * 4096 * 4096 + 3 * 4096 * 14336 + 2 * 4096)  # elements of the longest list of gradients


def _mp():
    import mixed_precision_numerics_gb300 as mp

    return mp


# ---- the cases ---------------------------------------------------------------------
# ffn: p, the gated product of both projections, in 16 bits (p="16") or in FP8 with one scale for 128 or 32 elements;
#      save: what the backward pass will read: nothing, gate and up in 16 bits, or their 8-bit checkpoint.
# ffn_bwd: from gate and up in 16 bits, from their 8-bit checkpoint, or (save="no") from x alone.
# clip: the norm of `layers` layers' gradients and the clipped gradients, written in the type `out`.


def listed():
    return [
        # one token of a decoding step: the weights are read once
        dict(name="ffn 1 token", op="ffn", rows=1, width=4096, hidden=14336, dtype="bf16", p="16", save="no"),
        # a ragged decoding batch in FP16 with a microscaled product
        dict(name="ffn 37 tokens f16 mx", op="ffn", rows=37, width=5120, hidden=12288, dtype="f16", p="32", save="no"),
        # the example's blocks: FP8 product and 8-bit checkpoint, rows that end inside a 128-tile
        dict(name="ffn 2048x256x688 saved", op="ffn", rows=2048, width=256, hidden=688, dtype="bf16", p="128", save="8"),
        # a training micro-batch of the 8B-sized parameter list, FP8 product and 8-bit checkpoint
        dict(name="ffn 8192x4096x14336 saved", op="ffn", rows=8192, width=4096, hidden=14336, dtype="bf16", p="128", save="8"),
        # a ragged FP16 batch with everything kept in 16 bits
        dict(name="ffn 1000x2048x5504 kept", op="ffn", rows=1000, width=2048, hidden=5504, dtype="f16", p="16", save="16"),
        # a small FP16 model with odd sizes
        dict(name="bwd 301x1040x1456 kept", op="ffn_bwd", rows=301, width=1040, hidden=1456, dtype="f16", save="16"),
        # the example's blocks, from the 8-bit checkpoint
        dict(name="bwd 2048x256x688 saved", op="ffn_bwd", rows=2048, width=256, hidden=688, dtype="bf16", save="8"),
        # the training micro-batch's backward pass from the 8-bit checkpoint
        dict(name="bwd 8192x4096x14336 saved", op="ffn_bwd", rows=8192, width=4096, hidden=14336, dtype="bf16", save="8"),
        # the same with nothing saved but x
        dict(name="bwd 2048x4096x14336 again", op="ffn_bwd", rows=2048, width=4096, hidden=14336, dtype="bf16", save="no"),
        # the example's 4 blocks: many small tensors
        dict(name="clip 4 small layers", op="clip", layers=4, width=256, hidden=688, dtype="bf16", out="bf16", max_norm=1.0),
        # gradients accumulated in FP32, clipped into the FP16 ones that the optimizer step reads
        dict(name="clip 12 layers f32 to f16", op="clip", layers=12, width=1040, hidden=1456, dtype="f32", out="f16", max_norm=1.0),
        # four layers of the 8B-sized list
        dict(name="clip 4 layers of 4096", op="clip", layers=4, width=4096, hidden=14336, dtype="bf16", out="bf16", max_norm=1.0),
    ]


def draw(rng):
    op = rng.choice(["ffn", "ffn", "ffn_bwd", "ffn_bwd", "clip"])
    if op == "clip":
        width = 8 * round(2 ** rng.uniform(3.0, 9.0))
        hidden = 8 * round(width * rng.uniform(2.0, 4.0) / 8)
        dtype, out = rng.choice([("bf16", "bf16"), ("f16", "f16"), ("f32", "f32"), ("f32", "bf16"), ("f32", "f16")])
        layers = round(2 ** rng.uniform(0.0, 5.0))
        cap = MOST_GRADS // (1 if dtype != "f32" else 4 if out == "f32" else 2)
        layers = max(1, min(layers, cap // _elements(1, width, hidden)))
        return dict(op=op, layers=layers, width=width, hidden=hidden, dtype=dtype, out=out,
                    max_norm=rng.choice([0.25, 1.0, 1.0, 1e6]))
    rows = round(2 ** rng.uniform(0.0, 13.0))
    width = 16 * max(1, round(2 ** rng.uniform(1.0, 8.4)))
    p = rng.choice(["16", "128", "32"]) if op == "ffn" else "16"
    step = 32 if p == "32" else 16
    hidden = step * max(1, round(2 ** rng.uniform(5.0, 13.8) / step))
    rows = max(1, min(rows, MOST // (width * hidden)))
    case = dict(op=op, rows=rows, width=width, hidden=hidden, dtype=rng.choice(["bf16", "bf16", "f16"]),
                save=rng.choice(["no", "16", "8"]))
    if op == "ffn":
        case["p"] = p
    return case


def _shapes(layers, width, hidden):
    """What a layer of a model with a gated feed-forward block has gradients of."""
    layer = [(width,), (2 * width, width), (2 * hidden, width), (width, hidden), (width,)]
    return layer * layers


def _elements(layers, width, hidden):
    return layers * (2 * width * width + 3 * width * hidden + 2 * width)


def _size(dtype):
    return 4 if dtype == "f32" else 2


def work(case):
    if case["op"] == "clip":  # every gradient in, every clipped one out
        n = _elements(case["layers"], case["width"], case["hidden"])
        return {"bytes": n * (_size(case["dtype"]) + _size(case["out"])) + 4, "flops": 3 * n}
    rows, width, hidden = case["rows"], case["width"], case["hidden"]
    n = rows * hidden
    tiles = 4 * rows * -(-hidden // 128)  # FP32 scales of one 8-bit [rows, hidden]
    kept = {"no": 0, "16": 4 * n, "8": 2 * n + 2 * tiles}[case["save"]]
    product = rows * width * hidden
    weights = 4 * hidden * width
    if case["op"] == "ffn":
        p = {"16": 2 * n, "128": n + tiles, "32": n + n // 32}[case["p"]]
        return {"bytes": 2 * rows * width + weights + p + kept, "flops": 4 * product + 10 * n}
    # dp, x, both weights and what was saved in; dx and both weights' gradients out
    again = 4 * product if case["save"] == "no" else 0
    return {"bytes": 2 * n + 4 * rows * width + 2 * weights + kept, "flops": 8 * product + again + 14 * n}


# ---- inputs ------------------------------------------------------------------------


def _normal(gen, *shape, sigma=1.0):
    return torch.randn(*shape, generator=gen, device="cuda") * sigma


def _empty(*shape, dtype):
    return torch.empty(*shape, dtype=dtype, device="cuda")


def _views(flat, shapes, step):
    """Tensors in one buffer, each at a multiple of `step` elements."""
    out, at = [], 0
    for shape in shapes:
        n = shape[0] * (shape[1] if len(shape) > 1 else 1)
        out.append(flat[at:at + n].view(shape))
        at += -(-n // step) * step
    return out


def _prepare_clip(case, gen):
    shapes = _shapes(case["layers"], case["width"], case["hidden"])
    dt, out = TORCH[case["dtype"]], TORCH[case["out"]]
    step = 64
    total = sum(-(-(s[0] * (s[1] if len(s) > 1 else 1)) // step) * step for s in shapes)
    flat = torch.zeros(total, dtype=dt, device="cuda")
    grads = _views(flat, shapes, step)
    for g in grads:
        sigma = 1e-3 * float(2.0 ** (4.0 * torch.rand(1, generator=gen, device="cuda") - 2.0))  # tensors differ in size
        g.copy_(torch.randn(g.shape, generator=gen, device="cuda").mul_(sigma))
    clipped = torch.zeros(total, dtype=out, device="cuda")  # the padding between tensors stays as it is
    s = dict(case, grads=grads, flat=clipped, clipped=_views(clipped, shapes, step))
    s["norm"] = _empty(1, dtype=torch.float32)
    s["plan"] = None  # the list as the library takes it, and its workspace: made once, as a program makes them
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "clip":
        return _prepare_clip(case, gen)
    rows, width, hidden, dt = case["rows"], case["width"], case["hidden"], TORCH[case["dtype"]]
    tiles, save, f8, f32 = -(-hidden // 128), case["save"], torch.float8_e4m3fn, torch.float32
    s = dict(case)
    s["x"] = _normal(gen, rows, width).to(dt)  # rows as a norm leaves them
    w = _normal(gen, 2 * hidden, width, sigma=width**-0.5).to(dt)
    s["w_gate"], s["w_up"] = w[:hidden], w[hidden:]
    if case["op"] == "ffn":
        if case["p"] == "16":
            s["p_out"], s["p_scales"] = _empty(rows, hidden, dtype=dt), None
        elif case["p"] == "128":
            s["p_out"], s["p_scales"] = _empty(rows, hidden, dtype=f8), _empty(rows, tiles, dtype=f32)
        else:
            s["p_out"] = _empty(rows, hidden, dtype=f8)
            s["p_scales"] = _empty(rows, hidden // 32, dtype=torch.float8_e8m0fnu)
        if save == "16":
            kept = _empty(rows, 2 * hidden, dtype=dt)
            s["gate"], s["up"] = kept[:, :hidden], kept[:, hidden:]
        elif save == "8":
            s["ckpt"], s["ckpt_scales"] = _empty(2, rows, hidden, dtype=f8), _empty(2, rows, tiles, dtype=f32)
        return s
    s["dp"] = _normal(gen, rows, hidden, sigma=1e-2).to(dt)
    if save != "no":
        kept = s["x"].float() @ w.float().t()
        if save == "16":
            kept = kept.to(dt)
            s["gate"], s["up"] = kept[:, :hidden], kept[:, hidden:]
        else:
            pairs = [_quantize(v, 128) for v in (kept[:, :hidden], kept[:, hidden:])]
            s["ckpt"] = torch.stack([c.view(torch.uint8) for c, _ in pairs]).view(f8)
            s["ckpt_scales"] = torch.stack([v for _, v in pairs])
    s["dx"], s["dw"] = _empty(rows, width, dtype=dt), _empty(2 * hidden, width, dtype=dt)
    s["workspace"] = None  # scratch; its size is the operator's to say
    return s


# ---- the plain forms ---------------------------------------------------------------


def _quantize(v, block):
    """E4M3 codes of a float32 [rows, cols] with one scale for `block` elements of a row."""
    rows, cols = v.shape
    pad = -cols % block
    t = torch.cat([v, v.new_zeros(rows, pad)], 1) if pad else v
    t = t.reshape(rows, -1, block)
    amax = t.abs().amax(2, keepdim=True)
    if block == 128:
        scale = (amax / FP8_MAX)[..., 0]
        q = t * torch.where(amax > 0, FP8_MAX / amax, 0.0)
    else:
        e = (torch.frexp(amax.clamp(min=2.0**-126))[1] - 1 - FP8_EMAX).clamp(min=-127)
        q = torch.ldexp(t, -e)
        scale = (e[..., 0] + 127).to(torch.uint8).view(torch.float8_e8m0fnu)
    codes = q.clamp(-FP8_MAX, FP8_MAX).reshape(rows, -1)[:, :cols].contiguous().to(torch.float8_e4m3fn)
    return codes, scale


def _plain_ffn(s):
    dt, x = TORCH[s["dtype"]], s["x"].float()
    g, u = x @ s["w_gate"].float().t(), x @ s["w_up"].float().t()
    p = g / (1.0 + torch.exp(-g)) * u
    if s["p"] == "16":
        out = dict(p=p.to(dt))
    else:
        codes, scales = _quantize(p, int(s["p"]))
        out = dict(p=codes, p_scales=scales)
    if s["save"] == "16":
        out["gate"], out["up"] = g.to(dt), u.to(dt)
    elif s["save"] == "8":
        (gc, gs), (uc, us) = _quantize(g, 128), _quantize(u, 128)
        out["ckpt"] = torch.stack([gc.view(torch.uint8), uc.view(torch.uint8)]).view(torch.float8_e4m3fn)
        out["ckpt_scales"] = torch.stack([gs, us])
    return out


def _plain_ffn_bwd(s):
    dt, x = TORCH[s["dtype"]], s["x"].float()
    wg, wu = s["w_gate"].float(), s["w_up"].float()
    if s["save"] == "16":
        g, u = s["gate"].float(), s["up"].float()
    elif s["save"] == "8":
        cols = s["ckpt"].shape[-1]
        g, u = s["ckpt"].float() * s["ckpt_scales"].repeat_interleave(128, -1)[..., :cols]
    else:
        g, u = x @ wg.t(), x @ wu.t()
    d = s["dp"].float()
    sig = 1.0 / (1.0 + torch.exp(-g))
    dg, du = d * u * (sig * (1.0 + g * (1.0 - sig))), d * (g * sig)
    return dict(dx=(dg @ wg + du @ wu).to(dt), dw_gate=(dg.t() @ x).to(dt), dw_up=(du.t() @ x).to(dt))


def _plain_clip(s):
    norm = torch.stack([g.double().square().sum() for g in s["grads"]]).sum().sqrt()
    coef = (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0).float()
    [c.copy_(g.float() * coef) for g, c in zip(s["grads"], s["clipped"])]
    return dict(norm=norm.float().reshape(1), clipped=s["flat"])


# ---- the library's calls -----------------------------------------------------------


def _own_ffn(s):
    mp = _mp()
    mp.linear_swiglu(s["x"], s["w_gate"], s["w_up"], s["p_out"], p_scales=s["p_scales"], gate=s.get("gate"),
                     up=s.get("up"), ckpt=s.get("ckpt"), ckpt_scales=s.get("ckpt_scales"),
                     scale_block=32 if s["p"] == "32" else 128)
    out = dict(p=s["p_out"])
    if s["p"] != "16":
        out["p_scales"] = s["p_scales"]
    return out | {k: s[k] for k in {"no": (), "16": ("gate", "up"), "8": ("ckpt", "ckpt_scales")}[s["save"]]}


def _own_ffn_bwd(s):
    mp = _mp()
    if s["workspace"] is None:  # made once, as a program makes it, and kept
        s["workspace"] = mp.new_linear_swiglu_workspace(s["rows"], s["width"], s["hidden"])
    dwg, dwu = s["dw"][:s["hidden"]], s["dw"][s["hidden"]:]
    mp.linear_swiglu_backward(s["dp"], s["x"], s["w_gate"], s["w_up"], s["dx"], dwg, dwu, s["workspace"],
                              gate=s.get("gate"), up=s.get("up"), ckpt=s.get("ckpt"), ckpt_scales=s.get("ckpt_scales"))
    return dict(dx=s["dx"], dw_gate=dwg, dw_up=dwu)


def _own_clip(s):
    mp = _mp()
    if s["plan"] is None:
        grads = mp.make_grad_array(s["grads"], s["clipped"])
        s["plan"] = grads, mp.new_grad_norm_workspace(grads)
    grads, workspace = s["plan"]
    mp.mp_grad_norm(grads, s["norm"], workspace)
    mp.mp_grad_clip(grads, s["norm"], s["max_norm"])
    return dict(norm=s["norm"], clipped=s["flat"])


_PLAIN = {"ffn": _plain_ffn, "ffn_bwd": _plain_ffn_bwd, "clip": _plain_clip}
_OWN = {"ffn": _own_ffn, "ffn_bwd": _own_ffn_bwd, "clip": _own_clip}


def run(state):
    return (_OWN if own else _PLAIN)[state["op"]](state)


# ---- the definitions in 64 bits ----------------------------------------------------


def _exact_codes(v, block):
    """Unrounded values of the codes, and the scales they are relative to."""
    rows, cols = v.shape
    width = -(-cols // block) * block
    t = torch.nn.functional.pad(v, (0, width - cols)).view(rows, width // block, block)
    amax = t.abs().max(-1).values
    if block == 128:
        scale = amax / FP8_MAX
    else:
        scale = torch.exp2((torch.floor(torch.log2(amax)) - FP8_EMAX).clamp(min=-127))
    codes = (t / scale.unsqueeze(-1)).nan_to_num(0.0).clamp(-FP8_MAX, FP8_MAX)  # a block of zeros: 0 / 0
    return codes.view(rows, width)[:, :cols], scale


def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "clip":
        squares = torch.zeros((), dtype=f64, device="cuda")
        for g in s["grads"]:
            squares += torch.linalg.vector_norm(g.to(f64)) ** 2
        norm = squares.pow(0.5)
        factor = min(1.0, case["max_norm"] / (float(norm) + 1e-6))
        clipped = torch.zeros(s["flat"].numel(), dtype=f64, device="cuda")
        start = s["flat"].data_ptr()
        for g, c in zip(s["grads"], s["clipped"]):
            at = (c.data_ptr() - start) // c.element_size()
            clipped[at:at + g.numel()] = g.to(f64).reshape(-1) * factor
        return dict(norm=norm.reshape(1), clipped=clipped)
    x, wg, wu = (s[k].to(f64) for k in ("x", "w_gate", "w_up"))
    if case["op"] == "ffn_bwd" and case["save"] == "16":
        g, u = s["gate"].to(f64), s["up"].to(f64)
    elif case["op"] == "ffn_bwd" and case["save"] == "8":
        at = torch.arange(case["hidden"], device="cuda") // 128
        g, u = (s["ckpt"][k].to(f64) * s["ckpt_scales"][k].to(f64)[:, at] for k in (0, 1))
    else:
        g, u = torch.einsum("rk,hk->rh", x, wg), torch.einsum("rk,hk->rh", x, wu)
    sig = torch.special.expit(g)
    if case["op"] == "ffn_bwd":
        d = s["dp"].to(f64)
        dg, du = d * u * sig * (1 + g - g * sig), d * g * sig
        dx = torch.einsum("rh,hk->rk", dg, wg) + torch.einsum("rh,hk->rk", du, wu)
        return dict(dx=dx, dw_gate=torch.einsum("rh,rk->hk", dg, x), dw_up=torch.einsum("rh,rk->hk", du, x))
    p = g * sig * u
    if case["p"] == "16":
        out = dict(p=p)
    else:
        out = dict(zip(("p", "p_scales"), _exact_codes(p, int(case["p"]))))
    if case["save"] == "16":
        out.update(gate=g, up=u)
    elif case["save"] == "8":
        pairs = [_exact_codes(v, 128) for v in (g, u)]
        out["ckpt"], out["ckpt_scales"] = (torch.stack(v) for v in zip(*pairs))
    return out
