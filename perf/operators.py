"""The cases on which the block operators with 8-bit outputs and 8-bit
checkpoints are measured: root-mean-square norm with the residual's addition,
the SwiGLU product, and the backward passes of both.

``run`` computes a case either in its plain form (elementary torch operations
in binary32) or, with ``own`` set, through the library's entry points.
Hidden sizes 4096 and 5120, the feed-forward size 14336, the width 12288 and
the token counts 8192 and 16384 are those of this repository's workloads; the
others are generic.
"""
import torch

own = False

EPS = 1e-5
TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
FP8_MAX = {"e4m3": 448.0, "e5m2": 57344.0}
FP8_EMAX = {"e4m3": 8, "e5m2": 15}
MOST = 8192 * 14336  # elements of the largest case


def _mp():
    import mixed_precision_numerics_gb300 as mp

    return mp


# ---- the cases ---------------------------------------------------------------------


def listed():
    return [
        # one token of a decoding step: the norm before a block, its FP8 input for the next product, nothing saved
        dict(name="norm 1 token", op="norm", rows=1, cols=4096, dtype="bf16", fp8="e4m3", block=128, save=False),
        # a ragged decoding batch in FP16, microscaled output
        dict(name="norm 37 tokens f16 mx", op="norm", rows=37, cols=5120, dtype="f16", fp8="e4m3", block=32, save=False),
        # a training micro-batch of the 8B-sized parameter list, checkpointed in 8 bits
        dict(name="norm 8192x4096 saved", op="norm", rows=8192, cols=4096, dtype="bf16", fp8="e4m3", block=128, save=True),
        # the activation shape of the quantiser workload, microscaled output, checkpointed
        dict(name="norm 16384x5120 mx saved", op="norm", rows=16384, cols=5120, dtype="bf16", fp8="e4m3", block=32, save=True),
        # a small FP32 model with a row length that ends inside a 128-tile; the stream saved as it is
        dict(name="norm_bwd 301x1040 f32", op="norm_bwd", rows=301, cols=1040, dtype="f32", save=False),
        # the training micro-batch's backward pass from the 8-bit checkpoint
        dict(name="norm_bwd 8192x4096 saved", op="norm_bwd", rows=8192, cols=4096, dtype="bf16", save=True),
        # the same at the largest token count
        dict(name="norm_bwd 16384x5120 saved", op="norm_bwd", rows=16384, cols=5120, dtype="bf16", save=True),
        # one token of a decoding step through the gated feed-forward product
        dict(name="swiglu 1 token", op="swiglu", rows=1, cols=14336, dtype="bf16", fp8="e4m3", block=128, save=False),
        # the training micro-batch: FP8 product for the down projection, gate and up checkpointed in 8 bits
        dict(name="swiglu 8192x14336 saved", op="swiglu", rows=8192, cols=14336, dtype="bf16", fp8="e4m3", block=128, save=True),
        # a small FP16 model whose rows end inside a 128-tile
        dict(name="swiglu_bwd 301x1456 f16", op="swiglu_bwd", rows=301, cols=1456, dtype="f16", save=True),
        # the training micro-batch's backward pass from the 8-bit checkpoint
        dict(name="swiglu_bwd 8192x14336 saved", op="swiglu_bwd", rows=8192, cols=14336, dtype="bf16", save=True),
        # gate and up kept in 16 bits, without a checkpoint
        dict(name="swiglu_bwd 2048x12288 kept", op="swiglu_bwd", rows=2048, cols=12288, dtype="bf16", save=False),
    ]


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "swiglu", "swiglu_bwd"])
    rows = round(2 ** rng.uniform(0.0, 14.0))
    save = rng.random() < 0.6
    fwd = op in ("norm", "swiglu")
    block = rng.choice([128, 32]) if fwd else 128
    step = 32 if block == 32 else 16  # what the row length has to be a multiple of
    cols = max(1, round(2 ** rng.uniform(5.0, 14.0) / step)) * step
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    cap = MOST // 2 if dtype == "f32" else MOST
    rows = max(1, min(rows, cap // cols))
    case = dict(op=op, rows=rows, cols=cols, dtype=dtype, save=save)
    if fwd:
        case.update(fp8=rng.choice(["e4m3", "e4m3", "e5m2"]), block=block)
    return case


def work(case):
    n, rows, cols = case["rows"] * case["cols"], case["rows"], case["cols"]
    es = 4 if case["dtype"] == "f32" else 2
    saved = n + 4 * rows * -(-cols // 128)  # one 8-bit checkpoint: codes and FP32 scales
    op = case["op"]
    if op in ("norm", "swiglu"):
        out = n + (rows * (cols // 32) if case["block"] == 32 else 4 * rows * -(-cols // 128))
    if op == "norm":  # x, residual, h, weight, rstd
        return {"bytes": 3 * es * n + out + saved * case["save"] + es * cols + 4 * rows, "flops": 8 * n}
    if op == "norm_bwd":  # dy, dh, dx, the stream, weight, dweight, rstd
        return {"bytes": 3 * es * n + (saved if case["save"] else es * n) + 2 * es * cols + 4 * rows, "flops": 12 * n}
    if op == "swiglu":  # gate, up
        return {"bytes": 2 * es * n + out + 2 * saved * case["save"], "flops": 10 * n}
    return {"bytes": 3 * es * n + (2 * saved if case["save"] else 2 * es * n), "flops": 14 * n}


# ---- inputs ------------------------------------------------------------------------


def _normal(gen, *shape, sigma=1.0):
    return torch.randn(*shape, generator=gen, device="cuda") * sigma


def _checkpoint(v):
    """8-bit codes and scales of 1x128 tiles, as a program has them from the forward pass."""
    codes, scales = _quantize(v.float(), "e4m3", 128)
    return codes, scales


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rows, cols, dt = case["rows"], case["cols"], TORCH[case["dtype"]]
    op, save = case["op"], case["save"]
    tiles = -(-cols // 128)

    def empty(*shape, dtype=dt):
        return torch.empty(*shape, dtype=dtype, device="cuda")

    s = dict(case)
    if op in ("norm", "norm_bwd"):
        # a few channels carry much larger values than the others
        channel = 1.0 + 20.0 * (torch.rand(cols, generator=gen, device="cuda") < 0.01)
        s["weight"] = (1.0 + _normal(gen, cols, sigma=0.1)).to(dt)
        stream = (_normal(gen, rows, cols) * channel).to(dt)
    if op == "norm":
        s["x"], s["residual"] = _normal(gen, rows, cols, sigma=0.3).to(dt), stream
        s["h"] = empty(rows, cols)
        s["rstd"] = empty(rows, dtype=torch.float32)
    elif op == "norm_bwd":
        s["dy"] = _normal(gen, rows, cols, sigma=1e-2).to(dt)
        s["dh"] = _normal(gen, rows, cols, sigma=1e-2).to(dt)
        s["rstd"] = 1.0 / torch.sqrt(stream.float().square().mean(1) + EPS)
        if save:
            s["ckpt"], s["ckpt_scales"] = _checkpoint(stream)
        else:
            s["h"] = stream
        s["dx"], s["dweight"] = empty(rows, cols), empty(cols)
        # the sums over rows are formed in here; its size is the operator's to say
        s["workspace"] = None
    elif op == "swiglu":
        gate_up = _normal(gen, rows, 2 * cols, sigma=1.5).to(dt)  # one product gives both halves
        s["gate"], s["up"] = gate_up[:, :cols], gate_up[:, cols:]
    else:
        s["dp"] = _normal(gen, rows, cols, sigma=1e-2).to(dt)
        gate_up = _normal(gen, rows, 2 * cols, sigma=1.5).to(dt)
        s["gate"], s["up"] = gate_up[:, :cols], gate_up[:, cols:]
        if save:
            pairs = [_checkpoint(s.pop("gate")), _checkpoint(s.pop("up"))]
            s["ckpt"] = torch.stack([c.view(torch.uint8) for c, _ in pairs]).view(torch.float8_e4m3fn)
            s["ckpt_scales"] = torch.stack([v for _, v in pairs])
        d = empty(rows, 2 * cols)
        s["dgate"], s["dup"] = d[:, :cols], d[:, cols:]
    if op in ("norm", "swiglu"):
        s["y"] = empty(rows, cols, dtype=FP8[case["fp8"]])
        if case["block"] == 32:
            s["y_scales"] = empty(rows, cols // 32, dtype=torch.float8_e8m0fnu)
        else:
            s["y_scales"] = empty(rows, tiles, dtype=torch.float32)
        if save:
            lead = (2,) if op == "swiglu" else ()
            s["ckpt"] = empty(*lead, rows, cols, dtype=torch.float8_e4m3fn)
            s["ckpt_scales"] = empty(*lead, rows, tiles, dtype=torch.float32)
    return s


# ---- the plain forms ---------------------------------------------------------------


def _tiles(v, block):
    rows, cols = v.shape
    pad = -cols % block
    if pad:
        v = torch.cat([v, v.new_zeros(rows, pad)], 1)
    return v.reshape(rows, -1, block)


def _quantize(v, fp8, block):
    """8-bit codes of a float32 [rows, cols] with one scale for `block` elements of a row."""
    rows, cols = v.shape
    t = _tiles(v, block)
    amax = t.abs().amax(2, keepdim=True)
    top = FP8_MAX[fp8]
    if block == 128:
        scale = amax / top
        q = t * torch.where(amax > 0, top / amax, 0.0)
        scale = scale[..., 0]
    else:
        e = (torch.frexp(amax.clamp(min=2.0**-126))[1] - 1 - FP8_EMAX[fp8]).clamp(min=-127)
        q = torch.ldexp(t, -e)
        scale = (e[..., 0] + 127).to(torch.uint8).view(torch.float8_e8m0fnu)
    codes = q.clamp(-top, top).reshape(rows, -1)[:, :cols].contiguous().to(FP8[fp8])
    return codes, scale


def _dequantize(codes, scales):
    """float32 values of 1x128 tiles; any leading dimensions."""
    cols = codes.shape[-1]
    return codes.float() * scales.repeat_interleave(128, -1)[..., :cols]


def _plain_norm(s):
    dt = TORCH[s["dtype"]]
    h = (s["x"].float() + s["residual"].float()).to(dt)  # the stream that the next block reads
    v = h.float()
    rstd = 1.0 / torch.sqrt((v * v).mean(1) + EPS)
    y, y_scales = _quantize(v * rstd[:, None] * s["weight"].float(), s["fp8"], s["block"])
    out = dict(h=h, y=y, y_scales=y_scales, rstd=rstd)
    if s["save"]:
        out["ckpt"], out["ckpt_scales"] = _quantize(v, "e4m3", 128)
    return out


def _plain_norm_bwd(s):
    dt = TORCH[s["dtype"]]
    dy = s["dy"].float()
    v = _dequantize(s["ckpt"], s["ckpt_scales"]) if s["save"] else s["h"].float()
    xhat = v * s["rstd"][:, None]
    g = dy * s["weight"].float()
    c = (g * xhat).mean(1, keepdim=True)
    dx = s["rstd"][:, None] * (g - xhat * c) + s["dh"].float()
    return dict(dx=dx.to(dt), dweight=(dy * xhat).sum(0).to(dt))


def _plain_swiglu(s):
    g, u = s["gate"].float(), s["up"].float()
    y, y_scales = _quantize(g / (1.0 + torch.exp(-g)) * u, s["fp8"], s["block"])
    out = dict(y=y, y_scales=y_scales)
    if s["save"]:
        gc, gs = _quantize(g, "e4m3", 128)
        uc, us = _quantize(u, "e4m3", 128)
        out["ckpt"] = torch.stack([gc.view(torch.uint8), uc.view(torch.uint8)]).view(torch.float8_e4m3fn)
        out["ckpt_scales"] = torch.stack([gs, us])
    return out


def _plain_swiglu_bwd(s):
    dt = TORCH[s["dtype"]]
    if s["save"]:
        g, u = _dequantize(s["ckpt"], s["ckpt_scales"])
    else:
        g, u = s["gate"].float(), s["up"].float()
    d = s["dp"].float()
    sig = 1.0 / (1.0 + torch.exp(-g))
    dgate = d * u * (sig * (1.0 + g * (1.0 - sig)))
    return dict(dgate=dgate.to(dt), dup=(d * (g * sig)).to(dt))


# ---- the library's calls -----------------------------------------------------------


def _own_norm(s):
    mp = _mp()
    mp.rmsnorm_residual_fp8(s["x"], s["weight"], s["y"], s["y_scales"], residual=s["residual"], h=s["h"],
                            rstd=s["rstd"], ckpt=s.get("ckpt"), ckpt_scales=s.get("ckpt_scales"), eps=EPS,
                            fp8_dtype=mp.MP_E4M3 if s["fp8"] == "e4m3" else mp.MP_E5M2, scale_block=s["block"])
    keys = ("h", "y", "y_scales", "rstd") + (("ckpt", "ckpt_scales") if s["save"] else ())
    return {k: s[k] for k in keys}


def _own_norm_bwd(s):
    mp = _mp()
    if s["workspace"] is None:  # made once, as a program makes it, and kept
        s["workspace"] = mp.new_rmsnorm_workspace(s["rows"], s["cols"])
    mp.rmsnorm_residual_backward(s["dy"], s["weight"], s["rstd"], s["dx"], s["dweight"], s["workspace"],
                                 h=s.get("h"), ckpt=s.get("ckpt"), ckpt_scales=s.get("ckpt_scales"), dh=s["dh"])
    return dict(dx=s["dx"], dweight=s["dweight"])


def _own_swiglu(s):
    mp = _mp()
    mp.swiglu_fp8(s["gate"], s["up"], s["y"], s["y_scales"], ckpt=s.get("ckpt"), ckpt_scales=s.get("ckpt_scales"),
                  fp8_dtype=mp.MP_E4M3 if s["fp8"] == "e4m3" else mp.MP_E5M2, scale_block=s["block"])
    return {k: s[k] for k in ("y", "y_scales") + (("ckpt", "ckpt_scales") if s["save"] else ())}


def _own_swiglu_bwd(s):
    _mp().swiglu_backward(s["dp"], s["dgate"], s["dup"], gate=s.get("gate"), up=s.get("up"), ckpt=s.get("ckpt"),
                          ckpt_scales=s.get("ckpt_scales"))
    return dict(dgate=s["dgate"], dup=s["dup"])


_PLAIN = {"norm": _plain_norm, "norm_bwd": _plain_norm_bwd, "swiglu": _plain_swiglu, "swiglu_bwd": _plain_swiglu_bwd}
_OWN = {"norm": _own_norm, "norm_bwd": _own_norm_bwd, "swiglu": _own_swiglu, "swiglu_bwd": _own_swiglu_bwd}


def run(state):
    return (_OWN if own else _PLAIN)[state["op"]](state)


# ---- the definitions in 64 bits ----------------------------------------------------


def _exact_codes(v, case):
    """Unrounded values of the codes, and the scales they are relative to."""
    rows, cols = v.shape
    fp8, block = case["fp8"], case["block"]
    width = -(-cols // block) * block
    t = torch.nn.functional.pad(v, (0, width - cols)).view(rows, width // block, block)
    amax = t.abs().max(-1).values
    if block == 128:
        scale = amax / FP8_MAX[fp8]
    else:
        scale = torch.exp2((torch.floor(torch.log2(amax)) - FP8_EMAX[fp8]).clamp(min=-127))
    codes = (t / scale.unsqueeze(-1)).nan_to_num(0.0).clamp(-FP8_MAX[fp8], FP8_MAX[fp8])  # a tile of zeros: 0 / 0
    return codes.view(rows, width)[:, :cols], scale


def _exact_saved(s, which=None):
    codes, scales = s["ckpt"], s["ckpt_scales"]
    if which is not None:
        codes, scales = codes[which], scales[which]
    at = torch.arange(codes.shape[1], device=codes.device) // 128
    return codes.to(torch.float64) * scales.to(torch.float64)[:, at]


def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    ckpt = dict(case, fp8="e4m3", block=128)
    op = case["op"]
    if op == "norm":
        # h is the stored stream: the sum rounded to its type, which the rest is a function of
        h = (s["x"].to(f64) + s["residual"].to(f64)).to(TORCH[case["dtype"]]).to(f64)
        rstd = (h.pow(2).sum(1) / case["cols"] + EPS).rsqrt()
        y, y_scales = _exact_codes(torch.einsum("rc,r,c->rc", h, rstd, s["weight"].to(f64)), case)
        out = dict(h=h, y=y, y_scales=y_scales, rstd=rstd)
        if case["save"]:
            out["ckpt"], out["ckpt_scales"] = _exact_codes(h, ckpt)
        return out
    if op == "norm_bwd":
        v = _exact_saved(s) if case["save"] else s["h"].to(f64)
        dy, r = s["dy"].to(f64), s["rstd"].to(f64)
        dweight = torch.einsum("rc,rc,r->c", dy, v, r)
        dy = dy * s["weight"].to(f64)
        dot = torch.einsum("rc,rc->r", dy, v)
        dx = dy * r[:, None] - v * (dot * r.pow(3) / case["cols"])[:, None]
        return dict(dx=dx + s["dh"].to(f64), dweight=dweight)
    if op == "swiglu":
        g, u = s["gate"].to(f64), s["up"].to(f64)
        y, y_scales = _exact_codes(g * torch.special.expit(g) * u, case)
        out = dict(y=y, y_scales=y_scales)
        if case["save"]:
            pairs = [_exact_codes(v, ckpt) for v in (g, u)]
            out["ckpt"], out["ckpt_scales"] = (torch.stack(v) for v in zip(*pairs))
        return out
    if case["save"]:
        g, u = _exact_saved(s, 0), _exact_saved(s, 1)
    else:
        g, u = s["gate"].to(f64), s["up"].to(f64)
    d, sig = s["dp"].to(f64), torch.special.expit(g)
    return dict(dgate=d * u * sig * (1 + g - g * sig), dup=d * g * sig)
