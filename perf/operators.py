"""Cases of the normalisation and gradient-clipping operators, for timing.

Two operators of a training step around the spectral layers:

* group norm with an activation (none, GELU, SiLU), forward and backward.  A
  field is channels last [B, ..., C] (where channel MLPs keep it) or channels
  first [B, C, ...] (where the transforms read it); input and output each have
  their own layout, and a 16-bit field may leave as float32;
* the global norm of all gradients of a model and the clipping by it:
  complex64 spectral weights beside float32, bfloat16 or float16 tensors.

With `own` false run() computes plain forms in elementary torch operations;
with `own` true it calls fft_spectral_convolution_amd.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZES = {"f32": 4, "bf16": 2, "f16": 2}


def _gn(name, backward, B, C, grid, groups, act, dtype, out_dtype, last, out_last):
    case = {"op": "group_norm", "backward": backward, "B": B, "C": C, "grid": grid, "groups": groups, "act": act,
            "dtype": dtype, "out_dtype": out_dtype, "last": last, "out_last": out_last}
    return dict(case, name=name) if name else case


def _clip(name, mode, layers, width, mx, my, dtype, lift):
    case = {"op": "clip", "mode": mode, "layers": layers, "width": width, "mx": mx, "my": my, "dtype": dtype,
            "lift": lift}
    return dict(case, name=name) if name else case


def listed():
    return [
        # the 32 x 32 workload's field, one small model step: latency
        _gn("gn_32x32_last_f32", False, 2, 4, "32x32", 2, "gelu", "f32", "f32", True, True),
        # the 64 x 64 workload's field kept in 16 bits between channel MLPs
        _gn("gn_64x64_last_bf16", False, 16, 32, "64x64", 8, "gelu", "bf16", "bf16", True, True),
        # the 128 x 128 workload, channels last
        _gn("gn_128x128_last_f32", False, 32, 64, "128x128", 8, "gelu", "f32", "f32", True, True),
        # the same field as the spectral convolution writes and reads it
        _gn("gn_128x128_first_f32", False, 32, 64, "128x128", 32, "silu", "f32", "f32", False, False),
        # from a 16-bit channels-last MLP into the float32 channels-first transforms
        _gn("gn_128x128_cross_bf16", False, 32, 64, "128x128", 8, "gelu", "bf16", "f32", True, False),
        # the 2048 x 2048 workload: two large images
        _gn("gn_2048x2048_last_f32", False, 2, 16, "2048x2048", 4, "silu", "f32", "f32", True, True),
        # training: the backward pass of the 128 x 128 field
        _gn("gn_bwd_128x128_last_f32", True, 32, 64, "128x128", 8, "gelu", "f32", "f32", True, True),
        # training: the 1D workload's sequences, channels first
        _gn("gn_bwd_4096_first_f32", True, 256, 64, "4096", 16, "none", "f32", "f32", False, False),
        # training on an odd grid and channel count in 16 bits
        _gn("gn_bwd_61x47_last_f16", True, 3, 30, "61x47", 5, "silu", "f16", "f16", True, True),
        # gradients of one small layer: latency
        _clip("clip_small", "clip", 1, 4, 8, 8, "f32", 16),
        # gradients of a four-layer model of the 128 x 128 workload, clipped into the optimizer's buffers
        _clip("clip_128x128_model", "clip", 4, 64, 32, 32, "f32", 128),
        # many small tensors, norm below the limit: a usual step late in training, nothing to change
        _clip("norm_many_bf16", "below", 48, 96, 5, 5, "bf16", 384),
    ]


def _loguniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.3:
        mode = rng.choice(["clip", "below", "two_step"])
        width, layers = _loguniform(rng, 4, 96), _loguniform(rng, 1, 48)
        mx, my = _loguniform(rng, 1, 16), _loguniform(rng, 1, 16)
        while 4 * layers * mx * my * width * width > 1 << 26:
            mx, my = max(1, mx // 2), max(1, my // 2)
        return _clip(None, mode, layers, width, mx, my, rng.choice(list(DTYPES)), _loguniform(rng, 1, 4 * width))
    backward = rng.random() < 0.5
    total = _loguniform(rng, 1 << 10, 1 << 25)
    C = _loguniform(rng, 1, 512)
    B = min(_loguniform(rng, 1, 64), max(1, total // C))
    P = max(1, total // (B * C))
    groups = rng.choice([g for g in range(1, C + 1) if C % g == 0])
    if P * (C // groups) < 4:      # a group of one or two values has no spread worth measuring
        groups = 1
    if rng.random() < 0.5:
        grid = str(P)
    else:
        W = max(1, min(P, int(math.sqrt(P) * rng.uniform(0.5, 2.0))))
        grid = "%dx%d" % (max(1, P // W), W)
    dtype = rng.choice(list(DTYPES))
    out_dtype = rng.choice([dtype, "f32"])
    last = rng.random() < 0.6
    out_last = last if rng.random() < 0.7 else not last
    return _gn(None, backward, B, C, grid, groups, rng.choice(["none", "gelu", "silu"]), dtype, out_dtype, last,
               out_last)


def _grid(case):
    return [int(v) for v in case["grid"].split("x")]


def _shape(case, last):
    grid = _grid(case)
    return [case["B"], *grid, case["C"]] if last else [case["B"], case["C"], *grid]


def _relayout(t, last, out_last):
    if last == out_last:
        return t
    return t.movedim(-1, 1) if last else t.movedim(1, -1)


def _tensor_shapes(case):
    """Shapes and types of one model's gradients: lifting, per layer spectral and pointwise weights and a norm, and
    projection."""
    w, dt = case["width"], DTYPES[case["dtype"]]
    shapes = [((3, w), dt), ((w,), dt)]
    for _ in range(case["layers"]):
        shapes += [((2, case["mx"], case["my"], w, w), torch.complex64), ((w, w), dt), ((w,), dt),
                   ((w,), torch.float32), ((w,), torch.float32)]
    return shapes + [((w, case["lift"]), dt), ((case["lift"],), dt), ((case["lift"], 1), dt), ((1,), dt)]


def _flat_types(case):
    return list(dict.fromkeys(d for _, d in _tensor_shapes(case)))


def _views(flat, shapes):
    """The model's tensors as slices of one packed buffer per type, as gradient buckets hold them."""
    at = dict.fromkeys(flat, 0)
    views = []
    for s, d in shapes:
        n = math.prod(s)
        views.append(flat[d][at[d]:at[d] + n].view(s))
        at[d] += n
    return views


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    if case["op"] == "clip":
        shapes = _tensor_shapes(case)
        # a model's gradient norm is a few units whatever its size
        n = sum(math.prod(s) * (2 if d.is_complex else 1) for s, d in shapes)
        std = 3.0 / math.sqrt(n)
        flat = {}
        for d in _flat_types(case):
            m = sum(math.prod(s) for s, t in shapes if t == d)
            flat[d] = torch.view_as_complex(randn(m, 2).mul_(std)) if d.is_complex else randn(m).mul_(std).to(d)
        # the limit is exceeded, or far away
        state = {"case": case, "flat": flat, "grads": _views(flat, shapes), "max_norm": 1.0, "outs": None}
        if case["mode"] == "below":
            state["max_norm"] = 100.0
        else:
            state["flat_out"] = {d: torch.empty_like(f) for d, f in flat.items()}
            state["outs"] = _views(state["flat_out"], shapes)
        return state

    B, C, last = case["B"], case["C"], case["last"]
    cshape = [1] * (len(_grid(case)) + 1) + [C] if last else [1, C] + [1] * len(_grid(case))
    # every channel has its own level and spread
    scale, level = torch.exp(0.5 * randn(C)).view(cshape), randn(C).view(cshape)
    x = (randn(*_shape(case, last)) * scale + level).to(DTYPES[case["dtype"]])
    state = {"case": case, "x": x, "weight": 1.0 + 0.2 * randn(C), "bias": 0.2 * randn(C), "eps": 1e-5}
    if case["backward"]:
        # what the forward call left: mean and 1 / deviation of each group, [B, groups, 2]
        xg = x.float().view(B, -1, case["groups"], C // case["groups"]) if last else \
            x.float().view(B, case["groups"], -1)
        dims = (1, 3) if last else (2,)
        mean = xg.mean(dims, keepdim=True)
        var = (xg - mean).square_().mean(dims)
        state["stats"] = torch.stack([mean.view(B, -1), torch.rsqrt(var + state["eps"]).view(B, -1)], dim=2)
        state["grad_out"] = randn(*_shape(case, case["out_last"])).to(DTYPES[case["out_dtype"]])
    return state


def _channel_view(v, case, last):
    n = len(_grid(case))
    return v.view([1] * (n + 1) + [case["C"]] if last else [1, case["C"]] + [1] * n)


def _per_channel(stat, case, last):
    """[B, groups] -> broadcastable over the field."""
    full = stat.repeat_interleave(case["C"] // case["groups"], dim=1)
    n = len(_grid(case))
    return full.view([case["B"]] + [1] * n + [case["C"]] if last else [case["B"], case["C"]] + [1] * n)


def _act(z, act):
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    return z / (1.0 + torch.exp(-z)) if act == "silu" else z


def _act_slope(z, act):
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (0.5 / math.pi) ** 0.5
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    return torch.ones_like(z)


def _group_norm(state):
    case, last = state["case"], state["case"]["last"]
    B, C, groups = case["B"], case["C"], case["groups"]
    x = state["x"].float()
    xg = x.view(B, -1, groups, C // groups) if last else x.view(B, groups, -1)
    dims = (1, 3) if last else (2,)
    mean = xg.mean(dims, keepdim=True)
    var = (xg - mean).square().mean(dims).view(B, groups)
    mean = mean.view(B, groups)
    rstd = torch.rsqrt(var + state["eps"])
    z = (x - _per_channel(mean, case, last)) * _per_channel(rstd, case, last)
    z = z * _channel_view(state["weight"], case, last) + _channel_view(state["bias"], case, last)
    y = _relayout(_act(z, case["act"]), last, case["out_last"]).contiguous()
    return {"out": y.to(DTYPES[case["out_dtype"]]), "stats": torch.stack([mean, rstd], dim=2)}


def _group_norm_backward(state):
    case, last = state["case"], state["case"]["last"]
    B, C, groups = case["B"], case["C"], case["groups"]
    x = state["x"].float()
    dy = _relayout(state["grad_out"].float(), case["out_last"], last)
    mean, rstd = state["stats"].unbind(2)
    w = _channel_view(state["weight"], case, last)
    xh = (x - _per_channel(mean, case, last)) * _per_channel(rstd, case, last)
    g = dy * _act_slope(xh * w + _channel_view(state["bias"], case, last), case["act"])
    chan = tuple(d for d in range(x.dim()) if d != (x.dim() - 1 if last else 1))
    grad_w, grad_b = (g * xh).sum(chan), g.sum(chan)
    gw = (g * w).contiguous()
    split = (B, -1, groups, C // groups) if last else (B, groups, -1)
    dims = (1, 3) if last else (2,)
    s1 = gw.view(split).mean(dims).view(B, groups)
    s2 = (gw * xh).view(split).mean(dims).view(B, groups)
    gx = (gw - _per_channel(s1, case, last) - xh * _per_channel(s2, case, last)) * _per_channel(rstd, case, last)
    return {"grad_x": gx.to(DTYPES[case["dtype"]]), "grad_weight": grad_w,
            "grad_bias": grad_b}


def _real(g):
    return torch.view_as_real(g) if g.is_complex() else g


def _clip_plain(state):
    grads = state["grads"]
    # long sums in 64 bits
    norm = torch.stack([_real(g).float().square().sum(dtype=torch.float64) for g in grads]).sum().sqrt()
    coef = torch.clamp(state["max_norm"] / (norm + 1e-6), max=1.0).float()
    outs = state["grads"] if state["outs"] is None else state["outs"]
    for g, o in zip(grads, outs):
        _real(o).copy_(_real(g).float() * coef)
    return _clip_outputs(state, norm.float())


def _clip_outputs(state, norm):
    flat = state["flat"] if state["outs"] is None else state["flat_out"]
    return {"norm": norm, **{str(d).split(".")[1]: f for d, f in flat.items()}}


def run(state):
    case = state["case"]
    if not own:
        if case["op"] == "clip":
            return _clip_plain(state)
        return _group_norm_backward(state) if case["backward"] else _group_norm(state)
    import fft_spectral_convolution_amd as fno
    if case["op"] == "clip":
        grads = state["grads"]
        if case["mode"] == "two_step":     # the norm is looked at (or reduced over ranks) before the clipping
            norm = fno.fno_grad_norm(grads)
            fno.fno_clip_grad_norm(grads, state["max_norm"], norm=norm, out=state["outs"])
            return _clip_outputs(state, norm)
        norm = fno.fno_clip_grad_norm(grads, state["max_norm"], out=state["outs"])
        return _clip_outputs(state, norm)
    layout = {"channels_last": case["last"], "out_channels_last": case["out_last"]}
    if case["backward"]:
        gx, gw, gb = fno.fno_group_norm_backward(state["x"], state["stats"], state["grad_out"], case["groups"],
                                                 weight=state["weight"], bias=state["bias"], act=case["act"],
                                                 **layout)
        return {"grad_x": gx, "grad_weight": gw, "grad_bias": gb}
    out, stats = fno.fno_group_norm(state["x"], case["groups"], weight=state["weight"], bias=state["bias"],
                                    eps=state["eps"], act=case["act"], out_dtype=DTYPES[case["out_dtype"]], **layout)
    return {"out": out, "stats": stats}


def work(case):
    if case["op"] == "clip":
        shapes = _tensor_shapes(case)
        n = sum(math.prod(s) * (2 if d.is_complex else 1) for s, d in shapes)
        moved = sum(math.prod(s) * d.itemsize for s, d in shapes)
        below = case["mode"] == "below"
        return {"bytes": moved * (1 if below else 2), "flops": n * (2 if below else 3)}
    n = math.prod(_shape(case, True))
    size, out_size = SIZES[case["dtype"]], SIZES[case["out_dtype"]]
    stats = 8 * case["B"] * case["groups"]
    if case["backward"]:
        return {"bytes": n * (2 * size + out_size) + stats + 16 * case["C"], "flops": 20 * n}
    return {"bytes": n * (size + out_size) + stats + 8 * case["C"], "flops": 10 * n}


def exact(case, seed):
    """The definitions in float64: the norm over explicit [B, G, D, P] groups, gradients by differentiation."""
    state = prepare(case, seed)
    if case["op"] == "clip":
        wide = {d: f.to(torch.complex128 if d.is_complex else torch.float64) for d, f in state["flat"].items()}
        norm = math.sqrt(sum(float(torch.linalg.vector_norm(f)) ** 2 for f in wide.values()))
        coef = min(1.0, state["max_norm"] / (norm + 1e-6))
        return {"norm": torch.tensor(norm, dtype=torch.float64, device="cuda"),
                **{str(d).split(".")[1]: f * coef for d, f in wide.items()}}

    B, C, G = case["B"], case["C"], case["groups"]

    def groups_of(t, last):
        flat = t.double().reshape(B, -1, C).transpose(1, 2) if last else t.double().reshape(B, C, -1)
        return flat.reshape(B, G, C // G, -1)

    def layout_of(t, last):
        flat = t.reshape(B, C, -1)
        return (flat.transpose(1, 2) if last else flat).reshape(_shape(case, last))

    x = groups_of(state["x"], case["last"])
    w = state["weight"].double().view(1, G, C // G, 1)
    b = state["bias"].double().view(1, G, C // G, 1)
    leaves = (x, w, b)
    if case["backward"]:
        for t in leaves:
            t.requires_grad_(True)
    mean = x.mean((2, 3), keepdim=True)
    rstd = ((x - mean).pow(2).mean((2, 3), keepdim=True) + state["eps"]).rsqrt()
    z = (x - mean) * rstd * w + b
    if case["act"] == "gelu":
        y = z * torch.special.ndtr(z)
    else:
        y = z * torch.sigmoid(z) if case["act"] == "silu" else z
    if not case["backward"]:
        return {"out": layout_of(y, case["out_last"]), "stats": torch.stack([mean.view(B, G), rstd.view(B, G)], 2)}
    gx, gw, gb = torch.autograd.grad(y, leaves, groups_of(state["grad_out"], case["out_last"]))
    return {"grad_x": layout_of(gx, case["last"]), "grad_weight": gw.reshape(C), "grad_bias": gb.reshape(C)}
