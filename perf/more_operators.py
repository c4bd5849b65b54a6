"""Cases of the channel product and of the optimizer's step, for timing.

What a training step of a spectral model does beside its transforms and norms:

* the channel product of a field, out = act(W x + bias + branch) or act(W x + bias) + branch at every position (the
  pointwise branch of a layer, channel MLPs, lifting and projection), forward and backward.  Fields are channels last
  [B, ..., C] or channels first [B, C, ...]; input and output each have their own layout, and a 16-bit field may leave
  as float32;
* AdamW over all tensors of a model, moments held in 32 bits or in 8, with the gradients clipped by a given norm and
  16-bit copies of the new parameters written on the way.

With `own` false run() computes plain forms in elementary torch operations;
with `own` true it calls fft_spectral_convolution_amd.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZES = {"f32": 4, "bf16": 2, "f16": 2}
BLOCK = 128            # values of an 8-bit moment that share a power of two


def _cl(name, backward, B, cin, cout, grid, act, branch, dtype, out_dtype, last, out_last, bias=True):
    case = {"op": "channels", "backward": backward, "B": B, "cin": cin, "cout": cout, "grid": grid, "act": act,
            "branch": branch, "bias": bias, "dtype": dtype, "out_dtype": out_dtype, "last": last,
            "out_last": out_last}
    return dict(case, name=name) if name else case


def _adamw(name, bits, layers, width, mx, my, dtype, lift, copies, clip, step):
    case = {"op": "adamw", "bits": bits, "layers": layers, "width": width, "mx": mx, "my": my, "dtype": dtype,
            "lift": lift, "copies": copies, "clip": clip, "step": step}
    return dict(case, name=name) if name else case


def listed():
    return [
        # the 32 x 32 workload's layer, one small model step: latency
        _cl("cl_32x32_first_f32", False, 2, 4, 4, "32x32", "gelu", "before", "f32", "f32", False, False),
        # lifting: three data channels, stored last, to the field the transforms read
        _cl("cl_lift_128x128_f32", False, 32, 3, 64, "128x128", "none", "none", "f32", "f32", True, False),
        # the 128 x 128 workload's layer: the pointwise branch joined to the spectral one
        _cl("cl_128x128_first_f32", False, 32, 64, 64, "128x128", "gelu", "before", "f32", "f32", False, False),
        # the widening half of a channel MLP on the same field, 16 bits
        _cl("cl_mlp_128x128_bf16", False, 32, 64, 256, "128x128", "gelu", "none", "bf16", "bf16", True, True),
        # wide channels along sequences, the residual added behind the activation
        _cl("cl_4096_wide_bf16", False, 16, 256, 256, "4096", "silu", "after", "bf16", "bf16", True, True),
        # training: the backward pass of the 128 x 128 layer
        _cl("cl_bwd_128x128_first_f32", True, 32, 64, 64, "128x128", "gelu", "before", "f32", "f32", False, False),
        # training: the widening half of a channel MLP, 16 bits
        _cl("cl_bwd_mlp_128x128_bf16", True, 32, 64, 128, "128x128", "gelu", "none", "bf16", "bf16", True, True),
        # training on an odd grid and odd channel counts, 16 bits
        _cl("cl_bwd_61x47_last_f16", True, 3, 30, 50, "61x47", "silu", "after", "f16", "f16", True, True),
        # the optimizer's step of one small layer: latency
        _adamw("adamw_small", 32, 1, 4, 8, 8, "f32", 16, False, False, 10),
        # four layers of the 128 x 128 workload: clipped, moments in 32 bits
        _adamw("adamw_128x128_model", 32, 4, 64, 32, 32, "f32", 128, False, True, 1000),
        # the same model with its moments in 8 bits and 16-bit copies of the pointwise weights
        _adamw("adamw8_128x128_model", 8, 4, 64, 32, 32, "f32", 128, True, True, 1000),
        # many small tensors in 16 bits, moments in 8
        _adamw("adamw8_many_bf16", 8, 48, 96, 5, 5, "bf16", 384, False, False, 20000),
    ]


def _loguniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.35:
        width, layers = _loguniform(rng, 4, 96), _loguniform(rng, 1, 48)
        mx, my = _loguniform(rng, 1, 16), _loguniform(rng, 1, 16)
        while 4 * layers * mx * my * width * width > 1 << 25:
            mx, my = max(1, mx // 2), max(1, my // 2)
        dtype = rng.choice(list(DTYPES))
        return _adamw(None, rng.choice([8, 32]), layers, width, mx, my, dtype, _loguniform(rng, 1, 4 * width),
                      dtype == "f32" and rng.random() < 0.5, rng.random() < 0.5, _loguniform(rng, 1, 100000))
    backward = rng.random() < 0.5
    cin, cout = _loguniform(rng, 1, 384), _loguniform(rng, 1, 384)
    total = _loguniform(rng, 1 << 6, 1 << 19)
    # never more than half of the largest listed case's products
    total = max(1, min(total, (1 << 32) // (cin * cout), (1 << 26) // (cin + cout)))
    B = min(_loguniform(rng, 1, 64), total)
    P = max(1, total // B)
    if rng.random() < 0.5:
        grid = str(P)
    else:
        W = max(1, min(P, int(math.sqrt(P) * rng.uniform(0.5, 2.0))))
        grid = "%dx%d" % (max(1, P // W), W)
    dtype = rng.choice(list(DTYPES))
    out_dtype = rng.choice([dtype, "f32"])
    last = rng.random() < 0.5
    out_last = last if rng.random() < 0.7 else not last
    return _cl(None, backward, B, cin, cout, grid, rng.choice(["none", "gelu", "silu"]),
               rng.choice(["none", "before", "after"]), dtype, out_dtype, last, out_last, rng.random() < 0.8)


def _grid(case):
    return [int(v) for v in case["grid"].split("x")]


def _shape(case, channels, last):
    grid = _grid(case)
    return [case["B"], *grid, channels] if last else [case["B"], channels, *grid]


# ---- the tensors of a model, packed ----------------------------------------------------------------------------


def _tensor_shapes(case):
    """Shapes and types of one model's parameters, those of a type together: spectral weights; pointwise weights and
    biases, lifting and projection; norms."""
    w, dt, n = case["width"], DTYPES[case["dtype"]], case["layers"]
    return ([((2, case["mx"], case["my"], w, w), torch.complex64)] * n
            + [((w, 3), dt), ((w,), dt)] + [((w, w), dt), ((w,), dt)] * n
            + [((case["lift"], w), dt), ((case["lift"],), dt), ((1, case["lift"]), dt), ((1,), dt)]
            + [((w,), torch.float32)] * (2 * n))


def _floats(shape, dtype):
    return math.prod(shape) * (2 if dtype.is_complex else 1)


def _moment_bytes(n):
    """An 8-bit moment of n values: the codes of whole blocks, a byte for each block's power of two, whole 16 bytes."""
    blocks = -(-n // BLOCK)
    return -(-(blocks * BLOCK + blocks) // 16) * 16


def _flat_sizes(shapes):
    sizes = {}
    for s, d in shapes:
        sizes[d] = sizes.get(d, 0) + math.prod(s)
    return sizes


def _views(flat, shapes):
    """The model's tensors as slices of one packed buffer a type."""
    at = dict.fromkeys(flat, 0)
    views = []
    for s, d in shapes:
        n = math.prod(s)
        views.append(flat[d][at[d]:at[d] + n].view(s))
        at[d] += n
    return views


def _slices(buffer, sizes):
    at, out = 0, []
    for n in sizes:
        out.append(buffer[at:at + n])
        at += n
    return out


def _real(t):
    return torch.view_as_real(t) if t.is_complex() else t


def _packed(flat):
    """All values in the list's order, as float32."""
    return torch.cat([_real(f).reshape(-1).float() for f in flat.values()])


# ---- moments in 8 bits --------------------------------------------------------------------------------------------
# A block's values are y 2^e with e its largest value's exponent, kept as a byte (e + 127, at least 1, for second
# moments at least 31; 0 for a block of zeros).  A code is 0 for zero, else exponent and three bits of fraction
# together, (1 + (c & 7) / 8) 2^((c >> 3) - 14 + e) for first moments (bit 7 the sign), - 30 for second ones.


def _decode(codes, exps, signed):
    c = codes.int()
    if signed:
        sign, c, top = 1.0 - 2.0 * (c >> 7), c & 127, 14
    else:
        sign, top = 1.0, 30
    e = (c >> 3) - top + exps.int() - 127
    return torch.where(c == 0, 0.0, sign * torch.ldexp(1.0 + (c & 7) / 8.0, e.double()))


def _encode(values, bits16, signed):
    """Codes [blocks, 128] and exponent bytes of float64 values [blocks, 128].  `bits16` (0 to 65535) rounds up where
    the dropped part (17 bits) and 2 bits16 + 1 pass a whole."""
    top, least = (14, 1) if signed else (30, 31)
    bits = values.abs().view(torch.int64)
    largest = bits.amax(1, keepdim=True)
    e = ((largest >> 52) - 1023 + 127).clamp(least, 254)
    e = torch.where(largest == 0, torch.zeros_like(e), e)
    # the high half of the value over 2^e: sign, 11 bits of exponent, 20 of fraction
    high = (bits >> 32) - ((e - 127) << 20)
    c = ((high + 2 * bits16 + 1) >> 17) - ((1023 - top) << 3)
    c = c.clamp(0, 126) if signed else c.clamp(1, 254)
    c = torch.where(bits == 0, torch.zeros_like(c), c)
    if signed:
        c = c | ((values < 0) & (c > 0)).long() << 7
    return c.to(torch.uint8), e.to(torch.uint8)


def _mix(x):
    x = x & 0xFFFFFFFF
    x = ((x ^ (x >> 16)) * 0x6A09E667) & 0xFFFFFFFF
    x = ((x ^ (x >> 15)) * 0xBB67AE85) & 0xFFFFFFFF
    return x ^ (x >> 16)


def _block_maps(shapes):
    """For every place of every tensor's blocks: the value's place among all values, its tensor and its number there,
    and the places of its code and of its block's byte among all moments' bytes."""
    dev = "cuda"
    n = torch.tensor([_floats(s, d) for s, d in shapes], device=dev)
    blocks = (n + BLOCK - 1) // BLOCK
    size = (blocks * (BLOCK + 1) + 15) // 16 * 16
    start, at, first = n.cumsum(0) - n, size.cumsum(0) - size, blocks.cumsum(0) - blocks
    tensor = torch.arange(len(shapes), device=dev).repeat_interleave(blocks)
    block = torch.arange(len(tensor), device=dev) - first[tensor]
    number = block[:, None] * BLOCK + torch.arange(BLOCK, device=dev)
    used = number < n[tensor][:, None]
    return {"value": torch.where(used, number + start[tensor][:, None], 0), "used": used, "tensor": tensor[:, None],
            "number": number, "code": number + at[tensor][:, None],
            "exp": (at + blocks * BLOCK)[tensor][:, None] + block[:, None]}


def _store_moment(out, maps, values, bits16, signed):
    c, e = _encode(values, bits16, signed)
    out[maps["code"]] = c
    out[maps["exp"]] = e


def _load_moment(held, maps, signed):
    return _decode(held[maps["code"]], held[maps["exp"]], signed)


# ---- inputs ---------------------------------------------------------------------------------------------------------


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    def rand(*shape):
        return torch.rand(*shape, generator=gen, device="cuda")

    if case["op"] == "adamw":
        shapes = _tensor_shapes(case)
        sizes = _flat_sizes(shapes)
        n = sum(_floats(s, d) for s, d in shapes)
        std = 3.0 / math.sqrt(n)               # a model's gradient norm is a few units whatever its size

        def flat(scale):
            return {d: torch.view_as_complex(randn(m, 2).mul_(scale)) if d.is_complex else randn(m).mul_(scale).to(d)
                    for d, m in sizes.items()}

        state = {"case": case, "shapes": shapes, "flat": flat(0.05), "flat_grad": flat(std)}
        state["flat_out"] = {d: torch.empty_like(f) for d, f in state["flat"].items()}
        state["norm"] = torch.full((), 3.0, device="cuda") if case["clip"] else None
        # some steps in: a mean of a few gradients, squares within a factor of ten of each other
        # (both stand near zero before the first step)
        seen = 1.0 - 0.9 ** (case["step"] - 1)
        m = randn(n).mul_(0.3 * std * seen)
        v = torch.exp(rand(n).mul_(2.3)).mul_(0.3 * std * std * (1.0 - 0.999 ** (case["step"] - 1)))
        if case["bits"] == 8:
            state["maps"] = maps = _block_maps(shapes)
            moment = [_moment_bytes(_floats(s, d)) for s, d in shapes]
            for key, values, signed in (("m", m, True), ("v", v, False)):
                held = torch.zeros(sum(moment), dtype=torch.uint8, device="cuda")
                wide = torch.where(maps["used"], values[maps["value"]].double(), 0.0)
                half = torch.full_like(maps["number"], 32768)
                _store_moment(held, maps, wide, half, signed)
                state[key], state[key + "_out"] = held, torch.zeros_like(held)
                state[key + "_read"] = torch.empty(n, device="cuda")
        else:
            moment = [_floats(s, d) for s, d in shapes]
            for key, values in (("m", m), ("v", v)):
                state[key], state[key + "_out"] = values, torch.empty_like(values)
        state["copy"] = {d: torch.empty(k, dtype=torch.bfloat16, device="cuda") for d, k in sizes.items()
                         if not d.is_complex} if case["copies"] else None
        # the lists a training program holds
        state["lists"] = {"params": _views(state["flat"], shapes), "grads": _views(state["flat_grad"], shapes),
                          "outs": _views(state["flat_out"], shapes)}
        for key in ("m", "v", "m_out", "v_out"):
            state["lists"][key] = _slices(state[key], moment)
        if case["bits"] == 8:
            for key in ("m_read", "v_read"):
                state["lists"][key] = _slices(state[key], [_floats(s, d) for s, d in shapes])
        if case["copies"]:
            dense = iter(_views(state["copy"], [s for s in shapes if not s[1].is_complex]))
            state["lists"]["copies"] = [None if d.is_complex else next(dense) for _, d in shapes]
        return state

    cin, cout, dt, out_dt = case["cin"], case["cout"], DTYPES[case["dtype"]], DTYPES[case["out_dtype"]]
    state = {"case": case, "x": randn(*_shape(case, cin, case["last"])).to(dt),
             "weight": (randn(cout, cin) / math.sqrt(cin)).to(dt), "bias": 0.2 * randn(cout) if case["bias"] else None,
             "branch": None}
    if case["branch"] != "none":
        state["branch"] = randn(*_shape(case, cout, case["out_last"])).to(out_dt)
    if case["backward"]:
        state["grad_out"] = randn(*_shape(case, cout, case["out_last"])).to(out_dt)
    return state


# ---- plain forms ------------------------------------------------------------------------------------------------------


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


def _product(w, t, last):
    """w [M, K] times the channels of a flattened float32 field: [B, P, K] or [B, K, P]."""
    if last:
        return torch.matmul(t.reshape(-1, w.shape[1]), w.t().contiguous()).view(t.shape[0], -1, w.shape[0])
    return torch.matmul(w, t)


def _flat(t, last):
    return t.reshape(t.shape[0], -1, t.shape[-1]) if last else t.reshape(t.shape[0], t.shape[1], -1)


def _turned(t, last, out_last):
    return t if last == out_last else t.transpose(1, 2).contiguous()


def _pre_activation(state):
    """W x + bias, and branch where it is inside, in out's layout, flattened."""
    case = state["case"]
    z = _product(state["weight"].float(), _flat(state["x"].float(), case["last"]), case["last"])
    z = _turned(z, case["last"], case["out_last"])
    if state["bias"] is not None:
        z = z + (state["bias"] if case["out_last"] else state["bias"][:, None])
    if case["branch"] == "before":
        z = z + _flat(state["branch"].float(), case["out_last"])
    return z


def _channels(state):
    case = state["case"]
    y = _act(_pre_activation(state), case["act"])
    if case["branch"] == "after":
        y = y + _flat(state["branch"].float(), case["out_last"])
    return {"out": y.view(_shape(case, case["cout"], case["out_last"])).to(DTYPES[case["out_dtype"]])}


def _channels_backward(state):
    case, last, out_last = state["case"], state["case"]["last"], state["case"]["out_last"]
    g = _flat(state["grad_out"].float(), out_last)
    if case["act"] != "none":
        g = g * _act_slope(_pre_activation(state), case["act"])
    outputs = {}
    if case["branch"] == "before":
        shape = _shape(case, case["cout"], out_last)
        outputs["grad_branch"] = g.view(shape).to(DTYPES[case["out_dtype"]])
    gx = _product(state["weight"].float().t().contiguous(), g, out_last)
    gx = _turned(gx, out_last, last).view(_shape(case, case["cin"], last))
    outputs["grad_x"] = gx.to(DTYPES[case["dtype"]])
    # a product for each item, their sum in 64 bits
    g_first = _turned(g, out_last, False)
    x_last = _turned(_flat(state["x"].float(), last), last, True)
    outputs["grad_weight"] = torch.matmul(g_first, x_last).sum(0, dtype=torch.float64).float()
    if state["bias"] is not None:
        outputs["grad_bias"] = g_first.sum(2).sum(0, dtype=torch.float64).float()
    return outputs


HYPER = {"lr": 1e-3, "betas": (0.9, 0.999), "eps": 1e-8, "weight_decay": 1e-2}
MAX_NORM = 1.0
SEED = 0x1234567890


def _clip_factor(norm):
    return torch.clamp(MAX_NORM / (norm.double() + 1e-6), max=1.0).float()


def _rounding_bits(case, maps):
    """32 random bits for each place: a hash of seed, step, tensor and number."""
    key = _mix(torch.full_like(maps["tensor"], SEED & 0xFFFFFFFF)) + (SEED >> 32)
    key = _mix(_mix(_mix(key) + case["step"]) + maps["tensor"])
    return _mix((maps["number"] & 0xFFFFFFFF) ^ _mix(key + (maps["number"] >> 32)))


def _adamw_plain(state):
    case, (b1, b2) = state["case"], HYPER["betas"]
    p, g = _packed(state["flat"]), _packed(state["flat_grad"])
    if state["norm"] is not None:
        g = g * _clip_factor(state["norm"])
    outputs = {}
    if case["bits"] == 8:
        maps = state["maps"]
        # in 64 bits: a code is that of the value, whatever its neighbour
        gb = torch.where(maps["used"], g[maps["value"]], 0.0).double()
        m = b1 * _load_moment(state["m"], maps, True) + (1.0 - b1) * gb
        v = b2 * _load_moment(state["v"], maps, False) + (1.0 - b2) * (gb * gb)
        r = _rounding_bits(case, maps)
        _store_moment(state["m_out"], maps, m, r & 0xFFFF, True)
        _store_moment(state["v_out"], maps, v, r >> 16, False)
        used = maps["used"]
        outputs["m"] = _load_moment(state["m_out"], maps, True)[used].float()
        outputs["v"] = _load_moment(state["v_out"], maps, False)[used].float()
        m, v = m[used].float(), v[used].float()
    else:
        m = outputs["m"] = b1 * state["m"] + (1.0 - b1) * g
        v = outputs["v"] = b2 * state["v"] + (1.0 - b2) * (g * g)
    c1, c2 = 1.0 - b1 ** case["step"], 1.0 - b2 ** case["step"]
    p = p * (1.0 - HYPER["lr"] * HYPER["weight_decay"]) \
        - (HYPER["lr"] / c1) * m / (torch.sqrt(v) / math.sqrt(c2) + HYPER["eps"])
    return {**outputs, **_unpacked(state, p)}


def _unpacked(state, p):
    """New parameters, a packed buffer a type, and their copies."""
    flat = state["flat"]
    parts = torch.split(p, [f.numel() * (2 if d.is_complex else 1) for d, f in flat.items()])
    outputs = {_key(d): torch.view_as_complex(v.view(-1, 2)) if d.is_complex else v.to(d)
               for d, v in zip(flat, parts)}
    if state["copy"] is not None:
        outputs.update({"copy_" + _key(d): v.to(torch.bfloat16) for d, v in zip(flat, parts) if not d.is_complex})
    return outputs


def _key(dtype):
    return str(dtype).split(".")[1]


def _adamw_own(state):
    import fft_spectral_convolution_amd as fno
    case, lists = state["case"], state["lists"]
    fno.fno_adamw(lists["params"], lists["grads"], lists["m"], lists["v"], case["step"], **HYPER,
                  norm=state["norm"], max_norm=MAX_NORM if case["clip"] else None, copies=lists.get("copies"),
                  seed=SEED, out=(lists["outs"], lists["m_out"], lists["v_out"]))
    outputs = {"m": state["m_out"], "v": state["v_out"]}
    if case["bits"] == 8:
        fno.fno_adamw_moments(lists["m_out"], lists["v_out"], out=(lists["m_read"], lists["v_read"]))
        outputs = {"m": state["m_read"], "v": state["v_read"]}
    outputs.update({_key(d): f for d, f in state["flat_out"].items()})
    if state["copy"] is not None:
        outputs.update({"copy_" + _key(d): f for d, f in state["copy"].items()})
    return outputs


def run(state):
    case = state["case"]
    if not own:
        if case["op"] == "adamw":
            return _adamw_plain(state)
        return _channels_backward(state) if case["backward"] else _channels(state)
    if case["op"] == "adamw":
        return _adamw_own(state)
    import fft_spectral_convolution_amd as fno
    options = {"bias": state["bias"], "branch": state["branch"], "branch_after": case["branch"] == "after",
               "act": case["act"], "channels_last": case["last"], "out_channels_last": case["out_last"]}
    if case["backward"]:
        gx, gw, gb, gr = fno.fno_channel_linear_backward(state["x"], state["weight"], state["grad_out"], **options)
        outputs = {"grad_x": gx, "grad_weight": gw}
        if state["bias"] is not None:
            outputs["grad_bias"] = gb
        if case["branch"] == "before":
            outputs["grad_branch"] = gr
        return outputs
    return {"out": fno.fno_channel_linear(state["x"], state["weight"], out_dtype=DTYPES[case["out_dtype"]],
                                          **options)}


def work(case):
    if case["op"] == "adamw":
        shapes = _tensor_shapes(case)
        n = sum(_floats(s, d) for s, d in shapes)
        moved = 3 * sum(math.prod(s) * d.itemsize for s, d in shapes)          # parameters in and out, gradients
        if case["bits"] == 8:
            moved += 4 * sum(_moment_bytes(_floats(s, d)) for s, d in shapes) + 8 * n     # and their values read out
        else:
            moved += 16 * n
        if case["copies"]:
            moved += 2 * sum(_floats(s, d) for s, d in shapes if not d.is_complex)
        return {"bytes": moved, "flops": 15 * n}
    n, cin, cout = case["B"] * math.prod(_grid(case)), case["cin"], case["cout"]
    size, out_size = SIZES[case["dtype"]], SIZES[case["out_dtype"]]
    weights = cin * cout
    bias = 4 * cout if case["bias"] else 0
    act = case["act"] != "none"
    if case["backward"]:
        # grad_out is its own gradient of a branch behind the activation; z is not needed where its slope is 1
        inside = case["branch"] == "before"
        fields = 2 * n * cin * size + n * cout * out_size * (1 + inside * (1 + act))
        return {"bytes": fields + weights * (size + 4) + bias * (1 + act),
                "flops": (6 if act else 4) * n * cin * cout}
    branch = n * cout * out_size if case["branch"] != "none" else 0
    return {"bytes": n * (cin * size + cout * out_size) + branch + weights * size + bias, "flops": 2 * n * cin * cout}


# ---- definitions in 64 bits -----------------------------------------------------------------------------------------------


def _exact_code_value(y, fraction, top, signed):
    """The value that the code of y (float64, its block's largest below 2) stands for, over 2^e."""
    mantissa, e = torch.frexp(y.abs())                                  # [0.5, 1)
    steps = torch.floor(mantissa * 2.0 ** 21) / 2.0 ** 17               # eighths, 8 to 16, cut at 17 bits behind
    whole = torch.floor(steps)
    up = (steps - whole) * 2.0 ** 17 + 2 * fraction + 1 >= 2.0 ** 17
    whole = whole + up.double()
    value = torch.ldexp(whole / 8.0, (e - 1).double())
    least = 2.0 ** -top                                                 # where codes of first moments end in zero
    if signed:
        value = torch.where(value > least, value, 0.0)
    else:
        value = torch.where(value > least, value, 1.125 * least)
    return torch.where(y == 0, 0.0, torch.sign(y) * value)


def _exact_moment(values, fraction, top, least, signed):
    big = values.abs().amax(1, keepdim=True)
    e = (torch.frexp(big)[1] - 1).clamp(least, 127).double()
    return torch.ldexp(_exact_code_value(torch.ldexp(values, -e), fraction, top, signed), e)


def _exact_adamw(case, state):
    b1, b2 = HYPER["betas"]
    p, g = _packed(state["flat"]).double(), _packed(state["flat_grad"])
    if state["norm"] is not None:
        factor = min(1.0, MAX_NORM / (float(state["norm"]) + 1e-6))
        # (the factor is a float32, and so is a clipped gradient)
        g = g * torch.tensor(factor, dtype=torch.float32, device="cuda")
    g = g.double()
    t = case["step"]
    outputs = {}
    if case["bits"] == 8:
        maps = state["maps"]
        used = maps["used"]
        m, v = (_load_moment(state[k], maps, k == "m")[used] for k in "mv")
    else:
        m, v = state["m"].double(), state["v"].double()
    m = m * b1 + g * (1.0 - b1)
    v = v * b2 + g ** 2 * (1.0 - b2)
    p = p - HYPER["lr"] * (HYPER["weight_decay"] * p + (m / (1.0 - b1 ** t)) / ((v / (1.0 - b2 ** t)).sqrt()
                                                                              + HYPER["eps"]))
    if case["bits"] == 8:
        r = _rounding_bits(case, maps)
        for key, values, fraction, top, least, signed in (("m", m, r & 0xFFFF, 14, -126, True),
                                                          ("v", v, r >> 16, 30, -96, False)):
            wide = torch.zeros(used.shape, dtype=torch.float64, device="cuda").masked_scatter_(used, values)
            outputs[key] = _exact_moment(wide, fraction.double(), top, least, signed)[used]
    else:
        outputs["m"], outputs["v"] = m, v
    at = 0
    for d, f in state["flat"].items():
        k = f.numel() * (2 if d.is_complex else 1)
        part = p[at:at + k]
        outputs[_key(d)] = torch.view_as_complex(part.view(-1, 2)) if d.is_complex else part
        if state["copy"] is not None and not d.is_complex:
            outputs["copy_" + _key(d)] = part
        at += k
    return outputs


def exact(case, seed):
    """The definitions in float64: fields as [B, P, C] and gradients by differentiation; moments and parameters."""
    state = prepare(case, seed)
    if case["op"] == "adamw":
        return _exact_adamw(case, state)
    B = case["B"]

    def points(t, last):
        t = t.double()
        return t.reshape(B, -1, t.shape[-1]) if last else t.reshape(B, t.shape[1], -1).transpose(1, 2)

    def laid(t, last):
        return (t if last else t.transpose(1, 2)).reshape(_shape(case, t.shape[2], last))

    leaves = {"grad_x": points(state["x"], case["last"]), "grad_weight": state["weight"].double()}
    if state["bias"] is not None:
        leaves["grad_bias"] = state["bias"].double()
    if case["branch"] == "before":
        leaves["grad_branch"] = points(state["branch"], case["out_last"])
    if case["backward"]:
        leaves = {k: t.clone().requires_grad_(True) for k, t in leaves.items()}
    z = torch.nn.functional.linear(leaves["grad_x"], leaves["grad_weight"], leaves.get("grad_bias"))
    if case["branch"] == "before":
        z = z + leaves["grad_branch"]
    if case["act"] == "gelu":
        y = z * torch.special.ndtr(z)
    else:
        y = z * torch.sigmoid(z) if case["act"] == "silu" else z
    if not case["backward"]:
        if case["branch"] == "after":
            y = y + points(state["branch"], case["out_last"])
        return {"out": laid(y, case["out_last"])}
    grads = dict(zip(leaves, torch.autograd.grad(y, list(leaves.values()), points(state["grad_out"],
                                                                                case["out_last"]))))
    grads["grad_x"] = laid(grads["grad_x"], case["last"])
    if "grad_branch" in grads:
        grads["grad_branch"] = laid(grads["grad_branch"], case["out_last"])
    return grads
