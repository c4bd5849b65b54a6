"""fno_group_norm and fno_group_norm_backward against their definitions in
float64, over types, layouts, odd sizes and the kernels that serve them.

Tolerances, elementwise, from the rounding of float32 (u = 2^-24): a sum of
n values is accumulated in chains of at most K = 512 additions (per thread,
then across threads and chunks), so a mean is off by at most K u mean|x| and
a variance by a relative K u; (x - mean) rstd w + b then carries

    z_err = |w| (|xh| K u + rstd (K u mean|x| + 2 u |x|)) + 2 u (|z| + |b|).

GELU and SiLU have slopes below 1.13 and are formed with a relative error
below 16 u of max(|z|, |y|); their slopes have second derivatives below 1 and
an error below 16 u (1 + z^2/2) (the exponential of z^2/2 carries its
argument's rounding).  A 16-bit output adds half a step of its type.
"""
import pytest

torch = pytest.importorskip("torch")

import fft_spectral_convolution_amd as fno  # noqa: E402

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
K = 512
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _gpu_present():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    fno.lib()


def to_groups(t, groups, last):
    """Any field -> float64 [B, G, D, P]."""
    b, c = t.shape[0], (t.shape[-1] if last else t.shape[1])
    flat = t.double().reshape(b, -1, c).transpose(1, 2) if last else t.double().reshape(b, c, -1)
    return flat.reshape(b, groups, c // groups, -1)


def to_field(g, shape, last):
    flat = g.reshape(g.shape[0], g.shape[1] * g.shape[2], g.shape[3])
    return (flat.transpose(1, 2) if last else flat).reshape(shape)


def act_of(z, act):
    if act == "gelu":
        return z * torch.special.ndtr(z)
    return z * torch.sigmoid(z) if act == "silu" else z


def slope_of(z, act):
    if act == "gelu":
        return torch.special.ndtr(z) + z * torch.exp(-0.5 * z * z) / (2 * torch.pi) ** 0.5
    if act == "silu":
        s = torch.sigmoid(z)
        return s * (1 + z * (1 - s))
    return torch.ones_like(z)


class Reference:
    def __init__(self, x, groups, weight, bias, eps, act, last):
        self.xg = to_groups(x, groups, last)
        b, g, d, p = self.xg.shape
        one = torch.ones(g * d, dtype=torch.float64, device=x.device)
        self.w = (one if weight is None else weight.double()).view(1, g, d, 1)
        self.b = (0 * one if bias is None else bias.double()).view(1, g, d, 1)
        self.act = act
        self.mean = self.xg.mean((2, 3), keepdim=True)
        self.rstd = ((self.xg - self.mean).square().mean((2, 3), keepdim=True) + eps).rsqrt()
        self.xh = (self.xg - self.mean) * self.rstd
        self.z = self.xh * self.w + self.b
        self.stats = torch.stack([self.mean.view(b, g), self.rstd.view(b, g)], 2)
        self.xh_err = self.xh.abs() * K * U + self.rstd * U * (K * self.xg.abs().mean((2, 3), keepdim=True)
                                                               + 2 * self.xg.abs())
        self.z_err = self.w.abs() * self.xh_err + 2 * U * (self.z.abs() + self.b.abs())

    def out(self, out_dtype):
        y = act_of(self.z, self.act)
        # the definition's own sensitivity in eps-dominated groups is in xh_err through rstd
        err = 1.13 * self.z_err + 16 * U * torch.maximum(self.z.abs(), y.abs())
        return y, err * (1 + HALF_STEP[out_dtype]) + HALF_STEP[out_dtype] * y.abs() + TINY[out_dtype]

    def grads(self, dyg, x_dtype):
        slope = slope_of(self.z, self.act)
        g = dyg * slope
        g_err = dyg.abs() * (1.13 * self.z_err + 16 * U * (1 + 0.5 * self.z.square())) + U * g.abs()
        n = self.xg.shape[2] * self.xg.shape[3]
        gw, gb = (g * self.xh).sum((0, 3)).flatten(), g.sum((0, 3)).flatten()
        gw_err = (g_err * self.xh.abs() + g.abs() * self.xh_err + K * U * (g * self.xh).abs()).sum((0, 3)).flatten()
        gb_err = (g_err + K * U * g.abs()).sum((0, 3)).flatten()
        v, v_err = g * self.w, (g_err + 2 * U * g.abs()) * self.w.abs()
        s1, s2 = v.sum((2, 3), keepdim=True) / n, (v * self.xh).sum((2, 3), keepdim=True) / n
        s1_err = (v_err + K * U * v.abs()).sum((2, 3), keepdim=True) / n
        s2_err = (v_err * self.xh.abs() + v.abs() * self.xh_err
                  + K * U * (v * self.xh).abs()).sum((2, 3), keepdim=True) / n
        gx = self.rstd * (v - s1 - self.xh * s2)
        gx_err = self.rstd * (v_err + s1_err + self.xh.abs() * s2_err + self.xh_err * s2.abs()
                              + 4 * U * (v.abs() + s1.abs() + (self.xh * s2).abs())) + K * U * gx.abs()
        gx_err = gx_err * (1 + HALF_STEP[x_dtype]) + HALF_STEP[x_dtype] * gx.abs() + TINY[x_dtype]
        return (gx, gx_err), (gw, gw_err + TINY[F32]), (gb, gb_err + TINY[F32])


def close(got, want, err, what):
    bad = ~((got.double() - want).abs() <= err)
    worst = ((got.double() - want).abs() / err).max().item()
    print(f"  {what}: worst error / tolerance {worst:.3f}", flush=True)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst {worst:.3g}"


def field(shape, dtype, seed, level=0.0, spread=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (level + spread * torch.randn(shape, generator=g, device=DEV)).to(dtype)


def params(c, seed, on=True):
    if not on:
        return None, None
    return 1.0 + 0.3 * field((c,), F32, seed + 1), 0.3 * field((c,), F32, seed + 2)


def shape_of(b, c, grid, last):
    return (b, *grid, c) if last else (b, c, *grid)


def check(b, c, grid, groups, act="gelu", dtype=F32, out_dtype=None, last=True, out_last=None, affine=True,
          eps=1e-5, level=0.0, seed=0, backward=True):
    out_last = last if out_last is None else out_last
    out_dtype = dtype if out_dtype is None else out_dtype
    x = field(shape_of(b, c, grid, last), dtype, seed, level)
    w, bias = params(c, seed, affine)
    opts = dict(weight=w, bias=bias, act=act, channels_last=last, out_channels_last=out_last)
    ref = Reference(x, groups, w, bias, eps, act, last)
    oshape = shape_of(b, c, grid, out_last)
    out, stats = fno.fno_group_norm(x, groups, eps=eps, out_dtype=out_dtype, **opts)
    torch.cuda.synchronize()
    assert tuple(out.shape) == oshape and out.dtype == out_dtype
    y, err = ref.out(out_dtype)
    close(to_groups(out, groups, out_last), y, err, "out")
    m_err = K * U * ref.xg.abs().mean((2, 3)) + U * ref.stats[..., 0].abs()
    close(stats[..., 0], ref.stats[..., 0], m_err, "mean")
    close(stats[..., 1], ref.stats[..., 1], ref.stats[..., 1] * K * U, "rstd")
    if not backward:
        return
    dy = field(oshape, out_dtype, seed + 7)
    gx, gw, gb = fno.fno_group_norm_backward(x, ref.stats.float(), dy, groups, **opts)
    torch.cuda.synchronize()
    (rx, ex), (rw, ew), (rb, eb) = ref.grads(to_groups(dy, groups, out_last), dtype)
    assert gx.shape == x.shape and gx.dtype == dtype
    close(to_groups(gx, groups, last), rx, ex, "grad_x")
    if affine:
        close(gw, rw, ew, "grad_weight")
        close(gb, rb, eb, "grad_bias")
    else:
        assert gw is None and gb is None


LAYOUTS = [(True, True), (False, False), (True, False), (False, True)]


@pytest.mark.parametrize("last,out_last", LAYOUTS)
@pytest.mark.parametrize("dtype,out_dtype", [(F32, F32), (BF16, BF16), (BF16, F32), (F16, F16), (F16, F32)])
def test_types_and_layouts(dtype, out_dtype, last, out_last):
    check(3, 24, (17, 11), 4, "gelu", dtype, out_dtype, last, out_last)


@pytest.mark.parametrize("last,out_last", LAYOUTS)
@pytest.mark.parametrize("act", ["none", "gelu", "silu"])
def test_activations(act, last, out_last):
    check(2, 16, (32, 32), 4, act, F32, None, last, out_last, seed=3)


@pytest.mark.parametrize("last,out_last", LAYOUTS)
@pytest.mark.parametrize("b,c,grid,groups", [
    (1, 1, (2,), 1),              # the smallest group with a spread
    (2, 8, (), 2),                # no positions axis: [B, C]
    (1, 6, (1,), 3),
    (2, 3, (5,), 1),              # everything odd
    (5, 33, (7, 9), 11),
    (2, 30, (61, 47), 5),
    (4, 7, (1000,), 7),           # one channel a group
    (3, 130, (19,), 1),           # one group
    (1, 64, (65, 63), 32),        # two channels a group, vectors over several groups
    (2, 36, (50,), 12),           # three channels a group
    (300, 4, (3,), 2),            # many items, few positions
    (2, 511, (9,), 7),
])
def test_shapes(b, c, grid, groups, last, out_last):
    check(b, c, grid, groups, "silu", F32, None, last, out_last, seed=11)
    check(b, c, grid, groups, "gelu", F16, None, last, out_last, seed=12)


@pytest.mark.parametrize("last,out_last", LAYOUTS)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_wide_channels(dtype, last, out_last):
    check(2, 5000, (6,), 10, "gelu", dtype, None, last, out_last, seed=20)
    check(1, 2049, (8,), 3, "none", dtype, None, last, out_last, seed=21)
    check(1, 9000, (4,), 9000, "none", dtype, None, last, out_last, seed=22)


@pytest.mark.parametrize("last,out_last", LAYOUTS)
@pytest.mark.parametrize("b,c,grid,groups,dtype", [
    (2, 32, (128, 128), 8, F32),
    (8, 16, (64, 64), 4, BF16),
    (1, 16, (512, 300), 4, F32),
    (3, 12, (4099,), 3, F32),
    (1, 3, (100003,), 1, F16),
    (1, 1, (300001,), 1, F32),
    (40, 32, (32, 32), 8, F32),
    (2, 256, (33, 31), 32, BF16),
])
def test_larger_fields(b, c, grid, groups, dtype, last, out_last):
    check(b, c, grid, groups, "gelu", dtype, F32, last, out_last, seed=30)


@pytest.mark.parametrize("last,out_last", LAYOUTS)
def test_without_weight_and_bias(last, out_last):
    check(2, 12, (40, 9), 3, "gelu", F32, None, last, out_last, affine=False, seed=40)


@pytest.mark.parametrize("last", [True, False])
def test_one_of_weight_and_bias(last):
    x = field(shape_of(2, 8, (31,), last), F32, 41)
    w, b = params(8, 41)
    dy = field(x.shape, F32, 42)
    for weight, bias in ((w, None), (None, b)):
        ref = Reference(x, 2, weight, bias, 1e-5, "silu", last)
        out, stats = fno.fno_group_norm(x, 2, weight=weight, bias=bias, act="silu", channels_last=last)
        y, err = ref.out(F32)
        close(to_groups(out, 2, last), y, err, "out")
        gx, gw, gb = fno.fno_group_norm_backward(x, stats, dy, 2, weight=weight, bias=bias, act="silu",
                                                 channels_last=last)
        (rx, ex), (rw, ew), (rb, eb) = ref.grads(to_groups(dy, 2, last), F32)
        close(to_groups(gx, 2, last), rx, ex, "grad_x")
        assert (gw is None) == (weight is None) and (gb is None) == (bias is None)
        if weight is not None:
            close(gw, rw, ew, "grad_weight")
        else:
            close(gb, rb, eb, "grad_bias")


@pytest.mark.parametrize("last", [True, False])
@pytest.mark.parametrize("b,c,grid,groups", [(2, 16, (64, 64), 4), (2, 8, (300, 300), 2)])
def test_level_far_above_the_spread(b, c, grid, groups, last):
    """Mean 1000, deviation 1: squares about zero would lose the variance."""
    check(b, c, grid, groups, "none", F32, None, last, level=1000.0, seed=50)


@pytest.mark.parametrize("last,out_last", LAYOUTS)
@pytest.mark.parametrize("n", [1, 7, 5000])
def test_constant_groups(n, last, out_last):
    """No spread: out = act(bias), and the gradient stays finite."""
    x = torch.full(shape_of(2, 6, (n,), last), 3.25, device=DEV)
    w, b = params(6, 60)
    out, stats = fno.fno_group_norm(x, 3, weight=w, bias=b, act="none", channels_last=last,
                                    out_channels_last=out_last)
    want = b.view(1, 1, 6) if out_last else b.view(1, 6, 1)
    assert torch.equal(out, want.expand_as(out))
    assert torch.equal(stats[..., 0], torch.full_like(stats[..., 0], 3.25))
    dy = field(out.shape, F32, 61)
    gx, _, _ = fno.fno_group_norm_backward(x, stats, dy, 3, weight=w, bias=b, channels_last=last,
                                           out_channels_last=out_last)
    assert torch.isfinite(gx).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("last,out_last", LAYOUTS)
@pytest.mark.parametrize("grid", [(9,), (64, 64), (200, 300)])
def test_non_finite_value_stays_in_its_group(grid, last, out_last, bad):
    x = field(shape_of(2, 12, grid, last), F32, 70)
    good, gstats = fno.fno_group_norm(x, 4, act="gelu", channels_last=last, out_channels_last=out_last)
    y = x.clone()
    if last:
        y.view(2, -1, 12)[1, 4, 5] = bad       # item 1, channel 5: group 1
    else:
        y.view(2, 12, -1)[1, 5, 4] = bad
    out, stats = fno.fno_group_norm(y, 4, act="gelu", channels_last=last, out_channels_last=out_last)
    a, b = to_groups(out, 4, out_last), to_groups(good, 4, out_last)
    assert torch.isnan(a[1, 1]).all()
    a[1, 1] = b[1, 1]
    assert torch.equal(a, b)
    assert torch.isnan(stats[1, 1, 1])
    stats[1, 1] = gstats[1, 1]
    assert torch.equal(stats, gstats)
    dy = field(out.shape, F32, 71)
    opts = dict(act="gelu", channels_last=last, out_channels_last=out_last)
    gx0, _, _ = fno.fno_group_norm_backward(x, gstats, dy, 4, **opts)
    _, stats = fno.fno_group_norm(y, 4, **opts)
    gx, _, _ = fno.fno_group_norm_backward(y, stats, dy, 4, **opts)
    a, b = to_groups(gx, 4, last), to_groups(gx0, 4, last)
    assert torch.isnan(a[1, 1]).all()
    a[1, 1] = b[1, 1]
    assert torch.equal(a, b)


@pytest.mark.parametrize("last,out_last", LAYOUTS)
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("b,c,grid,groups", [(2, 5, (7, 3), 5), (3, 16, (50, 41), 4), (2, 32, (128, 65), 2)])
def test_slices_of_packed_buffers(b, c, grid, groups, dtype, last, out_last):
    """Fields aligned to their elements only; nothing around the outputs is written."""
    n = b * c
    for v in grid:
        n *= v
    xs, os_ = shape_of(b, c, grid, last), shape_of(b, c, grid, out_last)

    def packed(t):
        buf = torch.full((n + 64,), -7.0, dtype=dtype, device=DEV)
        buf[33:33 + n] = t.reshape(-1)
        return buf, buf[33:33 + n].view(t.shape)

    x = field(xs, dtype, 80)
    w, bias = params(c, 80)
    opts = dict(weight=w, bias=bias, act="silu", channels_last=last, out_channels_last=out_last)
    want, stats = fno.fno_group_norm(x, groups, **opts)
    dy = field(os_, dtype, 81)
    wx, ww, wb = fno.fno_group_norm_backward(x, stats, dy, groups, **opts)
    _, xv = packed(x)
    obuf, ov = packed(torch.zeros(os_, dtype=dtype, device=DEV))
    _, st = fno.fno_group_norm(xv, groups, out=ov, **opts)
    assert torch.equal(ov, want) and torch.equal(st, stats)
    _, dv = packed(dy)
    gbuf, gv = packed(torch.zeros(xs, dtype=dtype, device=DEV))
    _, gw, gb = fno.fno_group_norm_backward(xv, stats, dv, groups, grad_x=gv, **opts)
    assert torch.equal(gv, wx) and torch.equal(gw, ww) and torch.equal(gb, wb)
    for buf in (obuf, gbuf):
        assert (buf[:33] == -7).all() and (buf[33 + n:] == -7).all()


@pytest.mark.parametrize("last,out_last", LAYOUTS)
def test_chosen_gradients_only(last, out_last):
    x = field(shape_of(3, 16, (40, 40), last), F32, 90)
    w, b = params(16, 90)
    opts = dict(weight=w, bias=b, act="gelu", channels_last=last, out_channels_last=out_last)
    out, stats = fno.fno_group_norm(x, 4, **opts)
    dy = field(out.shape, F32, 91)
    gx, gw, gb = fno.fno_group_norm_backward(x, stats, dy, 4, **opts)
    hx, hw, hb = fno.fno_group_norm_backward(x, stats, dy, 4, need_w=False, **opts)
    assert torch.equal(hx, gx) and hw is None and hb is None
    hx, hw, hb = fno.fno_group_norm_backward(x, stats, dy, 4, need_x=False, **opts)
    assert hx is None and torch.equal(hw, gw) and torch.equal(hb, gb)


@pytest.mark.parametrize("last,out_last", LAYOUTS)
@pytest.mark.parametrize("act", ["gelu", "silu"])
def test_gradients_against_differences(act, last, out_last):
    """Directional derivatives of L = sum(out dy) by central differences.  The
    step h = 2^-7 leaves a third-order term below h^2 times a few units and
    the float32 rounding of out, u sum|out dy| / h in the worst case; both are
    far below 1 % of the norm of the gradients here."""
    x = field(shape_of(2, 8, (13, 5), last), F32, 100)
    w, b = params(8, 100)
    lay = dict(act=act, channels_last=last, out_channels_last=out_last)
    out, stats = fno.fno_group_norm(x, 2, weight=w, bias=b, **lay)
    dy = field(out.shape, F32, 101)
    grads = fno.fno_group_norm_backward(x, stats, dy, 2, weight=w, bias=b, **lay)

    def loss(x, w, b):
        return (fno.fno_group_norm(x, 2, weight=w, bias=b, **lay)[0].double() * dy.double()).sum().item()

    h = 2.0 ** -7
    for i, (t, grad) in enumerate(zip((x, w, b), grads)):
        v = field(t.shape, F32, 102 + i)
        up = [x, w, b]
        dn = [x, w, b]
        up[i], dn[i] = t + h * v, t - h * v
        diff = (loss(*up) - loss(*dn)) / (2 * h)
        want = (grad.double() * v.double()).sum().item()
        assert abs(diff - want) <= 0.01 * grad.double().norm().item() * v.double().norm().item() / t.numel() ** 0.5, i


@pytest.mark.parametrize("last,out_last", LAYOUTS)
@pytest.mark.parametrize("b,c,grid,groups", [(2, 4, (32, 32), 2), (6, 64, (64, 64), 8), (2, 16, (400, 400), 4)])
def test_same_bits_again(b, c, grid, groups, last, out_last):
    x = field(shape_of(b, c, grid, last), F32, 110)
    w, bias = params(c, 110)
    opts = dict(weight=w, bias=bias, act="gelu", channels_last=last, out_channels_last=out_last)
    out, stats = fno.fno_group_norm(x, groups, **opts)
    dy = field(out.shape, F32, 111)
    first = (out, stats, *fno.fno_group_norm_backward(x, stats, dy, groups, **opts))
    for _ in range(3):
        o, s = fno.fno_group_norm(x, groups, **opts)
        again = (o, s, *fno.fno_group_norm_backward(x, stats, dy, groups, **opts))
        assert all(torch.equal(p, q) for p, q in zip(first, again))


@pytest.mark.parametrize("last,out_last", LAYOUTS)
@pytest.mark.parametrize("b,c,grid,groups", [(2, 4, (32, 32), 2), (4, 32, (200, 100), 8)])
def test_captured_and_replayed(b, c, grid, groups, last, out_last):
    """Two graphs captured on one stream, without an eager call before, each
    replayed several times with new inputs and eager work in between."""
    w, bias = params(c, 120)
    opts = dict(weight=w, bias=bias, act="gelu", channels_last=last, out_channels_last=out_last)
    stream = torch.cuda.Stream()
    runs = []
    for k in range(2):
        x = field(shape_of(b, c, grid, last), F32, 121 + k)
        dy = field(shape_of(b, c, grid, out_last), F32, 123 + k)
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=stream):
            out, stats = fno.fno_group_norm(x, groups, **opts)
            grads = fno.fno_group_norm_backward(x, stats, dy, groups, **opts)
        runs.append((g, x, dy, (out, stats, *grads)))
    for rep in range(3):
        wants = []
        for k, (g, x, dy, _) in enumerate(runs):
            x.copy_(field(x.shape, F32, 130 + 2 * rep + k))
            dy.copy_(field(dy.shape, F32, 140 + 2 * rep + k))
            out, stats = fno.fno_group_norm(x, groups, **opts)
            wants.append((out, stats, *fno.fno_group_norm_backward(x, stats, dy, groups, **opts)))
        torch.cuda.synchronize()
        # both at once, each on a stream of its own
        lanes = [torch.cuda.Stream(), torch.cuda.Stream()]
        for lane, (g, _, _, _) in zip(lanes, runs):
            with torch.cuda.stream(lane):
                g.replay()
        torch.cuda.synchronize()
        for (_, _, _, got), want in zip(runs, wants):
            assert all(torch.equal(p, q) for p, q in zip(got, want)), rep


@pytest.mark.parametrize("b,c,grid,groups,dtype", [
    (1, 32, (200, 200), 4, F32),       # one item over all workgroups
    (5, 48, (64, 61), 6, F32),
    (3, 30, (101, 67), 5, F16),        # incomplete super-rows
    (32, 64, (128, 128), 8, F32),      # several rounds of items
    (70, 32, (64, 64), 8, BF16),
])
@pytest.mark.parametrize("out_last", [True, False])
def test_workgroups_that_do_not_wait(b, c, grid, groups, dtype, out_last, monkeypatch):
    """Items spread over workgroups: one that does not see another's sums in
    time forms them itself.  With no time at all, most do; the bits are the same."""
    x = field((b, *grid, c), dtype, 180, 0.5)
    w, bias = params(c, 180)
    opts = dict(weight=w, bias=bias, act="gelu", channels_last=True, out_channels_last=out_last)
    out, stats = fno.fno_group_norm(x, groups, **opts)
    dy = field(out.shape, dtype, 181)
    want = (out, stats, *fno.fno_group_norm_backward(x, stats, dy, groups, **opts))
    for spin in ("0", "1"):
        monkeypatch.setenv("FNO_GN_SPIN", spin)
        out, stats = fno.fno_group_norm(x, groups, **opts)
        got = (out, stats, *fno.fno_group_norm_backward(x, stats, dy, groups, **opts))
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_streams_at_once():
    """Calls in flight on two streams share nothing."""
    cases = [(4, 64, (96, 96), 8, True, True), (4, 64, (96, 96), 8, False, True)]
    wants, xs = [], []
    for b, c, grid, groups, last, out_last in cases:
        x = field(shape_of(b, c, grid, last), F32, 150)
        xs.append(x)
        wants.append(fno.fno_group_norm(x, groups, act="gelu", channels_last=last, out_channels_last=out_last))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[], []]
    for _ in range(5):
        for i, (b, c, grid, groups, last, out_last) in enumerate(cases):
            with torch.cuda.stream(streams[i]):
                got[i].append(fno.fno_group_norm(xs[i], groups, act="gelu", channels_last=last,
                                                 out_channels_last=out_last))
    torch.cuda.synchronize()
    for want, results in zip(wants, got):
        for r in results:
            assert torch.equal(r[0], want[0]) and torch.equal(r[1], want[1])


@pytest.mark.parametrize("last,out_last", LAYOUTS)
def test_offsets_past_32_bits(last, out_last):
    """2^32 + 2^27 elements in 16 bits; the last group is checked whole."""
    b, c, p = 33, 4, 1 << 25
    x = torch.empty(shape_of(b, c, (p,), last), dtype=BF16, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(160)
    for i in range(b):
        x[i] = torch.randn(x[i].shape, generator=g, device=DEV) + i
    w, bias = params(c, 160)
    opts = dict(weight=w, bias=bias, act="silu", channels_last=last, out_channels_last=out_last)
    out, stats = fno.fno_group_norm(x, 2, **opts)
    ref = Reference(x[-1:], 2, w, bias, 1e-5, "silu", last)
    # a chain of additions grows with the positions a thread takes: none is longer than 2^13
    scale = 2 ** 13 / K
    y, err = ref.out(BF16)
    close(to_groups(out[-1:], 2, out_last), y, err * scale, "out of the last item")
    close(stats[-1:, :, 0], ref.stats[..., 0], scale * K * U * ref.xg.abs().mean((2, 3)), "mean")
    del y, err
    gx, _, _ = fno.fno_group_norm_backward(x, stats, out, 2, **opts)
    (rx, ex), _, _ = ref.grads(to_groups(out[-1:], 2, out_last), BF16)
    close(to_groups(gx[-1:], 2, last), rx, ex * scale, "grad_x of the last item")


@pytest.mark.parametrize("last", [True, False])
def test_between_spectral_layers(last):
    """A training step as a model runs it: spectral convolution with its tail,
    group norm, a loss, and everything backward, clipped at the end."""
    b, c, n, m, groups = 3, 16, 64, 12, 4
    x = field((b, c, n, n), F32, 170)
    w = torch.view_as_complex(field((2, m, m, c, c, 2), F32, 171, 0.0, 1.0 / c))
    gamma, beta = params(c, 172)
    h = fno.fno_spectral_conv2d(x, w, m, m)
    y, stats = fno.fno_group_norm(h, groups, weight=gamma, bias=beta, act="gelu", out_channels_last=last)
    dy = field(y.shape, F32, 173)
    gh, ggamma, gbeta = fno.fno_group_norm_backward(h, stats, dy, groups, weight=gamma, bias=beta, act="gelu",
                                                    out_channels_last=last)
    gx, gw = fno.fno_spectral_conv2d_backward(x, w, gh, m, m)
    grads = [gw, ggamma, gbeta]
    raw = [g.clone() for g in grads]
    norm = fno.fno_clip_grad_norm(grads, 1.0)
    torch.cuda.synchronize()

    # the same step by float64 definitions, on the CPU (whose complex-to-real transform leaves out the imaginary
    # parts of the ky = 0 and Nyquist bins, as the operator's definition does)
    xd, wd = x.cpu().double().requires_grad_(True), w.cpu().to(torch.complex128).requires_grad_(True)
    gd, bd = gamma.cpu().double().requires_grad_(True), beta.cpu().double().requires_grad_(True)
    f = torch.fft.rfft2(xd, norm="ortho")
    kx = list(range(m)) + list(range(n - m, n))
    kept = f[:, :, kx, :m].reshape(b, c, 2, m, m)
    mixed = (kept.permute(2, 3, 4, 0, 1) @ wd).permute(3, 4, 0, 1, 2).reshape(b, c, 2 * m, m)
    spec = torch.zeros(b, c, n, n // 2 + 1, dtype=torch.complex128)
    spec = spec.index_put((torch.arange(b).view(-1, 1, 1, 1), torch.arange(c).view(1, -1, 1, 1),
                           torch.tensor(kx).view(1, 1, -1, 1), torch.arange(m).view(1, 1, 1, -1)), mixed)
    hd = torch.fft.irfft2(spec, s=(n, n), norm="ortho")
    hg = hd.reshape(b, groups, -1)
    xh = ((hg - hg.mean(2, keepdim=True)) * (hg.var(2, unbiased=False, keepdim=True) + 1e-5).rsqrt()).view_as(hd)
    z = xh * gd.view(1, c, 1, 1) + bd.view(1, c, 1, 1)
    yd = z * torch.special.ndtr(z)
    dyd = dy.cpu().double().permute(0, 3, 1, 2) if last else dy.cpu().double()
    wants = torch.autograd.grad((yd * dyd).sum(), [wd, gd, bd, xd])
    # the transforms' own bar: relative L2 error 1e-5
    for got, want, what in zip(raw + [gx], wants, ("grad_w", "grad_weight", "grad_bias", "grad_x")):
        rel = ((got.cpu() - want).abs().square().sum() / want.abs().square().sum()).sqrt().item()
        print(f"  {what}: rel_l2={rel:.2e}", flush=True)
        assert rel <= 1e-5, what
    total = sum(g.abs().double().square().sum() for g in raw).sqrt()
    assert abs(norm.item() - total.item()) <= 2 * U * total.item()
    coef = min(1.0, 1.0 / (total.item() + 1e-6))
    for got, g in zip(grads, raw):
        assert torch.allclose(got, g * coef, rtol=4 * U, atol=0)


@pytest.mark.parametrize("last", [True, False])
def test_thousands_of_chunks(last):
    """One item of 3 10^8 values: its statistics come from more chunks than a
    workgroup joins at a time.  (Chains as in test_offsets_past_32_bits.)"""
    c, p = 2, 150_000_001
    x = torch.empty(shape_of(1, c, (p,), last), dtype=BF16, device=DEV)
    x.normal_(3.0, 1.0, generator=torch.Generator(device=DEV).manual_seed(190))
    out, stats = fno.fno_group_norm(x, 1, act="silu", channels_last=last)
    xd = x.double()
    mean, var = xd.mean(), xd.var(unbiased=False)
    assert abs(stats[0, 0, 0].item() - mean.item()) <= 2 ** 13 * U * mean.item()
    assert abs(stats[0, 0, 1].item() - (var + 1e-5).rsqrt().item()) <= 2 ** 13 * U
    z = (xd - mean) * (var + 1e-5).rsqrt()
    del xd
    want = z * torch.sigmoid(z)
    err = (out.double() - want).abs_()
    assert (err <= 2 ** -8 * want.abs() + 2 ** 14 * U * (1 + z.abs())).all()
    del z, want, err
    dy = torch.ones_like(out)
    gx, _, _ = fno.fno_group_norm_backward(x, stats, dy, 1, channels_last=last)
    # without an activation a constant gradient is taken back out by the mean: only roundings stay
    assert gx.float().abs().max().item() <= 2 ** 14 * U


SCHEDULES = {
    # (b, c, grid, groups, dtype, last, out_last): kernels of the forward and of the backward call
    (2, 4, (32, 32), 2, F32, True, True): (["gn_fused"], ["gn_bwd_fused", "gn_bwd_finish"]),
    (2, 4, (32, 32), 2, F32, False, False): (["gn_fused"], ["gn_bwd_fused", "gn_bwd_finish"]),
    (4, 32, (64, 64), 4, F32, True, True): (["gn_clear", "gn_once"], ["gn_clear", "gn_bwd_once", "gn_bwd_finish"]),
    (4, 32, (64, 64), 4, F32, True, False): (["gn_clear", "gn_once"],
                                             ["gn_bwd_sums_cross", "gn_bwd_apply_cross"]),
    (1, 6, (30, 30), 2, F32, True, False): (["gn_clear", "gn_once"], ["gn_bwd_sums_cross", "gn_bwd_apply_cross"]),
    (1, 6, (30, 30), 2, F32, False, True): (["gn_stats", "gn_apply_cross"],
                                            ["gn_bwd_sums_cross", "gn_bwd_apply_cross"]),
    (3, 30, (61, 47), 5, F16, True, True): (["gn_stats", "gn_apply"], ["gn_bwd_sums", "gn_bwd_apply"]),
    # the fewest chunks that give every CU work, and no more than a workgroup has looks for
    (1, 64, (256, 256), 8, F32, True, True): (["gn_clear", "gn_once"], ["gn_clear", "gn_bwd_once", "gn_bwd_finish"]),
    (1, 64, (512, 512), 64, F32, True, True): (["gn_stats", "gn_finish", "gn_apply"],
                                               ["gn_bwd_sums", "gn_bwd_finish", "gn_bwd_apply"]),
    (2, 16, (300, 300), 2, F32, False, False): (["gn_stats", "gn_apply"], ["gn_bwd_sums", "gn_bwd_apply"]),
    (2, 64, (512, 512), 2, F32, False, False): (["gn_stats", "gn_finish", "gn_apply"],
                                                ["gn_bwd_sums", "gn_bwd_finish", "gn_bwd_apply"]),
    (2, 64, (512, 512), 2, F32, False, True): (["gn_stats", "gn_finish", "gn_apply_cross"],
                                               ["gn_bwd_sums_cross", "gn_bwd_finish", "gn_bwd_apply_cross"]),
    (1, 2049, (8,), 3, F32, True, True): (["gn_stats_wide", "gn_finish", "gn_apply"],
                                          ["gn_bwd_sums", "gn_bwd_finish", "gn_bwd_apply"]),
    (1, 2049, (8,), 3, F32, True, False): (["gn_stats_wide", "gn_finish", "gn_apply_cross"],
                                           ["gn_bwd_sums_cross", "gn_bwd_finish", "gn_bwd_apply_cross"]),
}


@pytest.mark.parametrize("key", SCHEDULES, ids=str)
def test_schedules(key):
    """Which kernels a call runs, and that each schedule is right."""
    b, c, grid, groups, dtype, last, out_last = key
    x = field(shape_of(b, c, grid, last), dtype, 200)
    w, bias = params(c, 200)
    opts = dict(weight=w, bias=bias, act="gelu", channels_last=last, out_channels_last=out_last)
    out, stats = fno.fno_group_norm(x, groups, **opts)
    forward = fno.fno_last_kernels()
    fno.fno_group_norm_backward(x, stats, out, groups, **opts)
    assert (forward, fno.fno_last_kernels()) == SCHEDULES[key]
    check(b, c, grid, groups, "gelu", dtype, None, last, out_last, seed=201)


def test_host_threads_at_once():
    import threading
    x = field((4, 64, 64, 32), F32, 210)
    want, stats = fno.fno_group_norm(x, 8, act="gelu", channels_last=True)
    grads = [field((1000, 7), F32, 211), field((33,), BF16, 212)]
    norm = fno.fno_grad_norm(grads)
    results, errors = [], []

    def work():
        try:
            for _ in range(20):
                out, _ = fno.fno_group_norm(x, 8, act="gelu", channels_last=True)
                results.append((out, fno.fno_grad_norm(grads)))
        except Exception as e:          # noqa: BLE001 (shown below)
            errors.append(e)

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors and len(results) == 80
    assert all(torch.equal(o, want) and torch.equal(n, norm) for o, n in results)


@pytest.mark.parametrize("b,c,grid,groups", [
    (2, 4100, (701,), 41),         # several chunks of positions, the last one short
    (3, 2050, (1031,), 2050),      # a group a channel
    (1, 70000, (9,), 1),           # a group of more than 65536 channels
    (2, 131072 + 2, (3,), 2),
    (1, 2051, (5000,), 7),
])
@pytest.mark.parametrize("dtype", [F32, F16])
def test_wide_channels_in_chunks(b, c, grid, groups, dtype):
    check(b, c, grid, groups, "silu", dtype, None, True, True, seed=220)


def test_wide_channels_of_one_value():
    """A chunk's mean is its values' own, so a constant group has no deviation."""
    x = torch.full((2, 300, 4100), 1234.5678, device="cuda")
    out, stats = fno.fno_group_norm(x, 41, channels_last=True)
    assert torch.equal(out, torch.zeros_like(out))
    assert torch.equal(stats[..., 0], torch.full_like(stats[..., 0], 1234.5678))


def test_groups_of_many_pairs():
    """Groups whose partial sums a workgroup joins, and those a wave does."""
    for c, grid, groups in ((64, (512, 512), 1), (16, (512, 2048), 4), (64, (512, 512), 64)):
        check(1, c, grid, groups, "gelu", F32, None, True, True, seed=230)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("b,c,grid,groups", [
    (32, 64, (128, 128), 8),
    (64, 64, (64, 64), 8),
    (1, 145, (132, 126), 1),       # rows of odd length, eight at a time
    (13, 600, (2161,), 3),
])
def test_16_bit_fields_with_float32_grad_out(b, c, grid, groups, dtype):
    """Larger fields that stay in 16 bits on one side only, in one layout."""
    check(b, c, grid, groups, "gelu", dtype, F32, True, True, seed=240)


@pytest.mark.parametrize("b,c,grid,groups,last", [
    (4, 133, (128, 128), 19, False),       # group 18 lies in two tiles of 64 channels, group 9 too
    (2, 130, (16384,), 10, False),
    (1, 192, (16384,), 2, False),          # of 96 channels
    (2, 66, (128, 129), 33, False),
    (3, 150, (2001,), 6, True),            # 2001 positions: two passes
])
@pytest.mark.parametrize("seed", range(4))
def test_groups_in_two_tiles(b, c, grid, groups, last, seed):
    """A group whose output several workgroups write, each joining the chunks itself, has one set of statistics: every
    output is, to the bit, what the stored ones make of its value."""
    x = field(shape_of(b, c, grid, last), F32, 250 + seed)
    opts = dict(channels_last=last, out_channels_last=not last)
    out, stats = fno.fno_group_norm(x, groups, **opts)
    assert fno.fno_last_kernels() == ["gn_stats", "gn_apply_cross"]
    mean, rstd = (s.repeat_interleave(c // groups, 1).view(b, c, 1) for s in stats.unbind(2))
    flat = x.view(b, -1, c).transpose(1, 2) if last else x.view(b, c, -1)
    want = (flat - mean) * rstd
    got = out.view(b, c, -1) if last else out.view(b, -1, c).transpose(1, 2)
    assert torch.equal(got, want)
    again, st = fno.fno_group_norm(x, groups, **opts)
    assert torch.equal(again, out) and torch.equal(st, stats)


# every schedule of the backward pass, with remainders of vectors, rows, tiles and chunks
SUMS = [
    (2, 4, (32, 32), 2), (5, 33, (7, 9), 11), (300, 4, (3,), 2), (2, 511, (9,), 7), (3, 30, (61, 47), 5),
    (4, 32, (64, 64), 4), (70, 32, (64, 64), 8), (32, 64, (128, 128), 8), (256, 64, (4096,), 16),
    (1, 3, (100003,), 1), (8, 128, (16384,), 32), (1, 64, (512, 512), 64), (2, 16, (1031, 1033), 4),
    (4, 133, (128, 127), 19), (1, 2049, (8,), 3), (2, 4100, (701,), 41), (1, 2051, (5000,), 7),
]


@pytest.mark.parametrize("last,out_last", LAYOUTS)
@pytest.mark.parametrize("dtype,out_dtype", [(F32, F32), (BF16, BF16), (F16, F32)])
@pytest.mark.parametrize("b,c,grid,groups", SUMS)
def test_parameter_gradients_of_whole_numbers(b, c, grid, groups, dtype, out_dtype, last, out_last):
    """With whole numbers x (mean 0 and deviation 1 prescribed) and grad_out the sums are whole numbers below 2^24 and
    exact in float32 in any order.  All are positive: no position can be lost or counted twice."""
    g = torch.Generator(device=DEV).manual_seed(260)
    x = torch.randint(1, 3, shape_of(b, c, grid, last), generator=g, device=DEV).to(dtype)
    dy = torch.randint(1, 4, shape_of(b, c, grid, out_last), generator=g, device=DEV).to(out_dtype)
    w, bias = params(c, 261)
    stats = torch.tensor([0.0, 1.0], device=DEV).expand(b, groups, 2).contiguous()
    xg, yg = to_groups(x, groups, last), to_groups(dy, groups, out_last)
    want_b, want_w = yg.sum((0, 3)).flatten(), (xg * yg).sum((0, 3)).flatten()
    assert want_w.max().item() < 2 ** 24
    for need_x in (True, False):
        _, gw, gb = fno.fno_group_norm_backward(x, stats, dy, groups, weight=w, bias=bias, channels_last=last,
                                                out_channels_last=out_last, need_x=need_x)
        assert torch.equal(gb.double(), want_b) and torch.equal(gw.double(), want_w), need_x


@pytest.mark.parametrize("last,out_last", LAYOUTS)
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("b,c,grid,groups", SUMS)
def test_statistics_of_the_ends(b, c, grid, groups, dtype, last, out_last):
    """Ones at an item's first and last 61 positions and zeros between: with a share k of ones the mean is k and the
    variance k (1 - k).  One of the at most 122 positions lost or counted twice changes both by a hundredth.  A
    thread's sums of these whole numbers are exact; the joins of threads and chunks, fewer than 64 additions in a row,
    leave 64 u."""
    p = 1
    for v in grid:
        p *= v
    at = torch.arange(p, device=DEV)
    line = ((at < 61) | (at >= p - 61)).to(dtype)
    x = (line.view(1, p, 1).expand(b, p, c) if last else line.view(1, 1, p).expand(b, c, p)).contiguous()
    x = x.view(shape_of(b, c, grid, last))
    _, stats = fno.fno_group_norm(x, groups, eps=1e-5, channels_last=last, out_channels_last=out_last)
    k = line.sum().item() / p
    mean = torch.full((b, groups), k, dtype=torch.float64, device=DEV)
    rstd = torch.full_like(mean, (k * (1 - k) + 1e-5) ** -0.5)
    close(stats[..., 0], mean, 64 * U * mean, "mean")
    # the squares about a mean that is itself off by 64 u of at most 1, where all values are ones
    close(stats[..., 1], rstd, rstd * 64 * U + rstd ** 3 * (64 * U) ** 2, "rstd")


@pytest.mark.parametrize("last,out_last", LAYOUTS)
def test_parameter_gradients_of_many_values(last, out_last):
    """26 million values of either sign a channel.  A value's rounding errors are random; one of an addition has a
    deviation of 0.45 u times the sum it leaves.  n values in chains of L, whose sums are added pairwise over l levels,
    then carry 0.45 u (L / 2 + l)^1/2 n^1/2 rms: 2.5 u n^1/2 rms for chains of 16 and, together, 20 levels.  Over 64
    channels the root mean square is within a third of that; 4 is allowed (chains of hundreds give more)."""
    b, c, p, groups = 25, 64, 1 << 20, 8
    x = torch.empty(shape_of(b, c, (p,), last), device=DEV)
    dy = torch.empty(shape_of(b, c, (p,), out_last), device=DEV)
    g = torch.Generator(device=DEV).manual_seed(270)
    x.normal_(generator=g)
    dy.normal_(generator=g)
    stats = torch.tensor([0.0, 1.0], device=DEV).expand(b, groups, 2).contiguous()
    w, bias = params(c, 271)
    _, gw, gb = fno.fno_group_norm_backward(x, stats, dy, groups, weight=w, bias=bias, channels_last=last,
                                            out_channels_last=out_last, need_x=False)
    want_w, want_b, sq_w, sq_b = (torch.zeros(c, dtype=torch.float64, device=DEV) for _ in range(4))
    for i in range(b):
        xi = x[i].double() if last else x[i].double().t()
        yi = dy[i].double() if out_last else dy[i].double().t()
        want_b += yi.sum(0)
        sq_b += yi.square().sum(0)
        xi = xi * yi
        want_w += xi.sum(0)
        sq_w += xi.square_().sum(0)
    for got, want, sq, what in ((gw, want_w, sq_w, "grad_weight"), (gb, want_b, sq_b, "grad_bias")):
        rms = ((got.double() - want).square() / sq).mean().sqrt().item() / U
        print(f"  {what}: root mean square error {rms:.2f} u n^1/2 rms", flush=True)
        assert rms <= 4.0, what


@pytest.mark.parametrize("key", [*SUMS, (1, 64, (256, 256), 8), (2, 64, (512, 512), 2)], ids=str)
@pytest.mark.parametrize("last,out_last", LAYOUTS)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_squares_beyond_float32(key, last, out_last, dtype):
    """Finite values whose squares are not: the deviation is infinite, out = act(bias), and the gradient is zero."""
    b, c, grid, groups = key
    p = 1
    for v in grid:
        p *= v
    w, bias = params(c, 281)
    opts = dict(weight=w, bias=bias, channels_last=last, out_channels_last=out_last)
    want = to_groups(bias.to(dtype).view(1, c, 1), groups, False).expand(b, -1, -1, p)
    # one magnitude, the sign alternating at every so many positions: each thread's values have the same mean
    for period in (1, 2, 4, 16, 64, 256, 1024):
        line = 1e21 * (1 - 2 * (torch.arange(p, device=DEV) // period % 2))
        line = (line.view(1, p, 1).expand(b, p, c) if last else line.view(1, 1, p).expand(b, c, p)).contiguous()
        x = line.to(dtype).view(shape_of(b, c, grid, last))
        out, stats = fno.fno_group_norm(x, groups, **opts)
        assert torch.isfinite(stats[..., 0]).all()
        if period >= p:
            continue              # no deviation at all
        assert (stats[..., 1] == 0).all(), period
        assert torch.equal(to_groups(out, groups, out_last), want.double()), period
        gx, _, _ = fno.fno_group_norm_backward(x, stats, torch.ones_like(out), groups, **opts)
        assert (gx == 0).all()
