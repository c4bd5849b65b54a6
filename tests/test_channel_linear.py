"""Channel products of fields on the GPU, forward and backward, against float64.

Bounds count rounding steps.  A sum of K float32 products (each as good as
float32's: what the six part products leave out is below 2^-26) is within
(K + 8) 2^-24 of the sum S of the products' sizes; an activation passes on at most
1.13 of it and adds a few half steps of its own; slopes differ by at most 0.8
of what z does.  Whole numbers have exact sums and must come out equal.
"""
import itertools

import pytest

torch = pytest.importorskip("torch")

import fft_spectral_convolution_amd as fno  # noqa: E402

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
EPS = 2.0 ** -24
HALF_STEP = {F32: 2.0 ** -24, BF16: 2.0 ** -8, F16: 2.0 ** -11}
TYPES = [(F32, F32), (BF16, BF16), (BF16, F32), (F16, F16), (F16, F32)]
LAYOUTS = list(itertools.product((False, True), repeat=2))


@pytest.fixture(scope="module", autouse=True)
def _gpu_present():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    fno.lib()


def shape_of(B, C, grid, last):
    return (B, *grid, C) if last else (B, C, *grid)


def points(t, last):
    """[B P, C] in float64 on the CPU."""
    t = t.double().cpu()
    C = t.shape[-1] if last else t.shape[1]
    return (t if last else t.movedim(1, -1)).reshape(-1, C)


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


class Case:
    def __init__(self, B, cin, cout, grid, types=(F32, F32), last=False, out_last=False, act="none", branch="none",
                 bias=True, seed=0, whole=False):
        gen = torch.Generator().manual_seed(seed)

        def draw(*shape):
            if whole:
                return torch.randint(-3, 4, shape, generator=gen).float()
            return torch.randn(*shape, generator=gen)

        self.types, self.last, self.out_last, self.act, self.branch_at = types, last, out_last, act, branch
        x_type, out_type = types
        self.x = draw(*shape_of(B, cin, grid, last)).to(x_type).to(DEV)
        self.w = (draw(cout, cin) if whole else draw(cout, cin) * cin ** -0.5).to(x_type).to(DEV)
        self.bias = draw(cout).to(DEV) if bias else None
        self.branch = draw(*shape_of(B, cout, grid, out_last)).to(out_type).to(DEV) if branch != "none" else None
        self.grad_out = draw(*shape_of(B, cout, grid, out_last)).to(out_type).to(DEV)
        X, W = points(self.x, last), self.w.double().cpu()
        self.z = X @ W.t()
        size = X.abs() @ W.abs().t()
        if bias:
            self.z = self.z + self.bias.double().cpu()
            size = size + self.bias.double().cpu().abs()
        if branch == "before":
            self.z = self.z + points(self.branch, out_last)
            size = size + points(self.branch, out_last).abs()
        self.z_bound = (cin + 8) * EPS * size
        self.X, self.W = X, W

    def options(self):
        return dict(bias=self.bias, branch=self.branch, branch_after=self.branch_at == "after", act=self.act,
                    channels_last=self.last, out_channels_last=self.out_last)

    def forward(self, **more):
        return fno.fno_channel_linear(self.x, self.w, out_dtype=self.types[1], **self.options(), **more)

    def check_forward(self, out=None):
        out = self.forward() if out is None else out
        want = act_of(self.z, self.act)
        bound = 1.13 * self.z_bound + (8 * EPS * self.z.abs() + 1e-30 if self.act != "none" else 0)
        if self.branch_at == "after":
            r = points(self.branch, self.out_last)
            want = want + r
            bound = bound + EPS * want.abs()
        half = HALF_STEP[self.types[1]]
        bound = bound * 1.01 + half * want.abs() * 1.01 + (2.0 ** -25 if self.types[1] == F16 else 0)
        assert out.dtype == self.types[1]
        close(points(out, self.out_last), want, bound, "out")

    def backward(self, **more):
        return fno.fno_channel_linear_backward(self.x, self.w, self.grad_out, **self.options(), **more)

    def check_backward(self, got=None):
        gx, gw, gb, gr = self.backward() if got is None else got
        go = points(self.grad_out, self.out_last)
        g = go * slope_of(self.z, self.act)
        if self.act == "none":
            g_bound = torch.zeros_like(g)
        else:      # the slope's own error: a few half steps of values up to 1.13, 1.5e-7 of erf
            g_bound = go.abs() * (0.8 * self.z_bound + 12 * EPS)
        X, W = self.X, self.W
        n, cout = g.shape
        half = HALF_STEP[self.types[0]]
        want = g @ W
        # for grad_x, g of a 16-bit field is two bfloat16 parts.  Each is the nearest with 8 bits of fraction to what
        # is left: |g - hi| <= 2^-9 |g|, |g - hi - lo| <= 2^-9 2^-9 |g| = 2^-18 |g|.  Of float16 weights, two parts as
        # well (w = w1 + w2, |w2| <= 2^-9 |w|), the product lo w2 is left out: another 2^-18.
        parts = 2.0 ** -17 if self.types[0] != F32 else 0.0
        bound = g_bound @ W.abs() + ((cout + 8) * EPS + parts) * (g.abs() @ W.abs())
        bound = bound * 1.01 + half * want.abs() * 1.01 + (2.0 ** -24 if self.types[0] == F16 else 0)
        close(points(gx, self.last), want, bound, "grad_x")
        assert gw.dtype == F32 and gw.shape == self.w.shape
        bound = g_bound.t() @ X.abs() + (n + 64) * EPS * (g.abs().t() @ X.abs())
        close(gw.double().cpu(), g.t() @ X, bound, "grad_weight")
        if self.bias is not None:
            bound = g_bound.sum(0) + (n + 64) * EPS * g.abs().sum(0)
            close(gb.double().cpu(), g.sum(0), bound, "grad_bias")
        else:
            assert gb is None
        if self.branch is None:
            assert gr is None
        elif self.branch_at == "after" or self.act == "none":
            assert gr is self.grad_out
        else:
            bound = g_bound + HALF_STEP[self.types[1]] * g.abs() * 1.01 + (2.0 ** -25 if self.types[1] == F16 else 0)
            close(points(gr, self.out_last), g, bound, "grad_branch")


def close(got, want, bound, what):
    bad = ~((got - want).abs() <= bound)
    worst = float(((got - want).abs() / (bound + 1e-300)).max())
    assert not bool(bad.any()), (what, int(bad.sum()), bad.numel(), worst, bad.nonzero()[:4].tolist())


SIZES = [(1, 1, 1, (1,)), (2, 4, 4, (32, 32)), (3, 3, 64, (7, 9)), (1, 64, 1, (65,)), (2, 17, 33, (5, 13)),
         (1, 30, 50, (127,)), (2, 64, 64, (64,)), (5, 32, 32, (31,)), (1, 65, 100, (3, 43)), (2, 128, 130, (100,)),
         (7, 200, 40, (2,)), (1, 300, 260, (70,)), (1, 16, 16, (1000,)),
         (2, 70, 20, (50,)), (1, 33, 127, (97,)), (3, 129, 66, (400,))]


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("last,out_last", LAYOUTS)
def test_whole_numbers(size, last, out_last):
    """Every place of every size, layout and type exactly: whole numbers, nothing to round."""
    for types in TYPES:
        c = Case(*size, types=types, last=last, out_last=out_last, branch="before", whole=True)
        if types[1] == F32 or c.z.abs().max() <= (256 if types[1] == BF16 else 2048):
            assert torch.equal(points(c.forward(), out_last), c.z)
        gx, gw, gb, gr = c.backward()
        g = points(c.grad_out, out_last)
        want = g @ c.W
        if types[0] == F32 or want.abs().max() <= (256 if types[0] == BF16 else 2048):
            assert torch.equal(points(gx, last), want)
        assert torch.equal(gw.double().cpu(), g.t() @ c.X) and torch.equal(gb.double().cpu(), g.sum(0))


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("types", TYPES)
def test_forward(size, types):
    for k, (last, out_last) in enumerate(LAYOUTS):
        act = ("gelu", "silu", "none", "gelu")[k]
        for branch in ("none", "before", "after"):
            Case(*size, types=types, last=last, out_last=out_last, act=act, branch=branch, seed=k,
                 bias=branch != "after").check_forward()


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("types", TYPES)
def test_backward(size, types):
    for k, (last, out_last) in enumerate(LAYOUTS):
        act = ("silu", "gelu", "gelu", "none")[k]
        for branch in ("none", "before", "after"):
            Case(*size, types=types, last=last, out_last=out_last, act=act, branch=branch, seed=k,
                 bias=branch != "after").check_backward()


def test_gradient_by_differences():
    c = Case(2, 5, 7, (3, 11), act="gelu", branch="before", seed=3)
    gx, gw, gb, gr = c.backward()
    go = points(c.grad_out, False)

    def loss(z):
        return (act_of(z, "gelu") * go).sum()

    gen = torch.Generator().manual_seed(5)
    e = 1e-4
    dX, dW = torch.randn(c.X.shape, generator=gen).double(), torch.randn(c.W.shape, generator=gen).double()
    db = torch.randn(7, generator=gen).double()
    dr = torch.randn(c.z.shape, generator=gen).double()
    rest = c.z - c.X @ c.W.t()

    def at(s):
        return loss((c.X + s * dX) @ (c.W + s * dW).t() + rest + s * (db + dr))

    slope = (at(e) - at(-e)) / (2 * e)
    got = (points(gx, False) * dX).sum() + (gw.double().cpu() * dW).sum() + (gb.double().cpu() * db).sum() \
        + (points(gr, False) * dr).sum()
    # differences: e^2 times a third derivative of a few hundred terms of order one
    assert abs(got - slope) < 1e-4 * (1 + abs(slope))


@pytest.mark.parametrize("types", [(F32, F32), (BF16, BF16), (F16, F16)])
@pytest.mark.parametrize("last,out_last", LAYOUTS)
def test_not_finite_values_stay_at_their_position(types, last, out_last):
    c = Case(2, 20, 70, (9, 15), types=types, last=last, out_last=out_last, act="gelu")
    clean = points(c.forward(), out_last)
    bad = {17: float("nan"), 134: float("inf"), 200: float("-inf")}
    flat = points(c.x, last).clone()
    for p, v in bad.items():
        flat[p, p % 20] = v
    x = flat.reshape(2, 9, 15, 20)
    c.x = (x if last else x.movedim(-1, 1)).contiguous().to(types[0]).to(DEV)
    out = points(c.forward(), out_last)
    touched = torch.zeros(len(flat), dtype=torch.bool)
    touched[list(bad)] = True
    assert torch.equal(out[~touched], clean[~touched])
    assert bool(torch.isnan(out[17]).all())


@pytest.mark.parametrize("size", [(2, cin, cout, (9, 15)) for cin, cout in ((20, 50), (70, 20), (40, 100), (130, 70))])
@pytest.mark.parametrize("last,out_last", LAYOUTS)
def test_not_finite_gradients_stay_at_their_position(size, last, out_last):
    """A NaN of grad_out, of the branch or of x reaches grad_x and grad_branch at its own position alone."""
    for types in ((F32, F32), (BF16, BF16), (F16, F32)):
        c = Case(*size, types=types, last=last, out_last=out_last, act="silu", branch="before")
        clean = c.backward(need_w=False)
        B, cin, cout, grid = size
        at = {"grad_out": 17, "branch": 18, "x": 133}
        for name, p in at.items():
            is_last = last if name == "x" else out_last
            t = getattr(c, name)
            flat = points(t, is_last)
            flat[p] = float("nan")
            t2 = flat.reshape(B, *grid, -1)
            setattr(c, name, (t2 if is_last else t2.movedim(-1, 1)).contiguous().to(t.dtype).to(DEV))
        got = c.backward(need_w=False)
        touched = torch.zeros(B * 135, dtype=torch.bool)
        touched[list(at.values())] = True
        for k, is_last in ((0, last), (3, out_last)):
            g, w = points(got[k], is_last), points(clean[k], is_last)
            assert torch.equal(g[~touched], w[~touched])
            assert bool(torch.isnan(g[touched]).all())


def test_large_and_tiny_values():
    c = Case(1, 40, 70, (200,), seed=4)
    for scale in (2.0 ** 100, 2.0 ** -100):
        d = Case(1, 40, 70, (200,), seed=4, bias=False)
        d.x = d.x * scale
        got = points(d.forward(), False) / scale
        close(got, d.z, d.z_bound * 1.01 + HALF_STEP[F32] * d.z.abs(), scale)
    assert c.x is not None


def test_slices_at_any_offset():
    """Fields need the alignment of their elements only."""
    for types in TYPES:
        for last in (False, True):
            c = Case(2, 24, 40, (130,), types=types, last=last, out_last=last, act="silu", branch="after")

            def moved(t, k):
                buf = torch.zeros(t.numel() + 8, dtype=t.dtype, device=DEV)
                v = buf[k:k + t.numel()].view(t.shape)
                v.copy_(t)
                return v

            c.x, c.w, c.branch, c.grad_out = moved(c.x, 1), moved(c.w, 3), moved(c.branch, 5), moved(c.grad_out, 7)
            buf = torch.full((c.grad_out.numel() + 8,), 7.0, dtype=types[1], device=DEV)
            out = buf[3:3 + c.grad_out.numel()].view(c.grad_out.shape)
            c.check_forward(c.forward(out=out))
            assert bool((buf[:3] == 7).all()) and bool((buf[-5:] == 7).all())
            c.check_backward()


@pytest.mark.parametrize("last", [False, True])
def test_fields_beyond_32_bits(last):
    """More than 2^32 bytes and 2^31 values: the last items as the call on them alone."""
    B, C, P = 66, 8, 1 << 22
    shape = (B, P, C) if last else (B, C, P)
    x = torch.empty(shape, dtype=BF16, device=DEV).normal_()
    w = torch.randn(C, C, device=DEV).to(BF16)
    out = fno.fno_channel_linear(x, w, act="gelu", channels_last=last)
    tail = fno.fno_channel_linear(x[-2:].contiguous(), w, act="gelu", channels_last=last)
    assert torch.equal(out[-2:], tail)
    g = out
    gx, gw, _, _ = fno.fno_channel_linear_backward(x, w, g, act="gelu", channels_last=last)
    tail = fno.fno_channel_linear_backward(x[-2:].contiguous(), w, g[-2:].contiguous(), act="gelu",
                                           channels_last=last, need_w=False)[0]
    assert torch.equal(gx[-2:], tail)
    parts = sum(fno.fno_channel_linear_backward(x[k:k + 11], w, g[k:k + 11], act="gelu", channels_last=last,
                                                need_x=False)[1].double() for k in range(0, B, 11))
    # sums of 2.8e8 terms of either sign, in float32 over up to 10^6 of them at a time
    assert (gw.double() - parts).norm() <= 1e-4 * parts.norm()


def test_equal_bits_and_other_stream():
    c = Case(4, 48, 96, (61, 47), types=(BF16, BF16), last=True, out_last=True, act="gelu")
    a, b = c.forward(), c.backward()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        d, e = c.forward(), c.backward()
    s.synchronize()
    assert torch.equal(a, d)
    assert all(torch.equal(u, v) for u, v in zip(b[:3], e[:3]))


def test_captured():
    c = Case(3, 20, 36, (11, 13), act="gelu", branch="before", seed=8)
    graph = torch.cuda.CUDAGraph()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream), torch.cuda.graph(graph, stream=stream):
        out, grads = c.forward(), c.backward()
    for k in range(3):
        c.x.copy_(torch.randn_like(c.x))
        c.grad_out.copy_(torch.randn_like(c.grad_out))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, c.forward())
        assert all(torch.equal(u, v) for u, v in zip(grads, c.backward()))


def test_chosen_gradients():
    c = Case(2, 12, 20, (40,), act="silu", branch="before")
    full = c.backward()
    gx, gw, gb, gr = c.backward(need_w=False, need_branch=False)
    assert torch.equal(gx, full[0]) and gw is gb is gr is None
    gx, gw, gb, gr = c.backward(need_x=False)
    assert gx is None and torch.equal(gw, full[1]) and torch.equal(gb, full[2]) and torch.equal(gr, full[3])
    gx, gw, gb, gr = c.backward(need_x=False, need_w=False)
    assert torch.equal(gr, full[3])
    with pytest.raises(ValueError):
        c.backward(need_x=False, need_w=False, need_branch=False)


def test_refusals():
    c = Case(2, 12, 20, (40,), branch="before")
    x, w, b, r = c.x, c.w, c.bias, c.branch
    for bad in ({"act": "relu"}, {"bias": b[:3]}, {"branch": r[:1]}, {"out": torch.empty(2, 40, 20, device=DEV)}):
        with pytest.raises(ValueError):
            fno.fno_channel_linear(x, w, **bad)
    for bad in ({"bias": b.to(BF16)}, {"branch": r.to(BF16)}, {"out_dtype": torch.float64},
                {"out": torch.empty(2, 20, 40, device=DEV, dtype=BF16), "out_dtype": F32}):
        with pytest.raises(TypeError):
            fno.fno_channel_linear(x, w, **bad)
    with pytest.raises(TypeError):
        fno.fno_channel_linear(x, w.to(BF16))
    with pytest.raises(ValueError):
        fno.fno_channel_linear(x, w[:, :5].contiguous())
    with pytest.raises(ValueError):
        fno.fno_channel_linear(x.transpose(1, 2), w)
    with pytest.raises(ValueError):
        fno.fno_channel_linear(x.cpu(), w)
    with pytest.raises(fno.FnoError) as e:
        fno.fno_channel_linear(x, w, out_dtype=BF16)             # float32 in, bfloat16 out
    assert e.value.status == -12
    square = torch.eye(12, device=DEV)
    with pytest.raises(fno.FnoError) as e:
        fno.fno_channel_linear(x, square, out=x)
    assert e.value.status == -4
    with pytest.raises(fno.FnoError) as e:
        fno.fno_channel_linear(x[:0], w)
    assert e.value.status == -2
    with pytest.raises(ValueError):
        fno.fno_channel_linear_backward(x, w, c.grad_out[:1])
    with pytest.raises(ValueError):
        fno.fno_channel_linear_backward(x, w, c.grad_out, grad_x=torch.empty(3, device=DEV))
