"""Every form of the channel product's kernels against float64 on the GPU: 32, 64 or 128 output channels a wave;
four waves with the whole weight in LDS, eight (`wide`), or the weight a chunk at a time (`staged`); more tiles
than the device holds waves.  The names of a call's kernels carry the form that ran, so each test says which
one it is for.

Bounds count rounding steps.  One rounding of a value v to 32 bits is off by at most 2^-24 |v|.  A sum of K
products is formed by N K additions, N the number of part products, each off by at most 2^-24 S with S the sum
of the products' sizes; what the parts leave out is `omitted` S (see part_errors).
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
LEAST = {F32: 2.0 ** -149, BF16: 2.0 ** -133, F16: 2.0 ** -24}           # steps of the smallest values
TYPES = [(F32, F32), (BF16, BF16), (BF16, F32), (F16, F16), (F16, F32)]
LAYOUTS = list(itertools.product((False, True), repeat=2))


@pytest.fixture(scope="module", autouse=True)
def _gpu_present():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    fno.lib()


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


def points(t, last):
    """[B P, C] in float64."""
    t = t.double()
    C = t.shape[-1] if last else t.shape[1]
    return (t if last else t.movedim(1, -1)).reshape(-1, C).contiguous()


def parts(x_type, out_type=F32):
    """(part products of a product of x's type, what they leave out of it).

    bfloat16 keeps 8 bits: a rounding leaves up to 2^-8 of a value, two of them up to 2^-17, three none of
    float32's 24.  float32 x float32: six products, without x1 w2 + x2 w1 + x2 w2, up to 2 2^-25 + 2^-34.  g of
    two parts x a float16 weight of two: up to 2^-17 of g and, x1 w1, 2^-16; x a bfloat16 weight 2^-17."""
    if x_type == F32 and out_type == F16:
        return 3, 2.0 ** -17 + 2.0 ** -16
    if x_type == F32 and out_type == BF16:
        return 2, 2.0 ** -17
    return (6, 2.0 ** -24 + 2.0 ** -34) if x_type == F32 else (4, 0.0)


class Case:
    def __init__(self, B, cin, cout, P, types=(F32, F32), last=False, out_last=False, act="none", branch="none",
                 bias=True, seed=0, whole=False):
        gen = torch.Generator(device=DEV).manual_seed(seed)

        def draw(*shape):
            if whole:
                return torch.randint(-3, 4, shape, generator=gen, device=DEV).float()
            return torch.randn(*shape, generator=gen, device=DEV)

        def field(C, is_last):
            return draw(*((B, P, C) if is_last else (B, C, P)))

        x_type, out_type = self.types = types
        self.last, self.out_last, self.act, self.branch_at = last, out_last, act, branch
        self.x = field(cin, last).to(x_type)
        self.w = (draw(cout, cin) if whole else draw(cout, cin) * cin ** -0.5).to(x_type)
        self.bias = draw(cout) if bias else None
        self.branch = field(cout, out_last).to(out_type) if branch != "none" else None
        self.grad_out = field(cout, out_last).to(out_type)
        self.X, self.W = points(self.x, last), self.w.double()
        self.z = self.X @ self.W.t().contiguous()
        size = self.X.abs() @ self.W.t().abs().contiguous()
        for t in (self.bias.double() if bias else 0, points(self.branch, out_last) if branch == "before" else 0):
            self.z, size = self.z + t, size + abs(t)
        products, omitted = parts(x_type)
        self.z_bound = ((products * cin + 2) * EPS + omitted) * size

    def options(self):
        return dict(bias=self.bias, branch=self.branch, branch_after=self.branch_at == "after", act=self.act,
                    channels_last=self.last, out_channels_last=self.out_last)

    def forward(self):
        out = fno.fno_channel_linear(self.x, self.w, out_dtype=self.types[1], **self.options())
        return out, fno.fno_last_kernels()

    def backward(self, **more):
        grads = fno.fno_channel_linear_backward(self.x, self.w, self.grad_out, **self.options(), **more)
        return grads, fno.fno_last_kernels()

    def check_forward(self, out):
        # an activation passes on at most 1.13 of z's error and adds 3e-7 (GELU) or a few steps (SiLU) of its own
        want, bound = act_of(self.z, self.act), 1.13 * self.z_bound
        if self.act != "none":
            bound = bound + 8 * EPS * (1 + self.z.abs())
        if self.branch_at == "after":
            r = points(self.branch, self.out_last)
            want, bound = want + r, bound + EPS * (want + r).abs()
        close(points(out, self.out_last), want, bound, self.types[1], "out")

    def check_backward(self, grads):
        gx, gw, gb, gr = grads
        go = points(self.grad_out, self.out_last)
        g = go * slope_of(self.z, self.act)
        # slopes differ by at most 0.8 of what z does; their own error is a few steps and 1.5e-7 of erf
        g_bound = go.abs() * (0.8 * self.z_bound + 12 * EPS) if self.act != "none" else torch.zeros_like(g)
        n, cout = g.shape
        T, W, X = self.types[0], self.W, self.X
        products, omitted = parts(F32, T) if T != F32 else parts(F32)
        close(points(gx, self.last), g @ W,
              g_bound @ W.abs() + ((products * cout + 2) * EPS + omitted) * (g.abs() @ W.abs()), T, "grad_x")
        # six products; what is left out of them as for float32 (x of 16 bits has fewer parts)
        gt = g.t().contiguous()
        close(gw.double(), gt @ X, g_bound.t().contiguous() @ X.abs()
              + ((6 * n + 2) * EPS + 2.0 ** -23) * (gt.abs() @ X.abs()), F32, "grad_weight")
        if self.bias is not None:
            close(gb.double(), g.sum(0), g_bound.sum(0) + (3 * n + 2) * EPS * g.abs().sum(0), F32, "grad_bias")
        if self.branch_at == "before" and self.act != "none":
            close(points(gr, self.out_last), g, g_bound, self.types[1], "grad_branch")


def close(got, want, bound, dtype, what):
    """Within the bound, and a rounding to dtype."""
    bound = bound + HALF_STEP[dtype] * (want.abs() + bound) + LEAST[dtype] / 2
    bad = ~((got - want).abs() <= bound)
    worst = float(((got - want).abs() / bound).max())
    assert not bool(bad.any()), (what, int(bad.sum()), bad.numel(), worst, bad.nonzero()[:4].tolist())


# (B, Cin, Cout, P), and the form of a float32 and of a 16-bit product of Cin channels to Cout.
FORWARD = [
    ((8, 40, 100, 4099), "128", "128"),
    ((3, 130, 300, 3700), "128_wide", "128"),
    ((5, 260, 200, 3333), "128_staged", "128_wide"),
    ((1, 500, 129, 17000), "128_staged", "128_staged"),
    ((4, 40, 50, 8200), "64", "64"),
    ((7, 180, 63, 4700), "64_wide", "64"),
    ((9, 500, 33, 3700), "64_staged", "64_wide"),
    ((1, 970, 60, 33000), "64_staged", "64_staged"),
    ((2, 330, 30, 500), "32_wide", "32"),
    ((3, 970, 70, 40), "32_staged", "32_wide"),
    ((1, 1930, 20, 333), "32_staged", "32_staged"),
]


@pytest.mark.parametrize("size,f32,half", FORWARD)
@pytest.mark.parametrize("types", TYPES)
def test_forward(size, f32, half, types):
    want = ["channels_" + (f32 if types[0] == F32 else half)]
    for k, (last, out_last) in enumerate(LAYOUTS):
        c = Case(*size, types=types, last=last, out_last=out_last, branch="before", whole=True, seed=k)
        out, names = c.forward()
        assert names == want
        # exact in float32, so rounded once
        assert torch.equal(points(out, out_last), c.z.float().to(types[1]).double())
        c = Case(*size, types=types, last=last, out_last=out_last, act=("gelu", "silu")[k % 2],
                 branch=("before", "after", "none", "before")[k], bias=k != 1, seed=k)
        out, names = c.forward()
        assert names == want
        c.check_forward(out)


# The four kernels of a backward pass: the form that forms g (Cin to Cout, by x's type), and that of
# grad_x (g's Cout channels to Cin): float32 with float32, bfloat16 and float16 weights, of one, two or three parts.
BACKWARD = [
    ((8, 100, 140, 4099), ("128_wide", "128", "128"), ("128_wide", "128", "128_wide")),
    ((3, 300, 300, 3700), ("128_staged", "128_wide", "128_wide"), ("128_staged", "128_wide", "128_staged")),
    ((1, 500, 490, 8400), ("128_staged",) * 3, ("128_staged",) * 3),
    ((9, 60, 330, 3700), ("128", "128", "128"), ("64_staged", "64", "64_wide")),
    ((9, 500, 40, 3700), ("64_staged", "64_wide", "64_wide"), ("128", "128", "128")),
    ((2, 33, 970, 400), ("32",) * 3, ("32_staged", "32_wide", "32_staged")),
]


@pytest.mark.parametrize("size,slope,grad_x", BACKWARD)
@pytest.mark.parametrize("types", TYPES)
def test_backward(size, slope, grad_x, types):
    k_type = (F32, BF16, F16).index(types[0])
    tail = ["channels_grad_w", "channels_grad_sum"]
    own = ["channels_slope_" + slope[k_type], "channels_grad_x_" + grad_x[k_type], *tail]
    for k, (last, out_last) in enumerate(LAYOUTS):
        c = Case(*size, types=types, last=last, out_last=out_last, whole=True, seed=k)
        (gx, gw, gb, _), names = c.backward()
        # without an activation grad_out is g: a product of grad_out's type
        assert len(names) == 3 and names[0].startswith("channels_grad_x_") and names[1:] == tail
        if types[1] == F32:
            assert names[0] == own[1]
        g = points(c.grad_out, out_last)
        assert torch.equal(points(gx, last), (g @ c.W).float().to(types[0]).double())
        assert torch.equal(gw.double(), g.t().contiguous() @ c.X) and torch.equal(gb.double(), g.sum(0))
        c = Case(*size, types=types, last=last, out_last=out_last, act=("silu", "gelu")[k % 2],
                 branch=("before", "none", "after", "before")[k], bias=k != 2, seed=k)
        grads, names = c.backward()
        assert names == own
        c.check_backward(grads)


# More than the 8192 waves that 256 CUs can hold at all, of 64 positions each: every wave of a launch goes through
# several tiles.
@pytest.mark.parametrize("cin,cout", [(5, 9), (20, 40), (9, 70), (70, 12), (200, 130)])
@pytest.mark.parametrize("types", [(F32, F32), (BF16, BF16), (F16, F32)])
def test_several_tiles_a_wave(cin, cout, types):
    B, P = 13, (1 << 17) // 3
    assert B * P > 64 * 8192
    for k, (last, out_last) in enumerate(LAYOUTS):
        c = Case(B, cin, cout, P, types=types, last=last, out_last=out_last, branch="before", whole=True, seed=k)
        out, _ = c.forward()
        assert torch.equal(points(out, out_last), c.z.float().to(types[1]).double())
        del out
        (gx, gw, gb, _), names = c.backward()
        assert names[0] == "channels_bwd" if max(cin, cout) <= 64 else names[-1] == "channels_grad_sum"
        g = points(c.grad_out, out_last)
        assert torch.equal(points(gx, last), (g @ c.W).float().to(types[0]).double())
        # whole numbers below 2^24, so exact
        assert torch.equal(gw.double(), g.t().contiguous() @ c.X) and torch.equal(gb.double(), g.sum(0))
        del gx, gw, gb, g, c
    c = Case(B, cin, cout, P, types=types, last=True, out_last=False, act="gelu", branch="before", seed=9)
    c.check_forward(c.forward()[0])
    c.check_backward(c.backward()[0])


# Parts of few positions or channels that do not exist beside several 128-channel parts that do.
@pytest.mark.parametrize("types", TYPES)
def test_staged_with_ragged_ends(types):
    for k, (last, out_last) in enumerate(LAYOUTS):
        c = Case(600, 497, 131, 37, types=types, last=last, out_last=out_last, act="silu", branch="after", seed=k)
        out, names = c.forward()
        assert names == ["channels_128_staged"]
        c.check_forward(out)
        grads, names = c.backward()
        assert names[0] == "channels_slope_128_staged"
        c.check_backward(grads)
