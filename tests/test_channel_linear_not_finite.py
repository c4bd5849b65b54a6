"""Where infinities and NaN of a field may reach in the gradients of a channel product's weight and bias (GPU):

  grad_weight[o][i] = sum over positions of g[o] x[i],  grad_bias[o] = sum of g[o],

so one of grad_out or of the branch in output channel o reaches row o alone, one of x in input channel i column i
alone, unless it reaches g by way of z.  Everything else has the bits that it has without them.
"""
import itertools

import pytest

torch = pytest.importorskip("torch")

import fft_spectral_convolution_amd as fno  # noqa: E402

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
TYPES = [(F32, F32), (BF16, BF16), (BF16, F32), (F16, F16), (F16, F32)]
LAYOUTS = list(itertools.product((False, True), repeat=2))
# one kernel for up to 64 x 64 channels, 64 x 128 of 16 bits; four for more
SIZES = [(20, 30), (40, 50), (33, 100), (128, 64), (130, 70), (70, 200)]
BAD = (float("nan"), float("inf"), float("-inf"))


@pytest.fixture(scope="module", autouse=True)
def _gpu_present():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    fno.lib()


class Call:
    """The parameters' gradients of fields of B items of P positions, many enough for several tiles a wave or few."""

    def __init__(self, cin, cout, types, last, out_last, act, B=3, P=135):
        gen = torch.Generator(device=DEV).manual_seed(cin)

        def draw(*shape):
            return torch.randn(*shape, generator=gen, device=DEV)

        self.x = draw(B, P, cin).to(types[0])                      # as [B, P, C]; laid out by the call
        self.w = (draw(cout, cin) * cin ** -0.5).to(types[0])
        self.bias = draw(cout)
        self.branch, self.grad_out = draw(B, P, cout).to(types[1]), draw(B, P, cout).to(types[1])
        self.last, self.out_last, self.act = last, out_last, act

    def __call__(self, **more):
        def laid(t, last):
            return t if last else t.transpose(1, 2).contiguous()

        x, branch, g = laid(self.x, self.last), laid(self.branch, self.out_last), laid(self.grad_out, self.out_last)
        return fno.fno_channel_linear_backward(x, self.w, g, bias=self.bias, branch=branch, act=self.act,
                                               channels_last=self.last, out_channels_last=self.out_last, **more)


def check(gw, gb, clean, rows, columns):
    """Nothing finite in the rows and columns given, the clean call's bits elsewhere."""
    touched = torch.zeros(gw.shape, dtype=torch.bool, device=DEV)
    touched[rows] = True
    touched[:, columns] = True
    assert torch.equal(gw[~touched], clean[1][~touched])
    assert not bool(torch.isfinite(gw[touched]).any())
    one = torch.zeros(len(gb), dtype=torch.bool, device=DEV)
    one[rows] = True
    assert torch.equal(gb[~one], clean[2][~one])
    assert not bool(torch.isfinite(gb[one]).any())


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("types", TYPES)
def test_grad_out(size, types):
    for (last, out_last), act in itertools.product(LAYOUTS, ("none", "silu")):
        c = Call(*size, types, last, out_last, act)
        clean = c()
        rows = [1, 17, size[1] - 1]
        for k, (o, v) in enumerate(zip(rows, BAD)):
            c.grad_out[k, 40 * k + 3, o] = v
        _, gw, gb, _ = c()
        check(gw, gb, clean, rows, [])
        # of the parameters alone
        _, gw, gb, _ = c(need_x=False, need_branch=False)
        check(gw, gb, clean, rows, [])


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("types", TYPES)
def test_branch(size, types):
    for last, out_last in LAYOUTS:
        c = Call(*size, types, last, out_last, "gelu")
        clean = c()
        c.branch[1, 77, 11] = c.branch[2, 134, size[1] - 2] = float("nan")
        _, gw, gb, _ = c()
        check(gw, gb, clean, [11, size[1] - 2], [])


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("types", TYPES)
def test_x(size, types):
    """Without an activation z is not part of the gradients."""
    for last, out_last in LAYOUTS:
        c = Call(*size, types, last, out_last, "none")
        clean = c()
        columns = [0, 18, size[0] - 1]
        for k, (i, v) in enumerate(zip(columns, BAD)):
            c.x[k, 134 - 31 * k, i] = v
        _, gw, gb, _ = c()
        check(gw, gb, clean, [], columns)
        c.grad_out[0, 50, 7] = float("nan")
        _, gw, gb, _ = c()
        check(gw, gb, clean, [7], columns)


@pytest.mark.parametrize("size", [(5, 9), (40, 60), (100, 130)])
def test_several_tiles_a_wave(size):
    """In the last of many tiles, and back to finite ones."""
    for types, (last, out_last) in itertools.product([(F32, F32), (BF16, BF16)], LAYOUTS):
        c = Call(*size, types, last, out_last, "none", B=2, P=1 << 17)
        clean = c()
        c.grad_out[1, -1, 2] = c.grad_out[0, 5, 2] = float("nan")
        c.x[1, 70000, 4] = float("inf")
        _, gw, gb, _ = c()
        check(gw, gb, clean, [2], [4])


@pytest.mark.parametrize("size", [(20, 30), (40, 50), (130, 70)])
def test_finite_values_whose_sums_are_not(size):
    """g near float32's largest values, x small: grad_bias passes float32, grad_weight does not."""
    for last, out_last in LAYOUTS:
        c = Call(*size, (F32, F32), last, out_last, "none")
        c.x *= 2.0 ** -40
        c.grad_out.abs_().clamp_(0.5, 1.0).mul_(2.0 ** 127)
        _, gw, gb, _ = c(need_x=False)
        g, x = c.grad_out.double().flatten(0, 1), c.x.double().flatten(0, 1)
        assert bool(torch.isinf(gb).all())
        # six part products of 405 terms, each addition off by up to 2^-24 of the terms' sizes
        bound = (6 * 405 + 4) * 2.0 ** -24 * (g.t().contiguous() @ x.abs())
        assert bool(((gw.double() - g.t().contiguous() @ x).abs() <= bound).all())
