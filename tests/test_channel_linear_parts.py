"""What the parts of the channel products' operands leave out, at the values where it is most.

A float32 value is three bfloat16 parts x0 + x1 + x2, each the nearest to what is left; bfloat16 has 8 bits,
so a part leaves up to half a step, 2^-8 of a value in [1, 2), two parts 2^-17, and three none of 24 bits.
 - float32 products leave out x1 w2 + x2 w1 + x2 w2: up to 2 2^-8 2^-17 + 2^-34;
 - grad_x of a bfloat16 field takes g in two parts: up to 2^-17;
 - that of a float16 field takes a weight in two parts as well, without their product: 2^-8 2^-8 more.
"""
import pytest

torch = pytest.importorskip("torch")

import fft_spectral_convolution_amd as fno  # noqa: E402

DEV = "cuda:0"
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
EPS = 2.0 ** -24
# a first part that leaves the most, and a second one as well
TIE, WORST = 1 + 2.0 ** -8, 1 + 2.0 ** -8 - 2.0 ** -17


def parts(v, count):
    """Parts of float32 values, in float64, and what they leave."""
    left, found = v.clone(), []
    for _ in range(count):
        found.append(left.bfloat16().float())
        left = left - found[-1]
    return [f.double() for f in found], left.double()


def test_every_fraction():
    """All 2^23 float32 values of [1, 2)."""
    v = (torch.arange(1 << 23, dtype=torch.int32) | 127 << 23).view(F32)
    for count, bound in ((1, 2.0 ** -8), (2, 2.0 ** -17), (3, 0.0)):
        _, left = parts(v, count)
        assert float(left.abs().max()) == bound
    # float16 has 11 bits: two parts hold it
    half = (torch.arange(1 << 10, dtype=torch.int16) | 15 << 10).view(F16).float()
    assert float(parts(half, 2)[1].abs().max()) == 0.0


def test_products_left_out():
    v = torch.tensor([WORST], dtype=F32)
    (x0, x1, x2), _ = parts(v, 3)
    left = float((x1 * x2 + x2 * x1 + x2 * x2).abs() / v.double() ** 2)
    assert 2.0 ** -24.02 < left <= 2.0 ** -24 + 2.0 ** -34


def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def whole(*values, dtype):
    t = torch.tensor(values, dtype=torch.float64)
    assert torch.equal(t, t.to(dtype).double())
    return t.to(dtype).to(DEV)


@pytest.mark.gpu
@pytest.mark.parametrize("cin,positions", [(1, 5), (1, 9000), (3, 40), (64, 129)])
def test_forward(cin, positions):
    """One sign, every operand at its worst: six products a channel, each addition off by EPS of the sum."""
    need_gpu()
    x = torch.full((positions, cin), WORST, dtype=F32, device=DEV)
    for cout in (1, 70):
        w = torch.full((cout, cin), WORST, dtype=F32, device=DEV)
        out = fno.fno_channel_linear(x, w, channels_last=True).double()
        want = cin * WORST ** 2
        assert float((out - want).abs().max()) <= (6 * cin * EPS + 2.0 ** -24 + 2.0 ** -34) * want
        g = torch.full_like(out, WORST, dtype=F32)
        gx, gw, _, _ = fno.fno_channel_linear_backward(x, w, g, channels_last=True)
        want = cout * WORST ** 2
        assert float((gx.double() - want).abs().max()) <= (6 * cout * EPS + 2.0 ** -24 + 2.0 ** -34) * want
        want = positions * WORST ** 2
        assert float((gw.double() - want).abs().max()) <= (6 * positions * EPS + 2.0 ** -24 + 2.0 ** -34) * want


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,left_out", [(BF16, 2.0 ** -17), (F16, 2.0 ** -17 + 2.0 ** -16)])
@pytest.mark.parametrize("cin", [2, 130])
def test_grad_x_of_16_bit_fields(dtype, left_out, cin):
    """g0 w0 - g1 w1 with most of it cancelled, so that what is left out is larger than the result's rounding."""
    need_gpu()
    w0 = TIE if dtype == F16 else 1.0
    for g0 in (TIE, WORST, 1 - 2.0 ** -9):
        g = whole(g0, 1.0, dtype=F32).expand(300, 2).contiguous()
        w = whole(w0, -1.0, dtype=dtype)[:, None].expand(2, cin).contiguous()
        x = torch.zeros(300, cin, dtype=dtype, device=DEV)
        gx = fno.fno_channel_linear_backward(x, w, g, channels_last=True, need_w=False)[0].double()
        want = g0 * w0 - 1.0
        size = g0 * w0 + 1.0
        bound = (left_out + 6 * EPS) * size
        half = torch.finfo(dtype).eps / 2
        assert float((gx - want).abs().max()) <= bound + half * (abs(want) + bound)
