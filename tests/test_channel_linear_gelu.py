"""GELU of channel products over its whole range, on the GPU: one channel of weight 1, so that z is x."""
import pytest

torch = pytest.importorskip("torch")

import fft_spectral_convolution_amd as fno  # noqa: E402

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _gpu_present():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    fno.lib()


@pytest.mark.parametrize("types", [(F32, F32), (BF16, F32), (BF16, BF16), (F16, F32), (F16, F16)])
def test_gelu(types):
    """3e-7, and 0.1% down to -5.5, 1e-10 below, as include/fno.h says; then the rounding to the result's type."""
    x_type, out_type = types
    sizes = 10.0 ** torch.linspace(-30, 4, 999)
    x = torch.cat([torch.linspace(-40, 40, 1 << 20), torch.linspace(-7, -5, 1 << 18), sizes, -sizes]).to(x_type).to(DEV)
    x = x[torch.isfinite(x)]
    y = fno.fno_channel_linear(x[:, None], torch.ones(1, 1, dtype=x_type, device=DEV), act="gelu", out_dtype=out_type,
                               channels_last=True)[:, 0]
    z = x.double()
    want = z * torch.special.ndtr(z)
    # one rounding to float32 of values above 1 that it is formed in, and of Phi next to it
    own = torch.where(z >= -5.5, torch.minimum(1e-3 * want.abs(), 3e-7 + 2.0 ** -23 * want.abs()), 1e-10)
    half = torch.finfo(out_type).eps / 2
    least = {F32: 2.0 ** -126, BF16: 2.0 ** -126, F16: 2.0 ** -25}[out_type]        # (small ones may be flushed)
    bound = own + half * (want.abs() + own) + least
    bad = ~((y.double() - want).abs() <= bound)
    assert not bool(bad.any()), (x[bad][:5], y[bad][:5], want[bad][:5])
    # of the sign of z
    assert bool((y[z < 0] <= 0).all()) and bool((y[z > 0] >= 0).all())


def test_gelu_far_out():
    """Finite from the largest negative value up, and the value itself far up."""
    for dtype in (F32, BF16, F16):
        x = torch.tensor([-3e38 if dtype != F16 else -6e4, -1e4, 1e4, 3e38 if dtype != F16 else 6e4], dtype=dtype,
                         device=DEV)
        y = fno.fno_channel_linear(x[:, None], torch.ones(1, 1, dtype=dtype, device=DEV), act="gelu",
                                   channels_last=True)[:, 0]
        assert bool((y[:2].abs() <= 1e-28).all()) and torch.equal(y[2:], x[2:])
