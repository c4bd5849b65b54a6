"""Channel products of the largest weights on the GPU."""
import pytest

torch = pytest.importorskip("torch")

import fft_spectral_convolution_amd as fno  # noqa: E402

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _gpu_present():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    fno.lib()


@pytest.mark.parametrize("cin,cout", [(32768, 32768), (32771, 33000)])
def test_more_weights_than_a_grid_has_threads(cin, cout):
    """2^30 weights and more: their gradients' sums are joined 64 a workgroup of 256 threads, and a grid's threads are
    counted in 32 bits.  Whole numbers of two positions: every sum is exact."""
    gen = torch.Generator(device=DEV).manual_seed(3)

    def draw(*shape):
        return torch.randint(-3, 4, shape, generator=gen, device=DEV).to(torch.bfloat16)

    x, g = draw(2, cin), draw(2, cout)
    w = torch.empty(cout, cin, dtype=torch.bfloat16, device=DEV)
    for k in range(0, cout, 4096):
        w[k:k + 4096] = draw(*w[k:k + 4096].shape)
    gx, gw, gb, _ = fno.fno_channel_linear_backward(x, w, g, bias=torch.zeros(cout, device=DEV), channels_last=True)
    assert fno.fno_last_kernels()[-1] == "channels_grad_sum"
    assert torch.equal(gb, g.float().sum(0))
    wx = torch.zeros(2, cin, dtype=torch.float64, device=DEV)
    for k in range(0, cout, 4096):
        gk = g[:, k:k + 4096].double()
        assert torch.equal(gw[k:k + 4096], (gk.t().contiguous() @ x.double()).float()), k
        wx += gk @ w[k:k + 4096].double()
    # sums of up to 2^18: exact in float32, rounded once
    assert torch.equal(gx, wx.to(torch.float32).to(torch.bfloat16))
