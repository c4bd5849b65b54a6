"""The rounding of 8-bit moments of AdamW before they are coded: one fma in float64 (GPU)."""
from fractions import Fraction

import pytest

torch = pytest.importorskip("torch")

import fft_spectral_convolution_amd as fno  # noqa: E402
from test_adamw import code_values, encode, random_bits  # noqa: E402

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
B1, B2 = 0.9, 0.999


@pytest.fixture(scope="module", autouse=True)
def _gpu_present():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    fno.lib()


def fma(a, b, c):
    """a b + c rounded once: a quotient of whole numbers is rounded correctly."""
    return float(Fraction(a) * Fraction(b) + Fraction(c))


@pytest.mark.parametrize("ratio", [-9, -9 * (1 + 2.0 ** -12), 1])
def test_sums_are_rounded_once(ratio):
    """g = -9 m leaves of beta1 m + (1 - beta1) g only what the products' rounding does: a product rounded by itself
    gives other codes nearly everywhere."""
    n = 128 * 9
    gen = torch.Generator().manual_seed(12)
    held = []
    for signed in (True, False):
        codes = torch.randint(8 * (12 if signed else 27), 8 * (15 if signed else 31), (n,), generator=gen)
        if signed:
            codes |= torch.randint(0, 2, (n,), generator=gen) << 7
        exps = torch.randint(120, 131, (n // 128,), generator=gen)
        data = torch.zeros(-(-(n + n // 128) // 16) * 16, dtype=torch.uint8)
        data[:n], data[n:n + n // 128] = codes.to(torch.uint8), exps.to(torch.uint8)
        held.append(data)
    m, v = code_values(held[0], n, True), code_values(held[1], n, False)
    g = (m * ratio).float()
    ms, vs = [held[0].to(DEV)], [held[1].to(DEV)]
    fno.fno_adamw([torch.zeros(n, device=DEV)], [g.to(DEV)], ms, vs, 3, betas=(B1, B2), seed=21)
    q = g.double()
    r = random_bits(21, 3, 0, n)
    new_m = torch.tensor([fma(B1, a, (1 - B1) * b) for a, b in zip(m.tolist(), q.tolist())], dtype=torch.float64)
    new_v = torch.tensor([fma(B2, a, (1 - B2) * (b * b)) for a, b in zip(v.tolist(), q.tolist())], dtype=torch.float64)
    want = encode(new_m, r & 0xFFFF, True)
    assert torch.equal(ms[0].cpu()[:len(want)], want)
    want_v = encode(new_v, r >> 16, False)
    assert torch.equal(vs[0].cpu()[:len(want_v)], want_v)
    if ratio == -9:
        apart = encode(B1 * m + (1 - B1) * q, r & 0xFFFF, True)
        assert int((apart[:n] != want[:n]).sum()) > n // 2
