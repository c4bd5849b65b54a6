"""fno_grad_norm and fno_clip_grad_norm against float64.

The squares are summed in float64, so the norm is off by its one rounding to
float32 (u = 2^-24); the factor adds one rounding and each product one more
(3 u relative with the norm's), and a 16-bit output half a step of its type.
"""
import math

import pytest

torch = pytest.importorskip("torch")

import fft_spectral_convolution_amd as fno  # noqa: E402

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
HALF_STEP = {torch.float32: U, torch.complex64: U, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -149, torch.complex64: 2.0 ** -149, torch.bfloat16: 2.0 ** -133,
        torch.float16: 2.0 ** -24}
F32, BF16, F16, C64 = torch.float32, torch.bfloat16, torch.float16, torch.complex64


@pytest.fixture(scope="module", autouse=True)
def _gpu_present():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    fno.lib()


def make(shapes, seed=0, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    out = []
    for shape, dtype in shapes:
        if dtype == C64:
            out.append(torch.view_as_complex(torch.randn((*shape, 2), generator=g, device=DEV) * scale))
        else:
            out.append((torch.randn(shape, generator=g, device=DEV) * scale).to(dtype))
    return out


def wide(t):
    return torch.view_as_real(t).double() if t.dtype == C64 else t.double()


def norm_of(grads):
    return math.sqrt(sum(wide(g).square().sum().item() for g in grads))


def check_scaled(got, grads, coef):
    for o, g in zip(got, grads):
        want = wide(g) * coef
        tol = want.abs() * (4 * U + HALF_STEP[g.dtype]) + TINY[g.dtype]
        assert o.dtype == g.dtype and o.shape == g.shape
        assert ((wide(o) - want).abs() <= tol).all()


LISTS = {
    "one value": [((1,), F32)],
    "a scalar": [((), BF16)],
    "odd sizes": [((3,), F32), ((17, 5), BF16), ((4097,), F16), ((2, 3, 5), C64), ((8193,), BF16)],
    "chunk borders": [((4096,), F32), ((4095,), F32), ((4097,), F32), ((8192,), F16), ((8191,), BF16), ((2048,), C64),
                      ((2049,), C64)],
    "empty ones": [((0,), F32), ((5,), F32), ((3, 0), BF16), ((0,), C64), ((7,), C64), ((0,), F16)],
    "one layer": [((2, 8, 8, 4, 4), C64), ((4, 4), F32), ((4,), F32)],
    "more than one table": [((i % 37 + 1,), (F32, BF16, F16, C64)[i % 4]) for i in range(300)],
    "large and small": [((1 << 22,), F32), ((3,), F32), ((1 << 21, 3), BF16), ((64, 64), C64)] * 2,
    "just a table": [((100,), F32)] * 128,
    "one past a table": [((100,), F32)] * 129,
    "middling": [((300, 301), F32), ((77, 300), F16)],
}


@pytest.mark.parametrize("name", LISTS)
@pytest.mark.parametrize("mode", ["in place", "out", "given"])
def test_clip(name, mode):
    grads = make(LISTS[name], 1)
    norm = norm_of(grads)
    limit = 0.37 * norm
    raw = [g.clone() for g in grads]
    got = fno.fno_grad_norm(grads)
    assert got.shape == () and got.dtype == F32
    assert abs(got.item() - norm) <= 2 * U * norm
    if mode == "out":
        outs = [torch.full_like(g, float("nan")) for g in grads]
        n = fno.fno_clip_grad_norm(grads, limit, out=outs)
        assert all(torch.equal(a, b) for a, b in zip(grads, raw))
    elif mode == "given":
        outs = grads
        given = torch.tensor(2.0 * norm, device=DEV)
        n = fno.fno_clip_grad_norm(grads, limit, norm=given)
        assert n is given and n.item() == torch.tensor(2.0 * norm).item()
        norm *= 2.0
    else:
        outs = grads
        n = fno.fno_clip_grad_norm(grads, limit)
    assert abs(n.item() - norm) <= 2 * U * norm
    check_scaled(outs, raw, min(1.0, limit / (norm + 1e-6)))


@pytest.mark.parametrize("name", ["one value", "odd sizes", "more than one table", "middling", "large and small"])
def test_below_the_limit(name):
    """In place nothing changes, not one bit; into other tensors it is a copy."""
    grads = make(LISTS[name], 2)
    raw = [g.clone() for g in grads]
    norm = fno.fno_clip_grad_norm(grads, 1e9)
    assert abs(norm.item() - norm_of(raw)) <= 2 * U * norm_of(raw)
    assert all(torch.equal(a, b) for a, b in zip(grads, raw))
    outs = [torch.zeros_like(g) for g in grads]
    fno.fno_clip_grad_norm(grads, float("inf"), out=outs)
    assert all(torch.equal(a, b) for a, b in zip(outs, raw))


def test_no_tensors_and_empty_tensors():
    assert fno.fno_grad_norm([]).item() == 0.0
    assert fno.fno_clip_grad_norm([], 1.0).item() == 0.0
    empty = [torch.empty((0, 3), device=DEV), torch.empty((0,), dtype=C64, device=DEV)]
    assert fno.fno_grad_norm(empty).item() == 0.0
    assert fno.fno_clip_grad_norm(empty, 1.0).item() == 0.0


def test_zero_gradients_and_zero_limit():
    grads = [torch.zeros(1000, device=DEV)]
    assert fno.fno_clip_grad_norm(grads, 1.0).item() == 0.0
    assert (grads[0] == 0).all()
    grads = make([((1000,), F32), ((99,), BF16)], 3)
    fno.fno_clip_grad_norm(grads, 0.0)
    assert all((g == 0).all() for g in grads)


@pytest.mark.parametrize("scale", [1e-30, 1e25])
@pytest.mark.parametrize("n", [77, 200000])
def test_squares_outside_float32(scale, n):
    """Squares that vanish or overflow in float32."""
    grads = make([((n,), F32), ((n // 7, 3), C64)], 4, scale)
    norm = norm_of(grads)
    got = fno.fno_grad_norm(grads).item()
    assert abs(got - norm) <= 2 * U * norm


@pytest.mark.parametrize("n", [50, 300000])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_non_finite(bad, n):
    """NaN makes all NaN; infinity makes zeros, and NaN where it stands."""
    grads = make([((n,), F32), ((n + 3,), BF16)], 5)
    grads[0][n // 2] = bad
    norm = fno.fno_clip_grad_norm(grads, 1.0)
    if math.isnan(bad):
        assert math.isnan(norm.item())
        assert all(torch.isnan(g).all() for g in grads)
    else:
        assert norm.item() == float("inf")
        assert torch.isnan(grads[0][n // 2]) and torch.isnan(grads[0]).sum() == 1
        grads[0][n // 2] = 0
        assert all((g == 0).all() for g in grads)


def test_slices_of_one_buffer():
    """Neighbours in a packed bucket, at every alignment; nothing else is written."""
    for dtype in (F32, BF16, F16):
        buf = torch.full((60000,), 5.0, dtype=dtype, device=DEV)
        views, at, spans = [], 1, []
        for n in (1, 3, 5000, 8191, 7, 16385, 2, 20001):
            views.append(buf[at:at + n])
            spans.append((at, n))
            at += n + (n % 3)
        keep = torch.ones(60000, dtype=torch.bool, device=DEV)
        for a, n in spans:
            keep[a:a + n] = False
        raw = [v.clone() for v in views]
        norm = norm_of(raw)
        got = fno.fno_clip_grad_norm(views, 1.0)
        assert abs(got.item() - norm) <= 2 * U * norm
        check_scaled(views, raw, 1.0 / (norm + 1e-6))
        assert (buf[keep] == 5.0).all()
        # into a buffer of another alignment
        outs = [torch.empty(v.numel() + 1, dtype=dtype, device=DEV)[1:] for v in views]
        for v, r in zip(views, raw):
            v.copy_(r)
        fno.fno_clip_grad_norm(views, 1.0, out=outs)
        check_scaled(outs, raw, 1.0 / (norm + 1e-6))


def test_some_in_place_some_not():
    grads = make(LISTS["odd sizes"], 6)
    raw = [g.clone() for g in grads]
    outs = [g if i % 2 else torch.empty_like(g) for i, g in enumerate(grads)]
    norm = norm_of(raw)
    fno.fno_clip_grad_norm(grads, 0.5, out=outs)
    check_scaled(outs, raw, 0.5 / (norm + 1e-6))
    for i, (g, r) in enumerate(zip(grads, raw)):
        if i % 2 == 0:
            assert torch.equal(g, r)


def test_same_tensor_twice():
    """Counted twice in the norm; not scaled twice."""
    g = make([((1000,), F32)], 7)[0]
    assert abs(fno.fno_grad_norm([g, g]).item() - math.sqrt(2.0) * norm_of([g])) <= 4 * U * norm_of([g])
    with pytest.raises(fno.FnoError) as e:
        fno.fno_clip_grad_norm([g, g], 1.0)
    assert e.value.status == -4


def test_offsets_past_32_bits():
    g = torch.full(((1 << 32) + 12345,), 0.5, dtype=BF16, device=DEV)
    g[-5:] = 3.0
    n = g.numel()
    want = math.sqrt(0.25 * (n - 5) + 45.0)
    assert abs(fno.fno_clip_grad_norm([g], want / 2).item() - want) <= 2 * U * want
    # the half of both values is exact in the type, up to the 1e-6 of the formula
    assert (g[-5:] == 1.5).all() and (g[:1000] == 0.25).all() and (g[1 << 31:(1 << 31) + 1000] == 0.25).all()


def test_same_bits_again():
    grads = make(LISTS["large and small"], 8)
    first = fno.fno_grad_norm(grads)
    assert all(torch.equal(fno.fno_grad_norm(grads), first) for _ in range(5))


@pytest.mark.parametrize("name", ["one layer", "more than one table", "large and small"])
def test_captured_and_replayed(name):
    """Two graphs captured on one stream, without an eager call before, replayed
    together several times with new gradients."""
    stream = torch.cuda.Stream()
    runs = []
    for k in range(2):
        grads = make(LISTS[name], 10 + k)
        outs = [torch.empty_like(g) for g in grads]
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=stream):
            norm = fno.fno_clip_grad_norm(grads, 1.0, out=outs)
        runs.append((g, grads, outs, norm))
    for rep in range(3):
        wants = []
        for k, (_, grads, _, _) in enumerate(runs):
            for g, n in zip(grads, make(LISTS[name], 20 + 2 * rep + k)):
                g.copy_(n)
            o = [torch.empty_like(g) for g in grads]
            wants.append((o, fno.fno_clip_grad_norm(grads, 1.0, out=o)))
        torch.cuda.synchronize()
        lanes = [torch.cuda.Stream(), torch.cuda.Stream()]
        for lane, (g, _, _, _) in zip(lanes, runs):
            with torch.cuda.stream(lane):
                g.replay()
        torch.cuda.synchronize()
        for (_, _, outs, norm), (o, n) in zip(runs, wants):
            assert torch.equal(norm, n)
            assert all(torch.equal(a, b) for a, b in zip(outs, o))


def test_norm_over_a_gradient_is_refused():
    g = torch.full((), 3.0, device=DEV)
    packed = torch.ones(8, device=DEV)
    for grads, out in (([g], g), ([packed], packed[5]), ([packed[:3], packed[3:]], packed[7])):
        with pytest.raises(fno.FnoError) as e:
            fno.fno_grad_norm(grads, out=out)
        assert e.value.status == -4
    assert fno.fno_grad_norm([packed[:5]], out=packed[5]) is not None
    torch.cuda.synchronize()
    assert g.item() == 3.0 and (packed[:5] == 1).all() and abs(packed[5].item() - 5 ** 0.5) < 4 * U


def test_given_norm_among_the_gradients():
    g = torch.tensor([3.0, 4.0], device=DEV)
    out = torch.empty_like(g)
    assert fno.fno_clip_grad_norm([g], 1.5, norm=g[0], out=[out]).item() == 3.0
    check_scaled([out], [g], 1.5 / (3.0 + 1e-6))


@pytest.mark.parametrize("count", [129, 1000, 3000])
def test_every_kernel_of_a_long_list_is_counted(count):
    tables = (count + 127) // 128
    grads = make([((100,), F32)] * count, 12)
    norm = norm_of(grads)
    raw = [g.clone() for g in grads]
    got = fno.fno_clip_grad_norm(grads, 0.5)
    assert fno.fno_last_kernels() == ["grad_sumsq"] * tables + ["grad_finish"] + ["grad_scale"] * tables
    assert abs(got.item() - norm) <= 2 * U * norm
    check_scaled(grads, raw, 0.5 / (norm + 1e-6))
