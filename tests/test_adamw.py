"""AdamW over many tensors on the GPU, against the formulas in float64.

Moments of 32 bits, parameters and copies are roundings of float32 sums: the
bounds count half steps.  Codes of 8-bit moments are integers and compared as
such: the oracle forms the new moment in float64 and codes it from the words of
its bits, the random bits from the documented hash.
"""
import math

import pytest

torch = pytest.importorskip("torch")

import fft_spectral_convolution_amd as fno  # noqa: E402

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F32, BF16, F16, C64 = torch.float32, torch.bfloat16, torch.float16, torch.complex64
HALF_STEP = {F32: 2.0 ** -24, BF16: 2.0 ** -8, F16: 2.0 ** -11}


@pytest.fixture(scope="module", autouse=True)
def _gpu_present():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    fno.lib()


def rand(shape, dtype, gen, scale=1.0):
    if dtype == C64:
        return torch.view_as_complex(torch.randn(*shape, 2, generator=gen) * scale).to(DEV)
    return (torch.randn(*shape, generator=gen) * scale).to(dtype).to(DEV)


def wide(t):
    """float64 values on the CPU, complex ones as pairs."""
    t = torch.view_as_real(t) if t.is_complex() else t
    return t.double().cpu().reshape(-1)


def mix(x):
    x &= 0xFFFFFFFF
    x = ((x ^ (x >> 16)) * 0x6A09E667) & 0xFFFFFFFF
    x = ((x ^ (x >> 15)) * 0xBB67AE85) & 0xFFFFFFFF
    return x ^ (x >> 16)


def random_bits(seed, step, tensor, n):
    k = mix(mix(mix(mix(seed & 0xFFFFFFFF) + (seed >> 32)) + step) + tensor)
    i = torch.arange(n)
    return mix((i & 0xFFFFFFFF) ^ mix(torch.tensor(k) + (i >> 32)))


def code_values(held, n, signed):
    """float64 values of an 8-bit moment's bytes (no NaN codes)."""
    held = held.cpu().long()
    whole = -(-n // 128) * 128
    c, e = held[:whole], held[whole:whole + whole // 128].repeat_interleave(128) - 127
    u, top = (c & 127, 14) if signed else (c, 30)
    v = torch.ldexp(1.0 + (u & 7).double() / 8, ((u >> 3) - top + e).double())
    v = torch.where(u == 0, 0.0, v)
    return (torch.where(c >= 128, -v, v) if signed else v)[:n]


def encode(values, r, signed):
    """Bytes of an 8-bit moment of float64 values with the random halves r, by Python's own frexp."""
    n = len(values)
    blocks = -(-n // 128)
    top, least = (14, -126) if signed else (30, -96)
    codes, exps = [0] * (128 * blocks), [0] * blocks
    for b in range(blocks):
        part = values[128 * b:128 * b + 128].tolist()
        big = max(map(abs, part))
        if big == 0.0:
            continue
        e = min(127, max(least, math.frexp(big)[1] - 1))
        exps[b] = e + 127
        for j, v in enumerate(part):
            if v == 0.0:
                continue
            f, x = math.frexp(abs(v))
            x -= 1 + e                                   # the value is (1 + fraction) 2^(x + e)
            fraction = int((2 * f - 1) * 2 ** 20)
            c = (x + top) * 8 + (fraction >> 17)
            c += (fraction & 0x1FFFF) + 2 * int(r[128 * b + j]) + 1 >= 1 << 17
            c = max(0 if signed else 1, min(c, 8 * (top + 1) - (e == 127)))      # 2^128 is no float32
            codes[128 * b + j] = c | (128 if signed and c and v < 0 else 0)
    return torch.tensor(codes + exps, dtype=torch.uint8)


class Reference:
    """The formulas in float64, over one tensor."""

    def __init__(self, step, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=1e-2):
        self.step, self.lr, self.betas, self.eps, self.wd = step, lr, betas, eps, weight_decay

    def __call__(self, p, g, m, v):
        b1, b2 = self.betas
        m = b1 * m + (1 - b1) * g
        v = b2 * v + (1 - b2) * g * g
        u = m / (1 - b1 ** self.step) / ((v / (1 - b2 ** self.step)).sqrt() + self.eps)
        return p - self.lr * (self.wd * p + u), m, v, self.lr * u.abs()


def check_params(got, want, old, update, dtype):
    # p' is a product, a quotient of a few float32 operations (16 half steps of the update
    # cover them) and one rounding to the stored type; p (1 - lr wd) one more of float32
    bound = 16 * 2.0 ** -24 * update + 2 * 2.0 ** -24 * old.abs() + HALF_STEP[dtype] * want.abs() * 1.01 + 1e-30
    if dtype == F16:
        bound = bound + 2.0 ** -25            # half of the least step
    assert ((got - want).abs() <= bound).all(), ((got - want).abs() / bound).max()


SHAPES = [((3, 5), F32), ((1,), F32), ((0,), F32), ((4097,), BF16), ((129,), F16), ((2, 3, 4, 5), C64), ((8191,), F32),
          ((127,), BF16), ((64, 64), F32)]


def make(shapes, bits, seed, grad_types=None, scale=1.0):
    gen = torch.Generator().manual_seed(seed)
    params = [rand(s, d, gen, 0.1) for s, d in shapes]
    grads = [rand(s, d if grad_types is None or d == C64 else grad_types[i % len(grad_types)], gen, scale)
             for i, (s, d) in enumerate(shapes)]
    ms, vs = fno.fno_adamw_states(params, bits)
    return params, grads, ms, vs


@pytest.mark.parametrize("out_of_place", [False, True])
@pytest.mark.parametrize("grad_types", [None, [F32, BF16, F16]])
def test_steps_in_32_bits(out_of_place, grad_types):
    params, grads, ms, vs = make(SHAPES, 32, 1, grad_types)
    for step in (1, 2, 3):
        ref = Reference(step, lr=0.01)
        want = [ref(wide(p), wide(g), wide(m), wide(v)) for p, g, m, v in zip(params, grads, ms, vs)]
        old = [wide(p) for p in params]
        kept = [t.clone() for t in (*params, *ms, *vs)]
        out = tuple([torch.full_like(t, 7) for t in ts] for ts in (params, ms, vs)) if out_of_place else None
        fno.fno_adamw(params, grads, ms, vs, step, lr=0.01, out=out)
        if out_of_place:
            assert all(torch.equal(a, b) for a, b in zip(kept, (*params, *ms, *vs)))
            params, ms, vs = out
        for (s, d), p, m, v, o, (wp, wm, wv, u) in zip(SHAPES, params, ms, vs, old, want):
            check_params(wide(p), wp, o, u, F32 if d == C64 else d)
            # two products and a sum (three half steps) of factors that are rounded themselves (two)
            size_m = 0.9 * wm.abs() + wm.abs() + 1.0
            assert ((wide(m) - wm).abs() <= 5 * 2.0 ** -24 * size_m).all()
            assert ((wide(v) - wv).abs() <= 6 * 2.0 ** -24 * (wv + 1e-30)).all()


@pytest.mark.parametrize("scale", [1.0, 1e-6, 3e4])
def test_codes_in_8_bits(scale):
    shapes = [(s, d if scale < 2e4 or d != F16 else F32) for s, d in SHAPES]
    params, grads, ms, vs = make(shapes, 8, 2, scale=scale)
    seed = 0xABCDEF0123456789
    for step in (1, 2, 7):
        ref = Reference(step)
        sizes = [g.numel() * (2 if g.is_complex() else 1) for g in grads]
        want = [ref(wide(p), wide(g), code_values(m, n, True), code_values(v, n, False))
                for p, g, m, v, n in zip(params, grads, ms, vs, sizes)]
        old = [wide(p) for p in params]
        fno.fno_adamw(params, grads, ms, vs, step, seed=seed)
        for i, (n, (wp, wm, wv, u)) in enumerate(zip(sizes, want)):
            r = random_bits(seed, step, i, n)
            for held, w, half, signed in ((ms[i], wm, r & 0xFFFF, True), (vs[i], wv, r >> 16, False)):
                code = encode(w, half, signed)
                assert torch.equal(held.cpu()[:len(code)], code), (i, step, signed)
            d = shapes[i][1]
            check_params(wide(params[i]), wp, old[i], u, F32 if d == C64 else d)
        read = fno.fno_adamw_moments(ms, vs, numels=sizes)
        for held, got, signed in ((ms, read[0], True), (vs, read[1], False)):
            for h, q, n in zip(held, got, sizes):
                assert torch.equal(q.double().cpu(), code_values(h, n, signed))


def test_rounding_is_by_chance():
    """A moment that stands still between two codes is coded as either, in proportion; seeds and steps differ."""
    n = 1 << 16
    g = torch.full((n,), 1.0 + 3 / 32, device=DEV)         # a quarter of the way between codes 1 and 1 1/8 ... 3/4
    p = torch.zeros(n, device=DEV)
    seen = []
    for seed, step in ((1, 1), (2, 1), (1, 2)):
        ms, vs = fno.fno_adamw_states([p], 8)
        fno.fno_adamw([p.clone()], [g], ms, vs, step, betas=(0.0, 0.0), seed=seed)
        m = code_values(ms[0], n, True)
        assert set(m.tolist()) == {1.0, 1.125}
        up = (m == 1.125).double().mean().item()
        assert abs(up - 0.75) < 5 * math.sqrt(0.75 * 0.25 / n)
        seen.append(m)
    for a, b in ((0, 1), (0, 2), (1, 2)):
        both = ((seen[a] == 1.125) & (seen[b] == 1.125)).double().mean().item()
        assert abs(both - 0.75 ** 2) < 5 * math.sqrt(0.25 / n)


def test_second_moment_decays_in_8_bits():
    """Rounding to nearest would leave a moment that shrinks by 0.1% a step where it is for ever."""
    n = 1 << 14
    p, ms, vs = [torch.zeros(n, device=DEV)], *fno.fno_adamw_states([torch.zeros(n, device=DEV)], 8)
    g = torch.ones(n, device=DEV)
    g[::128] = 16.0                                        # holds the block's power of two
    fno.fno_adamw(p, [g], ms, vs, 1, betas=(0.9, 0.0))     # v = g^2
    small = torch.zeros(n, device=DEV)
    small[::128] = 16.0
    steps = 400
    for t in range(steps):
        fno.fno_adamw(p, [small], ms, vs, 2 + t, seed=5)
    v = code_values(vs[0], n, False).view(-1, 128)[:, 1:]
    want = 0.999 ** steps                                  # 0.67
    # a step moves v by 0.1% on average, in jumps of at most an eighth of it: its variance is at most 0.001 / 8
    spread = math.sqrt(steps * 0.001 * 0.125)
    assert abs(v.mean().item() - want) < 6 * spread / math.sqrt(v.numel()) + 1e-3


def test_clipping_and_copies():
    shapes = [((65, 33), F32), ((17,), F32), ((3, 4), C64), ((300,), BF16)]
    for bits in (32, 8):
        params, grads, ms, vs = make(shapes, bits, 3)
        twin = [p.clone() for p in params]
        tm, tv = [m.clone() for m in ms], [v.clone() for v in vs]
        copies = [torch.zeros_like(params[0], dtype=BF16), torch.zeros_like(params[1], dtype=F16), None, None]
        norm = fno.fno_grad_norm(grads)
        fno.fno_adamw(params, grads, ms, vs, 1, norm=norm, max_norm=0.5, copies=copies, seed=9)
        # float32 gradients: the same as clipping them first
        clipped = [g.clone() for g in grads]
        fno.fno_clip_grad_norm(clipped[:3], 0.5, norm=norm)
        fno.fno_adamw(twin[:3], clipped[:3], tm[:3], tv[:3], 1, seed=9)
        for a, b in zip((*params[:3], *ms[:3], *vs[:3]), (*twin[:3], *tm[:3], *tv[:3])):
            assert torch.equal(a, b)
        assert torch.equal(copies[0], params[0].to(BF16)) and torch.equal(copies[1], params[1].to(F16))
        # a norm below the limit changes nothing
        p2, g2, m2, v2 = make(shapes, bits, 4)
        p3, g3, m3, v3 = make(shapes, bits, 4)
        fno.fno_adamw(p2, g2, m2, v2, 1, norm=norm, max_norm=1e9, seed=1)
        fno.fno_adamw(p3, g3, m3, v3, 1, seed=1)
        assert all(torch.equal(a, b) for a, b in zip((*p2, *m2, *v2), (*p3, *m3, *v3)))


def test_many_tensors_and_packed_slices():
    """More tensors than a table, slices of packed buffers at any offset, moments of both kinds in one call."""
    sizes = [(37 * i) % 300 + 1 for i in range(130)]
    gen = torch.Generator().manual_seed(6)
    flat_p, flat_g = rand((sum(sizes),), F32, gen), rand((sum(sizes),), BF16, gen)
    params, grads = list(flat_p.split(sizes)), list(flat_g.split(sizes))
    m32, v32 = fno.fno_adamw_states(params, 32)
    m8, v8 = fno.fno_adamw_states(params, 8)
    ms = [a if i % 3 else b for i, (a, b) in enumerate(zip(m32, m8))]
    vs = [a if i % 3 else b for i, (a, b) in enumerate(zip(v32, v8))]
    before = wide(flat_p)
    fno.fno_adamw(params, grads, ms, vs, 1, seed=3)
    wp, wm, wv, u = Reference(1)(before, wide(flat_g), torch.zeros_like(before), torch.zeros_like(before))
    check_params(wide(flat_p), wp, before, u, F32)
    at = 0
    for i, n in enumerate(sizes):
        if i % 3 == 0:
            code = encode(wm[at:at + n], random_bits(3, 1, i, n) & 0xFFFF, True)
            assert torch.equal(ms[i].cpu()[:len(code)], code), i
        at += n
    assert len(fno.fno_last_kernels()) == 3


@pytest.mark.parametrize("bits", [32, 8])
def test_step_and_rate_in_memory_and_graph(bits):
    """A captured step with its number and rate on the device: every replay as the eager call."""
    shapes = [((100, 7), F32), ((5,), C64)]
    params, grads, ms, vs = make(shapes, bits, 7)
    eager = [[t.clone() for t in ts] for ts in (params, ms, vs)]
    step = torch.zeros((), dtype=torch.int64, device=DEV)
    lr = torch.zeros((), device=DEV)
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        with torch.cuda.graph(graph, stream=stream):
            step += 1
            fno.fno_adamw(params, grads, ms, vs, step, lr=lr, seed=11)
    for t in range(1, 5):
        rate = 0.01 / t
        lr.fill_(rate)
        for g in grads:
            g.mul_(0.9)
        graph.replay()
        torch.cuda.synchronize()
        fno.fno_adamw(eager[0], grads, eager[1], eager[2], t, lr=torch.tensor(rate, dtype=F32).item(), seed=11)
        for a, b in zip((*params, *ms, *vs), (*eager[0], *eager[1], *eager[2])):
            if bits == 8 and a.dtype == torch.uint8:
                assert torch.equal(a, b)
            else:        # 1 - b^t by another exponential: last bits of the rate
                torch.testing.assert_close(a, b, rtol=4e-7, atol=1e-9)
        # the next step starts from the same values
        for a, b in zip((*params, *ms, *vs), (*eager[0], *eager[1], *eager[2])):
            b.copy_(a)


def test_not_finite_and_zero():
    n = 300
    for bits in (32, 8):
        p = [torch.ones(n, device=DEV)]
        g = [torch.ones(n, device=DEV)]
        g[0][3], g[0][200], g[0][5] = float("nan"), float("inf"), 0.0
        ms, vs = fno.fno_adamw_states(p, bits)
        fno.fno_adamw(p, g, ms, vs, 1)
        m, v = (ms, vs) if bits == 32 else fno.fno_adamw_moments(ms, vs, numels=[n])
        bad = torch.zeros(n, dtype=torch.bool, device=DEV)
        bad[3] = bad[200] = True
        ok = ~bad
        assert torch.isfinite(p[0][ok]).all() and torch.isfinite(m[0][ok]).all() and torch.isfinite(v[0][ok]).all()
        assert torch.isnan(p[0][bad]).all()
        assert not torch.isfinite(m[0][bad]).any() and not torch.isfinite(v[0][bad]).any()
        assert p[0][5] == 1.0 - 1e-3 * 1e-2 and m[0][5] == 0 and v[0][5] == 0
        # ones have a code of their own
        if bits == 8:
            fno.fno_adamw([torch.ones(n, device=DEV)], [torch.zeros(n, device=DEV)], ms, vs, 2)
            m, v = fno.fno_adamw_moments(ms, vs, numels=[n])
            assert torch.isnan(m[0][bad]).all() and torch.isnan(v[0][bad]).all() and torch.isfinite(m[0][ok]).all()


def test_tiny_and_huge_values_in_8_bits():
    """Blocks below and above the range of the exponent byte, and a block of both."""
    g = torch.zeros(512, device=DEV)
    g[:128] = 1e-30                    # squares below 2^-96
    g[128:256] = 1e25                  # squares beyond float32
    g[256] = 1e10
    g[257:384] = 1e-10                 # far below the block's largest
    ms, vs = fno.fno_adamw_states([g], 8)
    p = torch.zeros(512, device=DEV)
    fno.fno_adamw([p], [g], ms, vs, 1, betas=(0.0, 0.0))
    wide_g = wide(g)
    r = random_bits(0, 1, 0, 512)
    assert torch.equal(ms[0].cpu()[:516], encode(wide_g, r & 0xFFFF, True))
    assert torch.equal(vs[0].cpu()[:516], encode(wide_g * wide_g, r >> 16, False))
    m, v = fno.fno_adamw_moments(ms, vs, numels=[512])
    assert bool(torch.isfinite(m[0]).all()) and bool(torch.isfinite(v[0]).all())
    assert bool((v[0][:384] > 0).all()) and bool((v[0][384:] == 0).all())


def test_tensor_beyond_32_bits():
    """A tensor of more than 2^32 values: its last blocks' codes, whose numbers take more than 32 bits."""
    n = (1 << 32) + 5000
    p, g = torch.zeros(n, dtype=BF16, device=DEV), torch.zeros(n, dtype=BF16, device=DEV)
    tail = 5000 + 128
    g[-tail:] = torch.randn(tail, generator=torch.Generator().manual_seed(8)).to(BF16).to(DEV)
    ms, vs = fno.fno_adamw_states([p], 8)
    fno.fno_adamw([p], [g], ms, vs, 1, seed=77)
    first = n - tail                                   # a whole number of blocks
    assert first % 128 == 0
    wide_g = wide(g[-tail:])
    k = mix(mix(mix(mix(77)) + 1))
    i = torch.arange(first, n)
    r = mix((i & 0xFFFFFFFF) ^ mix(torch.tensor(k) + (i >> 32)))
    codes = -(-tail // 128) * 128
    blocks = codes // 128
    whole = -(-n // 128) * 128
    for held, w, half, signed in ((ms[0], (1 - 0.9) * wide_g, r & 0xFFFF, True),
                                  (vs[0], (1 - 0.999) * wide_g * wide_g, r >> 16, False)):
        want = encode(w, half, signed)
        assert torch.equal(held[first:first + codes].cpu(), want[:codes])
        exps = whole + first // 128
        assert torch.equal(held[exps:exps + blocks].cpu(), want[codes:])
        assert int(held[:first].max()) == 0
    assert float(p[:first].abs().max()) == 0 and bool((p[-tail:] != 0).any())


def test_refusals():
    p, g, m, v = make([((4, 4), F32), ((8,), C64)], 32, 1)
    m8, v8 = fno.fno_adamw_states(p, 8)
    with pytest.raises(ValueError):
        fno.fno_adamw(p, g[:1], m, v, 1)
    with pytest.raises(ValueError):
        fno.fno_adamw(p, g, m, v, 0)
    with pytest.raises(TypeError):
        fno.fno_adamw(p, g, m, v8, 1)
    with pytest.raises(ValueError):
        fno.fno_adamw(p, g, [m[0][:2], m[1]], v, 1)
    with pytest.raises(TypeError):
        fno.fno_adamw(p, [g[0], torch.view_as_real(g[1])[:, 0].contiguous()], m, v, 1)
    with pytest.raises(TypeError):
        fno.fno_adamw(p, g, [t.to(F16) for t in m], v, 1)
    with pytest.raises(ValueError):
        fno.fno_adamw(p, g, m, v, 1, norm=fno.fno_grad_norm(g))
    with pytest.raises(TypeError):
        fno.fno_adamw(p, g, m, v, 1, copies=[None, torch.zeros(8, dtype=BF16, device=DEV)])
    with pytest.raises(TypeError):
        fno.fno_adamw(p, g, m, v, torch.ones((), device=DEV))
    with pytest.raises(ValueError):
        fno.fno_adamw([p[0].t()[:, :3], p[1]], g, m, v, 1)
    with pytest.raises(fno.FnoError) as e:                    # the same tensor twice
        fno.fno_adamw([p[0], p[0]], [g[0], g[0]], [m[0], m[0]], [v[0], v[0]], 1)
    assert e.value.status == -4
    with pytest.raises(fno.FnoError) as e:
        fno.fno_adamw([p[0]], [p[0]], [m[0]], [v[0]], 1)       # its own gradient, overwritten
    assert e.value.status == -4
    for bad in ({"betas": (1.0, 0.999)}, {"betas": (0.9, -0.1)}, {"eps": -1.0}, {"lr": float("nan")},
                {"weight_decay": float("inf")}):
        with pytest.raises(fno.FnoError) as e:
            fno.fno_adamw(p, g, m, v, 1, **bad)
        assert e.value.status == -12
    fno.fno_adamw([], [], [], [], 1)
