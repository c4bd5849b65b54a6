"""A training step of a small model as the calls are used together: lifting,
two layers (spectral product joined to the channel product, norm), projection;
the backward pass; the norm of all gradients; AdamW with the clipping in it and
16-bit copies.  Against the same model in float64 with torch's FFT and automatic
differentiation.
"""
import pytest

torch = pytest.importorskip("torch")

import fft_spectral_convolution_amd as fno  # noqa: E402

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
B, H, W, C, M = 2, 16, 32, 12, 4


@pytest.fixture(scope="module", autouse=True)
def _gpu_present():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    fno.lib()


def make_params(gen):
    def r(*shape, scale=1.0):
        return torch.randn(*shape, generator=gen) * scale

    p = {"lift_w": r(C, 3, scale=0.6), "lift_b": r(C, scale=0.1)}
    for k in range(2):
        p[f"spec{k}"] = torch.view_as_complex(r(2, M, M, C, C, 2, scale=0.3))
        p[f"w{k}"], p[f"b{k}"] = r(C, C, scale=0.3), r(C, scale=0.1)
        p[f"gamma{k}"], p[f"beta{k}"] = 1 + r(C, scale=0.1), r(C, scale=0.1)
    p.update(proj_w=r(1, C, scale=0.3), proj_b=r(1, scale=0.1))
    return p


def forward(p, data):
    """Calls of the library; returns the output and what the backward pass reads."""
    kept = []
    x = fno.fno_channel_linear(data, p["lift_w"], p["lift_b"], channels_last=True, out_channels_last=False)
    for k in range(2):
        s = fno.fno_spectral_conv2d(x, p[f"spec{k}"], M, M)
        y = fno.fno_channel_linear(x, p[f"w{k}"], p[f"b{k}"], branch=s, act="gelu")
        n, stats = fno.fno_group_norm(y, 3, weight=p[f"gamma{k}"], bias=p[f"beta{k}"], act="silu")
        kept.append((x, s, y, stats))
        x = n
    out = fno.fno_channel_linear(x, p["proj_w"], p["proj_b"], out_channels_last=True)
    return out, kept, x


def backward(p, data, kept, last, grad):
    g = {}
    gx, g["proj_w"], g["proj_b"], _ = fno.fno_channel_linear_backward(last, p["proj_w"], grad, bias=p["proj_b"],
                                                                     out_channels_last=True)
    for k in (1, 0):
        x, s, y, stats = kept[k]
        gy, g[f"gamma{k}"], g[f"beta{k}"] = fno.fno_group_norm_backward(
            y, stats, gx, 3, weight=p[f"gamma{k}"], bias=p[f"beta{k}"], act="silu")
        gx, g[f"w{k}"], g[f"b{k}"], gs = fno.fno_channel_linear_backward(x, p[f"w{k}"], gy, bias=p[f"b{k}"], branch=s,
                                                                         act="gelu")
        g2, g[f"spec{k}"] = fno.fno_spectral_conv2d_backward(x, p[f"spec{k}"], gs, M, M)
        gx = gx + g2
    _, g["lift_w"], g["lift_b"], _ = fno.fno_channel_linear_backward(
        data, p["lift_w"], gx, bias=p["lift_b"], channels_last=True, out_channels_last=False, need_x=False)
    return g


def reference(p, data):
    x = torch.einsum("bhwi,oi->bohw", data, p["lift_w"]) + p["lift_b"].view(1, -1, 1, 1)
    for k in range(2):
        X = torch.fft.rfft2(x, norm="ortho")
        rows = list(range(M)) + list(range(H - M, H))
        kept = X[:, :, rows, :M].reshape(B, C, 2, M, M)
        Y = torch.einsum("bisrk,srkio->bosrk", kept, p[f"spec{k}"])
        full = torch.zeros(B, C, H, W // 2 + 1, dtype=torch.complex128)
        full[:, :, :M, :M], full[:, :, H - M:, :M] = Y[:, :, 0], Y[:, :, 1]
        s = torch.fft.irfft2(full, s=(H, W), norm="ortho")
        z = torch.einsum("bihw,oi->bohw", x, p[f"w{k}"]) + p[f"b{k}"].view(1, -1, 1, 1) + s
        y = z * torch.special.ndtr(z)
        n = torch.nn.functional.group_norm(y, 3, p[f"gamma{k}"], p[f"beta{k}"], 1e-5)
        x = n * torch.sigmoid(n)
    return torch.einsum("bihw,oi->bhwo", x, p["proj_w"]) + p["proj_b"]


@pytest.mark.parametrize("bits", [32, 8])
def test_training_step(bits):
    gen = torch.Generator().manual_seed(21)
    host = make_params(gen)
    data, target = torch.randn(B, H, W, 3, generator=gen), torch.randn(B, H, W, 1, generator=gen)
    names = list(host)
    p = {k: v.to(DEV) for k, v in host.items()}
    ms, vs = fno.fno_adamw_states(p.values(), bits)
    copies = [torch.zeros_like(v, dtype=torch.bfloat16) if not v.is_complex() else None for v in p.values()]
    x, t = data.to(DEV), target.to(DEV)
    for step in (1, 2):
        leaves = {k: v.detach().cpu().to(torch.complex128 if v.is_complex() else torch.float64).requires_grad_(True)
                  for k, v in p.items()}
        want_out = reference(leaves, data.double())
        loss = 0.5 * ((want_out - target.double()) ** 2).sum()
        want = dict(zip(names, torch.autograd.grad(loss, list(leaves.values()))))
        out, kept, last = forward(p, x)
        # a chain of about twenty float32 steps, each good to a few 2^-24 of its largest values
        assert (out.cpu().double() - want_out).norm() <= 1e-5 * want_out.norm()
        g = backward(p, x, kept, last, out - t)
        for k in names:
            err = (g[k].cpu().to(want[k].dtype) - want[k]).norm()
            assert err <= 2e-5 * want[k].norm(), (k, float(err / want[k].norm()))
        grads = [g[k] for k in names]
        norm = fno.fno_grad_norm(grads)
        total = sum(float(torch.linalg.vector_norm(w)) ** 2 for w in want.values()) ** 0.5
        assert abs(float(norm) - total) <= 2e-5 * total
        old = {k: v.clone() for k, v in p.items()}
        before = [(m.clone(), v.clone()) for m, v in zip(ms, vs)]
        fno.fno_adamw(list(p.values()), grads, ms, vs, step, lr=0.01, norm=norm, max_norm=0.1, copies=copies, seed=4)
        factor = min(1.0, 0.1 / (float(norm) + 1e-6))
        for i, k in enumerate(names):
            q, gr, new = [(torch.view_as_real(t) if t.is_complex() else t).reshape(-1).cpu().double()
                          for t in (old[k], g[k], p[k])]
            if bits == 8:
                n = len(q)
                m0, v0 = (f[0].cpu().double() for f in fno.fno_adamw_moments(
                    [before[i][0]], [before[i][1]], numels=[n]))
            else:
                m0, v0 = (f.cpu().double().reshape(-1) for f in before[i])
            gr = (gr.float() * torch.tensor(factor, dtype=torch.float64).float()).double()
            m, v = 0.9 * m0 + 0.1 * gr, 0.999 * v0 + 0.001 * gr * gr
            step_size = 0.01 * (m / (1 - 0.9 ** step)) / ((v / (1 - 0.999 ** step)).sqrt() + 1e-8)
            after = q * (1 - 0.01 * 0.01) - step_size
            # float32 operations: 16 half steps of the update, three of the parameter; the factor's last bit
            bound = 2.0 ** -20 * step_size.abs() + 3 * 2.0 ** -24 * (q.abs() + after.abs()) + 1e-12
            assert bool(((new - after).abs() <= bound).all()), k
        for c, v in zip(copies, p.values()):
            if c is not None:
                assert torch.equal(c, v.to(torch.bfloat16))
    # the copies are what 16-bit products read
    half = fno.fno_channel_linear(x.to(torch.bfloat16), copies[names.index("lift_w")], p["lift_b"], channels_last=True)
    full = fno.fno_channel_linear(x, p["lift_w"], p["lift_b"], channels_last=True)
    assert (half.float() - full).norm() <= 2.0 ** -7 * full.norm()
