"""Host-side checks of the group norm and gradient clipping calls (no GPU):
bad arguments are refused before the device is touched.  Pointers are fake
addresses."""
import ctypes
import os

import pytest

import fft_spectral_convolution_amd as fno

NULL, SHAPE, ALIAS, ALIGN, WORKSPACE, VALUE = -1, -2, -4, -5, -8, -12

X, W, B, O, S, G = (0x10000000 * k for k in range(1, 7))
GW, GB, WS = 0x70000000, 0x71000000, 0x72000000
BIG = 1 << 20


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(fno.library_path()):
        pytest.skip("libfno.so not built (run __graft_entry__.build())")
    return fno.lib()


def norm(lib, x=X, w=W, b=B, out=O, stats=S, dims=(2, 8, 10, 4), eps=1e-5, act=0, x_last=1, out_last=1, x_type=0,
         out_type=0, ws=WS, ws_bytes=BIG):
    return lib.fno_group_norm(x, w, b, out, stats, *dims, eps, act, x_last, out_last, x_type, out_type, ws, ws_bytes,
                              None)


def back(lib, x=X, w=W, b=B, stats=S, dy=O, gx=G, gw=GW, gb=GB, dims=(2, 8, 10, 4), act=0, x_last=1, out_last=1,
         x_type=0, out_type=0, ws=WS, ws_bytes=BIG):
    return lib.fno_group_norm_backward(x, w, b, stats, dy, gx, gw, gb, *dims, act, x_last, out_last, x_type, out_type,
                                       ws, ws_bytes, None)


@pytest.mark.parametrize("call", [norm, back])
def test_group_norm_sizes_and_options(lib, call):
    for dims in ((0, 8, 10, 4), (2, 0, 10, 4), (2, 8, 0, 4), (2, 8, 10, 0), (2, 8, 10, 3), (2, 8, 10, 16),
                 (-1, 8, 10, 4), (2, 8, -10, 4), (65536, 65536, 1, 1), (1 << 20, 1 << 10, 1 << 20, 1),
                 (1, (1 << 24) + 1, 1, 1), (1, 1, (1 << 30) + 1, 1)):
        assert call(lib, dims=dims) == SHAPE, dims
        assert lib.fno_group_norm_workspace_size(*dims, 1, 1, 0, 0) == 0
    assert call(lib, act=3) == VALUE and call(lib, act=-1) == VALUE
    assert call(lib, x_last=2) == VALUE and call(lib, out_last=-1) == VALUE
    assert call(lib, x_type=3) == VALUE and call(lib, x_type=-1) == VALUE
    assert call(lib, x_type=0, out_type=1) == VALUE          # float32 in, bfloat16 out
    assert call(lib, x_type=1, out_type=2) == VALUE
    # float32 in the one layout, out or grad_out in the other: chunks' sums in the workspace
    need = lib.fno_group_norm_workspace_size(2, 8, 10, 4, 1, 0, 0, int(call is back))
    assert need > 0
    assert call(lib, out_last=0, ws=None) == WORKSPACE and call(lib, out_last=0, ws_bytes=need - 1) == WORKSPACE
    assert call(lib, ws=WS + 16) == ALIGN
    assert lib.fno_group_norm_workspace_size(2, 8, 10, 4, 1, 0, 3, 0) == 0
    assert lib.fno_group_norm_workspace_size(2, 8, 10, 4, 2, 0, 0, 0) == 0


def test_group_norm_eps(lib):
    for eps in (0.0, -1e-5, float("nan"), float("inf")):
        assert norm(lib, eps=eps) == VALUE


def test_group_norm_pointers(lib):
    for k in ("x", "out", "stats"):
        assert norm(lib, **{k: None}) == NULL
    assert norm(lib, x=X + 2) == ALIGN and norm(lib, out=O + 1, x_type=1, out_type=1) == ALIGN
    assert norm(lib, w=W + 2) == ALIGN and norm(lib, b=B + 1) == ALIGN and norm(lib, stats=S + 2) == ALIGN
    n = 2 * 8 * 10 * 4
    assert norm(lib, out=X) == ALIAS and norm(lib, out=X + n - 4) == ALIAS and norm(lib, out=X - n + 4) == ALIAS
    assert norm(lib, out=W - n + 8) == ALIAS and norm(lib, stats=B) == ALIAS and norm(lib, stats=O + 64) == ALIAS
    assert norm(lib, ws=X, ws_bytes=BIG) == ALIAS and norm(lib, out=WS + 4096) == ALIAS


def test_group_norm_backward_pointers(lib):
    for k in ("x", "dy", "stats"):
        assert back(lib, **{k: None}) == NULL
    assert back(lib, gx=None, gw=None, gb=None) == NULL
    assert back(lib, gx=G + 2) == ALIGN and back(lib, gw=GW + 2) == ALIGN and back(lib, gb=GB + 3) == ALIGN
    assert back(lib, gx=X) == ALIAS and back(lib, gx=O) == ALIAS and back(lib, gw=W) == ALIAS
    assert back(lib, gw=GW, gb=GW + 4) == ALIAS and back(lib, gb=S) == ALIAS


def table(entries):
    n = len(entries)
    return ((ctypes.c_void_p * n)(*[e[0] for e in entries]), (ctypes.c_longlong * n)(*[e[1] for e in entries]),
            (ctypes.c_int * n)(*[e[2] for e in entries]))


def clip(lib, entries, outs=None, limit=1.0, given=None, n=O, ws=WS, ws_bytes=BIG, count=None):
    p, m, t = table(entries)
    q = p if outs is None else (ctypes.c_void_p * len(outs))(*outs)
    return lib.fno_clip_grad_norm(p, q, m, t, len(entries) if count is None else count, limit, given, n, ws, ws_bytes,
                                  None)


def total(lib, entries, n=O, ws=WS, ws_bytes=BIG, count=None):
    p, m, t = table(entries)
    return lib.fno_grad_norm(p, m, t, len(entries) if count is None else count, n, ws, ws_bytes, None)


@pytest.mark.parametrize("call", [total, clip])
def test_grad_norm_refusals(lib, call):
    assert call(lib, [(X, 10, 0)], count=-1) == SHAPE
    assert call(lib, [(X, -1, 0)]) == SHAPE and call(lib, [(X, (1 << 35) + 1, 0)]) == SHAPE
    assert call(lib, [(X, 10, 4)]) == VALUE and call(lib, [(X, 10, -1)]) == VALUE
    assert call(lib, [(None, 10, 0)]) == NULL
    assert call(lib, [(X + 2, 10, 0)]) == ALIGN and call(lib, [(X + 1, 10, 1)]) == ALIGN
    assert call(lib, [(X, 10, 0)], n=None) == NULL
    assert call(lib, [(X, 10, 0)], n=O + 2) == ALIGN
    assert call(lib, [(X, 10, 0)], ws=None) == WORKSPACE and call(lib, [(X, 10, 0)], ws_bytes=64) == WORKSPACE
    assert call(lib, [(X, 10, 0)], ws=WS + 8) == ALIGN
    assert lib.fno_grad_norm(None, None, None, 1, O, WS, BIG, None) == NULL
    assert lib.fno_grad_norm_workspace_size(-1) == 0


def test_clip_refusals(lib):
    one = [(X, 100, 0)]
    for limit in (-1.0, float("nan")):
        assert clip(lib, one, limit=limit) == VALUE
    assert clip(lib, one, outs=[None]) == NULL
    assert clip(lib, one, outs=[G + 1]) == ALIGN
    assert clip(lib, one, outs=[X + 4]) == ALIAS                       # not in place, not apart
    assert clip(lib, one, outs=[X + 396]) == ALIAS
    assert clip(lib, [(X, 100, 0), (X, 100, 0)]) == ALIAS              # one tensor twice, in place
    assert clip(lib, [(X, 100, 0), (X + 200, 4, 0)]) == ALIAS          # a part of another
    assert clip(lib, [(X, 100, 0), (G, 100, 0)], outs=[GW, GW + 396]) == ALIAS
    assert clip(lib, [(X, 100, 0), (G, 100, 0)], outs=[G, X]) == ALIAS # swapped
    assert clip(lib, one, n=X + 40) == ALIAS
    assert clip(lib, one, n=None, given=X + 40) == ALIAS
    assert clip(lib, one, ws=X - 256) == ALIAS


def test_binding_refuses_before_the_device():
    torch = pytest.importorskip("torch")
    x = torch.zeros((1, 4, 8))
    with pytest.raises(ValueError):
        fno.fno_group_norm(x, 2)
    with pytest.raises(ValueError):
        fno.fno_group_norm_backward(x, torch.zeros(1, 2, 2), x, 2)
    with pytest.raises(ValueError):
        fno.fno_grad_norm([x])
    with pytest.raises(ValueError):
        fno.fno_clip_grad_norm([x], 1.0)
    with pytest.raises(TypeError):
        fno.fno_grad_norm([1.0])
    with pytest.raises(TypeError):
        fno.fno_group_norm([1.0], 1)


# Fields far apart, and a workspace that is off its alignment by 16 bytes: a call that finds it large enough is refused
# for that (ALIGN), one that needs more for its size (WORKSPACE), and none is launched.
FAR = [k << 44 for k in range(1, 9)]
OFF = (9 << 44) + 16


def _queried_size_serves(lib, dims, x_last, out_last, x_type):
    for backward in (0, 1):
        need = lib.fno_group_norm_workspace_size(*dims, x_last, out_last, x_type, backward)
        for out_type in sorted({x_type, 0}):
            opts = dict(dims=dims, x_last=x_last, out_last=out_last, x_type=x_type, out_type=out_type, ws=OFF,
                        ws_bytes=need)
            rc = back(lib, *FAR, **opts) if backward else norm(lib, *FAR[:5], **opts)
            assert rc == ALIGN, (backward, out_type, need)


@pytest.mark.parametrize("x_type", [0, 1, 2])
@pytest.mark.parametrize("x_last,out_last", [(1, 1), (0, 0), (1, 0), (0, 1)])
@pytest.mark.parametrize("dims", [
    (32, 64, 16384, 8), (16, 64, 16384, 8), (8, 64, 16384, 8), (64, 64, 4096, 8), (1, 145, 16632, 1),
    (2, 4, 1024, 2), (3, 30, 2867, 5), (2, 16, 1 << 22, 4), (4, 8192, 1024, 8), (256, 64, 4096, 16), (1, 1, 1, 1),
])
def test_queried_workspace_serves_every_type(lib, dims, x_last, out_last, x_type):
    _queried_size_serves(lib, dims, x_last, out_last, x_type)


@pytest.mark.parametrize("seed", range(4))
def test_queried_workspace_serves_random_fields(lib, seed):
    import random
    rng = random.Random(seed)
    for _ in range(500):
        c = int(2 ** rng.uniform(0, 13))
        groups = rng.choice([g for g in range(1, c + 1) if c % g == 0])
        dims = (int(2 ** rng.uniform(0, 8)), c, int(2 ** rng.uniform(0, 20)), groups)
        _queried_size_serves(lib, dims, rng.randint(0, 1), rng.randint(0, 1), rng.randint(0, 2))


def test_looks_are_bounded(lib, monkeypatch):
    """The wait for another workgroup's sums ends, whatever is asked for."""
    for looks in (-1, 4097, 2 ** 31 - 1, -2 ** 31):
        assert lib.fno_set_exchange_looks(looks) == VALUE
    asked = []
    monkeypatch.setattr(fno, "lib", lambda: type("L", (), {"fno_set_exchange_looks": lambda self, n: asked.append(n)
                                                           or lib.fno_set_exchange_looks(n)})())
    for value, want in (("0", [0]), ("0", []), ("-5", []), ("17", [17]), ("2147483647", [4096]), ("99999999999", []),
                        ("1", [1]), (None, [4096])):
        asked.clear()
        if value is None:
            monkeypatch.delenv("FNO_GN_SPIN")
        else:
            monkeypatch.setenv("FNO_GN_SPIN", value)
        fno._follow_looks()
        assert asked == want, value
    # nothing in the library follows the environment, which other threads may be changing
    src = os.path.join(os.path.dirname(fno.__file__), "csrc")
    for name in os.listdir(src):
        assert "getenv" not in open(os.path.join(src, name)).read(), name


def test_norm_written_over_a_gradient(lib):
    """fno_grad_norm writes its norm and workspace and nothing else."""
    grads = [(X, 100, 0), (G, 100, 3), (B, 0, 0)]
    for n in (X, X + 396, G + 796):
        assert total(lib, grads, n=n) == ALIAS, hex(n)
    assert total(lib, grads, ws=X - 256) == ALIAS and total(lib, grads, ws=G + 512) == ALIAS
    assert total(lib, grads, n=WS + 1024) == ALIAS
    # next to them, on an empty one, and a gradient twice: taken (and then refused for the workspace's alignment)
    for n in (X - 4, X + 400, G + 800, B):
        assert total(lib, grads, n=n, ws=WS + 8) == ALIGN, hex(n)
    assert total(lib, [(X, 100, 0), (X, 100, 0), (X + 4, 9, 0)], ws=WS + 8) == ALIGN


def test_given_norm_is_only_read(lib):
    """It may be one of the gradients that are only read, not of those written, nor in the workspace."""
    two, apart = [(X, 100, 0), (G, 100, 0)], [GW, GW + 400]
    assert clip(lib, two, outs=apart, given=X + 40, ws=WS + 8) == ALIGN           # taken up to the workspace's alignment
    assert clip(lib, two, outs=apart, given=O, ws=WS + 8) == ALIGN                # norm itself
    assert clip(lib, two, outs=[X, GW], given=X + 40) == ALIAS
    assert clip(lib, two, outs=apart, given=GW + 796) == ALIAS
    assert clip(lib, two, outs=apart, given=WS + 512) == ALIAS
    assert clip(lib, two, outs=apart, given=O + 2) == ALIAS


@pytest.mark.parametrize("groups", [2 ** 32 + 2, -2 ** 32 + 2, 2 ** 31, 2 ** 63])
def test_groups_beyond_32_bits(groups, monkeypatch):
    """Refused by the binding: the call would see the low 32 bits, here a divisor of the channels."""
    torch = pytest.importorskip("torch")
    monkeypatch.setattr(fno, "_field_type", lambda *a: 0)         # a CPU tensor stands for the field
    with pytest.raises(ValueError):
        fno._group_norm_args(torch, torch.zeros(1, 8, 4), groups, None, None, "none", False, None)
