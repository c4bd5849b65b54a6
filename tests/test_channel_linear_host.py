"""Host-side checks of the channel product calls (no GPU): bad arguments are
refused before the device is touched.  Pointers are fake addresses."""
import os

import pytest

import fft_spectral_convolution_amd as fno

NULL, SHAPE, ALIAS, ALIGN, WORKSPACE, VALUE = -1, -2, -4, -5, -8, -12

X, W, B, R, O, GX, GR = (0x10000000 * k for k in range(1, 8))
GW, GB, WS = 0x80000000, 0x81000000, 0x82000000
BIG = 1 << 24
DIMS = (2, 8, 12, 10)          # B, Cin, Cout, P


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(fno.library_path()):
        pytest.skip("libfno.so not built (run __graft_entry__.build())")
    return fno.lib()


def forward(lib, x=X, w=W, b=B, branch=R, out=O, dims=DIMS, act=1, after=0, x_last=1, out_last=1, x_type=0, out_type=0):
    return lib.fno_channel_linear(x, w, b, branch, out, *dims, act, after, x_last, out_last, x_type, out_type, None)


def backward(lib, x=X, w=W, b=B, branch=R, out=O, gx=GX, gw=GW, gb=GB, gr=GR, dims=DIMS, act=1, after=0, x_last=1,
             out_last=1, x_type=0, out_type=0, ws=WS, ws_bytes=BIG):
    return lib.fno_channel_linear_backward(x, w, b, branch, out, gx, gw, gb, gr, *dims, act, after, x_last, out_last,
                                           x_type, out_type, ws, ws_bytes, None)


@pytest.mark.parametrize("call", [forward, backward])
def test_sizes_and_options(lib, call):
    for dims in ((0, 8, 12, 10), (2, 0, 12, 10), (2, 8, 0, 10), (2, 8, 12, 0), (-1, 8, 12, 10), (2, 8, 12, -5),
                 (2, (1 << 16) + 1, 12, 10), (2, 8, (1 << 16) + 1, 10), (2, 8, 12, (1 << 30) + 1),
                 (1 << 20, 1, 2, 1 << 20), (1 << 12, 1, 1, (1 << 23) + 1)):
        assert call(lib, dims=dims) == SHAPE, dims
        assert lib.fno_channel_linear_workspace_size(*dims, 1, 1, 1, 0, 0) == 0
    for last in ((0, 0), (0, 1), (1, 0)):
        assert call(lib, dims=(1, 8, 12, (1 << 24) + 1), x_last=last[0], out_last=last[1]) == SHAPE
    for bad in ({"act": 3}, {"act": -1}, {"after": 2}, {"x_last": 2}, {"out_last": -1}, {"x_type": 3}, {"x_type": -1},
                {"out_type": 1}, {"x_type": 1, "out_type": 2}):
        assert call(lib, **bad) == VALUE, bad


@pytest.mark.parametrize("call", [forward, backward])
def test_pointers(lib, call):
    for k in ("x", "w", "out"):
        assert call(lib, **{k: None}) == NULL
        assert call(lib, **{k: 0x90000002}) == ALIGN
    assert call(lib, b=B + 2) == ALIGN and call(lib, branch=R + 1) == ALIGN
    assert call(lib, x=X + 1, x_type=1, out_type=1) == ALIGN


def test_forward_overlaps(lib):
    n = 2 * 12 * 10 * 4
    for k, size in ((X, 2 * 8 * 10 * 4), (W, 8 * 12 * 4), (B, 12 * 4), (R, n)):
        assert forward(lib, out=k) == ALIAS and forward(lib, out=k + size - 4) == ALIAS
        assert forward(lib, out=k - n + 4) == ALIAS


def test_backward_pointers(lib):
    assert backward(lib, gx=None, gw=None, gb=None, gr=None) == NULL
    for k in ("gx", "gw", "gb", "gr"):
        assert backward(lib, **{k: 0x90000002}) == ALIGN
        for other in (X, W, B, R, O):
            assert backward(lib, **{k: other}) == ALIAS, (k, other)
    assert backward(lib, gw=GW, gb=GW + 8) == ALIAS and backward(lib, gx=GR) == ALIAS
    assert backward(lib, ws=X, ws_bytes=BIG) == ALIAS and backward(lib, gw=WS + 256) == ALIAS
    # a branch behind the activation, or without one, has grad_out for its gradient
    assert backward(lib, after=1) == VALUE and backward(lib, act=0) == VALUE


def test_workspace(lib):
    for act in (0, 1, 2):
        need = lib.fno_channel_linear_workspace_size(*DIMS, act, 1, 1, 0, 0)
        assert need > 0
        given = {"act": act, "gr": None}
        assert backward(lib, ws=None, **given) == WORKSPACE
        assert backward(lib, ws_bytes=need - 1, **given) == WORKSPACE
        assert backward(lib, ws=WS + 16, **given) == ALIGN
    assert lib.fno_channel_linear_workspace_size(*DIMS, 1, 2, 1, 0, 0) == 0
    assert lib.fno_channel_linear_workspace_size(*DIMS, 1, 1, 1, 0, 1) == 0
