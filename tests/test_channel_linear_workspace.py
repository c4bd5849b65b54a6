"""The workspace of a channel product's backward pass (no GPU)."""
import os

import pytest

import fft_spectral_convolution_amd as fno


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(fno.library_path()):
        pytest.skip("libfno.so not built (run __graft_entry__.build())")
    return fno.lib()


# channels of the one-kernel pass and of the four-kernel one
@pytest.mark.parametrize("cin,cout", [(20, 30), (64, 60), (300, 20), (20, 300), (200, 200)])
@pytest.mark.parametrize("act", [0, 1])
def test_channels_last_positions_are_one_run(lib, cin, cout, act):
    """Both sides channels last: B items of P positions are the same call as one item of B P."""
    for B, P in ((2048, 1), (700, 3), (33, 31), (1000, 33)):
        for types in ((0, 0), (1, 1), (2, 0)):
            assert lib.fno_channel_linear_workspace_size(B, cin, cout, P, act, 1, 1, *types) \
                == lib.fno_channel_linear_workspace_size(1, cin, cout, B * P, act, 1, 1, *types)


def test_shares_hold_a_tile_a_wave(lib):
    """Sums of the weight's gradient in shares of four waves' tiles of 32 positions: 2048 positions are 16 of them."""
    share = (300 + 1) * 20 * 4
    assert lib.fno_channel_linear_workspace_size(2048, 300, 20, 1, 0, 1, 1, 0, 0) == -(-16 * share // 256) * 256
