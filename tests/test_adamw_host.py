"""Host-side checks of the AdamW calls (no GPU): bad arguments are refused before
the device is touched.  Pointers are fake addresses."""
import array
import ctypes
import os

import pytest

import fft_spectral_convolution_amd as fno

NULL, SHAPE, ALIAS, ALIGN, VALUE = -1, -2, -4, -5, -12

NAMES = ("params", "out_params", "grads", "exp_avgs", "out_exp_avgs", "exp_avg_sqs", "out_exp_avg_sqs", "copies")


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(fno.library_path()):
        pytest.skip("libfno.so not built (run __graft_entry__.build())")
    return fno.lib()


def entry(k, n=100, ptype=0, gtype=0, bits=32, ctype=1, copy=0, **pointers):
    base = 0x100000000 * (k + 1)
    e = {name: base + 0x10000000 * i for i, name in enumerate(NAMES)}
    e["copies"] = copy
    e.update(pointers)
    return {**e, "numels": n, "param_types": ptype, "grad_types": gtype, "state_bits": bits, "copy_types": ctype}


def adamw(lib, entries, count=None, drop=(), **options):
    columns = {n: array.array("Q", [e[n] for e in entries]) for n in NAMES}
    columns["numels"] = array.array("q", [e["numels"] for e in entries])
    for n in ("param_types", "grad_types", "state_bits", "copy_types"):
        columns[n] = array.array("i", [e[n] for e in entries])
    t = fno._AdamwTensors(**{n: c.buffer_info()[0] for n, c in columns.items() if n not in drop})
    given = {"lr": 1e-3, "beta1": 0.9, "beta2": 0.999, "eps": 1e-8, "weight_decay": 0.01, "step": 1, **options}
    o = fno._AdamwOptions(**given)
    return lib.fno_adamw(ctypes.addressof(t), len(entries) if count is None else count, ctypes.addressof(o), None)


def test_options(lib):
    one = [entry(0)]
    nan, inf = float("nan"), float("inf")
    for bad in ({"lr": -1.0}, {"lr": nan}, {"lr": inf}, {"beta1": 1.0}, {"beta1": -0.1}, {"beta2": 1.0},
                {"beta2": nan}, {"eps": -1e-8}, {"eps": inf}, {"weight_decay": -0.1}, {"weight_decay": nan},
                {"step": 0}, {"step": -3}, {"norm": 0x70000000, "max_norm": -1.0},
                {"norm": 0x70000000, "max_norm": nan}):
        assert adamw(lib, one, **bad) == VALUE, bad
    for bad in ({"norm": 0x70000002, "max_norm": 1.0}, {"lr_device": 0x70000001}, {"step_device": 0x70000004}):
        assert adamw(lib, one, **bad) == ALIGN, bad
    assert lib.fno_adamw(None, 1, None, None) == NULL
    assert adamw(lib, one, count=-1) == SHAPE


def test_entries(lib):
    for n in NAMES[:7]:
        assert adamw(lib, [entry(0), entry(1, **{n: 0})]) == NULL, n
        assert adamw(lib, [entry(0)], drop=(n,)) == NULL, n
        assert adamw(lib, [entry(0, **{n: 0x700000002})]) == ALIGN, n
    for n in ("numels", "param_types", "grad_types", "state_bits", "copy_types"):
        assert adamw(lib, [entry(0)], drop=(n,)) == NULL, n
    assert adamw(lib, [entry(0, n=-1)]) == SHAPE and adamw(lib, [entry(0, n=(1 << 35) + 1)]) == SHAPE
    for bad in ({"ptype": 4}, {"ptype": -1}, {"gtype": 4}, {"ptype": 3}, {"gtype": 3}, {"bits": 16}, {"bits": 0},
                {"copy": 0x900000000, "ctype": 0}, {"copy": 0x900000000, "ctype": 3},
                {"copy": 0x900000000, "ptype": 3, "gtype": 3}):
        assert adamw(lib, [entry(0, **bad)]) == VALUE, bad
    assert adamw(lib, [entry(0, bits=8, exp_avgs=0x700000008)]) == ALIGN
    assert adamw(lib, [entry(0, copy=0x700000001)]) == ALIGN


def test_overlaps(lib):
    a = entry(0)
    for n in ("out_params", "out_exp_avgs", "out_exp_avg_sqs"):
        for other in ("grads", "exp_avg_sqs", "params", "exp_avgs"):
            if other == n[4:] + "" or n == "out_" + other:
                continue
            assert adamw(lib, [entry(0, **{n: a[other] + 396})]) == ALIAS, (n, other)
            assert adamw(lib, [entry(0), entry(1, **{n: a[other]})]) == ALIAS, (n, other)
    # in place, the same tensor twice
    same = {n: a[n.replace("out_", "")] for n in NAMES if n.startswith("out_")}
    assert adamw(lib, [entry(0, **same), entry(0, **same)]) == ALIAS
    # in place, but not quite
    assert adamw(lib, [entry(0, out_params=a["params"] + 4)]) == ALIAS
    assert adamw(lib, [entry(0, copy=a["out_params"])]) == ALIAS
    assert adamw(lib, [entry(0)], norm=a["out_params"] + 4, max_norm=1.0) == ALIAS
    assert adamw(lib, [entry(0)], lr_device=a["out_exp_avgs"]) == ALIAS
    assert adamw(lib, [entry(0)], step_device=a["out_exp_avg_sqs"] + 8) == ALIAS
    # the bytes of an 8-bit moment: 256 codes and 2 exponents in whole 16 bytes
    end = a["out_exp_avgs"] + 272
    assert adamw(lib, [entry(0, n=256, bits=8), entry(1, out_params=end - 4)]) == ALIAS


def test_moments(lib):
    def call(m=0x10000000, v=0x20000000, mo=0x30000000, vo=0x40000000, n=100, count=1):
        columns = [array.array("Q", [p]) for p in (m, v, mo, vo)] + [array.array("q", [n])]
        return lib.fno_adamw_moments(*[c.buffer_info()[0] for c in columns], count, None)

    assert call(count=-1) == SHAPE and call(n=-1) == SHAPE and call(n=(1 << 36) + 1) == SHAPE
    for k in ("m", "v", "mo", "vo"):
        assert call(**{k: 0}) == NULL and call(**{k: 0x50000002}) == ALIGN
    assert call(m=0x50000008) == ALIGN
    assert call(mo=0x10000000) == ALIAS and call(mo=0x40000000) == ALIAS and call(vo=0x20000000 + 128) == ALIAS
    assert lib.fno_adamw_moments(None, None, None, None, None, 1, None) == NULL
    assert lib.fno_adamw_moments(None, None, None, None, None, 0, None) == 0


def test_moment_sizes(lib):
    for n, t, size in ((0, 0, 0), (1, 0, 144), (128, 1, 144), (129, 2, 272), (64, 3, 144), (65, 3, 272),
                       (2048, 0, 2064), (2049, 0, 2208), (-1, 0, 0), (1, 4, 0), (1, -1, 0), ((1 << 35) + 1, 0, 0)):
        assert lib.fno_adamw_moment_size(n, t) == size, (n, t)
        if 0 <= t <= 2 and 0 <= n <= 1 << 35:
            assert fno._moment_bytes(n) == size


def test_tensor_lists(lib):
    """What the reader of tensor lists refuses, by its kind of error (of tensors on the CPU, the device)."""
    torch = pytest.importorskip("torch")
    with pytest.raises(TypeError, match="must be torch tensors"):
        fno._read_tensors(torch, [3], "grads")
    with pytest.raises(TypeError, match="must be torch tensors"):
        fno._read_tensors(torch, [None], "grads")
    with pytest.raises(ValueError, match="one GPU device"):
        fno._read_tensors(torch, (torch.zeros(3),), "grads")
    assert fno._read_tensors(torch, [None, None], "copies", fno._HALVES, optional=True)[3].tolist() == [-1, -1]
    assert fno._read_tensors(torch, iter([]), "grads")[4] is None
    for call in (fno.fno_grad_norm, fno.fno_adamw_states):
        with pytest.raises(ValueError):
            call([torch.zeros(3)])
