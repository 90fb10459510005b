"""The 8-bit layer's calls refuse bad arguments on the host, before anything is
launched, and its 64-bit reference is itself pinned (no GPU)."""

import ctypes

import numpy as np
import pytest

from tests import _fp8_ref as ref

FAKE = 0x10000  # 16-byte aligned, never dereferenced: validation fails first
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    from bit_w4a4_quantized_smooth_b200 import build, binding
    build.build()
    return binding.load()


def _bad(args, i, v):
    return tuple(v if j == i else a for j, a in enumerate(args))


def test_sizes(lib):
    from bit_w4a4_quantized_smooth_b200 import SvdqError, fp8_sizes
    assert fp8_sizes(4608, 3072) == (4608 * 3072, 36 * 6 * 512)
    assert fp8_sizes(1, 16) == (16, 512)
    assert fp8_sizes(129, 528) == (129 * 528, 2 * 2 * 512)
    assert fp8_sizes(0, 64) == (0, 0)
    for rows, K, status in ((1, 24, 2), (1, 0, 1), (-1, 64, 1), ((1 << 22) + 1, 64, 2), (1, (1 << 20) + 16, 2)):
        with pytest.raises(SvdqError) as e:
            fp8_sizes(rows, K)
        assert e.value.status == status


def test_pack_refusals(lib):
    f = lib.svdq_pack_weight_fp8
    ok = (P(FAKE), 0, 64, 16, P(FAKE), P(FAKE), None)
    for i, v, status in ((0, None, 1), (4, None, 1), (5, None, 1), (1, 2, 1), (2, 0, 1), (3, -8, 1), (2, 72, 2),
                         (3, 12, 2), (2, (1 << 20) + 16, 2), (3, (1 << 22) + 8, 2), (0, P(FAKE + 8), 3),
                         (4, P(FAKE + 4), 3), (5, P(FAKE + 1), 3)):
        assert f(*_bad(ok, i, v)) == status, (i, v)


def test_quantize_refusals(lib):
    f = lib.svdq_quantize_fp8
    ok = (P(FAKE), 64, 4, 64, 0, P(FAKE), P(FAKE), None)
    for i, v, status in ((0, None, 1), (5, None, 1), (6, None, 1), (1, 56, 1), (2, 0, 1), (3, 0, 1), (4, 2, 1),
                         (1, 68, 2), (3, 40, 2), (2, (1 << 22) + 1, 2), (0, P(FAKE + 2), 3), (5, P(FAKE + 8), 3),
                         (6, P(FAKE + 8), 3)):
        assert f(*_bad(ok, i, v)) == status, (i, v)


def test_rmsnorm_refusals(lib):
    f = lib.svdq_rmsnorm
    ok = (P(FAKE), 64, P(FAKE), 0, P(FAKE), 1e-6, 4, 64, P(FAKE), P(FAKE), P(FAKE), P(FAKE), None)
    for i, v, status in ((0, None, 1), (1, 48, 1), (6, 0, 1), (7, 0, 1), (3, 7, 1), (5, -1.0, 1),
                         (5, float("nan"), 1), (5, float("inf"), 1),
                         (2, None, 1),        # residual_out without a residual
                         (8, None, 1),        # a residual without residual_out
                         (10, None, 1),       # scales without codes
                         (11, None, 1),       # codes without scales
                         (1, 68, 2), (7, 40, 2), (6, (1 << 22) + 1, 2), (0, P(FAKE + 4), 3), (2, P(FAKE + 4), 3),
                         (4, P(FAKE + 2), 3), (8, P(FAKE + 8), 3), (9, P(FAKE + 8), 3), (10, P(FAKE + 8), 3)):
        assert f(*_bad(ok, i, v)) == status, (i, v)
    big = _bad(_bad(ok, 7, 32784), 1, 32784)
    assert f(*big) == 2
    no_out = tuple(None if i in (9, 10, 11) else a for i, a in enumerate(ok))
    assert f(*no_out) == 1


@pytest.mark.parametrize("name", ["svdq_linear_fp8", "svdq_linear_fp8_gelu"])
def test_linear_refusals(lib, name):
    f = getattr(lib, name)
    gelu = name.endswith("gelu")
    ok = (P(FAKE), P(FAKE), P(FAKE), P(FAKE), P(FAKE), 4, 64, 32, P(FAKE)) + ((P(FAKE),) if gelu else ()) + (None,)
    bad = [(0, None, 1), (1, None, 1), (2, None, 1), (3, None, 1), (8, None, 1), (5, 0, 1), (6, 0, 1), (7, 0, 1),
           (6, 40, 2), (7, 12, 2), (5, (1 << 22) + 1, 2), (6, (1 << 20) + 16, 2), (7, (1 << 22) + 16, 2),
           (0, P(FAKE + 8), 3), (1, P(FAKE + 8), 3), (2, P(FAKE + 8), 3), (3, P(FAKE + 8), 3), (4, P(FAKE + 2), 3),
           (8, P(FAKE + 8), 3)]
    if gelu:
        bad += [(9, None, 1), (9, P(FAKE + 8), 3), (7, 24, 2), (7, (1 << 20) + 16, 2)]
    for i, v, status in bad:
        assert f(*_bad(ok, i, v)) == status, (i, v)


def test_path_setting(lib):
    from bit_w4a4_quantized_smooth_b200 import set_linear_fp8_path
    assert lib.svdq_set_linear_fp8_path(3) == 1 and lib.svdq_set_linear_fp8_path(-1) == 1
    set_linear_fp8_path("small")
    set_linear_fp8_path("auto")


def test_splits_setting(lib):
    from bit_w4a4_quantized_smooth_b200 import SvdqError, set_linear_fp8_splits
    assert lib.svdq_set_linear_fp8_splits(9) == 1 and lib.svdq_set_linear_fp8_splits(-1) == 1
    with pytest.raises(SvdqError):
        set_linear_fp8_splits(9)
    set_linear_fp8_splits(8)
    set_linear_fp8_splits(0)


def test_binding_refuses_what_the_abi_cannot_see():
    """Types, shapes, strides and devices are checked before a pointer is taken."""
    import torch
    import bit_w4a4_quantized_smooth_b200 as svdq
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        svdq.quantize_fp8(bf(4, 64))
    with pytest.raises(ValueError, match="bfloat16"):
        svdq.quantize_fp8(torch.zeros(4, 64))
    with pytest.raises(ValueError, match="bfloat16"):
        svdq.rmsnorm(bf(2, 4, 64))
    with pytest.raises(ValueError, match="CUDA"):
        svdq.rmsnorm(bf(4, 64), bf(64))
    with pytest.raises(ValueError, match="CUDA"):
        svdq.pack_weight_fp8(bf(64, 16))
    with pytest.raises(ValueError, match="CUDA"):
        svdq.linear_fp8(u8(4, 64), u8(512), u8(16, 64), u8(512))
    with pytest.raises(ValueError, match="2-D"):
        svdq.linear_fp8_gelu(u8(4, 64), u8(512), u8(16), u8(512))


# ------------------------------------------------------- the reference's pins --
def test_reference_e4m3_matches_torch():
    import torch
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).to(torch.float64).numpy()
    assert np.array_equal(t, ref.E4M3, equal_nan=True)
    rng = np.random.default_rng(1)
    u = np.concatenate([rng.normal(size=20000) * 10.0 ** rng.uniform(-4, 2, 20000), ref._MID, -ref._MID, ref._POS])
    u = np.clip(u, -448, 448).astype(np.float32)
    want = torch.from_numpy(u).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ref.e4m3_encode(u.astype(np.float64)), want)


def test_reference_scale_is_the_smallest():
    rng = np.random.default_rng(2)
    a = np.concatenate([10.0 ** rng.uniform(-30, 30, 2000), 448.0 * 2.0 ** np.arange(-100, 100),
                        np.nextafter(448.0 * 2.0 ** np.arange(-100, 100), np.inf)])
    b = ref.scale_byte(a).astype(np.float64) - 127
    assert (a <= 448.0 * 2.0 ** b).all() and (a > 448.0 * 2.0 ** (b - 1)).all()
    assert ref.scale_byte(np.array([0.0, 1e-45]))[0] == 0 and ref.scale_byte(np.array([1e-45]))[0] == 0


def test_reference_tiles_round_trip():
    rng = np.random.default_rng(3)
    s = rng.integers(1, 255, (200, 9)).astype(np.uint8)
    flat = ref.tiles(s)
    back, rest = ref.untile(flat, 200, 9 * 128)
    assert np.array_equal(back, s) and not flat[rest].any() and rest.sum() == 256 * 12 - 200 * 9


def test_measured_cases_plain_forms_agree_with_this_reference(monkeypatch):
    """perf/operators.py's plain form and its 64-bit definition, on the CPU."""
    import importlib.util
    import os
    import torch
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "perf", "operators.py")
    spec = importlib.util.spec_from_file_location("operators_cases", path)
    M = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(M)
    rng = np.random.default_rng(4)
    v = rng.normal(size=(130, 656)) * 10.0 ** rng.uniform(-5, 5, (130, 1))
    v = v.astype(np.float32)
    v[3, 128:256] = 0.0
    codes, s = ref.encode(v.astype(np.float64))
    for fn, x in ((M._quantise, torch.from_numpy(v)), (M._exact_fp8, torch.from_numpy(v).double())):
        c, t = fn(x)
        assert np.array_equal(c.view(torch.uint8).numpy(), codes)
        assert np.array_equal(t.view(torch.uint8).numpy(), ref.tiles(s))
