"""The frequencies of scaled rotary positions against their definition, over original lengths from far below to far above the
base's wave lengths (on the host; no GPU)."""
import math

import numpy as np
import pytest


@pytest.fixture(scope="module")
def bd():
    import block_diffusion_gb300 as bd
    from block_diffusion_gb300 import build
    build.build()
    bd.load_library()
    return bd


def frequencies(r):
    return np.array(r.turns[:r.rot_dim // 2], np.float64) * 2.0 ** -64 * 2 * math.pi


def yarn_keep(rot, base, length, few, many):
    """How much of its own frequency each pair keeps: all of it up to the pair that makes `many` turns over the original
    length, nothing from the one that makes `few`, both rounded away from each other and kept within 0 .. rot - 1."""
    def pair(turns):        # real x with length * base^(-2 x / rot) = 2 pi turns
        return math.log(length / (2 * math.pi * turns), base) * rot / 2
    lo, hi = max(0, math.floor(pair(many))), min(rot - 1, math.ceil(pair(few)))
    assert lo < hi
    return np.interp(np.arange(rot // 2), [lo, hi], [1.0, 0.0])


@pytest.mark.parametrize("rot", [16, 64, 96, 128])
@pytest.mark.parametrize("base", [10000.0, 500000.0])
@pytest.mark.parametrize("length", [512, 4096, 32768, 65536, 131072, 1 << 20])
@pytest.mark.parametrize("factor", [1.0, 4.0, 40.0])
def test_yarn(bd, rot, base, length, factor):
    r = bd.bdlm_rotary_init(rot, False, base, bd.BDLM_ROTARY_YARN, factor, length, 1.0, 32.0)
    own = base ** (-2 * np.arange(rot // 2) / rot)
    keep = yarn_keep(rot, base, length, 1.0, 32.0)
    want = own * (keep + (1 - keep) / factor)
    assert np.all(np.abs(frequencies(r) - want) <= 1e-12 * want + 1e-18)


def test_yarn_of_a_long_original_length(bd):
    """Pairs that still make more than one turn when the last of them has: by hand, 128 dims, base 10000, 65536 tokens."""
    r = bd.bdlm_rotary_init(128, False, 10000.0, bd.BDLM_ROTARY_YARN, 8.0, 65536.0, 1.0, 32.0)
    ratio = frequencies(r) / 10000.0 ** (-np.arange(64) / 64)
    # pairs 40.2 (32 turns) and 64.3 (one): from 40 to 65
    assert ratio[40] == pytest.approx(1, rel=1e-12) and ratio[39] == pytest.approx(1, rel=1e-12)
    for i in (41, 52, 62, 63):
        assert ratio[i] == pytest.approx(1 - (i - 40) / 25 * 7 / 8, rel=1e-12)
    assert ratio[62] == pytest.approx(0.23, abs=1e-3) and ratio[63] == pytest.approx(0.195, abs=1e-3)


@pytest.mark.parametrize("length", [512.0, 1e5, 1e8])
def test_bands(bd, length):
    """By the turns themselves there is nothing to round or to keep within."""
    r = bd.bdlm_rotary_init(128, True, 10000.0, bd.BDLM_ROTARY_BANDS, 8.0, length, 1.0, 4.0)
    own = 10000.0 ** (-np.arange(64) / 64)
    keep = np.interp(length * own / (2 * math.pi), [1.0, 4.0], [0.0, 1.0])
    want = own * (keep + (1 - keep) / 8)
    assert np.all(np.abs(frequencies(r) - want) <= 1e-12 * want + 1e-18)


@pytest.mark.parametrize("amplitude", [1e-300, 1e-50, 1e-46, 1e-39])
def test_an_amplitude_that_no_float_holds_is_refused(bd, amplitude):
    """It would be 0, and so would all results, or have few bits left."""
    with pytest.raises(bd.BdlmError) as e:
        bd.bdlm_rotary_init(64, False, 10000.0, amplitude=amplitude)
    assert e.value.status == bd.BDLM_ERR_INVALID
    for good in (1.2e-38, 0.5, 3e38):
        assert bd.bdlm_rotary_init(64, False, 10000.0, amplitude=good).amplitude == np.float32(good)
