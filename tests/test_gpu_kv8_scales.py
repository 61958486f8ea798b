"""Attention over the 8-bit cache with page scales as far apart as they may be, and past that."""
import numpy as np
import pytest

import step_ref as R
import workloads as W
from test_gpu_kv8 import Cache, attend, f
from test_gpu_kv8_tails import SCALE, tolerance

pytestmark = pytest.mark.gpu

ROWS = [(1, 2, 2), (4, 8, 2), (8, 8, 2), (32, 8, 2), (64, 8, 2)]


@pytest.mark.parametrize("L,Hq,Hkv", ROWS)
@pytest.mark.parametrize("far", [6, 12, 20, 33, 46])
def test_a_page_far_above_the_others(lib, L, Hq, Hkv, far):
    """One page's V is 2^far times the others', with zeros in some dims: there the others' sums show, down to 2^-47 of the
    largest weight (2^-32 with more than 32 rows)."""
    rng = np.random.default_rng(far + L)
    G, lens = Hq // Hkv, np.array([1500, 90, 3000])
    c = Cache(rng, lens + L, Hkv)
    pages = [c.table[0, 3], c.table[1, 5], c.table[2, 180]]
    c.scales[:, :, 1] = 2.0 ** rng.uniform(-37, -36, c.scales.shape[:2])
    c.scales[pages, :, 1] *= 2.0 ** far
    c.v[pages, :, :, :40] = 0
    q = W._normal_bf16(rng, (3, L, Hq, 128), 1.0)
    got = f(attend(lib, c, q, L, Hq, Hkv))
    few = L * G <= 32
    for b, n in enumerate(c.lens):
        ids = c.table[b, :(n + 15) // 16]
        for g in range(Hkv):
            kk, codes = (R.E4M3[t[ids, g]].reshape(-1, 128)[:n] for t in (c.k, c.v))
            sk, sv = (np.repeat(c.scales[ids, g, i].astype(np.float64), 16)[:n] for i in range(2))
            kk = kk * sk[:, None]
            qq = R.f64(q[b, :, g * G:(g + 1) * G]).reshape(-1, 128)
            p = np.exp(qq @ kk.T * SCALE)
            p /= p.sum(1, keepdims=True)
            out = (p * sv) @ codes
            tol = tolerance(qq, kk, codes, sv, p, out, few)
            if few:
                tol = tol + 2.0 ** -47 * 1.01 * (p * sv).max(1, keepdims=True) * np.abs(codes).sum(0)
            excess = np.abs(got[b, :, g * G:(g + 1) * G].reshape(-1, 128) - out) - tol
            assert excess.max() <= 0, (b, g, excess.max())
    assert lib.bdlm_device_error() == 0


@pytest.mark.parametrize("L,Hq,Hkv", ROWS)
def test_scales_outside_their_range(lib, L, Hq, Hkv):
    """Below 2^-40 and NaN count as 2^-40, above 2^40 as that: the same bits as with those."""
    rng = np.random.default_rng(L)
    c = Cache(rng, np.array([300, 2000]) + L, Hkv)
    q = W._normal_bf16(rng, (2, L, Hq, 128), 1.0)
    pages = c.table[0, :5]
    c.scales[pages, :, 0] = [[x] * Hkv for x in (0.0, -1.0, np.nan, 1e-30, -np.inf)]
    c.scales[c.table[1, :4], :, 1] = [[x] * Hkv for x in (2.0 ** -41, np.nan, -3.0, 0.0)]
    c.scales[c.table[1, 50], :, 1] = np.inf
    got = f(attend(lib, c, q, L, Hq, Hkv))
    c.scales = np.clip(np.nan_to_num(c.scales, nan=0.0), 2.0 ** -40, 2.0 ** 40).astype(np.float32)
    want = f(attend(lib, c, q, L, Hq, Hkv))
    assert np.all(np.isfinite(got)) and np.array_equal(got, want)
    assert lib.bdlm_device_error() == 0
