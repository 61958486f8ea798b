"""Attention over the 8-bit cache against a bound of each output's own: what its weights, its queries and the tokens that they
are held next to allow, and no token's weight lost on another's account."""
import numpy as np
import pytest

import step_ref as R
import workloads as W
from test_gpu_kv8 import Cache, attend, f
from test_gpu_kv8_tails import SCALE, tolerance

pytestmark = pytest.mark.gpu


def check(c, q, got, L, Hq, Hkv, scale=SCALE):
    G = Hq // Hkv
    for b, n in enumerate(c.lens):
        ids = c.table[b, :(n + 15) // 16]
        for g in range(Hkv):
            kk, codes = (R.E4M3[t[ids, g]].reshape(-1, 128)[:n] for t in (c.k, c.v))
            sk, sv = (np.repeat(c.scales[ids, g, i].astype(np.float64), 16)[:n] for i in range(2))
            kk = kk * sk[:, None] * (scale / SCALE)
            qq = R.f64(q[b, :, g * G:(g + 1) * G]).reshape(-1, 128)
            x = qq @ kk.T * SCALE
            p = np.exp(x - x.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            out = (p * sv) @ codes
            excess = np.abs(got[b, :, g * G:(g + 1) * G].reshape(-1, 128) - out) - tolerance(qq, kk, codes, sv, p, out, L * G <= 32)
            assert excess.max() <= 0, (b, g, excess.max())


@pytest.mark.parametrize("L,Hq,Hkv,lens", [
    (1, 1, 1, [0]), (1, 32, 4, [1, 127, 2000, 20000]), (4, 16, 8, [0, 11, 13, 125, 700]), (3, 5, 5, [60, 3000]), (5, 24, 4, [33, 9000]),
    (8, 16, 4, [120, 1801]), (2, 32, 2, [0, 77, 900]), (7, 28, 7, [129]), (16, 8, 4, [5000, 112]), (33, 4, 2, [95, 500]), (64, 4, 2, [0, 64, 999]),
    (17, 24, 3, [7, 3333]), (64, 16, 4, [5000, 33]), (64, 3, 1, [192, 4100]), (40, 16, 1, [257, 600]), (64, 16, 1, [0, 130]),
])
@pytest.mark.parametrize("spread", [0.5, 6.0])
def test_every_output_within_its_own_bound(lib, L, Hq, Hkv, lens, spread):
    rng = np.random.default_rng(L * 100 + Hq)
    c = Cache(rng, np.array(lens) + L, Hkv, spread=spread)
    c.scales[:, :, 0] = 2.0 ** rng.uniform(-1, 1, c.scales.shape[:2]) / 110
    q = W._normal_bf16(rng, (len(lens), L, Hq, 128), 1.0)
    check(c, q, f(attend(lib, c, q, L, Hq, Hkv)), L, Hq, Hkv)
    assert lib.bdlm_device_error() == 0


@pytest.mark.parametrize("L,Hq,Hkv", [(1, 8, 8), (4, 32, 8), (8, 16, 4), (32, 8, 2), (64, 8, 2)])
@pytest.mark.parametrize("rising", [False, True])
def test_maxima_that_move_all_along(lib, L, Hq, Hkv, rising):
    """Scores that grow, or fall, by some hundred powers of two over the tokens: every chunk is far from the last."""
    rng = np.random.default_rng(L)
    n = 6000
    c = Cache(rng, np.array([n, 1000]) + L, Hkv)
    q = np.abs(rng.normal(size=(2, L, Hq, 128))).astype(np.float32)
    q[..., 0] = 4.0
    q = W.f32_to_bf16_bits(q)
    steps = np.linspace(-448, 448, c.cols) * (1 if rising else -1)
    for b in range(2):
        for col, page in enumerate(c.table[b, :(c.lens[b] + 15) // 16]):
            c.k[page, :, :, 0] = R.encode(np.full(16, steps[col]))
            c.scales[page, :, 0] = 0.5
            c.k[page, :, :, 1:] = R.encode(rng.normal(0, 0.05, (Hkv, 16, 127)))
    check(c, q, f(attend(lib, c, q, L, Hq, Hkv)), L, Hq, Hkv)
