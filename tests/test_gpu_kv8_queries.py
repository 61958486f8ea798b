"""Attention over the 8-bit cache for queries of zeros, of tiny values and of very different sizes."""
import numpy as np
import pytest

import step_ref as R
import workloads as W
from test_gpu_kv8 import Cache, attend, f
from test_gpu_kv8_tails import SCALE, tolerance

pytestmark = pytest.mark.gpu

# query rows per KV head: 1, 8, 16, 32, 128, 255, 256
ROWS = [(1, 2, 2), (4, 4, 2), (4, 8, 2), (8, 8, 2), (32, 8, 2), (64, 24, 6), (64, 8, 2)]


@pytest.mark.parametrize("L,Hq,Hkv", ROWS)
@pytest.mark.parametrize("size", [0.0, 2.0 ** -120])
def test_queries_of_zeros(lib, L, Hq, Hkv, size):
    """All queries of a sequence and KV head zero, or next to it: every token weighs the same, whatever pages the last
    tile of 128 tokens lacks.  (Factors of 2^-110 and of a missing page's 2^-40 met as 0, and 0 times -inf.)"""
    lens = [n for n in (65, 128, 129, 144, 240, 241, 16, 1000) if n >= L]
    rng = np.random.default_rng(L + Hq)
    c = Cache(rng, np.array(lens), Hkv)
    c.scales[c.table[0, 0]] = 2.0 ** -40                  # a page of zeros, as the write makes it
    c.k[c.table[0, 0]] = c.v[c.table[0, 0]] = 0
    q = W._normal_bf16(rng, (len(lens), L, Hq, 128), 1.0)
    q[:, :, :Hq // Hkv] = W.f32_to_bf16_bits(np.full(128, size, np.float32))
    q[1] = q[0, 0, 0]
    out = attend(lib, c, q, L, Hq, Hkv)
    R.check_attention(f(out), R.attention_kv8(q, c.k, c.v, c.scales, c.table, c.lens - L, Hkv))
    assert lib.bdlm_device_error() == 0


@pytest.mark.parametrize("L,Hq,Hkv", ROWS)
def test_a_tiny_softmax_scale(lib, L, Hq, Hkv):
    """A scale next to zero does the same to any queries, over bad pages too."""
    rng = np.random.default_rng(L + Hq + 1)
    c = Cache(rng, np.array([70, 333, 1200]) + L, Hkv)
    q = W._normal_bf16(rng, (3, L, Hq, 128), 1.0)
    c.table[1, 2], c.table[2, 7] = -1, c.pages
    out = attend(lib, c, q, L, Hq, Hkv, scale=1e-36)
    R.check_attention(f(out), R.attention_kv8(q, c.k, c.v, c.scales, c.table, c.lens - L, Hkv, scale=1e-36))
    assert lib.bdlm_device_error() == lib.BDLM_DEVERR_PAGE


@pytest.mark.parametrize("L,Hq,Hkv", [(2, 8, 2), (4, 8, 2), (8, 8, 2), (32, 8, 2), (33, 24, 6), (64, 16, 4), (40, 32, 2)])
@pytest.mark.parametrize("huge", [3000.0, 1e30, np.inf, np.nan])
def test_a_row_keeps_out_of_the_others(lib, L, Hq, Hkv, huge):
    """Rows that share a KV head, one or all heads of a position with values far from the others' (a padded slot's, say),
    others far smaller: each row comes out as if it were alone."""
    rng = np.random.default_rng(L * Hq)
    G, lens = Hq // Hkv, np.array([50, 777, 2100])
    c = Cache(rng, lens + L, Hkv)
    x = rng.normal(size=(3, L, Hq, 128)).astype(np.float32)
    x[:, :, 1] *= 2.0 ** -6
    x[:, -1] *= huge
    x[0, 0, 0, 3] = huge
    q = W.f32_to_bf16_bits(x)
    x = R.f64(q)
    apart = (~np.isfinite(x) | (np.abs(x) > 100)).any(-1)
    assert apart.any() and not apart.all()
    got = f(attend(lib, c, q, L, Hq, Hkv))
    for b, n in enumerate(c.lens):
        ids = c.table[b, :(n + 15) // 16]
        for g in range(Hkv):
            rows = ~apart[b, :, g * G:(g + 1) * G].reshape(-1)
            if not rows.any():
                continue
            kk, codes = (R.E4M3[t[ids, g]].reshape(-1, 128)[:n] for t in (c.k, c.v))
            sk, sv = (np.repeat(c.scales[ids, g, i].astype(np.float64), 16)[:n] for i in range(2))
            kk = kk * sk[:, None]
            qq = x[b, :, g * G:(g + 1) * G].reshape(-1, 128)[rows]
            p = np.exp(qq @ kk.T * SCALE)
            p /= p.sum(1, keepdims=True)
            out = (p * sv) @ codes
            excess = np.abs(got[b, :, g * G:(g + 1) * G].reshape(-1, 128)[rows] - out) - tolerance(qq, kk, codes, sv, p, out, L * G <= 32)
            assert excess.max() <= 0, (b, g, excess.max())


@pytest.mark.parametrize("L,Hq,Hkv", ROWS)
def test_the_largest_queries(lib, L, Hq, Hkv):
    """Elements up to the largest bf16, brought back by a small softmax scale."""
    rng = np.random.default_rng(L + Hq + 2)
    c = Cache(rng, np.array([300, 1000]) + L, Hkv)
    x = rng.uniform(-1, 1, (2, L, Hq, 128)) * 3.3895e38
    x[..., 5] = 3.3895e38
    q = W.f32_to_bf16_bits(x.astype(np.float32))
    assert np.isfinite(R.f64(q)).all() and R.f64(q).max() > 1.99 * 2.0 ** 127
    out = f(attend(lib, c, q, L, Hq, Hkv, scale=1e-39))
    small = W.f32_to_bf16_bits((R.f64(q) * 2.0 ** -128).astype(np.float32))
    scale = float(np.float32(1e-39)) * 2.0 ** 128
    for b, n in enumerate(c.lens):
        ids = c.table[b, :(n + 15) // 16]
        for g in range(Hkv):
            kk, codes = (R.E4M3[t[ids, g]].reshape(-1, 128)[:n] for t in (c.k, c.v))
            sk, sv = (np.repeat(c.scales[ids, g, i].astype(np.float64), 16)[:n] for i in range(2))
            kk = kk * sk[:, None] * (scale / SCALE)
            G = Hq // Hkv
            qq = R.f64(small[b, :, g * G:(g + 1) * G]).reshape(-1, 128)
            p = np.exp(qq @ kk.T * SCALE)
            p /= p.sum(1, keepdims=True)
            want = (p * sv) @ codes
            excess = np.abs(out[b, :, g * G:(g + 1) * G].reshape(-1, 128) - want) - tolerance(qq, kk, codes, sv, p, want, L * G <= 32)
            assert excess.max() <= 0, (b, g, excess.max())
