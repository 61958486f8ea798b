"""Attention over the 8-bit cache where one token has most of a row's weight and many others share the rest, as with a
first token that all queries attend to: the rest has to come out right, however long it is and however the lists are cut."""
import numpy as np
import pytest
from scipy.ndimage import maximum_filter1d

import step_ref as R
import workloads as W
from gpu_util import bf16_tensor, dev
from test_gpu_kv8 import f

pytestmark = pytest.mark.gpu

SCALE = 1 / np.sqrt(128)


def tolerance(q, k, codes, sv, p, out, few):
    """Of one KV head, q [rows, 128], k [n, 128], codes of V [n, 128], p [rows, n].  Derived from what is rounded:
    - scores: as step_ref.check_attention has it, with each row's own largest element;
    - a weight (p times its page's scale): two e4m3 parts of a float16 number, within 2^-8 + 2^-11 of itself, or with more
      than 32 rows that number, 2^-11;
    - small ones: at most 2^-23 of the largest weight that they are held next to, which lies within 896 tokens (two parts
      down to half of 2^-14, a largest one of 2^8), or 2^-32 of the row's largest (float16 down to half of 2^-24, 2^7);
    - sums in float32 (2^-14), the output in bf16."""
    a = np.abs(q)
    ds = (2.0 ** -17 * a.max(1, keepdims=True) * np.abs(k).sum(1).max() + (8 * 33 * 2.0 ** -23 + 2.0 ** -21) * (a @ np.abs(k).T).max(1, keepdims=True)) * SCALE
    w = p * sv
    A = w @ np.abs(codes)
    near = maximum_filter1d(w, 2 * 896 - 1, axis=1, mode="constant") if few else np.broadcast_to(w.max(1, keepdims=True), w.shape)
    floor = (2.0 ** -23 if few else 2.0 ** -32) * 1.01 * (near @ np.abs(codes))
    return (1.01 * ((2.0 ** -8 if few else 0) + 2.0 ** -11) + 2.0 ** -14 + np.expm1(2 * ds)) * A + floor + R.BF16 * 1.01 * np.abs(out)


def run(lib, B, L, Hq, Hkv, n, table, k, v, scales, q):
    """The same sequence B times: lists that one CTA has whole, and lists that are cut."""
    import torch
    d = lib.attn_desc(B, L, Hq, Hkv, 128, table.shape[0], k.shape[0])
    out = torch.full((B, L, Hq, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    lib.bdlm_attention_kv8(d, bf16_tensor(np.stack([q] * B)), dev(k), dev(v), dev(scales),
                           dev(np.stack([table] * B)), dev(np.full(B, n - L, np.int32)), out)
    assert lib.bdlm_device_error() == 0
    return f(out)


# 1, 8, 16, 32, 128 and 256 rows
@pytest.mark.parametrize("L,G", [(1, 1), (2, 4), (4, 4), (8, 4), (32, 4), (64, 4)])
@pytest.mark.parametrize("n,share", [(8192, 0.95), (32768, 0.9)])
@pytest.mark.parametrize("B", [1, 160])
def test_a_dominant_token(lib, L, G, n, share, B):
    """Token 5 has about `share` of the weight and a V of a twentieth of the others'."""
    rng = np.random.default_rng(n + L)
    Hkv, pages = 2, n // R.P
    table = rng.permutation(pages).astype(np.int32)
    k = R.encode(np.clip(rng.normal(0, 110, (pages, Hkv, R.P, 128)), -448, 448))
    v = R.encode(np.clip(rng.normal(55, 110, (pages, Hkv, R.P, 128)), -448, 448))
    scales = (2.0 ** rng.uniform(-1, 1, (pages, Hkv, 2)) / 110).astype(np.float32)
    q = W._normal_bf16(rng, (L, G * Hkv, 128), 1.0)
    q[..., 0] = W.f32_to_bf16_bits(np.array([8.0], np.float32))[0]
    k[..., 0] = 0
    page = table[0]
    k[page] = 0
    k[page, :, 5, 0] = 126                              # 448
    v[page, :, 5] = R.encode(rng.normal(0, 5.5, (Hkv, 128)))
    scales[page, :, 1] = 1 / 110
    flat = lambda x, g: R.E4M3[x[table, g]].reshape(n, 128)
    per_token = lambda g, c: np.repeat(scales[table, g, c].astype(np.float64), R.P)
    refs = []
    for g in range(Hkv):
        qq = R.f64(q[:, g * G:(g + 1) * G]).reshape(L * G, 128)
        rest = np.log(np.mean(np.sum(np.exp(qq @ (flat(k, g) * per_token(g, 0)[:, None]).T * SCALE), axis=1)))
        scales[page, g, 0] = (rest + np.log(share / (1 - share))) / (8 * 448 * SCALE)
        kk = flat(k, g) * per_token(g, 0)[:, None]
        x = qq @ kk.T * SCALE
        p = np.exp(x - x.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
        assert abs(np.median(p[:, 5]) - share) < 0.1
        out = (p * per_token(g, 1)) @ flat(v, g)
        refs.append((out, tolerance(qq, kk, flat(v, g), per_token(g, 1), p, out, L * G <= 32)))
    got = run(lib, B, L, G * Hkv, Hkv, n, table, k, v, scales, q)
    for g, (out, tol) in enumerate(refs):
        excess = np.abs(got[:, :, g * G:(g + 1) * G].reshape(B, L * G, 128) - out) - tol
        assert excess.max() <= 0, (g, excess.max(), np.abs(out).mean())


@pytest.mark.parametrize("L,G", [(1, 8), (4, 4), (8, 4), (32, 4), (64, 4)])
@pytest.mark.parametrize("at", [0, 70000, 131071])
def test_a_flat_tail(lib, L, G, at):
    """131072 tokens, all but one of them of the same score, 1.4 * 2^-22 of that one's weight: what one loses all lose."""
    n, Hkv, B = 131072, 2, 160
    rng = np.random.default_rng(L)
    # page 0 is all the tokens' but those of page 1, which has the one
    table = np.zeros(n // R.P, np.int32)
    table[at // R.P] = 1
    k = np.zeros((2, Hkv, R.P, 128), np.uint8)
    v = R.encode(np.clip(rng.normal(55, 110, (2, Hkv, R.P, 128)), -448, 448))
    v[1, :, at % R.P] = 0
    k[1, :, at % R.P, 0] = 126
    ratio = 1.4 * 2.0 ** -22
    scales = np.full((2, Hkv, 2), 1 / 128, np.float32)
    scales[1, :, 0] = -np.log(ratio) / (8 * 448 * SCALE)
    q = np.zeros((L, G * Hkv, 128), np.float32)
    q[..., 0] = 8
    q = W.f32_to_bf16_bits(q)
    got = run(lib, B, L, G * Hkv, Hkv, n, table, k, v, scales, q)
    for g in range(Hkv):
        codes, few = R.E4M3[v[:, g]].reshape(2 * R.P, 128), L * G <= 32
        count = np.repeat([float(n // R.P - 1), 1.0], R.P)
        p = np.where(np.arange(2 * R.P) == R.P + at % R.P, 1.0, np.exp(-8 * 448 * SCALE * float(scales[1, g, 0])))
        p /= (p * count).sum()
        out = (p * count / 128) @ codes
        A = (p * count / 128) @ np.abs(codes)
        near = np.minimum(count, 2 * 896 / R.P) if few else count         # tokens that the floor can meet
        floor = (2.0 ** -23 if few else 2.0 ** -32) * 1.01 * p.max() / 128 * (near @ np.abs(codes))
        ds = 16 * (8 * 33 * 2.0 ** -23 + 2.0 ** -21)                      # (q has one element, a power of two)
        tol = (1.01 * ((2.0 ** -8 if few else 0) + 2.0 ** -11) + 2.0 ** -14 + np.expm1(2 * ds)) * A + floor + R.BF16 * 1.01 * np.abs(out)
        excess = np.abs(got[:, :, g * G:(g + 1) * G].reshape(-1, 128) - out) - tol
        assert excess.max() <= 0, (g, excess.max(), np.abs(out).mean())
