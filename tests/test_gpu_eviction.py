"""Attention weights, eviction and the move of tokens, against 64-bit and plain forms."""
import numpy as np
import pytest

import cache_ref as R
import workloads as W
from gpu_util import bf16_tensor, dev, host

pytestmark = pytest.mark.gpu


def bits(t):
    import torch
    return host(t.view(torch.int16)).view(np.uint16)


@pytest.mark.parametrize("L,Hq,Hkv,lens", [
    (1, 16, 8, [0, 1, 127, 128, 129]), (4, 32, 8, [500, 17, 2048, 3000]), (5, 24, 8, [100, 1000]),
    (8, 32, 8, [700, 3]), (9, 32, 8, [300, 40]), (33, 16, 8, [260, 5]), (64, 32, 8, [4500, 64, 0]),
    (64, 16, 2, [400]), (64, 16, 1, [200, 900]), (17, 4, 4, [20000])])
@pytest.mark.parametrize("decay", [1.0, 0.0, 0.75])
def test_attention_weights(lib, L, Hq, Hkv, lens, decay):
    import torch
    rng = np.random.default_rng(L + Hq)
    B = len(lens)
    a = W.make_attention(rng, B, L, Hq, Hkv, 128, prefix_lens=np.array(lens), qkv_std=1.0)
    P = a.page_table_ref.shape[1]
    d = lib.attn_desc(B, L, Hq, Hkv, 128, P, a.k_ref.shape[0])
    q, k, t, n = bf16_tensor(a.q), bf16_tensor(a.k_ref), dev(a.page_table_ref), dev(a.prefix_lens)
    out = torch.empty((B, L, Hq, 128), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((B, L, Hq), device="cuda")
    lib.bdlm_tree_attention(d, q, k, bf16_tensor(a.v_ref), t, n, None, out, lse)
    w0 = rng.random((B, Hkv, P * 16)).astype(np.float32)
    w = dev(w0)
    lib.bdlm_attention_weights(d, q, k, t, n, lse, decay, w)
    torch.cuda.synchronize()
    assert lib.bdlm_device_error() == 0
    want, add, s1 = R.attention_weights(a.q, a.k_ref, a.page_table_ref, a.prefix_lens, host(lse), decay,
                                        w0, Hkv)
    # a term's exponent is off by the score's error and a few roundings of its size (|lse| and the
    # score below 2^7 in log2 units), 2^-22 for the exponential; sums of up to 1024 positive terms
    # and up to four launches add 2^-15 at most
    tol = add * (2 * R.score_error(s1) + 2.0 ** -15 + 3 * 2.0 ** -17) + 4 * 2.0 ** -24 * np.abs(want)
    got = host(w).astype(np.float64)
    assert np.all(np.abs(got - want) <= tol + 1e-30)
    for b in range(B):
        assert np.array_equal(host(w)[b, :, lens[b]:], w0[b, :, lens[b]:])


@pytest.mark.parametrize("L,Hq,Hkv", [(4, 16, 8), (5, 24, 2), (64, 32, 8)])
def test_weights_of_queries_left_out(lib, L, Hq, Hkv):
    """A query whose lse is +inf adds nothing, for few query rows and for many alike."""
    import torch
    rng = np.random.default_rng(L)
    a = W.make_attention(rng, 2, L, Hq, Hkv, 128, prefix_lens=np.array([300, 40]), qkv_std=1.0)
    P = a.page_table_ref.shape[1]
    d = lib.attn_desc(2, L, Hq, Hkv, 128, P, a.k_ref.shape[0])
    lse = (5 + rng.random((2, L, Hq))).astype(np.float32)
    lse[:, 0] = np.inf
    lse[1, :, 1] = np.inf
    lse[1, -1, -1] = 3.4e38   # as good as
    w0 = np.zeros((2, Hkv, P * 16), np.float32)
    w = dev(w0)
    lib.bdlm_attention_weights(d, bf16_tensor(a.q), bf16_tensor(a.k_ref), dev(a.page_table_ref),
                               dev(a.prefix_lens), dev(lse), 1.0, w)
    torch.cuda.synchronize()
    assert lib.bdlm_device_error() == 0
    want, add, s1 = R.attention_weights(a.q, a.k_ref, a.page_table_ref, a.prefix_lens, lse, 1.0, w0, Hkv)
    # as test_attention_weights
    tol = add * (2 * R.score_error(s1) + 2.0 ** -15 + 3 * 2.0 ** -17) + 4 * 2.0 ** -24 * np.abs(want)
    assert np.all(np.abs(host(w).astype(np.float64) - want) <= tol + 1e-30)


@pytest.mark.parametrize("L,Hq,Hkv", [(4, 16, 8), (16, 32, 8), (64, 16, 2)])
def test_weights_of_this_step_alone(lib, L, Hq, Hkv):
    """decay 0 reads nothing of what the weights held (rows up to 32, up to 256, two launches)."""
    import torch
    rng = np.random.default_rng(Hq)
    a = W.make_attention(rng, 2, L, Hq, Hkv, 128, prefix_lens=np.array([300, 40]), qkv_std=1.0)
    P = a.page_table_ref.shape[1]
    d = lib.attn_desc(2, L, Hq, Hkv, 128, P, a.k_ref.shape[0])
    lse = dev((5 + rng.random((2, L, Hq))).astype(np.float32))
    got = []
    for fill in (0.0, float("nan")):
        w = torch.full((2, Hkv, P * 16), fill, device="cuda")
        lib.bdlm_attention_weights(d, bf16_tensor(a.q), bf16_tensor(a.k_ref), dev(a.page_table_ref),
                                   dev(a.prefix_lens), lse, 0.0, w)
        torch.cuda.synchronize()
        got.append([host(w)[b, :, :n] for b, n in enumerate((300, 40))])
    assert all(np.array_equal(x, y) and np.all(x > 0) for x, y in zip(*got))


def test_weights_flag_bad_pages_and_lengths(lib):
    import torch
    rng = np.random.default_rng(2)
    a = W.make_attention(rng, 3, 4, 16, 8, 128, prefix_lens=np.array([200, 200, 200]))
    t, n = a.page_table_ref.copy(), a.prefix_lens.copy()
    t[0, 3] = -1
    n[1], n[2] = -1, 10 ** 6
    d = lib.attn_desc(3, 4, 16, 8, 128, t.shape[1], a.k_ref.shape[0])
    w = torch.full((3, 8, t.shape[1] * 16), 5.0, device="cuda")
    lib.bdlm_attention_weights(d, bf16_tensor(a.q), bf16_tensor(a.k_ref), dev(t), dev(n),
                               torch.full((3, 4, 16), 6.0, device="cuda"), 1.0, w)
    torch.cuda.synchronize()
    assert lib.bdlm_device_error() == lib.BDLM_DEVERR_PAGE | lib.BDLM_DEVERR_LENGTH
    w = host(w)
    assert np.all(w[0, :, 48:64] == 5.0) and np.all(w[0, :, :48] > 5.0) and np.all(w[0, :, 64:200] > 5.0)
    assert np.all(w[1:] == 5.0)


def cache(rng, lens, Hkv, max_tokens, extra):
    """A pool whose values name their slot, so that a wrong move shows."""
    B, cols = len(lens), (max_tokens + 15) // 16
    n = B * cols + extra
    perm = rng.permutation(n).astype(np.int32)
    k = rng.integers(0, 0x7F00, size=(n, 16, Hkv, 128)).astype(np.uint16)
    v = rng.integers(0, 0x7F00, size=(n, 16, Hkv, 128)).astype(np.uint16)
    return k, v, perm[:B * cols].reshape(B, cols).copy(), perm[B * cols:]


def plain_move(k, v, table, to, base, idx, counts, Hkv):
    k2, v2 = k.copy(), v.copy()
    for b in range(len(counts)):
        for h in range(Hkv):
            row = idx[b, h if idx.shape[1] > 1 else 0]
            for j in range(int(counts[b])):
                s, t = int(base[b]) + int(row[j]), int(base[b]) + j
                k2[to[b, t // 16], t % 16, h] = k[table[b, s // 16], s % 16, h]
                v2[to[b, t // 16], t % 16, h] = v[table[b, s // 16], s % 16, h]
    return k2, v2


def run_evict(lib, k, v, table, lens, w, keep, recent, to, in_place, stream=None):
    import torch
    B, Hkv = w.shape[:2]
    kd, vd, td, wd = bf16_tensor(k), bf16_tensor(v), dev(table), dev(w)
    to_d = td if in_place else dev(to)
    tw = wd if in_place else torch.full_like(wd, -3.0)
    kept = torch.full((B, Hkv, keep), -9, dtype=torch.int32, device="cuda")
    new = torch.full((B,), -9, dtype=torch.int32, device="cuda")
    d = lib.attn_desc(B, 1, Hkv, Hkv, 128, table.shape[1], k.shape[0])
    lib.bdlm_evict_kv(d, kd, vd, td, dev(lens), wd, keep, recent, to_d, tw, kept, new, stream=stream)
    torch.cuda.synchronize()
    return bits(kd), bits(vd), host(tw), host(kept), host(new)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("lens,keep,recent,kind", [
    ([1, 0, 5, 16], 4, 2, "random"), ([600, 100, 256, 257], 256, 32, "random"),
    ([600, 300], 100, 0, "random"), ([600, 300], 100, 100, "random"), ([50, 33], 1, 0, "random"),
    ([50, 33], 1, 1, "random"), ([700, 300, 40], 64, 5, "equal"), ([700, 300], 64, 5, "few"),
    ([3000, 2100], 1500, 64, "tail"), ([2000], 2000, 10, "random"), ([500], 499, 3, "random"),
    ([26000], 5000, 100, "random"), ([1100, 90], 80, 8, "odd"),
    # more lists than SMs, which move in a kernel of their own
    ([5 + 37 * i % 400 for i in range(70)], 150, 9, "random"), ([300] * 60, 200, 0, "tail")])
def test_eviction(lib, lens, keep, recent, kind, in_place):
    rng = np.random.default_rng(sum(lens) + keep)
    Hkv = 2 if max(lens) > 5000 else 3
    lens = np.array(lens, np.int32)
    k, v, table, free = cache(rng, lens, Hkv, max(int(lens.max()), keep), len(lens) * ((keep + 15) // 16))
    cols = table.shape[1]
    to = np.full((len(lens), cols), -1, np.int32)
    to[:, :(keep + 15) // 16] = free.reshape(len(lens), -1)
    w = rng.random((len(lens), Hkv, cols * 16)).astype(np.float32)
    if kind == "equal":
        w[:] = 0.25
    if kind == "few":
        w = rng.integers(0, 3, size=w.shape).astype(np.float32) - 1
        w[w == 0] = np.where(rng.random((w == 0).sum()) < 0.5, -0.0, 0.0)
    if kind == "tail":
        w = (rng.exponential(size=w.shape) ** 4).astype(np.float32)
    if kind == "odd":
        at = rng.random(w.shape)
        w[at < 0.1], w[(at > 0.1) & (at < 0.15)], w[at > 0.93] = np.nan, np.inf, -np.inf
    gk, gv, gw, kept, new = run_evict(lib, k, v, table, lens, w, keep, recent, to, in_place)
    assert lib.bdlm_device_error() == 0
    assert np.array_equal(new, np.minimum(lens, keep))
    want = np.full((len(lens), Hkv, keep), -1, np.int64)
    ww = w.copy() if in_place else np.full_like(w, -3.0)
    for b in range(len(lens)):
        for h in range(Hkv):
            r = R.evict(w[b, h], int(lens[b]), keep, recent)
            want[b, h, :len(r)] = r
            ww[b, h, :len(r)] = w[b, h, r]
    assert np.array_equal(kept, want)
    assert np.array_equal(gw, ww, equal_nan=True)
    k2, v2 = plain_move(k, v, table, table if in_place else to, np.zeros(len(lens), int), want, new, Hkv)
    assert np.array_equal(gk, k2) and np.array_equal(gv, v2)


@pytest.mark.parametrize("lens,keep", [([700, 90], 64), ([26000], 900)])
def test_eviction_of_weights_at_odd_addresses(lib, lens, keep):
    """Weights that start 4 bytes past 16, with zeros of both signs and NaN, keep their bits."""
    import torch
    rng = np.random.default_rng(keep)
    k, v, table, _ = cache(rng, lens, 2, max(lens), 0)
    B, stride = len(lens), table.shape[1] * 16
    w = rng.random((B, 2, stride)).astype(np.float32) * (rng.random((B, 2, stride)) < 0.05)
    w[:, :, ::7] *= -0.0
    w[:, 0, 3:9] = np.nan
    w[:, 0, 5:60].view(np.uint32)[...] |= np.uint32(1)
    flat = torch.zeros(w.size + 1, device="cuda")
    flat[1:] = dev(w).view(-1)
    wd = flat[1:].view(B, 2, stride)
    assert wd.data_ptr() % 16 == 4
    d = lib.attn_desc(B, 1, 2, 2, 128, table.shape[1], k.shape[0])
    kept = torch.empty((B, 2, keep), dtype=torch.int32, device="cuda")
    new = torch.empty((B,), dtype=torch.int32, device="cuda")
    tw, td = torch.full_like(wd, -3.0), dev(table)
    lib.bdlm_evict_kv(d, bf16_tensor(k), bf16_tensor(v), td, dev(np.array(lens, np.int32)), wd, keep, 5, td,
                      tw, kept, new)
    torch.cuda.synchronize()
    assert lib.bdlm_device_error() == 0
    for b, n in enumerate(lens):
        for h in range(2):
            want = R.evict(w[b, h], n, keep, 5)
            assert np.array_equal(host(kept)[b, h, :len(want)], want)
            assert np.array_equal(host(tw)[b, h, :len(want)].view(np.uint32), w[b, h][want].view(np.uint32))


def test_eviction_flags_bad_lengths_and_pages(lib):
    rng = np.random.default_rng(4)
    lens = np.array([300, -2, 10 ** 6], np.int32)
    k, v, table, _ = cache(rng, [300] * 3, 2, 300, 0)
    hole = table[0, 2]
    table[0, 2] = -1
    w = rng.random((3, 2, table.shape[1] * 16)).astype(np.float32)
    gk, gv, gw, kept, new = run_evict(lib, k, v, table, lens, w, 100, 4, table, True)
    assert lib.bdlm_device_error() == lib.BDLM_DEVERR_PAGE | lib.BDLM_DEVERR_LENGTH
    assert list(new) == [100, 0, 0] and np.all(kept[1:] == -1)
    assert np.array_equal(gk[hole], k[hole])
    assert np.array_equal(gk[table[1]], k[table[1]]) and np.array_equal(gw[1:], w[1:])


@pytest.mark.parametrize("heads", [1, 3])
@pytest.mark.parametrize("in_place", [False, True])
def test_compact(lib, heads, in_place):
    """The accepted path of a drafted tree: block positions after the prefix move up."""
    import torch
    rng = np.random.default_rng(6 + heads)
    B, Hkv, n_max = 5, 3, 150
    base = np.array([0, 7, 16, 100, 31], np.int32)
    counts = np.array([0, 1, 150, 64, 65], np.int32)
    k, v, table, free = cache(rng, [400] * B, Hkv, 400, B * 25)
    to = table if in_place else free.reshape(B, 25).copy()
    idx = np.sort(np.stack([[rng.permutation(250)[:n_max] for _ in range(heads)] for _ in range(B)]), -1)
    idx[3, 0, :64] = np.arange(64)                       # already in place
    idx = idx.astype(np.int32)
    kd, vd, td = bf16_tensor(k), bf16_tensor(v), dev(table)
    d = lib.attn_desc(B, 1, Hkv, Hkv, 128, table.shape[1], k.shape[0])
    lib.bdlm_compact_kv(d, kd, vd, td, dev(base), dev(idx), heads, n_max, dev(counts),
                        td if in_place else dev(to))
    torch.cuda.synchronize()
    assert lib.bdlm_device_error() == 0
    k2, v2 = plain_move(k, v, table, to, base, idx, counts, Hkv)
    assert np.array_equal(bits(kd), k2) and np.array_equal(bits(vd), v2)


@pytest.mark.parametrize("n_max", [1, 64, 513])
def test_compact_in_place_again_and_again(lib, n_max):
    """Every second, then every third token of long lists: each round's reads lie behind its writes."""
    import torch
    rng = np.random.default_rng(n_max)
    B, Hkv = 3, 4
    k, v, table, _ = cache(rng, [2000] * B, Hkv, 2000, 0)
    kd, vd, td = bf16_tensor(k), bf16_tensor(v), dev(table)
    d = lib.attn_desc(B, 1, Hkv, Hkv, 128, table.shape[1], k.shape[0])
    counts = np.array([n_max, n_max // 2, n_max], np.int32)
    for step in (2, 3):
        idx = np.tile((np.arange(n_max) * step + 1).astype(np.int32), (B, 1, 1))
        lib.bdlm_compact_kv(d, kd, vd, td, None, dev(idx), 1, n_max, dev(counts), td)
        k, v = plain_move(k, v, table, table, np.zeros(B, int), idx, counts, Hkv)
    torch.cuda.synchronize()
    assert lib.bdlm_device_error() == 0
    assert np.array_equal(bits(kd), k) and np.array_equal(bits(vd), v)


def test_compact_flags_bad_rows(lib):
    import torch
    rng = np.random.default_rng(7)
    k, v, table, _ = cache(rng, [64] * 2, 2, 64, 0)
    idx = np.array([[[-1, 3, 500]], [[1, 2, 3]]], np.int32)
    kd, vd, td = bf16_tensor(k), bf16_tensor(v), dev(table)
    d = lib.attn_desc(2, 1, 2, 2, 128, 4, k.shape[0])
    lib.bdlm_compact_kv(d, kd, vd, td, dev(np.array([10, -1], np.int32)), dev(idx), 1, 3,
                        dev(np.array([3, 3], np.int32)), td)
    torch.cuda.synchronize()
    assert lib.bdlm_device_error() == lib.BDLM_DEVERR_ROW | lib.BDLM_DEVERR_LENGTH
    k2 = k.copy()
    k2[table[0, 0], 11] = k[table[0, 0], 13]
    assert np.array_equal(bits(kd), k2)
