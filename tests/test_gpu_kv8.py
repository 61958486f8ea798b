"""The 8-bit cache: its writes, and attention over it, against plain 64-bit forms."""
import numpy as np
import pytest

import step_ref as R
import workloads as W
from gpu_util import bf16_tensor, dev, host

pytestmark = pytest.mark.gpu


def f(t):
    return host(t.float()).astype(np.float64)


class Cache:
    """A pool with a shuffled table; unused pages and slots hold NaN codes."""

    def __init__(self, rng, lens, Hkv, spread=2.0, spare=3, extra_cols=1):
        B = len(lens)
        self.lens = np.asarray(lens, np.int32)
        need = (self.lens + R.P - 1) // R.P
        self.cols = int(need.max()) + extra_cols
        n = int(need.sum()) + spare
        ids = rng.permutation(n)
        self.table = np.full((B, self.cols), -1, np.int32)
        self.k, self.v = (np.full((n, Hkv, R.P, R.D), 127, np.uint8) for _ in range(2))
        # scales that are no powers of two, from page to page and head to head
        self.scales = (2.0 ** rng.uniform(-spread, spread, (n, Hkv, 2)) / 110).astype(np.float32)
        at = 0
        for b in range(B):
            for col in range(need[b]):
                page = ids[at]
                at += 1
                self.table[b, col] = page
                live = min(R.P, self.lens[b] - col * R.P)
                for x in (self.k, self.v):
                    x[page, :, :live] = R.encode(np.clip(rng.normal(0, 110, (Hkv, live, R.D)), -448, 448))
        self.pages = n

    def dev(self):
        return dev(self.k), dev(self.v), dev(self.scales), dev(self.table)


def attend(lib, c, q, L, Hq, Hkv, out=None, scale=0.0, stream=None):
    import torch
    B = len(c.lens)
    d = lib.attn_desc(B, L, Hq, Hkv, 128, c.cols, c.pages, sm_scale=scale)
    k, v, s, t = c.dev()
    out = torch.full((B, L, Hq, 128), float("nan"), dtype=torch.bfloat16, device="cuda") if out is None else out
    lib.bdlm_attention_kv8(d, bf16_tensor(q), k, v, s, t, dev(c.lens - L), out, stream=stream)
    torch.cuda.synchronize()
    return out


# query rows per KV head 1 to 1024, prefixes of no token to several tiles, last pages of every fill
@pytest.mark.parametrize("L,Hq,Hkv,lens", [
    (1, 1, 1, [0]), (1, 8, 8, [0, 15, 16]), (1, 32, 4, [1, 127, 2000]), (4, 16, 8, [0, 1, 11, 12, 13, 124, 125, 700]),
    (4, 32, 8, [1500, 895, 896, 897, 891, 892]), (3, 5, 5, [60, 3000]), (5, 24, 4, [33, 1000]), (8, 16, 4, [120, 121, 1800]),
    (2, 32, 2, [0, 77, 900]), (7, 28, 7, [129]), (16, 16, 4, [0, 112, 240, 1111]), (33, 4, 2, [95, 500]),
    (64, 4, 2, [0, 64, 999]), (17, 24, 3, [7, 3333]), (32, 32, 8, [3100, 0]), (64, 16, 4, [5000, 33]),
    (64, 3, 1, [192, 4100]), (64, 10, 2, [65]), (40, 16, 1, [257, 600]), (64, 16, 1, [0, 130]),
])
def test_attention(lib, L, Hq, Hkv, lens):
    rng = np.random.default_rng(L * 1000 + Hq)
    c = Cache(rng, np.array(lens) + L, Hkv)
    q = W._normal_bf16(rng, (len(lens), L, Hq, 128), 1.0)
    out = attend(lib, c, q, L, Hq, Hkv)
    R.check_attention(f(out), R.attention_kv8(q, c.k, c.v, c.scales, c.table, c.lens - L, Hkv))
    assert lib.bdlm_device_error() == 0


@pytest.mark.parametrize("L,Hq,Hkv", [(1, 4, 2), (4, 32, 8), (12, 16, 8), (16, 16, 4), (64, 8, 4), (64, 16, 4)])
def test_attention_of_sharp_scores(lib, L, Hq, Hkv):
    """Large queries and scales far apart: one or two tokens take nearly all of a row's weight."""
    rng = np.random.default_rng(5)
    c = Cache(rng, np.array([2100, 40]) + L, Hkv, spread=5.0)
    q = W._normal_bf16(rng, (2, L, Hq, 128), 6.0)
    ref = R.attention_kv8(q, c.k, c.v, c.scales, c.table, c.lens - L, Hkv, scale=0.25)
    R.check_attention(f(attend(lib, c, q, L, Hq, Hkv, scale=0.25)), ref)


@pytest.mark.parametrize("L,Hq,Hkv", [(4, 8, 2), (64, 8, 2)])
def test_attention_of_extreme_scales(lib, L, Hq, Hkv):
    """V pages of 2^-40 (all zeros) and of 2^20 times the others, weights mostly on the zeros; heads of
    queries of very different magnitudes, one of zeros."""
    rng = np.random.default_rng(6)
    c = Cache(rng, np.array([400, 70]) + L, Hkv)
    for page in c.table[0, :4]:
        c.v[page] = 0
        c.scales[page, :, 1] = 2.0 ** -40
    c.scales[c.table[0, 9], :, 1] *= 2.0 ** 12
    c.scales[c.table[1, 0], :, 1] = 2.0 ** -30
    q = W._normal_bf16(rng, (2, L, Hq, 128), 1.0)
    q[:, :, 0] = 0
    q[:, :, 1] = W._normal_bf16(rng, (2, L, 128), 2.0 ** -12)
    R.check_attention(f(attend(lib, c, q, L, Hq, Hkv)), R.attention_kv8(q, c.k, c.v, c.scales, c.table, c.lens - L, Hkv))


@pytest.mark.parametrize("L,Hq,Hkv", [(4, 8, 2), (8, 8, 2), (32, 8, 2), (64, 16, 4)])
def test_attention_of_bad_pages_and_lengths(lib, L, Hq, Hkv):
    """A bad page reads as zeros; a length that does not fit is flagged; neither touches its neighbours."""
    import torch
    rng = np.random.default_rng(7)
    c = Cache(rng, np.array([300, 300, 300]) + L, Hkv, extra_cols=0)
    q = W._normal_bf16(rng, (3, L, Hq, 128), 1.0)
    c.table[0, 2], c.table[0, 5] = -1, c.pages
    out = attend(lib, c, q, L, Hq, Hkv)
    assert lib.bdlm_device_error() == lib.BDLM_DEVERR_PAGE
    R.check_attention(f(out), R.attention_kv8(q, c.k, c.v, c.scales, c.table, c.lens - L, Hkv))
    good = f(out)
    c.lens = c.lens.copy()
    c.lens[0] = c.cols * 16 + L
    out = attend(lib, c, q, L, Hq, Hkv)
    assert lib.bdlm_device_error() & lib.BDLM_DEVERR_LENGTH
    assert np.array_equal(f(out)[1:], good[1:])


def test_attention_repeats_and_streams(lib):
    """The same bits every time, on another stream, and from a captured graph over new inputs."""
    import torch
    rng = np.random.default_rng(8)
    L, Hq, Hkv = 4, 32, 8
    c = Cache(rng, np.array([3000, 17, 900]) + L, Hkv)
    q = W._normal_bf16(rng, (3, L, Hq, 128), 1.0)
    first = host(attend(lib, c, q, L, Hq, Hkv).view(torch.int16))
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        again = attend(lib, c, q, L, Hq, Hkv)
    assert np.array_equal(first, host(again.view(torch.int16)))
    d = lib.attn_desc(3, L, Hq, Hkv, 128, c.cols, c.pages)
    (k, v, sc, t), qd, n = c.dev(), bf16_tensor(q), dev(c.lens - L)
    out = torch.zeros((3, L, Hq, 128), dtype=torch.bfloat16, device="cuda")
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        lib.bdlm_attention_kv8(d, qd, k, v, sc, t, n, out)
    g.replay()
    torch.cuda.synchronize()
    assert np.array_equal(first, host(out.view(torch.int16)))
    q2 = W._normal_bf16(rng, (3, L, Hq, 128), 1.0)
    qd.copy_(bf16_tensor(q2))
    n.copy_(dev(np.array([2000, 3, 900], np.int32)))
    g.replay()
    torch.cuda.synchronize()
    R.check_attention(f(out), R.attention_kv8(q2, c.k, c.v, c.scales, c.table, np.array([2000, 3, 900]), Hkv))


@pytest.mark.parametrize("n,Hkv,lens", [(1, 1, [0]), (1, 8, [0, 1, 15, 16, 31]), (4, 8, [0, 3, 13, 14, 12, 160]), (16, 3, [0, 1, 16]),
                                        (33, 2, [0, 5, 31]), (300, 8, [0, 100, 7])])
@pytest.mark.parametrize("ragged", [False, True])
def test_write(lib, n, Hkv, lens, ragged):
    rng = np.random.default_rng(n * 10 + Hkv)
    lens = np.array(lens, np.int32)
    c = Cache(rng, lens + n, Hkv)
    c.scales[:] = 2.0 ** rng.integers(-9, 3, c.scales.shape)      # some of them power of two, then not
    c.scales[::2] *= np.float32(1.37)
    first, rows = None, len(lens) * n
    if ragged:
        counts = rng.integers(0, n + 1, len(lens))
        counts[rng.integers(len(lens))] = n
        first = np.concatenate(([0], np.cumsum(counts))).astype(np.int32)
        rows = int(first[-1])
    new = [W._normal_bf16(rng, (max(rows, 1), Hkv, 128), s) for s in (3.0, 0.02)]
    new[0][:, 0] = W._normal_bf16(rng, (max(rows, 1), 128), 1e-6)
    want = R.write_kv8(n, first, *new, c.k, c.v, c.scales, c.table, lens)
    d = lib.attn_desc(len(lens), 1, Hkv, Hkv, 128, c.cols, c.pages)
    k, v, s, t = c.dev()
    lib.bdlm_write_kv8(d, n, None if first is None else dev(first), rows, bf16_tensor(new[0]), bf16_tensor(new[1]), k, v, s, t, dev(lens))
    assert np.array_equal(host(s), want[2])
    assert R.same_codes(host(k), want[0]) and R.same_codes(host(v), want[1])
    assert lib.bdlm_device_error() == 0


def test_write_of_special_values(lib):
    """Zeros of both signs, values at the scale's borders, ties, infinities, NaN, the largest and smallest bf16."""
    Hkv, n = 6, 16
    x = np.zeros((n, Hkv, 128), np.float32)
    x[3, 0, 5] = -0.0
    x[:, 1, 0] = 448.0                                        # exactly the scale 1
    x[:, 1, 1:9] = [1.0625, 1.1875, 2.0 ** -9, 2.0 ** -10, 1.5 * 2.0 ** -9, 2.0 ** -11, -1.0625, 0.0]
    x[0, 2, 0], x[1, 2, 1], x[2, 2, 2] = 450.0, 448.0, 3.0    # just past it: the next scale
    x[0, 3, 0], x[0, 3, 1], x[1, 3, 0] = np.inf, -np.inf, 1.0
    x[0, 4, 0], x[1, 4, 1] = np.nan, 0.75
    x[0, 5, 0], x[0, 5, 1], x[0, 5, 2] = 3e38, 1e-38, -1.0
    bits = W.f32_to_bf16_bits(x)
    rng = np.random.default_rng(1)
    c = Cache(rng, [16], Hkv)
    want = R.write_kv8(n, None, bits, bits, c.k, c.v, c.scales, c.table, np.zeros(1, np.int32))
    d = lib.attn_desc(1, 1, Hkv, Hkv, 128, c.cols, c.pages)
    k, v, s, t = c.dev()
    z = dev(np.zeros(1, np.int32))
    lib.bdlm_write_kv8(d, n, None, 0, bf16_tensor(bits), bf16_tensor(bits), k, v, s, t, z)
    assert np.array_equal(host(s), want[2]) and R.same_codes(host(k), want[0]) and R.same_codes(host(v), want[1])
    page = c.table[0, 0]
    assert want[2][page, 0, 0] == 2.0 ** -40 and want[2][page, 1, 0] == 1.0 and want[2][page, 2, 0] == 2.0


def test_write_refuses_bad_rows_on_the_device(lib):
    """Bad page ids, lengths and row lists skip what they concern, and nothing else."""
    rng = np.random.default_rng(3)
    Hkv, n = 2, 20
    c = Cache(rng, np.full(4, 60), Hkv, extra_cols=0)
    d = lib.attn_desc(4, 1, Hkv, Hkv, 128, c.cols, c.pages)
    new = W._normal_bf16(rng, (4 * n, Hkv, 128), 1.0)
    x = bf16_tensor(new)

    def call(table, lens, first, rows=4 * n):
        k, v, s, _ = c.dev()
        lib.bdlm_write_kv8(d, n, None if first is None else dev(np.array(first, np.int32)), rows, x, x, k, v, s, dev(table), dev(lens))
        return host(k), host(v), host(s), lib.bdlm_device_error()

    lens = np.array([40, 0, 30, 20], np.int32)
    table = c.table.copy()
    table[1, 0], table[2, 2] = c.pages, -5
    k, v, s, err = call(table, lens, None)
    want = R.write_kv8(n, None, new, new, c.k, c.v, c.scales, c.table, lens)
    skipped = [c.table[1, 0], c.table[2, 2]]
    for got, w, was in ((k, want[0], c.k), (v, want[1], c.v)):
        w = w.copy()
        w[skipped] = was[skipped]
        assert R.same_codes(got, w)
    assert err == lib.BDLM_DEVERR_PAGE
    for bad, bit in (([-1, 45, 2 ** 31 - 1, 60], lib.BDLM_DEVERR_LENGTH),):
        k, v, s, err = call(c.table, np.array(bad, np.int32), None)
        assert err == bit and np.array_equal(k, c.k) and np.array_equal(v, c.v) and np.array_equal(s, c.scales)
    for first in ([5, 4, 3, 2, 1], [-3, -2, -1, -1, -1], [81, 90, 95, 99, 100], [0, 21, 42, 63, 84], [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1, 2 ** 31 - 1, -1]):
        k, v, s, err = call(c.table, np.zeros(4, np.int32), first)
        assert err & lib.BDLM_DEVERR_ROW, first


def test_blocks_written_again_and_again(lib):
    """A block's steps: each writes the block's new values over the last step's, the tokens before it stay."""
    import torch
    rng = np.random.default_rng(9)
    Hkv, n = 4, 4
    lens = np.array([13, 30, 45], np.int32)
    c = Cache(rng, lens + n, Hkv)
    c.scales[:] = 2.0 ** rng.integers(-8, -4, c.scales.shape)
    d = lib.attn_desc(3, n, Hkv, Hkv, 128, c.cols, c.pages)
    k, v, s, t = c.dev()
    wk, wv, ws = c.k, c.v, c.scales
    for step in range(4):
        new = [W._normal_bf16(rng, (3 * n, Hkv, 128), 2.0 ** (step % 3)) for _ in range(2)]
        lib.bdlm_write_kv8(d, n, None, 0, bf16_tensor(new[0]), bf16_tensor(new[1]), k, v, s, t, dev(lens))
        wk, wv, ws = R.write_kv8(n, None, *new, wk, wv, ws, c.table, lens)
    assert R.same_codes(host(k), wk) and R.same_codes(host(v), wv) and np.array_equal(host(s), ws)


def test_pages_past_two_gigabytes(lib):
    """Pages whose bytes lie past 2^31 and 2^32 in the pools."""
    import torch
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("no room")
    rng = np.random.default_rng(10)
    Hkv, L, Hq, n = 8, 4, 32, 20
    pages = (1 << 32) // (Hkv * 2048) + 70
    table = np.array([[pages - 1, 5, (1 << 31) // (Hkv * 2048) + 3], [pages - 20, pages - 3, 0]], np.int32)
    k, v = (torch.zeros((pages, Hkv, 16, 128), dtype=torch.uint8, device="cuda") for _ in range(2))
    s = torch.ones((pages, Hkv, 2), device="cuda")
    d = lib.attn_desc(2, L, Hq, Hkv, 128, 3, pages)
    new = [W._normal_bf16(rng, (2 * n, Hkv, 128), 1.0) for _ in range(2)]
    zero = dev(np.zeros(2, np.int32))
    lib.bdlm_write_kv8(d, n, None, 0, bf16_tensor(new[0]), bf16_tensor(new[1]), k, v, s, dev(table), zero)
    q = W._normal_bf16(rng, (2, L, Hq, 128), 1.0)
    out = torch.empty((2, L, Hq, 128), dtype=torch.bfloat16, device="cuda")
    lib.bdlm_attention_kv8(d, bf16_tensor(q), k, v, s, dev(table), dev(np.full(2, n - L, np.int32)), out)
    small = np.arange(6, dtype=np.int32).reshape(2, 3)
    blank = np.zeros((6, Hkv, 16, 128), np.uint8)
    wk, wv, ws = R.write_kv8(n, None, *new, blank, blank, np.ones((6, Hkv, 2), np.float32), small, np.zeros(2, np.int32))
    R.check_attention(f(out), R.attention_kv8(q, wk, wv, ws, small, np.full(2, n - L), Hkv))
    got = host(k[torch.from_numpy(table.reshape(-1).astype(np.int64)).cuda()])
    assert R.same_codes(got, wk)


@pytest.mark.parametrize("L,Hq,Hkv,B", [(1, 4, 1, 300), (2, 16, 1, 260), (12, 4, 1, 257), (64, 3, 1, 258)])
def test_attention_of_many_sequences(lib, L, Hq, Hkv, B):
    """More sequences than a warp keeps the tiles of."""
    rng = np.random.default_rng(B)
    lens = rng.integers(0, 200, B)
    lens[rng.integers(0, B, 5)] = 400
    c = Cache(rng, lens + L, Hkv)
    q = W._normal_bf16(rng, (B, L, Hq, 128), 1.0)
    out = attend(lib, c, q, L, Hq, Hkv)
    R.check_attention(f(out), R.attention_kv8(q, c.k, c.v, c.scales, c.table, c.lens - L, Hkv))
    assert lib.bdlm_device_error() == 0


@pytest.mark.parametrize("L,Hq,Hkv,lens", [(1, 2, 1, [50000]), (16, 2, 1, [30001, 5]), (64, 2, 1, [20000]), (64, 4, 1, [20010]),
                                           (3, 8, 2, [9000, 20000]), (1, 1, 1, [40000, 1, 700])])
def test_attention_of_lists_in_many_parts(lib, L, Hq, Hkv, lens):
    """Long lists that all CTAs share."""
    rng = np.random.default_rng(L)
    c = Cache(rng, np.array(lens) + L, Hkv)
    q = W._normal_bf16(rng, (len(lens), L, Hq, 128), 1.0)
    out = attend(lib, c, q, L, Hq, Hkv)
    R.check_attention(f(out), R.attention_kv8(q, c.k, c.v, c.scales, c.table, c.lens - L, Hkv))
    assert lib.bdlm_device_error() == 0


@pytest.mark.parametrize("L,Hq,Hkv", [(1, 8, 8), (4, 32, 8), (4, 64, 8), (8, 128, 16)])
def test_attention_repeats_bit_for_bit_beside_other_work(lib, L, Hq, Hkv):
    """Lists that borders cut are joined in their order, whoever comes last: no run differs from another."""
    import torch
    rng = np.random.default_rng(12)
    B = 40
    c = Cache(rng, rng.integers(1, 1500, B) + L, Hkv)
    q = W._normal_bf16(rng, (B, L, Hq, 128), 1.0)
    first = attend(lib, c, q, L, Hq, Hkv)
    R.check_attention(f(first), R.attention_kv8(q, c.k, c.v, c.scales, c.table, c.lens - L, Hkv))
    d = lib.attn_desc(B, L, Hq, Hkv, 128, c.cols, c.pages)
    (k, v, s, t), qd, n = c.dev(), bf16_tensor(q), dev(c.lens - L)
    outs = [torch.zeros_like(first) for _ in range(20)]
    busy = torch.randn(2048, 2048, device="cuda")
    other = torch.cuda.Stream()
    with torch.cuda.stream(other):
        for _ in range(50):
            busy @ busy
    for o in outs:
        lib.bdlm_attention_kv8(d, qd, k, v, s, t, n, o)
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o.view(torch.int16), first.view(torch.int16))


def test_write_of_a_far_larger_maximum(lib):
    """n_tokens is only the most that a packed sequence may have: the largest there is does no harm."""
    import torch
    rng = np.random.default_rng(13)
    c = Cache(rng, [40], 2)
    new = W._normal_bf16(rng, (21, 2, 128), 1.0)
    first = np.array([3, 20], np.int32)
    want = R.write_kv8(21, first, new, new, c.k, c.v, c.scales, c.table, np.array([5], np.int32))
    k, v, s, t = c.dev()
    d = lib.attn_desc(1, 1, 2, 2, 128, c.cols, c.pages)
    lib.bdlm_write_kv8(d, 2 ** 24 - 1, dev(first), 21, bf16_tensor(new), bf16_tensor(new), k, v, s, t, dev(np.array([5], np.int32)))
    assert np.array_equal(host(s), want[2]) and R.same_codes(host(k), want[0]) and R.same_codes(host(v), want[1])
    assert lib.bdlm_device_error() == 0


@pytest.mark.parametrize("L,Hq,Hkv,B", [(2, 8, 2, 9), (8, 8, 2, 5), (16, 8, 2, 6), (64, 8, 2, 3), (40, 2, 1, 300), (3, 2, 1, 300)])
@pytest.mark.parametrize("captured", [False, True])
def test_attention_right_behind_what_wrote_its_inputs(lib, L, Hq, Hkv, B, captured):
    """Lengths, tables, pages and queries that change from call to call, with nothing between their writers and the call
    that reads them: the same as with the GPU idle before each call."""
    import torch
    rng = np.random.default_rng(L)
    sets = []
    for i in range(2):
        c = Cache(rng, rng.integers(0, 60 + 500 * i, B) + L, Hkv)
        new = [bf16_tensor(W._normal_bf16(rng, (B * L, Hkv, 128), 2.0 ** (3 * i))) for _ in range(2)]
        sets.append((c, new, bf16_tensor(W._normal_bf16(rng, (B, L, Hq, 128), 1.0))))
    cols, pages = max(c.cols for c, _, _ in sets), max(c.pages for c, _, _ in sets)
    src = []
    for c, new, q in sets:
        t = np.full((B, cols), -1, np.int32)
        t[:, :c.cols] = c.table
        pad = lambda x: dev(np.concatenate([x, np.full((pages - c.pages,) + x.shape[1:], 127, x.dtype)]))
        src.append([pad(c.k), pad(c.v), pad(c.scales), dev(t), dev(c.lens - L), *new, q])
    d = lib.attn_desc(B, L, Hq, Hkv, 128, cols, pages)
    at = [torch.empty_like(x) for x in src[0]]
    steps = 8
    outs = [torch.zeros((B, L, Hq, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2 * steps)]

    def step(i, out, idle, stream=None):
        k, v, s, t, n, nk, nv, q = at
        for x, y in zip(at, src[i % 2]):
            x.copy_(y)
        if idle:
            torch.cuda.synchronize()
        lib.bdlm_write_kv8(d, L, None, 0, nk, nv, k, v, s, t, n, stream=stream)
        if idle:
            torch.cuda.synchronize()
        lib.bdlm_attention_kv8(d, q, k, v, s, t, n, out, stream=stream)

    for i in range(steps):
        step(i, outs[i], True)
    torch.cuda.synchronize()
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for i in range(steps):
                step(i, outs[steps + i], False, torch.cuda.current_stream())
        graph.replay()
    else:
        for i in range(steps):
            step(i, outs[steps + i], False)
    torch.cuda.synchronize()
    for i in range(steps):
        assert torch.equal(outs[i].view(torch.int16), outs[steps + i].view(torch.int16)), i
    assert not torch.equal(outs[0].view(torch.int16), outs[1].view(torch.int16))
    assert lib.bdlm_device_error() == 0
