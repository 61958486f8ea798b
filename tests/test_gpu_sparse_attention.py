"""Page bounds, page selection and the attention over the selected pages, against 64-bit forms."""
import numpy as np
import pytest

import cache_ref as R
import workloads as W
from gpu_util import bf16_tensor, dev, host

pytestmark = pytest.mark.gpu


def bits(t):
    import torch
    return host(t.view(torch.int16)).view(np.uint16)


def gpu_bounds(lib, a, frm, to, init):
    import torch
    t = bf16_tensor(init)
    d = lib.attn_desc(a.B, 1, a.Hkv, a.Hkv, 128, a.page_table_ref.shape[1], a.k_ref.shape[0])
    lib.bdlm_page_bounds(d, bf16_tensor(a.k_ref), dev(a.page_table_ref),
                         None if frm is None else dev(frm), dev(to), t)
    torch.cuda.synchronize()
    return bits(t)


@pytest.mark.parametrize("B,Hkv,hi", [(1, 8, 40), (5, 8, 700), (3, 1, 2000), (2, 3, 500), (200, 2, 64)])
def test_bounds(lib, B, Hkv, hi):
    rng = np.random.default_rng(B + Hkv)
    lens = rng.integers(0, hi, size=B)
    a = W.make_attention(rng, B, 1, Hkv, Hkv, 128, prefix_lens=lens)     # NaN past the last token
    to = (lens + 1).astype(np.int32)
    frm = rng.integers(0, to + 1).astype(np.int32)
    init = np.full((a.k_ref.shape[0], Hkv, 2, 128), 0x4242, np.uint16)
    for f in (None, frm):
        want = R.page_bounds(a.k_ref, a.page_table_ref, np.zeros(B, int) if f is None else f, to, init)
        got = gpu_bounds(lib, a, f, to, init)
        assert np.array_equal(R.f64(got), R.f64(want))
    assert lib.bdlm_device_error() == 0


def test_bounds_flags_bad_pages_and_lengths(lib):
    rng = np.random.default_rng(3)
    a = W.make_attention(rng, 3, 1, 8, 8, 128, prefix_lens=np.array([100, 100, 100]))
    good = a.page_table_ref.copy()
    a.page_table_ref[1, 2] = -1
    init = np.full((a.k_ref.shape[0], 8, 2, 128), 0x4242, np.uint16)
    frm, to = np.array([0, 0, 80], np.int32), np.array([101, 101, 40], np.int32)
    got = gpu_bounds(lib, a, frm, to, init)
    assert lib.bdlm_device_error() == lib.BDLM_DEVERR_PAGE | lib.BDLM_DEVERR_LENGTH
    assert np.all(got[good[1, 2]] == 0x4242) and np.all(got[good[2]] == 0x4242)
    assert np.all(got[good[0, :6]] != 0x4242)


class Pages:
    """A cache known by its page bounds only."""

    def __init__(self, rng, lens, L, Hq, Hkv, extra=3):
        self.lens = np.asarray(lens, np.int32)
        self.B, self.L, self.Hq, self.Hkv = len(lens), L, Hq, Hkv
        self.cols = (int(self.lens.max()) + L + 15) // 16
        n = int(np.sum((self.lens + L + 15) // 16)) + extra
        perm, c = rng.permutation(n).astype(np.int32), 0
        self.table = np.full((self.B, self.cols), -1, np.int32)
        for b in range(self.B):
            m = (int(self.lens[b]) + L + 15) // 16
            self.table[b, :m] = perm[c:c + m]
            c += m
        self.num = n
        self.q = W._normal_bf16(rng, (self.B, L, Hq, 128), 1.0)
        x = rng.normal(size=(n, Hkv, 1, 128)).astype(np.float32)
        y = np.abs(rng.normal(size=(n, Hkv, 2, 128))).astype(np.float32) + 0.5
        self.bounds = W.f32_to_bf16_bits(np.concatenate([x - y[:, :, :1], x + y[:, :, 1:]], 2))

    def run(self, lib, group, n_select, cols=None, table=None, lens=None, stream=None):
        import torch
        cols = n_select + (self.L + 30) // 16 if cols is None else cols
        sel = torch.full((self.B, self.L // group, self.Hkv, cols), -7, dtype=torch.int32, device="cuda")
        sl = torch.full((self.B, self.L // group), -7, dtype=torch.int32, device="cuda")
        d = lib.attn_desc(self.B, self.L, self.Hq, self.Hkv, 128, self.cols, self.num)
        lib.bdlm_select_pages(d, bf16_tensor(self.q), bf16_tensor(self.bounds),
                              dev(self.table if table is None else table),
                              dev(self.lens if lens is None else lens), group, n_select, cols, sel, sl,
                              stream=stream)
        torch.cuda.synchronize()
        return host(sel), host(sl)

    def check(self, lib, group, n_select, cols=None):
        cols = n_select + (self.L + 30) // 16 if cols is None else cols
        got, lens = self.run(lib, group, n_select, cols)
        want, want_lens = R.select_pages(self.q, self.bounds, self.table, self.lens, group, n_select,
                                         cols, self.Hkv)
        assert np.array_equal(lens, want_lens)
        assert np.array_equal(got, want)
        assert lib.bdlm_device_error() == 0


@pytest.mark.parametrize("L,group,Hq,Hkv", [(1, 1, 16, 8), (4, 4, 32, 8), (4, 1, 32, 8), (6, 3, 24, 8),
                                            (15, 5, 16, 2), (64, 64, 32, 8), (64, 8, 32, 8),
                                            (64, 16, 16, 1), (64, 1, 16, 1), (40, 40, 12, 2)])
def test_selection(lib, L, group, Hq, Hkv):
    rng = np.random.default_rng(L + group * 7 + Hq)
    p = Pages(rng, [0, 15, 16, 500, 2047, 2048 + 17, 4000], L, Hq, Hkv)
    for n in (1, 5, 128, 10000):
        p.check(lib, group, n, cols=min(n, 400) + 6 if n < 400 else n + 6)
    p.check(lib, group, 0)


@pytest.mark.parametrize("lens,n", [([40000, 33000], 200), ([300000], 1000), ([16384 * 16 + 5], 16000)])
def test_selection_long(lib, lens, n):
    """Lists past a run of tiles, past a tile, and past the keys that fit shared memory."""
    rng = np.random.default_rng(len(lens))
    Pages(rng, lens, 2, 4, 2).check(lib, 2, n)


def test_selection_of_equal_pages_takes_the_first(lib):
    rng = np.random.default_rng(8)
    p = Pages(rng, [3000, 24000], 2, 4, 2)
    p.bounds[:] = p.bounds[:1]                       # every page the same: 187 and 1500 near ties
    for n in (1, 50, 186, 1499):
        p.check(lib, 2, n)
    pool = p.bounds[rng.integers(0, 2, size=p.num)]  # two kinds
    p.bounds = pool
    p.bounds[p.table[1, 700:900], :, 1, 3] = W.f32_to_bf16_bits(np.full(1, 4.0, np.float32))
    for n in (1, 60, 400, 1100):
        p.check(lib, 1, n)


@pytest.mark.parametrize("L,group,G", [(4, 4, 4), (4, 1, 4), (16, 16, 4), (3, 3, 16), (10, 5, 8), (32, 32, 4)])
@pytest.mark.parametrize("ties", [False, True])
def test_selection_of_many_short_lists(lib, L, group, G, ties):
    """More lists than are worked on at once, of up to 64 query rows and of more."""
    rng = np.random.default_rng(L + G)
    p = Pages(rng, rng.integers(0, 1500, size=90), L, 8 * G, 8)
    if ties:   # few kinds of pages, one bf16 step apart in one dim
        p.bounds[:] = p.bounds[0]
        p.bounds[:, :, 1, 7] += rng.integers(0, 6, size=(p.num, 1)).astype(np.uint16)
    for n in (1, 30):
        p.check(lib, group, n)


@pytest.mark.parametrize("L,group,Hq,Hkv", [(64, 64, 32, 8), (32, 16, 64, 8), (5, 5, 16, 1), (48, 48, 4, 1)])
def test_selection_of_near_ties_over_many_rows(lib, L, group, Hq, Hkv):
    """Pages whose scores differ by a bf16 step of one or two bounds, for some rows only."""
    rng = np.random.default_rng(L + Hq)
    p = Pages(rng, [2500, 19000], L, Hq, Hkv)
    p.bounds[:] = p.bounds[0]
    for dim in (3, 90):
        p.bounds[:, :, :, dim] += rng.integers(0, 3, size=(p.num, 1, 2)).astype(np.uint16)
    for n in (1, 40, 155):
        p.check(lib, group, n)


def test_selection_tells_close_scores_apart(lib):
    """Scores that differ by less than float32 resolves at their size: one dim moves by a step of
    bf16 where the query is small."""
    rng = np.random.default_rng(9)
    p = Pages(rng, [1600], 1, 2, 2)
    p.q[..., 5] = W.f32_to_bf16_bits(np.full(1, 2.0 ** -22, np.float32))
    same = p.bounds[0].copy()
    p.bounds[:] = same
    steps = rng.permutation(p.num)
    p.bounds[:, :, 1, 5] = W.f32_to_bf16_bits((1 + steps % 100 / 128).astype(np.float32))[:, None]
    for n in (1, 13, 50, 99):
        p.check(lib, 1, n)


def test_selection_flags_bad_pages_and_lengths(lib):
    rng = np.random.default_rng(10)
    p = Pages(rng, [640, 640, 640], 4, 8, 2)
    t, n = p.table.copy(), p.lens.copy()
    t[0, 3], t[0, 20] = -5, 10 ** 7
    n[1], n[2] = -1, 10 ** 8
    sel, lens = p.run(lib, 4, 30, table=t, lens=n)
    assert lib.bdlm_device_error() == lib.BDLM_DEVERR_PAGE | lib.BDLM_DEVERR_LENGTH
    assert lens[0, 0] == 480 and list(lens[1:, 0]) == [-1, -1] and np.all(sel[1:] == -1)
    assert not np.isin(sel[0, 0, :, :30], [-5, 10 ** 7]).any()
    p.check(lib, 4, 30)


@pytest.mark.parametrize("lens", [[200, 640], [200, 9000]])
@pytest.mark.parametrize("n", [0, 40, 600])
def test_a_bad_page_is_flagged_whether_or_not_it_is_scored(lib, lens, n):
    """Short lists, which are scored and chosen from in one kernel, and longer ones."""
    rng = np.random.default_rng(11)
    p = Pages(rng, lens, 4, 8, 2)
    t = p.table.copy()
    t[0, 5] = p.num
    sel, _ = p.run(lib, 4, n, table=t)
    assert lib.bdlm_device_error() == lib.BDLM_DEVERR_PAGE
    assert np.array_equal(sel[0, 0, :, :min(n, 12)], np.tile(t[0, :min(n, 12)], (2, 1)))
    p.check(lib, 4, n)


@pytest.mark.parametrize("L,Hq,Hkv", [(64, 32, 8), (48, 8, 2), (5, 64, 4)])
def test_whole_tiles_of_bad_pages_hold_up_nothing(lib, L, Hq, Hkv):
    """Runs of 128 and more bad ids between good pages, scored for more than 64 rows a list: the choice
    among the good pages is theirs alone, and no wait runs out."""
    rng = np.random.default_rng(L)
    p = Pages(rng, [16 * 1100 + 3, 16 * 900, 40, 16 * 1300], L, Hq, Hkv)
    t = p.table.copy()
    for b, runs in ((0, [(128, 256), (512, 900)]), (1, [(0, 128), (256, 384), (512, 640), (768, 896)]),
                    (3, [(0, 1290)])):
        for lo, hi in runs:
            t[b, lo:hi] = np.where(np.arange(hi - lo) % 2, -1, p.num + 7)
    for n in (1, 100):
        sel, lens = p.run(lib, L, n, table=t)
        assert lib.bdlm_device_error() == lib.BDLM_DEVERR_PAGE
        for b in range(4):
            full = int(p.lens[b]) // 16
            good = np.flatnonzero((t[b, :full] >= 0) & (t[b, :full] < p.num))
            k = min(n, full)
            for h in range(Hkv):
                got = sel[b, 0, h, :k]
                if len(good) < k:   # every good page, and bad ones that make up the number
                    assert set(t[b, good]) <= set(got)
                    continue
                score = R.page_scores(p.q[b], p.bounds, t[b, good], h, Hq // Hkv)
                best = np.sort(good[np.argsort(-score, kind="stable")[:k]])
                assert np.array_equal(got, t[b, best])


@pytest.mark.parametrize("L,group,Hq,Hkv,n", [(1, 1, 16, 8, 8), (4, 4, 32, 8, 16), (4, 1, 32, 8, 16),
                                             (6, 3, 24, 8, 5), (64, 64, 32, 8, 12), (32, 8, 32, 8, 64),
                                             (16, 16, 16, 1, 30), (2, 1, 4, 4, 300)])
def test_sparse_attention(lib, L, group, Hq, Hkv, n):
    """Every KV head and group reads pages of its own; pages and slots outside the lists hold NaN."""
    import torch
    rng = np.random.default_rng(L + n)
    B = 3
    lens = np.array([0, 5 * 16 + 3, n * 16 + 200])
    a = W.make_attention(rng, B, L, Hq, Hkv, 128, prefix_lens=lens, qkv_std=1.0)
    S, cols = L // group, n + (L + 30) // 16
    sel = np.full((B, S, Hkv, cols), -1, np.int32)
    sl = np.zeros((B, S), np.int32)
    for b in range(B):
        full = int(lens[b]) // 16
        k = min(n, full)
        tail = a.page_table_ref[b, full:(int(lens[b]) + L + 15) // 16]
        for s in range(S):
            sl[b, s] = k * 16 + lens[b] % 16 + L - group
            for h in range(Hkv):
                pick = np.sort(rng.permutation(full)[:k])
                sel[b, s, h, :k] = a.page_table_ref[b, pick]
                sel[b, s, h, k:k + len(tail)] = tail
    out = torch.full((B, L, Hq, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    d = lib.attn_desc(B, L, Hq, Hkv, 128, 1, a.k_ref.shape[0])
    lib.bdlm_sparse_attention(d, bf16_tensor(a.q), bf16_tensor(a.k_ref), bf16_tensor(a.v_ref), group,
                              cols, dev(sel), dev(sl), out)
    torch.cuda.synchronize()
    assert lib.bdlm_device_error() == 0
    want, A, s1 = R.sparse_attention(a.q, a.k_ref, a.v_ref, sel, sl, group, Hkv)
    R.check_out(host(out.float()).astype(np.float64), want, A, s1)


def test_bounds_selection_and_attention_together(lib):
    """As a round uses them: bounds of the prompt, a selection, attention over it; with every page
    selected the result is block attention's."""
    import torch
    rng = np.random.default_rng(12)
    B, L, Hq, Hkv = 4, 4, 32, 8
    a = W.make_attention(rng, B, L, Hq, Hkv, 128, prefix_lens=np.array([17, 400, 1000, 1500]), qkv_std=1.0)
    P = a.page_table_ref.shape[1]
    q, k, v, t, n = (bf16_tensor(a.q), bf16_tensor(a.k_ref), bf16_tensor(a.v_ref), dev(a.page_table_ref),
                     dev(a.prefix_lens))
    d = lib.attn_desc(B, L, Hq, Hkv, 128, P, a.k_ref.shape[0])
    bounds = torch.zeros((a.k_ref.shape[0], Hkv, 2, 128), dtype=torch.bfloat16, device="cuda")
    lib.bdlm_page_bounds(d, k, t, None, n, bounds)
    block = torch.empty((B, L, Hq, 128), dtype=torch.bfloat16, device="cuda")
    lib.bdlm_block_attention(d, q, k, v, t, n, L, block)
    for n_sel in (10, 200):
        cols = n_sel + 2
        sel = torch.empty((B, 1, Hkv, cols), dtype=torch.int32, device="cuda")
        sl = torch.empty((B, 1), dtype=torch.int32, device="cuda")
        out = torch.empty_like(block)
        lib.bdlm_select_pages(d, q, bounds, t, n, L, n_sel, cols, sel, sl)
        lib.bdlm_sparse_attention(d, q, k, v, L, cols, sel, sl, out)
        torch.cuda.synchronize()
        want_sel, _ = R.select_pages(a.q, bits(bounds), a.page_table_ref, a.prefix_lens, L, n_sel, cols, Hkv)
        assert np.array_equal(host(sel), want_sel)
        want, A, s1 = R.sparse_attention(a.q, a.k_ref, a.v_ref, want_sel, host(sl), L, Hkv)
        R.check_out(host(out.float()).astype(np.float64), want, A, s1)
        if n_sel == 200:
            # the same keys in the same order: at most one more rounding of the output
            assert torch.allclose(out.float(), block.float(), rtol=2 ** -7, atol=2 ** -9)
    assert lib.bdlm_device_error() == 0
