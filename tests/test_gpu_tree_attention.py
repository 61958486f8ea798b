"""bdlm_tree_attention against the 64-bit form: visibility words of every kind, rows that see
nothing, garbage behind the mask, and the normalisers."""
import numpy as np
import pytest

import cache_ref as R
import workloads as W
from gpu_util import bf16_tensor, dev, host

pytestmark = pytest.mark.gpu


def masks(rng, B, L, kind):
    if kind == "path":        # each token sees the ones before it and itself
        m = np.array([(1 << (i + 1)) - 1 for i in range(L)], dtype=np.uint64)
        return np.broadcast_to(m, (B, L)).copy()
    if kind == "tree":
        m = np.zeros((B, L), np.uint64)
        for b in range(B):
            for i in range(L):
                up = int(rng.integers(-1, i)) if i else -1
                m[b, i] = np.uint64((int(m[b, up]) if up >= 0 else 0) | (1 << i))
        return m
    if kind == "self":
        return np.broadcast_to(np.array([1 << i for i in range(L)], np.uint64), (B, L)).copy()
    if kind == "none":
        return np.zeros((B, L), np.uint64)
    m = rng.integers(0, 2 ** 64, size=(B, L), dtype=np.uint64)     # bits past L too
    m[rng.random((B, L)) < 0.3] = 0
    return m


def run(lib, a, mask, k=None, v=None, lse=True, stream=None, sm_scale=0.0):
    import torch
    out = torch.full((a.B, a.L, a.Hq, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    ls = torch.full((a.B, a.L, a.Hq), float("nan"), device="cuda") if lse else None
    d = lib.attn_desc(a.B, a.L, a.Hq, a.Hkv, 128, a.page_table_ref.shape[1], a.k_ref.shape[0],
                      sm_scale=sm_scale)
    m = None if mask is None else dev(mask.view(np.int64))
    lib.bdlm_tree_attention(d, bf16_tensor(a.q), bf16_tensor(a.k_ref if k is None else k),
                            bf16_tensor(a.v_ref if v is None else v), dev(a.page_table_ref),
                            dev(a.prefix_lens), m, out, ls, stream=stream)
    torch.cuda.synchronize()
    assert lib.bdlm_device_error() == 0
    return host(out.float()).astype(np.float64), None if ls is None else host(ls).astype(np.float64)


def check(lib, a, mask, **kw):
    got, lse = run(lib, a, mask, **kw)
    out, ref_lse, A, s1 = R.tree_attention(a.q, a.k_ref if kw.get("k") is None else kw["k"],
                                           a.v_ref if kw.get("v") is None else kw["v"],
                                           a.page_table_ref, a.prefix_lens, mask, a.Hkv)
    R.check_out(got, out, A, s1)
    R.check_lse(lse, ref_lse, s1)


@pytest.mark.parametrize("kind", ["tree", "path", "self", "any", "none"])
@pytest.mark.parametrize("L,Hq,Hkv", [(1, 16, 8), (4, 32, 8), (8, 16, 8), (9, 16, 8), (5, 24, 8),
                                      (31, 8, 8), (16, 32, 8), (33, 4, 4), (40, 32, 8),
                                      (64, 32, 8), (20, 16, 1), (64, 8, 1)])
def test_shapes_and_masks(lib, L, Hq, Hkv, kind):
    rng = np.random.default_rng(L * 100 + Hq + len(kind))
    lens = np.array([0, int(rng.integers(1, 300)), 128 - L // 2, 127])
    a = W.make_attention(rng, 4, L, Hq, Hkv, 128, prefix_lens=lens, qkv_std=1.0)
    check(lib, a, masks(rng, 4, L, kind))


@pytest.mark.parametrize("L,Hq,lens", [(8, 16, [2500, 895, 896, 897]), (16, 16, [1790, 5000, 1]),
                                       (20, 32, [9000, 3200, 0]), (64, 32, [9000, 4032, 4090])])
def test_splits(lib, L, Hq, lens):
    """Prefixes cut into KV splits, with the block across a boundary of tiles or splits."""
    rng = np.random.default_rng(L + Hq)
    a = W.make_attention(rng, len(lens), L, Hq, 8, 128, prefix_lens=np.array(lens), qkv_std=1.0)
    check(lib, a, masks(rng, len(lens), L, "any"))


@pytest.mark.parametrize("L", [4, 64])
def test_whole_sequences(lib, L):
    rng = np.random.default_rng(5)
    lens = rng.integers(0, 300, size=80)
    a = W.make_attention(rng, 80, L, 32, 8, 128, prefix_lens=lens, qkv_std=1.0)
    got, lse = run(lib, a, mask := masks(rng, 80, L, "any"))
    for b in (0, 17, 79):
        out, rl, A, s1 = R.tree_attention(a.q[b:b + 1], a.k_ref, a.v_ref, a.page_table_ref[b:b + 1],
                                          lens[b:b + 1], mask[b:b + 1], 8)
        R.check_out(got[b:b + 1], out, A, s1)
        R.check_lse(lse[b:b + 1], rl, s1)


@pytest.mark.parametrize("L,Hq,prefix", [(8, 16, 100), (16, 32, 100), (40, 32, 1000), (8, 16, 5000)])
def test_nothing_leaks_from_unseen_tokens(lib, L, Hq, prefix):
    """K of a token is NaN or infinite for queries that do not see it; V of a token no query sees."""
    rng = np.random.default_rng(L)
    a = W.make_attention(rng, 2, L, Hq, 8, 128, prefix_lens=np.array([prefix, prefix - 3]), qkv_std=1.0)
    mask = masks(rng, 2, L, "any")
    hidden = [t for t in range(L) if t % 3 == 1]                 # seen by nobody
    for t in hidden:
        mask &= ~np.uint64(1 << t)
    k, v = a.k_ref.copy(), a.v_ref.copy()
    for b in range(2):
        for t in hidden:
            tok = int(a.prefix_lens[b]) + t
            page = a.page_table_ref[b, tok // 16]
            k[page, tok % 16] = [0x7FC0, 0x7F80, 0xFF80][t % 3]
            v[page, tok % 16] = [0x7F80, 0x7FC0, 0xFF80][t % 3]
    check(lib, a, mask, k=k, v=v)


def test_no_mask_is_block_attention(lib):
    import torch
    for L, Hq in [(4, 32), (8, 32), (16, 32), (50, 32)]:
        rng = np.random.default_rng(L)
        a = W.make_attention(rng, 5, L, Hq, 8, 128, prefix_range=(0, 4000))
        got, lse = run(lib, a, None)
        ones, lse1 = run(lib, a, np.full((5, L), 2 ** 64 - 1, np.uint64))
        only, _ = run(lib, a, None, lse=False)
        out = torch.empty((5, L, Hq, 128), dtype=torch.bfloat16, device="cuda")
        d = lib.attn_desc(5, L, Hq, 8, 128, a.page_table_ref.shape[1], a.k_ref.shape[0])
        lib.bdlm_block_attention(d, bf16_tensor(a.q), bf16_tensor(a.k_ref), bf16_tensor(a.v_ref),
                                 dev(a.page_table_ref), dev(a.prefix_lens), L, out)
        block = host(out.float()).astype(np.float64)
        assert np.array_equal(got, block) and np.array_equal(ones, block) and np.array_equal(only, block)
        assert np.array_equal(lse, lse1)


def test_bad_pages_and_lengths_are_flagged(lib):
    import torch
    rng = np.random.default_rng(1)
    a = W.make_attention(rng, 3, 8, 16, 8, 128, prefix_lens=np.array([100, 50, 70]))
    pt, pl = a.page_table_ref.copy(), a.prefix_lens.copy()
    pt[0, 2] = 10 ** 6
    pl[1], pl[2] = -4, 10 ** 7
    d = lib.attn_desc(3, 8, 16, 8, 128, pt.shape[1], a.k_ref.shape[0])
    out = torch.empty((3, 8, 16, 128), dtype=torch.bfloat16, device="cuda")
    lib.bdlm_tree_attention(d, bf16_tensor(a.q), bf16_tensor(a.k_ref), bf16_tensor(a.v_ref), dev(pt),
                            dev(pl), dev(masks(rng, 3, 8, "tree").view(np.int64)), out)
    torch.cuda.synchronize()
    assert lib.bdlm_device_error() == lib.BDLM_DEVERR_PAGE | lib.BDLM_DEVERR_LENGTH
    check(lib, a, masks(rng, 3, 8, "tree"))


@pytest.mark.parametrize("B,L,lo,hi", [(640, 4, 20, 200), (640, 8, 20, 200), (400, 16, 20, 200), (200, 40, 20, 200),
                                       (24, 8, 2000, 9000), (24, 40, 2000, 9000)])
def test_no_mask_is_block_attention_over_many_results(lib, B, L, lo, hi):
    """Bit for bit over millions of results, among which any other rounding of the quotient shows."""
    import torch
    torch.manual_seed(L)
    cols = (hi + L + 15) // 16
    lens = torch.randint(lo, hi, (B,), dtype=torch.int32, device="cuda")
    t = torch.randperm(B * cols, device="cuda").int().view(B, cols)
    k = torch.randn((B * cols, 16, 8, 128), device="cuda").bfloat16()
    v = torch.randn((B * cols, 16, 8, 128), device="cuda").bfloat16()
    q = torch.randn((B, L, 32, 128), device="cuda").bfloat16()
    block, tree = torch.empty_like(q), torch.empty_like(q)
    d = lib.attn_desc(B, L, 32, 8, 128, cols, B * cols)
    lib.bdlm_block_attention(d, q, k, v, t, lens, L, block)
    lib.bdlm_tree_attention(d, q, k, v, t, lens, None, tree)
    torch.cuda.synchronize()
    assert torch.equal(block, tree)
    assert lib.bdlm_device_error() == 0
