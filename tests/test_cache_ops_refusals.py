"""Refusals of the operators over part of the cache: arguments are checked on the host, before a
GPU is touched."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def so():
    from block_diffusion_gb300 import build, load_library
    build.build()
    return load_library()


P = 0x1000   # never dereferenced


def desc(B=2, L=4, Hq=32, Hkv=8, D=128, cols=10, num=100, **kw):
    import block_diffusion_gb300 as bd
    return ctypes.byref(bd.attn_desc(B, L, Hq, Hkv, D, cols, num, **kw))


def tree(so, d=None, q=P, k=P, v=P, t=P, n=P, m=P, out=P, lse=P):
    return so.bdlm_tree_attention(desc() if d is None else d, q, k, v, t, n, m, out, lse, None)


def bounds(so, d=None, k=P, t=P, f=P, to=P, b=P):
    return so.bdlm_page_bounds(desc() if d is None else d, k, t, f, to, b, None)


def select(so, d=None, q=P, b=P, t=P, n=P, group=4, n_sel=8, cols=10, sel=P, sl=P):
    return so.bdlm_select_pages(desc() if d is None else d, q, b, t, n, group, n_sel, cols, sel, sl, None)


def sparse(so, d=None, q=P, k=P, v=P, group=4, cols=10, sel=P, sl=P, out=P):
    return so.bdlm_sparse_attention(desc() if d is None else d, q, k, v, group, cols, sel, sl, out, None)


def weights(so, d=None, q=P, k=P, t=P, n=P, lse=P, decay=1.0, w=P):
    return so.bdlm_attention_weights(desc() if d is None else d, q, k, t, n, lse, decay, w, None)


def evict(so, d=None, k=P, v=P, t=P, n=P, w=P, keep=32, recent=4, to=P, tw=P, kept=P, new=P + 64):
    return so.bdlm_evict_kv(desc() if d is None else d, k, v, t, n, w, keep, recent, to, tw, kept, new, None)


def compact(so, d=None, k=P, v=P, t=P, base=P, idx=P, heads=1, n_max=4, c=P, to=P):
    return so.bdlm_compact_kv(desc() if d is None else d, k, v, t, base, idx, heads, n_max, c, to, None)


@pytest.mark.parametrize("call", [tree, select, sparse, weights])
def test_descriptors_of_attention(so, call):
    for bad in (dict(B=-1), dict(L=0), dict(L=65), dict(Hq=30), dict(Hq=0), dict(Hkv=0), dict(D=64),
                dict(Hq=32, Hkv=1), dict(num=0), dict(page_size=32), dict(sm_scale=float("inf")),
                dict(sm_scale=float("nan")), dict(B=2 ** 30, L=64)):
        assert call(so, desc(**bad)) == -1, bad
    assert call(so, desc(cols=0)) == -1


@pytest.mark.parametrize("call", [bounds, evict, compact])
def test_descriptors_of_the_cache(so, call):
    for bad in (dict(B=-1), dict(Hkv=0, Hq=8), dict(D=64), dict(cols=0), dict(num=0), dict(page_size=8),
                dict(cols=2 ** 28), dict(B=2 ** 29, Hkv=8)):
        assert call(so, desc(**bad)) == -1, bad


@pytest.mark.parametrize("call,optional", [(tree, ("m", "lse")), (bounds, ("f",)), (select, ()),
                                           (sparse, ()), (weights, ()), (evict, ()), (compact, ("base",))])
def test_null_and_misaligned_pointers(so, call, optional):
    import inspect
    names = [n for n, p in inspect.signature(call).parameters.items()
             if p.default in (P, P + 64) and p.default is not None]
    for name in names:
        if name not in optional:
            assert call(so, **{name: None}) == -1, name
    for name in {"q", "k", "v", "out", "b"} & set(names):
        assert call(so, **{name: P + 8}) == -1, name
    if call is tree:
        assert tree(so, m=P + 4) == -1


def test_sizes(so):
    for bad in (dict(group=0), dict(group=3), dict(n_sel=-1), dict(cols=9), dict(n_sel=2 ** 31 - 1)):
        assert select(so, **bad) == -1, bad
    assert select(so, desc(L=64, Hq=16, Hkv=1), group=64, cols=20) == -3      # 1024 rows in a group
    assert select(so, desc(cols=262145)) == -3
    assert select(so, desc(B=0, num=2 ** 27)) == -3 and select(so, desc(B=0, num=2 ** 27 - 1)) == 0
    for bad in (dict(group=0), dict(group=3), dict(cols=0), dict(cols=2 ** 28)):
        assert sparse(so, **bad) == -1, bad
    for bad in (dict(decay=float("nan")), dict(decay=float("inf"))):
        assert weights(so, **bad) == -1, bad
    for bad in (dict(keep=0), dict(keep=161), dict(recent=-1), dict(recent=33), dict(n=P + 64)):
        assert evict(so, **bad) == -1, bad
    for bad in (dict(heads=0), dict(heads=2), dict(n_max=-1)):
        assert compact(so, **bad) == -1, bad


@pytest.mark.parametrize("call", [bounds, weights, evict, compact])
def test_a_table_beyond_the_token_counters(so, call):
    assert call(so, desc(B=0, cols=2 ** 26 + 1)) == -3
    assert call(so, desc(B=0, cols=2 ** 26)) == 0


def test_counts_beyond_the_token_counters(so):
    assert compact(so, desc(B=0), n_max=2 ** 30 + 1) == -3
    assert compact(so, desc(B=0), n_max=2 ** 30) == 0


def test_moves_beyond_a_grid(so):
    """More moves to other pages than one launch has CTAs for (256 tokens of a list and head each)."""
    many = desc(B=2 ** 15, Hq=2 ** 15, Hkv=2 ** 15, cols=2 ** 15, num=1)
    assert compact(so, many, n_max=2 ** 19 - 31, to=P + 64) == -3      # 2^30 lists of 2^14 runs
    assert compact(so, many, n_max=2 ** 30, to=P + 64) == -3
    wide = desc(B=2 ** 4, Hq=2 ** 11, Hkv=2 ** 11, cols=2 ** 26, num=1)
    assert evict(so, wide, keep=2 ** 30, to=P + 64) == -3


def test_weights_refuse_a_vanishing_scale(so):
    for scale in (1e-38, 2.0 ** -65):
        assert weights(so, desc(B=0, sm_scale=scale)) == -3, scale
    assert weights(so, desc(B=0, sm_scale=2.0 ** -64)) == 0


def test_empty_calls_succeed_without_a_device(so):
    for call in (tree, bounds, select, sparse, weights, evict, compact):
        assert call(so, desc(B=0)) == 0
    assert compact(so, n_max=0) == 0


def binding_calls(bd):
    """Each operator's call of B = 0 sequences (nothing is launched), and its tensors' types by name."""
    d = bd.attn_desc(0, 4, 8, 8, 128, 2, 8)
    b, i, f, w = "bfloat16", "int32", "float32", "int64"
    return [
        (dict(q=b, k_pages=b, v_pages=b, page_table=i, prefix_lens=i, tree_mask=w, out=b, lse=f),
         lambda t: bd.bdlm_tree_attention(d, **t, stream=0)),
        (dict(k_pages=b, v_pages=b, page_table=i, base_lens=i, idx=i, counts=i, to_table=i),
         lambda t: bd.bdlm_compact_kv(d, **t, heads=1, n_max=4, stream=0)),
        (dict(k_pages=b, page_table=i, from_lens=i, to_lens=i, bounds=b),
         lambda t: bd.bdlm_page_bounds(d, **t, stream=0)),
        (dict(q=b, bounds=b, page_table=i, prefix_lens=i, sel_table=i, sel_lens=i),
         lambda t: bd.bdlm_select_pages(d, **t, group=4, n_select=2, sel_cols=4, stream=0)),
        (dict(q=b, k_pages=b, v_pages=b, sel_table=i, sel_lens=i, out=b),
         lambda t: bd.bdlm_sparse_attention(d, **t, group=4, sel_cols=4, stream=0)),
        (dict(q=b, k_pages=b, page_table=i, prefix_lens=i, lse=f, weights=f),
         lambda t: bd.bdlm_attention_weights(d, **t, decay=1.0, stream=0)),
        (dict(k_pages=b, v_pages=b, page_table=i, lens=i, weights=f, to_table=i, to_weights=f, kept=i,
              new_lens=i),
         lambda t: bd.bdlm_evict_kv(d, **t, keep=4, recent=1, stream=0)),
    ]


def test_binding_refuses_other_element_types(so, monkeypatch):
    """An address says nothing of the type behind it: int64 indices (of sort or nonzero), float64 weights
    or float16 queries would be read as something else."""
    import torch

    import block_diffusion_gb300 as bd
    monkeypatch.setattr(bd, "_device", lambda: -1)         # the CPU's tensors stand for the device's
    monkeypatch.setattr(bd, "_raw_stream", lambda dev: 0)
    every = [torch.bfloat16, torch.float16, torch.float32, torch.float64, torch.uint8, torch.int32,
             torch.int64]
    for types, call in binding_calls(bd):
        good = {n: torch.zeros(64, dtype=getattr(torch, t)) for n, t in types.items()}
        call(good)
        for name, t in types.items():
            for other in every:
                if other == getattr(torch, t):
                    continue
                with pytest.raises(bd.BdlmError) as e:
                    call(dict(good, **{name: torch.zeros(64, dtype=other)}))
                assert e.value.status == bd.BDLM_ERR_INVALID, (name, other)
        for name, t in types.items():                       # the same bits under another name pass
            if t == "bfloat16":
                call(dict(good, **{name: good[name].view(torch.int16)}))


@pytest.mark.gpu
def test_binding_refuses_tensors_an_address_would_misread():
    import torch

    import block_diffusion_gb300 as bd
    d = bd.attn_desc(2, 4, 8, 8, 128, 2, 8)
    q = torch.zeros((2, 4, 8, 128), dtype=torch.bfloat16, device="cuda")
    kv = torch.zeros((8, 16, 8, 128), dtype=torch.bfloat16, device="cuda")
    t = torch.zeros((2, 2), dtype=torch.int32, device="cuda")
    n = torch.zeros((2,), dtype=torch.int32, device="cuda")
    lse = torch.zeros((2, 8, 4), device="cuda")
    w = torch.zeros((2, 8, 32), device="cuda")
    for bad in (lse.transpose(1, 2), lse.transpose(1, 2).contiguous().cpu()):
        with pytest.raises(bd.BdlmError) as e:
            bd.bdlm_attention_weights(d, q, kv, t, n, bad, 1.0, w)
        assert e.value.status == bd.BDLM_ERR_INVALID
    bd.bdlm_attention_weights(d, q, kv, t, n, lse.transpose(1, 2).contiguous(), 1.0, w)
    torch.cuda.synchronize()
    assert bd.bdlm_device_error() == 0
