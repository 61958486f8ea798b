"""The operators over part of the cache as a program runs them together: after a prefill, over a
drafted block, through an eviction; captured into graphs, on another stream, and far into a pool."""
import numpy as np
import pytest

import cache_ref as R
import workloads as W
from gpu_util import bf16_tensor, dev, host

pytestmark = pytest.mark.gpu


def bits(t):
    import torch
    return host(t.view(torch.int16)).view(np.uint16)


def f(t):
    return host(t.float()).astype(np.float64)


def test_a_request_from_prompt_to_eviction(lib):
    """Prefill, a drafted tree verified and its accepted path kept, weights gathered, the cache cut
    back, bounds made, a selection and sparse attention over what is left."""
    import torch
    rng = np.random.default_rng(31)
    B, L, Hq, Hkv, prompt, cols = 3, 8, 8, 2, 192, 16
    pages = B * cols + 2
    table = rng.permutation(pages)[:B * cols].astype(np.int32).reshape(B, cols)
    d = lib.attn_desc(B, L, Hq, Hkv, 128, cols, pages)

    def rows(n, H):
        return W._normal_bf16(rng, (B, n, H, 128), 1.0)

    kp = bf16_tensor(np.zeros((pages, 16, Hkv, 128), np.uint16))
    vp = torch.zeros_like(kp)
    t, zero = dev(table), dev(np.zeros(B, np.int32))
    out = torch.empty((B, prompt, Hq, 128), dtype=torch.bfloat16, device="cuda")
    lib.bdlm_prefill_attention(d, prompt, bf16_tensor(rows(prompt, Hq)), bf16_tensor(rows(prompt, Hkv)),
                               bf16_tensor(rows(prompt, Hkv)), kp, vp, t, zero, out)
    # a drafted tree after the prompt
    lens = np.full(B, prompt, np.int32)
    q = rows(L, Hq)
    lib.bdlm_write_block_kv(d, bf16_tensor(rows(L, Hkv)), bf16_tensor(rows(L, Hkv)), kp, vp, t, dev(lens))
    up = [-1, 0, 0, 1, 1, 2, 3, 5]
    words = []
    for i, u in enumerate(up):
        words.append((words[u] if u >= 0 else 0) | 1 << i)
    mask = np.tile(np.array(words, np.uint64), (B, 1))
    o = torch.empty((B, L, Hq, 128), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((B, L, Hq), device="cuda")
    lib.bdlm_tree_attention(d, bf16_tensor(q), kp, vp, t, dev(lens), dev(mask.view(np.int64)), o, lse)
    k0, v0 = bits(kp), bits(vp)
    want, wl, A, s1 = R.tree_attention(q, k0, v0, table, lens, mask, Hkv)
    R.check_out(f(o), want, A, s1)
    R.check_lse(f(lse), wl, s1)
    # the weight its queries give the prompt
    w = torch.zeros((B, Hkv, cols * 16), device="cuda")
    lib.bdlm_attention_weights(d, bf16_tensor(q), kp, t, dev(lens), lse, 1.0, w)
    ww, add, s1 = R.attention_weights(q, k0, table, lens, host(lse), 1.0, np.zeros(w.shape), Hkv)
    assert np.all(np.abs(f(w) - ww) <= add * (2 * R.score_error(s1) + 2.0 ** -14) + 1e-30)
    # the accepted paths: tokens 0 2 5 7, 0 1, none
    idx = np.array([[[0, 2, 5, 7]], [[0, 1, 0, 0]], [[0, 0, 0, 0]]], np.int32)
    took = np.array([4, 2, 0], np.int32)
    lib.bdlm_compact_kv(d, kp, vp, t, dev(lens), dev(idx), 1, 4, dev(took), t)
    for b in range(B):
        for j in range(took[b]):
            to, frm = prompt + j, prompt + idx[b, 0, j]
            k0[table[b, to // 16], to % 16] = k0[table[b, frm // 16], frm % 16]
            v0[table[b, to // 16], to % 16] = v0[table[b, frm // 16], frm % 16]
    assert np.array_equal(bits(kp), k0) and np.array_equal(bits(vp), v0)
    lens = lens + took
    # cut back to 100 tokens, in place
    keep, recent = 100, 20
    kept = torch.empty((B, Hkv, keep), dtype=torch.int32, device="cuda")
    new = torch.empty((B,), dtype=torch.int32, device="cuda")
    w0 = host(w)
    lib.bdlm_evict_kv(d, kp, vp, t, dev(lens), w, keep, recent, t, w, kept, new)
    torch.cuda.synchronize()
    k1, v1 = k0.copy(), v0.copy()
    for b in range(B):
        for h in range(Hkv):
            r = R.evict(w0[b, h], int(lens[b]), keep, recent)
            assert np.array_equal(host(kept)[b, h], r)
            assert np.array_equal(host(w)[b, h, :keep], w0[b, h, r])
            for j, i in enumerate(r):
                k1[table[b, j // 16], j % 16, h] = k0[table[b, i // 16], i % 16, h]
                v1[table[b, j // 16], j % 16, h] = v0[table[b, i // 16], i % 16, h]
    assert np.array_equal(bits(kp), k1) and np.array_equal(bits(vp), v1)
    lens = host(new)
    assert list(lens) == [keep] * B
    # bounds of what is left, a selection per two queries, and the attention over it
    bounds = torch.zeros((pages, Hkv, 2, 128), dtype=torch.bfloat16, device="cuda")
    lib.bdlm_page_bounds(d, kp, t, None, new, bounds)
    zb = np.zeros((pages, Hkv, 2, 128), np.uint16)
    assert np.array_equal(R.f64(bits(bounds)), R.f64(R.page_bounds(k1, table, [0] * B, lens, zb)))
    sel = torch.empty((B, 4, Hkv, 6), dtype=torch.int32, device="cuda")
    sl = torch.empty((B, 4), dtype=torch.int32, device="cuda")
    lib.bdlm_write_block_kv(d, bf16_tensor(rows(L, Hkv)), bf16_tensor(rows(L, Hkv)), kp, vp, t, new)
    lib.bdlm_select_pages(d, bf16_tensor(q), bounds, t, new, 2, 4, 6, sel, sl)
    lib.bdlm_sparse_attention(d, bf16_tensor(q), kp, vp, 2, 6, sel, sl, o)
    torch.cuda.synchronize()
    ws, wsl = R.select_pages(q, bits(bounds), table, lens, 2, 4, 6, Hkv)
    assert np.array_equal(host(sel), ws) and np.array_equal(host(sl), wsl)
    want, A, s1 = R.sparse_attention(q, bits(kp), bits(vp), ws, wsl, 2, Hkv)
    R.check_out(f(o), want, A, s1)
    assert lib.bdlm_device_error() == 0


class Step:
    """Every operator once over one set of buffers; `__call__` enqueues them on a stream."""

    def __init__(self, lib, seed, B, L, Hq, Hkv, lens, n_sel, keep, at=0, pool=0):
        import torch
        rng = np.random.default_rng(seed)
        self.lib, self.group, self.n_sel, self.keep = lib, L, n_sel, keep
        a = W.make_attention(rng, B, L, Hq, Hkv, 128, prefix_lens=np.asarray(lens), qkv_std=1.0,
                             poison=False)
        cols, n = a.page_table_ref.shape[1], a.k_ref.shape[0]
        pool = max(pool, at + 2 * n)
        self.pool, self.n, self.at = pool, n, at
        self.k = torch.empty((pool, 16, Hkv, 128), dtype=torch.bfloat16, device="cuda")
        self.v = torch.empty_like(self.k)
        self.bounds = torch.empty((pool, Hkv, 2, 128), dtype=torch.bfloat16, device="cuda")
        for x in (self.k, self.v, self.bounds):
            x[at:] = 0
        self.k[at:at + n], self.v[at:at + n] = bf16_tensor(a.k_ref), bf16_tensor(a.v_ref)
        self.t = dev(np.where(a.page_table_ref >= 0, a.page_table_ref + at, -1).astype(np.int32))
        self.to = dev(np.where(a.page_table_ref >= 0, a.page_table_ref + at + n, -1).astype(np.int32))
        self.lens = dev(a.prefix_lens)
        self.q = bf16_tensor(a.q)
        self.d = lib.attn_desc(B, L, Hq, Hkv, 128, cols, pool)
        self.cols = n_sel + (L + 30) // 16

        def empty(*shape, dtype=torch.int32):
            return torch.zeros(shape, dtype=dtype, device="cuda")

        self.mask = dev(rng.integers(1, 2 ** 62, size=(B, L)))
        self.out, self.sparse = torch.zeros_like(self.q), torch.zeros_like(self.q)
        self.lse = empty(B, L, Hq, dtype=torch.float32)
        self.w = empty(B, Hkv, cols * 16, dtype=torch.float32)
        self.tw = torch.zeros_like(self.w)
        self.sel, self.sl = empty(B, 1, Hkv, self.cols), empty(B, 1)
        self.kept, self.new = empty(B, Hkv, keep), empty(B)

    def __call__(self, stream=None):
        lib, d = self.lib, self.d
        lib.bdlm_page_bounds(d, self.k, self.t, None, self.lens, self.bounds, stream=stream)
        lib.bdlm_select_pages(d, self.q, self.bounds, self.t, self.lens, self.group, self.n_sel,
                              self.cols, self.sel, self.sl, stream=stream)
        lib.bdlm_sparse_attention(d, self.q, self.k, self.v, self.group, self.cols, self.sel, self.sl,
                                  self.sparse, stream=stream)
        lib.bdlm_tree_attention(d, self.q, self.k, self.v, self.t, self.lens, self.mask, self.out,
                                self.lse, stream=stream)
        lib.bdlm_attention_weights(d, self.q, self.k, self.t, self.lens, self.lse, 0.5, self.w,
                                   stream=stream)
        lib.bdlm_evict_kv(d, self.k, self.v, self.t, self.lens, self.w, self.keep, 3, self.to, self.tw,
                          self.kept, self.new, stream=stream)

    def results(self):
        import torch
        torch.cuda.synchronize()
        sel = torch.where(self.sel >= 0, self.sel - self.at, -1)
        at = slice(self.at, self.at + 2 * self.n)
        return [x.clone() for x in (self.out, self.lse, self.sparse, sel, self.sl, self.w, self.tw,
                                    self.kept, self.new, self.k[at], self.v[at], self.bounds[at])]

    def clear(self):
        for x in (self.w, self.tw, self.out, self.sparse):
            x.zero_()
        self.kept.fill_(-5)


def same(a, b):
    import torch
    return all(torch.equal(x.view(torch.uint8).reshape(-1) if x.is_floating_point() else x,
                           y.view(torch.uint8).reshape(-1) if y.is_floating_point() else y)
               for x, y in zip(a, b))


SHAPES = [dict(B=2, L=4, Hq=16, Hkv=8, lens=[700, 90], n_sel=20, keep=64),
          dict(B=3, L=40, Hq=32, Hkv=8, lens=[5000, 0, 1800], n_sel=30, keep=100)]


@pytest.mark.parametrize("shape", SHAPES)
def test_graphs_replay_what_eager_calls_compute(lib, shape):
    """Captured on a side stream; a larger call grows the workspace between capture and replay; a
    second graph shares it; replays on another stream and after new inputs."""
    import torch
    x = Step(lib, 1, **shape)
    x()
    eager = x.results()
    x.clear()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        x()
    big = Step(lib, 2, B=8, L=64, Hq=32, Hkv=8, lens=[3000] * 8, n_sel=40, keep=200)
    big()
    want_big = big.results()
    big.clear()
    second = torch.cuda.CUDAGraph()
    with torch.cuda.graph(second, stream=side):
        big()
    for _ in range(2):
        x.clear()
        graph.replay()
        assert same(x.results(), eager)
        big.clear()
        second.replay()
        assert same(big.results(), want_big)
    # new inputs in the same buffers, replayed on another stream
    y = Step(lib, 3, **shape)
    y()
    want = y.results()
    for name in ("q", "k", "v", "t", "to", "lens", "mask", "bounds"):
        getattr(x, name).copy_(getattr(y, name))
    x.clear()
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        graph.replay()
    assert same(x.results(), want)
    assert lib.bdlm_device_error() == 0


def test_an_explicit_stream_and_the_current_one_agree(lib):
    import torch
    x = Step(lib, 5, **SHAPES[0])
    x()
    want = x.results()
    x.clear()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    x(stream=s)
    s.synchronize()
    assert same(x.results(), want)


def test_a_capture_that_would_need_memory_is_refused_and_stays_valid(lib):
    import torch
    x = Step(lib, 6, **SHAPES[1])
    x()
    want = x.results()
    x.clear()
    torch.cuda.synchronize()
    lib.bdlm_release()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        with pytest.raises(lib.BdlmError) as e:
            lib.bdlm_select_pages(x.d, x.q, x.bounds, x.t, x.lens, x.group, x.n_sel, x.cols, x.sel, x.sl)
        assert e.value.status == lib.BDLM_ERR_NOMEM
        x.w.add_(1.0)
    graph.replay()
    torch.cuda.synchronize()
    assert float(x.w.min()) == 1.0
    x.clear()
    x()
    assert same(x.results(), want)


def test_pages_far_into_a_pool(lib):
    """Page ids whose elements lie past 2^31: the same step at the pool's start and at its end."""
    import torch
    shape = dict(B=2, L=4, Hq=16, Hkv=8, lens=[900, 333], n_sel=20, keep=64)
    x = Step(lib, 7, **shape)
    x()
    want = x.results()
    y = Step(lib, 7, **shape, at=140000, pool=140000 + 2 * x.n + 1)
    y()
    assert same(y.results(), want)
    assert lib.bdlm_device_error() == 0
    del y
    torch.cuda.empty_cache()
