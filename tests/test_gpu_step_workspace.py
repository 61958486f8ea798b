"""The workspaces of the operators on the cache's side of a step: growth inside a capture, what captured graphs
keep, and graphs that share one."""
import numpy as np
import pytest

import step_ref as R
import workloads as W
from gpu_util import bf16_tensor, dev, host
from test_gpu_kv8 import Cache

pytestmark = pytest.mark.gpu


class Calls:
    """Small calls of every new entry point; attention in its three forms."""

    def __init__(self, lib, seed=0):
        import torch
        rng = np.random.default_rng(seed)
        self.lib = lib
        self.c = Cache(rng, np.array([2000, 70, 900]), 2)
        self.k, self.v, self.s, self.t = self.c.dev()
        i32 = dict(dtype=torch.int32, device="cuda")
        self.outs = []
        for L, Hq in ((1, 4), (16, 4), (64, 8)):
            q = bf16_tensor(W._normal_bf16(rng, (3, L, Hq, 128), 1.0))
            out = torch.zeros_like(q)
            self.outs.append(out)
            setattr(self, "attend%d" % L, self._attend(q, L, Hq, out))
        self.old, self.new = torch.zeros(3, **i32), dev(np.array([40, 0, 7], np.int32))
        self.free = torch.arange(20, **i32)
        self.table, self.lens, self.first = torch.full((3, 4), -1, **i32), torch.zeros(3, **i32), torch.zeros(4, **i32)
        self.pos, self.slots, self.next = torch.zeros(9000, **i32), torch.zeros(9000, **i32), torch.zeros(1, **i32)
        self.x, self.y = (bf16_tensor(W._normal_bf16(rng, (12, 2, 128), 1.0)) for _ in range(2))
        self.rot = lib.bdlm_rotary_init(64, False, 10000.0)
        self.turned = torch.zeros_like(self.x)
        self.outs += [self.table, self.lens, self.first, self.pos, self.slots, self.next, self.turned]

    def _attend(self, q, L, Hq, out):
        d, n = self.lib.attn_desc(3, L, Hq, 2, 128, self.c.cols, self.c.pages), dev(self.c.lens - L if L < 70 else self.c.lens)
        return lambda: self.lib.bdlm_attention_kv8(d, q, self.k, self.v, self.s, self.t, n, out)

    def tables(self):
        self.lib.bdlm_build_tables(self.lib.attn_desc(3, 1, 1, 1, 128, 4, 20), self.old, self.new, self.free, 20, None, self.table,
                                   self.lens, self.first, 9000, self.pos, self.slots, self.next)

    def few_tables(self):
        self.lib.bdlm_build_tables(self.lib.attn_desc(3, 1, 1, 1, 128, 4, 20), self.old, self.new, self.free, 20, None, self.table,
                                   self.lens, self.first, 100, self.pos, self.slots, self.next)

    def rotary(self):
        self.lib.bdlm_rotary(self.lib.attn_desc(3, 1, 2, 2, 128, 1, 1), self.rot, 4, None, 0, self.x, 0, self.old, None, False, None, self.turned)

    def write(self):
        self.lib.bdlm_write_kv8(self.lib.attn_desc(3, 1, 2, 2, 128, self.c.cols, self.c.pages), 4, None, 0, self.x, self.y, self.k, self.v,
                                self.s, self.t, self.old)


SCRATCH = ["attend1", "attend16", "attend64", "tables", "few_tables"]


@pytest.mark.parametrize("name", SCRATCH)
def test_growth_in_a_capture_is_refused_and_the_capture_stays_valid(lib, name):
    import torch
    c = Calls(lib)
    call = getattr(c, name)
    x = torch.zeros((), device="cuda")
    torch.cuda.synchronize()
    lib.bdlm_release()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        with pytest.raises(lib.BdlmError) as e:
            call()
        x.add_(1.0)
    assert e.value.status == lib.BDLM_ERR_NOMEM
    graph.replay()
    torch.cuda.synchronize()
    assert float(x) == 1.0
    call()
    want = [o.clone() for o in c.outs]
    for o in c.outs:
        o.zero_()
    with torch.cuda.graph(second := torch.cuda.CUDAGraph(), stream=torch.cuda.Stream()):
        call()
    c.table.fill_(-1)
    second.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(c.outs, want) if o is not c.table)
    assert lib.bdlm_device_error() == 0


def test_calls_without_scratch_are_captured_after_a_release(lib):
    """The rotary call and the write take nothing from the workspace."""
    import torch
    c = Calls(lib)
    torch.cuda.synchronize()
    c.rotary()
    c.write()
    want = c.turned.clone(), c.k.clone(), c.s.clone()
    torch.cuda.synchronize()
    lib.bdlm_release()
    c.turned.zero_()
    with torch.cuda.graph(graph := torch.cuda.CUDAGraph(), stream=torch.cuda.Stream()):
        c.rotary()
        c.write()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(c.turned, want[0]) and torch.equal(c.k, want[1]) and torch.equal(c.s, want[2])


def test_two_graphs_share_the_workspace_in_turn(lib):
    """Graphs of different forms and sizes, replayed in turn, between eager calls and after the workspace grew."""
    import torch
    a, b = Calls(lib, 1), Calls(lib, 2)
    steps = ["attend64", "tables", "attend1", "attend16"]
    torch.cuda.synchronize()
    lib.bdlm_release()
    graphs = []
    for c in (a, b):
        for name in steps:
            getattr(c, name)()
        torch.cuda.synchronize()
        c.want = [o.clone() for o in c.outs[:3]]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=torch.cuda.Stream()):
            for name in steps:
                getattr(c, name)()
        graphs.append(g)
    rng = np.random.default_rng(3)
    for turn in range(3):
        for c, g in zip((a, b), graphs):
            for o in c.outs[:3]:
                o.zero_()
            g.replay()
            g.replay()
        # a larger problem, with more lists than CTAs, between them
        B = 60 + 40 * turn
        big = Cache(rng, rng.integers(1, 300, B) + 4, 8)
        q = W._normal_bf16(rng, (B, 4, 16, 128), 1.0)
        k, v, s, t = big.dev()
        out = torch.empty((B, 4, 16, 128), dtype=torch.bfloat16, device="cuda")
        lib.bdlm_attention_kv8(lib.attn_desc(B, 4, 16, 8, 128, big.cols, big.pages), bf16_tensor(q), k, v, s, t, dev(big.lens - 4), out)
        torch.cuda.synchronize()
        for c in (a, b):
            assert all(torch.equal(o, w) for o, w in zip(c.outs, c.want))
        R.check_attention(host(out.float()).astype(np.float64),
                          R.attention_kv8(q, big.k, big.v, big.scales, big.table, big.lens - 4, 8))
    assert lib.bdlm_device_error() == 0


def test_the_old_and_the_new_attention_share_counters(lib):
    """bf16 block attention (whose scheduler counts in the same words) between calls of the 8-bit one."""
    import torch
    rng = np.random.default_rng(5)
    c = Calls(lib)
    n = W.make_attention(rng, 64, 4, 32, 8, 128, prefix_lens=rng.integers(0, 900, 64), poison=False)
    q, k, v = bf16_tensor(n.q), bf16_tensor(n.k_ref), bf16_tensor(n.v_ref)
    t, l = dev(n.page_table_ref), dev(n.prefix_lens)
    d = lib.attn_desc(64, 4, 32, 8, 128, n.page_table_ref.shape[1], n.k_ref.shape[0])
    out = torch.zeros_like(q)
    big = Cache(rng, rng.integers(1, 500, 80) + 1, 8)
    bq = bf16_tensor(W._normal_bf16(rng, (80, 1, 8, 128), 1.0))
    bk, bv, bs, bt = big.dev()
    bd, bl, bo = lib.attn_desc(80, 1, 8, 8, 128, big.cols, big.pages), dev(big.lens - 1), torch.zeros_like(bq)
    want = None
    for _ in range(4):
        lib.bdlm_block_attention(d, q, k, v, t, l, 4, out)
        lib.bdlm_attention_kv8(bd, bq, bk, bv, bs, bt, bl, bo)
        c.attend64()
        torch.cuda.synchronize()
        got = out.clone(), bo.clone(), c.outs[2].clone()
        if want is not None:
            assert all(torch.equal(a, b) for a, b in zip(got, want))
        want = got
    assert lib.bdlm_device_error() == 0
