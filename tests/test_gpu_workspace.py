"""The library workspace: growth inside a capture, allocations that fail, what a captured graph keeps
and what is given back."""
import os
import subprocess
import sys

import numpy as np
import pytest

import workloads as W
from gpu_util import bf16_tensor, dev, host

pytestmark = pytest.mark.gpu

P = 0x1000   # an address that no kernel gets: the calls that take it fail before any launch


class Calls:
    """One small call of every entry point that takes scratch from the workspace."""

    def __init__(self, lib):
        import torch
        rng = np.random.default_rng(21)
        a = W.make_attention(rng, 2, 4, 32, 8, 128, prefix_lens=np.array([9000, 64]), poison=False)
        self.lib, self.a = lib, a
        self.q, self.k, self.v = bf16_tensor(a.q), bf16_tensor(a.k_ref), bf16_tensor(a.v_ref)
        self.t, self.n = dev(a.page_table_ref), dev(a.prefix_lens)
        self.d = lib.attn_desc(2, 4, 32, 8, 128, a.page_table_ref.shape[1], a.k_ref.shape[0])
        self.out = torch.zeros_like(self.q)
        self.kn = torch.zeros((2, 4, 8, 128), dtype=torch.bfloat16, device="cuda")
        self.zero = dev(np.zeros(2, np.int32))
        self.mask = torch.ones((2, 4), dtype=torch.uint8, device="cuda")
        self.tok = torch.zeros((2, 4), dtype=torch.int32, device="cuda")
        self.conf = torch.zeros((2, 4), device="cuda")
        self.com = torch.zeros((2, 4), dtype=torch.uint8, device="cuda")
        self.hidden = torch.ones((8, 64), dtype=torch.bfloat16, device="cuda")
        self.w = torch.ones((512, 64), dtype=torch.bfloat16, device="cuda")
        self.rows = torch.arange(8, dtype=torch.int32, device="cuda")
        self.count = dev(np.array([8], np.int32))
        self.logits = torch.zeros((8, 512), dtype=torch.bfloat16, device="cuda")
        self.bounds = torch.zeros((a.k_ref.shape[0], 8, 2, 128), dtype=torch.bfloat16, device="cuda")
        self.sel = torch.zeros((2, 1, 8, 12), dtype=torch.int32, device="cuda")
        self.sl = torch.zeros((2, 1), dtype=torch.int32, device="cuda")

    def block_attention(self):
        self.lib.bdlm_block_attention(self.d, self.q, self.k, self.v, self.t, self.n, 4, self.out)

    def block_attention_kv(self):
        self.lib.bdlm_block_attention_kv(self.d, self.q, self.kn, self.kn, self.k, self.v, self.t,
                                         self.n, 4, self.out)

    def prefill(self):
        self.lib.bdlm_prefill_attention(self.d, 4, self.q, self.kn, self.kn, self.k, self.v, self.t,
                                        self.zero, self.out)

    def tree_attention(self):
        self.lib.bdlm_tree_attention(self.d, self.q, self.k, self.v, self.t, self.n, None, self.out)

    def select_pages(self):
        self.lib.bdlm_select_pages(self.d, self.q, self.bounds, self.t, self.n, 4, 10, 12, self.sel, self.sl)

    def commit(self):
        self.lib.bdlm_confidence_commit(self.logits, self.mask, 2, 4, 512, 0.5, 1.0, self.tok, self.conf,
                                        self.com)

    def commit_rule(self):
        self.lib.bdlm_confidence_commit_rule(self.logits, self.mask, 2, 4, 512,
                                             self.lib.BDLM_COMMIT_TOPK, 1, 0.5, 1.0, self.tok, self.conf,
                                             self.com)

    def lm_head(self):
        self.lib.bdlm_lm_head(self.hidden, self.w, self.rows, 8, 8, 64, 512, self.logits)

    def lm_head_device_count(self):
        self.lib.bdlm_lm_head_device_count(self.hidden, self.w, self.rows, self.count, 8, 8, 64, 512,
                                           self.logits)

    def lm_head_commit(self):
        self.lib.bdlm_lm_head_commit(self.hidden, self.w, self.mask, None, 2, 4, 64, 512,
                                     self.lib.BDLM_COMMIT_TOPK, 1, 0.5, 1.0, self.tok, self.conf, self.com)


def huge_selection(lib):
    """A selection whose scratch (3.3 TB) no GPU has."""
    d = lib.attn_desc(2048, 64, 8, 8, 128, 262144, 100)
    with pytest.raises(lib.BdlmError) as e:
        lib.bdlm_select_pages(d, P, P, P, P, 1, 8, 16, P, P)
    assert e.value.status == lib.BDLM_ERR_NOMEM


def test_an_allocation_that_failed_leaves_no_error_behind(lib):
    """The calls after it succeed and compute what they computed before."""
    import torch
    c = Calls(lib)
    names = [n for n in vars(Calls) if not n.startswith("_")]
    k, v = c.k.clone(), c.v.clone()
    c.block_attention()
    want = host(c.out.float())
    for name in names:
        huge_selection(lib)
        getattr(c, name)()
    huge_selection(lib)
    c.out.zero_()
    c.k.copy_(k)   # (two of the calls write K and V)
    c.v.copy_(v)
    c.block_attention()
    torch.cuda.synchronize()
    assert np.array_equal(host(c.out.float()), want)
    assert lib.bdlm_device_error() == 0
CAPTURED = ["block_attention", "block_attention_kv", "prefill", "tree_attention", "select_pages", "commit",
            "commit_rule", "lm_head", "lm_head_device_count", "lm_head_commit"]


@pytest.mark.parametrize("name", CAPTURED)
def test_growth_in_a_capture_is_refused_and_the_capture_stays_valid(lib, name):
    """Every entry point that takes scratch: with the workspace released the captured call is refused,
    and what is captured beside it replays; after a call outside it is captured and replays."""
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
    outs = (c.out, c.tok, c.conf, c.com, c.logits, c.sel, c.sl)
    want = [o.clone() for o in outs]
    for o in outs:
        o.zero_()
    with torch.cuda.graph(second := torch.cuda.CUDAGraph(), stream=torch.cuda.Stream()):
        call()
    second.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))
    assert lib.bdlm_device_error() == 0


def test_a_refused_prefill_has_written_nothing(lib):
    """Room for its prompts' table but not for its attention: the K/V write is not captured either."""
    import torch
    c = Calls(lib)
    torch.cuda.synchronize()
    lib.bdlm_release()
    c.prefill()
    wide = torch.zeros((2, 16384), dtype=torch.int32, device="cuda")
    wide[:, :c.t.shape[1]] = c.t
    d = lib.attn_desc(2, 4, 32, 8, 128, 16384, c.k.shape[0])
    c.k.fill_(3.0)
    with torch.cuda.graph(graph := torch.cuda.CUDAGraph(), stream=torch.cuda.Stream()):
        with pytest.raises(lib.BdlmError) as e:
            lib.bdlm_prefill_attention(d, 4, c.q, c.kn, c.kn, c.k, c.v, wide, c.zero, c.out)
        c.out.zero_()
    assert e.value.status == lib.BDLM_ERR_NOMEM
    graph.replay()
    torch.cuda.synchronize()
    assert float(c.k.float().min()) == 3.0
    assert lib.bdlm_device_error() == 0


def test_a_loop_relaunched_in_a_capture_is_refused_where_it_would_need_memory(lib):
    import torch
    from test_gpu_round_loop import Case
    c = Case(5, B=4)
    mask, den = dev(c.mask0), dev(c.den)
    tok = torch.zeros((c.S, c.B, c.L), dtype=torch.int32, device="cuda")
    conf = torch.zeros((c.S, c.B, c.L), device="cuda")
    com = torch.zeros((c.S, c.B, c.L), dtype=torch.uint8, device="cuda")
    done = torch.zeros((1,), dtype=torch.int32, device="cuda")
    loop = lib.bdlm_round_loop_create(lib.round_loop_desc(
        c.desc(lib), c.S, c.H, c.V, lib.BDLM_COMMIT_TOPK, 1, 0.5, 1.0, q_steps=c.q, k_new_steps=c.kn,
        v_new_steps=c.vn, hidden_steps=c.hid, k_pages=c.k0, v_pages=c.v0, page_table=c.pt,
        prefix_lens=c.pl, w=c.w, mask=mask, denoising=den, tok_steps=tok, conf_steps=conf,
        commit_steps=com, steps_done=done))
    try:
        torch.cuda.synchronize()
        lib.bdlm_release()
        x = torch.zeros((), device="cuda")
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
            with pytest.raises(lib.BdlmError) as e:
                lib.bdlm_round_loop_launch(loop)
            x.add_(1.0)
        assert e.value.status == lib.BDLM_ERR_NOMEM
        graph.replay()
        lib.bdlm_round_loop_launch(loop)
        torch.cuda.synchronize()
        assert float(x) == 1.0 and 1 <= int(done) <= c.S
    finally:
        lib.bdlm_round_loop_destroy(loop)


FIRST = """
import sys
sys.path[:0] = [{root!r}, {tests!r}]
import torch
import block_diffusion_gb300 as bd
from test_gpu_workspace import Calls
c = Calls(bd)
x = torch.zeros((), device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g, stream=torch.cuda.Stream()):
    try:
        c.lm_head()
        raise SystemExit("not refused")
    except bd.BdlmError as e:
        assert e.status == bd.BDLM_ERR_NOMEM, e
    x.add_(1.0)
g.replay()
c.lm_head()
torch.cuda.synchronize()
assert float(x) == 1.0 and float(c.logits.float().min()) == 64.0
assert bd.bdlm_device_error() == 0
print("fine")
"""


def test_a_process_whose_first_call_is_captured(lib):
    """The library's first call on a device sets up its error word, which is memory too."""
    tests = os.path.dirname(os.path.abspath(__file__))
    code = FIRST.format(root=os.path.dirname(tests), tests=tests)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "fine", r.stdout + r.stderr


def test_a_workspace_that_no_capture_used_is_given_back_when_it_grows(lib):
    """Growing from 0.8 to 1.6 GB leaves about a quarter more than the need held, not both buffers."""
    import torch
    table = torch.zeros((1, 262144), dtype=torch.int32, device="cuda")
    lens = dev(np.array([0], np.int32))

    def select(L, Hkv):   # scratch: 12 bytes per list and page of the table, L * Hkv lists
        q = torch.zeros((1, L, Hkv, 128), dtype=torch.bfloat16, device="cuda")
        bounds = torch.zeros((1, Hkv, 2, 128), dtype=torch.bfloat16, device="cuda")
        sel = torch.zeros((1, L, Hkv, 8), dtype=torch.int32, device="cuda")
        sl = torch.zeros((1, L), dtype=torch.int32, device="cuda")
        d = lib.attn_desc(1, L, Hkv, Hkv, 128, 262144, 1)
        lib.bdlm_select_pages(d, q, bounds, table, lens, 1, 2, 8, sel, sl)
        torch.cuda.synchronize()

    torch.cuda.synchronize()
    lib.bdlm_release()
    select(1, 8)
    lib.bdlm_release()
    torch.cuda.empty_cache()
    free = torch.cuda.mem_get_info()[0]
    for L in (32, 64, 64):
        select(L, 8)
    torch.cuda.empty_cache()
    held = free - torch.cuda.mem_get_info()[0]
    need = 64 * 8 * 262144 * 12
    assert need <= held <= 1.25 * need + 2 ** 28, held / need
    lib.bdlm_release()


def test_a_workspace_that_a_graph_uses_outlives_growth(lib):
    """The graph replays in the memory it was captured with; later growth, which no graph has seen,
    gives its buffers back."""
    import torch
    c = Calls(lib)
    torch.cuda.synchronize()
    lib.bdlm_release()
    c.block_attention()
    want = host(c.out.float())
    with torch.cuda.graph(graph := torch.cuda.CUDAGraph(), stream=torch.cuda.Stream()):
        c.block_attention()
    for rows in (512, 4096, 32768):
        hidden = torch.zeros((rows, 1024), dtype=torch.bfloat16, device="cuda")
        lib.bdlm_lm_head(hidden, hidden[:512], torch.arange(rows, dtype=torch.int32, device="cuda"), rows,
                         rows, 1024, 512, torch.empty((rows, 512), dtype=torch.bfloat16, device="cuda"))
        junk = torch.full((2 ** 24,), 7.0, device="cuda")   # whatever was freed gets written
        c.out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(host(c.out.float()), want)
        del junk
    assert lib.bdlm_device_error() == 0
