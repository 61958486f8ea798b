"""The library workspace: growth inside a capture, allocations that fail, what a captured graph keeps
and what is given back."""
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
        a = W.make_attention(rng, 2, 4, 32, 8, 128, prefix_lens=np.array([5000, 64]), poison=False)
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
