"""The rotary binding reads q and k by a stride that the caller gives: tensors laid out otherwise are refused (on the host; the
library's call is a stand-in that records what it gets)."""
import pytest


@pytest.fixture
def call(monkeypatch):
    import torch

    import block_diffusion_gb300 as bd
    monkeypatch.setattr(bd, "_device", lambda: -1)         # the CPU's tensors stand for the device's
    monkeypatch.setattr(bd, "_raw_stream", lambda dev: 0)

    class Library:
        def bdlm_rotary(self, desc, rotary, n, q, q_stride, k, k_stride, *rest):
            self.got = q, q_stride, k, k_stride
            return 0

        def bdlm_status_string(self, status):
            return b""

    lib = Library()
    monkeypatch.setattr(bd, "load_library", lambda: lib)
    start, out = torch.zeros(8, dtype=torch.int32), torch.zeros(1, dtype=torch.bfloat16)

    def rotary(B, n, q=None, q_stride=0, k=None, k_stride=0, Hq=4, Hkv=2):
        d = bd.attn_desc(B, 1, Hq, Hkv, 128, 1, 1)
        bd.bdlm_rotary(d, bd.RotaryDesc(), n, q, q_stride, k, k_stride, start, None, False, None if q is None else out, None if k is None else out)
        return lib.got

    def refused(*args, **kw):
        with pytest.raises(bd.BdlmError) as e:
            rotary(*args, **kw)
        assert e.value.status == bd.BDLM_ERR_INVALID

    rotary.refused = refused
    return rotary


def tensor(*shape):
    import torch
    return torch.zeros(shape, dtype=torch.bfloat16)


def test_slices_of_a_projection(call):
    qkv = tensor(3, 5, 8, 128)
    q, k, v = qkv[:, :, :4], qkv[:, :, 4:6], qkv[:, :, 6:]
    assert call(3, 5, q, 1024, k, 1024) == (q.data_ptr(), 1024, k.data_ptr(), 1024)
    call(15, 1, qkv.view(15, 8, 128)[:, :4], 1024)
    call(3, 5, k=v, k_stride=1024)
    for stride in (0, 512, 1016, 1032, 2048):             # 0: dense, which these are not
        call.refused(3, 5, q, stride)
        call.refused(3, 5, k=k, k_stride=stride)
    call(0, 5, q, 0)                                       # (nothing is read)


def test_tokens_of_a_longer_tensor(call):
    x = tensor(3, 9, 4, 128)
    call.refused(3, 5, x[:, :5], 0)                        # the second sequence's tokens are 9 further on, not 5
    call.refused(3, 5, x[:, :5], 9 * 512)
    call.refused(3, 5, x[:, ::2], 1024)
    call(1, 5, x[:1, :5], 0)                               # one sequence's do lie together,
    call(3, 1, x[:, :1], 9 * 512)                          # and single tokens at one distance
    call(3, 9, x, 0)
    call.refused(3, 1, x[:, :1], 0)
    call.refused(2, 9, x[1:].expand(2, 9, 4, 128).transpose(0, 1), 0)
    call.refused(3, 9, x[:1].expand(3, 9, 4, 128), 0)      # a broadcast one


def test_fewer_tokens_than_the_call_reads(call):
    x, wide = tensor(3, 5, 4, 128), tensor(3, 5, 8, 128)
    call.refused(3, 6, x, 0)
    call.refused(4, 5, x, 0)
    call.refused(3, 5, x, 1024)                            # a dense tensor is not 1024 apart
    call.refused(3, 6, wide[:, :, :4], 1024)
    call.refused(3, 5, wide[:, :, 5:], 1024)               # 3 heads of 4
    call.refused(3, 5, wide.view(-1)[:-1], 0, Hq=8)
    call(2, 5, x, 0)                                       # more of them than it reads


def test_dense_tensors_of_any_shape(call):
    x, wide = tensor(3, 5, 4, 128), tensor(3, 5, 8, 128)
    for shape in ((15, 4, 128), (15, 512), (60, 128), (3, 20, 128), (3, 5, 512), (-1,)):
        call(3, 5, x.view(shape), 0)
        call(3, 5, x.view(shape), 512)
    for shape in ((15, 8, 128), (15, 1024), (3, 5, 1024)):  # q as the first heads of whole rows
        call(3, 5, wide.view(shape), 1024)
    call(1, 1, tensor(4, 128), 4096)                       # one token: no stride
    call(3, 5, x.data_ptr(), 4096)                         # an address is the caller's


def test_heads_in_two_dimensions(call):
    """A token's heads as [Hkv, G]: packed in the wider tensor, or with others between them."""
    x = tensor(3, 5, 3, 2, 128)
    call(3, 5, x[:, :, :2], 768)
    call.refused(3, 5, x[:, :, :2], 0)
    call.refused(3, 5, x[:, :, :, :1], 768, Hq=3)
    call.refused(3, 5, x[:, :, :1], 768)
    call(15, 1, x.view(15, 3, 2, 128)[:, 1:], 768)
    call(3, 5, tensor(3, 5, 4, 1, 128)[:, :, 1:, :], 512, Hq=3)
