"""Refusals of the operators on the cache's side of a step, on the host, before a GPU is touched; the
frequencies that bdlm_rotary_init makes; and the plain forms' own pins."""
import ctypes
import inspect
import math

import numpy as np
import pytest

import step_ref as R


@pytest.fixture(scope="module")
def so():
    from block_diffusion_gb300 import build, load_library
    build.build()
    return load_library()


P = 0x1000   # never dereferenced


def desc(B=2, L=4, Hq=32, Hkv=8, D=128, cols=10, num=100, **kw):
    import block_diffusion_gb300 as bd
    return ctypes.byref(bd.attn_desc(B, L, Hq, Hkv, D, cols, num, **kw))


def rotary_desc(rot=128):
    import block_diffusion_gb300 as bd
    r = bd.RotaryDesc()
    r.rot_dim, r.amplitude = rot, 1.0
    return ctypes.byref(r)


def tables(so, d=None, old=P, new=P, free=P, n_free=4, frm=P, t=P, lens=P, first=P, rows=8, pos=P, slots=P, nxt=P):
    return so.bdlm_build_tables(desc() if d is None else d, old, new, free, n_free, frm, t, lens, first, rows, pos, slots, nxt, None)


def rotary(so, d=None, r=0, n=4, q=P, qs=0, k=P, ks=0, start=P, pos=P, inv=0, qo=P, ko=P):
    return so.bdlm_rotary(desc() if d is None else d, rotary_desc() if r == 0 else r, n, q, qs, k, ks, start, pos, inv, qo, ko, None)


def write(so, d=None, n=4, first=P, rows=8, kn=P, vn=P, k=P, v=P, sc=P, t=P, lens=P):
    return so.bdlm_write_kv8(desc() if d is None else d, n, first, rows, kn, vn, k, v, sc, t, lens, None)


def attend(so, d=None, q=P, k=P, v=P, sc=P, t=P, n=P, out=P):
    return so.bdlm_attention_kv8(desc() if d is None else d, q, k, v, sc, t, n, out, None)


@pytest.mark.parametrize("call,optional", [(tables, ("frm", "pos", "slots", "nxt")), (rotary, ("start", "pos")), (write, ("first",)), (attend, ())])
def test_null_pointers(so, call, optional):
    names = [n for n, p in inspect.signature(call).parameters.items() if p.default == P]
    for name in names:
        if name not in optional:
            assert call(so, **{name: None}) == -1, name


@pytest.mark.parametrize("call,names", [(rotary, ("q", "k", "qo", "ko")), (write, ("kn", "vn", "k", "v")), (attend, ("q", "k", "v", "out"))])
def test_misaligned_pointers(so, call, names):
    for name in names:
        assert call(so, **{name: P + 8}) == -1, name
    if call is not rotary:
        assert call(so, sc=P + 4) == -1


def test_attention_descriptors(so):
    for bad in (dict(B=-1), dict(L=0), dict(L=65), dict(Hq=30), dict(Hq=0), dict(Hkv=0), dict(D=64), dict(Hq=32, Hkv=1), dict(num=0),
                dict(page_size=32), dict(sm_scale=float("inf")), dict(sm_scale=float("nan")), dict(B=2 ** 30, L=64), dict(cols=0)):
        assert attend(so, desc(**bad)) == -1, bad
    assert attend(so, desc(B=0)) == 0
    assert attend(so, desc(B=0, num=2 ** 27)) == -3 and attend(so, desc(B=0, num=2 ** 27 - 1)) == 0      # 2^30 pages of a head
    assert attend(so, desc(B=1, cols=2 ** 26 + 1)) == -3


def test_write_sizes(so):
    for bad in (dict(B=-1), dict(Hkv=0, Hq=8), dict(D=64), dict(cols=0), dict(num=0), dict(page_size=8), dict(cols=2 ** 28), dict(B=2 ** 29, Hkv=8),
                dict(Hkv=4 * 65535 + 1)):
        assert write(so, desc(**bad)) == -1, bad
    assert write(so, n=0) == -1 and write(so, rows=-1) == -1
    assert write(so, desc(B=2 ** 27, Hkv=1, cols=1), n=2 ** 31 - 1) == -1
    assert write(so, desc(B=0)) == 0


def test_table_sizes(so):
    for bad in (dict(B=-1), dict(cols=0), dict(num=0), dict(page_size=8), dict(B=2 ** 21, cols=2 ** 10)):
        assert tables(so, desc(**bad)) == -1, bad
    assert tables(so, n_free=-1) == -1 and tables(so, rows=-1) == -1
    assert tables(so, desc(num=2 ** 27 + 1)) == -3 and tables(so, desc(B=0, num=2 ** 27)) == 0
    assert tables(so, desc(B=1, cols=2 ** 26 + 1)) == -3


def test_rotary_sizes(so):
    for bad in (dict(B=-1), dict(D=64), dict(Hq=0), dict(Hkv=0), dict(B=2 ** 30)):
        assert rotary(so, desc(**bad)) == -1, bad
    for bad in (dict(n=0), dict(qs=32 * 128 - 8), dict(ks=8 * 128 - 8), dict(qs=32 * 128 + 4), dict(qs=2 ** 41), dict(qs=-8),
                dict(r=None), dict(start=None, pos=None), dict(qo=None), dict(q=None), dict(r=rotary_desc(8)), dict(r=rotary_desc(136)),
                dict(r=rotary_desc(24)), dict(qs=32 * 128 + 8), dict(ks=8 * 128 + 8)):     # (the last: in place with a stride)
        assert rotary(so, **bad) == -1, bad
    assert rotary(so, desc(B=0)) == 0
    assert rotary(so, q=None, qo=None, k=None, ko=None) == 0


def test_rotary_init(so):
    import block_diffusion_gb300 as bd
    good = dict(rot_dim=64, interleaved=False, base=10000.0, scaling=4, factor=4.0, original_len=100.0, few=1.0, many=32.0)
    bd.bdlm_rotary_init(**good)
    nan, inf = float("nan"), float("inf")
    for bad in (dict(rot_dim=0), dict(rot_dim=8), dict(rot_dim=130), dict(rot_dim=144), dict(base=1.0), dict(base=nan), dict(base=inf),
                dict(scaling=-1), dict(scaling=5), dict(factor=0.5), dict(factor=nan), dict(factor=inf), dict(original_len=0.0),
                dict(few=0.0), dict(many=1.0), dict(many=nan), dict(amplitude=-1.0), dict(amplitude=inf), dict(amplitude=nan), dict(amplitude=1e39)):
        with pytest.raises(bd.BdlmError):
            bd.bdlm_rotary_init(**{**good, **bad})
    assert so.bdlm_rotary_init(None, 64, 0, 10000.0, 0, 1.0, 1.0, 1.0, 2.0, 0.0) == -1
    for rot in (16, 48, 128):
        for scaling in range(5):
            args = dict(scaling=scaling, factor=5.0, few=1.0, many=16.0)
            r = bd.bdlm_rotary_init(rot, True, 7000.0, original_len=3000.0, amplitude=0.0, **args)
            f = R.frequencies(rot, 7000.0, original=3000.0, **args)
            got = np.array([t for t in r.turns[:rot // 2]], np.float64) * 2.0 ** -64 * 2 * math.pi
            assert np.all(np.abs(got - f) <= 1e-13 * f + 1e-18)
            assert r.amplitude == pytest.approx(0.1 * math.log(5) + 1 if scaling == 4 else 1.0, rel=1e-6)
            assert r.turns[rot // 2:] == [0] * (64 - rot // 2)
    assert bd.bdlm_rotary_init(64, True, 7000.0, amplitude=1.25).amplitude == 1.25


def test_codes_of_the_plain_form():
    """The plain form's rounding against torch's own, ties and borders among the values."""
    import torch
    assert np.array_equal(R.E4M3[:127], np.sort(R.E4M3[:127])) and R.E4M3[126] == 448 and R.E4M3[1] == 2.0 ** -9
    mids = (R.E4M3[:126] + R.E4M3[1:127]) / 2
    x = np.concatenate((R.E4M3[:127], mids, mids * (1 + 1e-6), mids * (1 - 1e-6), np.random.default_rng(0).normal(0, 60, 5000)))
    x = np.clip(np.concatenate((x, -x)), -448, 448).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(R.encode(x.astype(np.float64)), want)
    assert R.exponent(448.0) == 0 and R.exponent(448.0001) == 1 and R.exponent(0.0) == -40 and R.exponent(1e30) == 40


def binding_calls(bd):
    """Each operator's call of B = 0 sequences (nothing is launched), and its tensors' types by name."""
    d, r = bd.attn_desc(0, 4, 8, 8, 128, 2, 8), bd.bdlm_rotary_init(64, False, 10000.0)
    b, i, f, e = "bfloat16", "int32", "float32", "float8_e4m3fn"
    return [
        (dict(old_lens=i, new_lens=i, free_pages=i, free_from=i, page_table=i, lens_out=i, first=i, positions=i, slots=i, free_next=i),
         lambda t: bd.bdlm_build_tables(d, **t, n_free=4, max_tokens=8, stream=0)),
        (dict(q=b, k=b, start=i, positions=i, q_out=b, k_out=b),
         lambda t: bd.bdlm_rotary(d, r, 4, **t, q_stride=0, k_stride=0, inverse=False, stream=0)),
        (dict(first=i, k_new=b, v_new=b, k_pages=e, v_pages=e, scales=f, page_table=i, prefix_lens=i),
         lambda t: bd.bdlm_write_kv8(d, 4, **t, n_rows=8, stream=0)),
        (dict(q=b, k_pages=e, v_pages=e, scales=f, page_table=i, prefix_lens=i, out=b),
         lambda t: bd.bdlm_attention_kv8(d, **t, stream=0)),
    ]


def test_bindings_refuse_other_element_types(so, monkeypatch):
    import torch

    import block_diffusion_gb300 as bd
    monkeypatch.setattr(bd, "_device", lambda: -1)         # the CPU's tensors stand for the device's
    monkeypatch.setattr(bd, "_raw_stream", lambda dev: 0)
    every = [torch.bfloat16, torch.float16, torch.float32, torch.float64, torch.int8, torch.int32, torch.int64, torch.float8_e4m3fn,
             torch.float8_e5m2]
    for types, call in binding_calls(bd):
        good = {n: torch.zeros((8, 8), dtype=getattr(torch, t)) for n, t in types.items()}
        call(good)
        for name, t in types.items():
            for other in every:
                if other != getattr(torch, t):
                    with pytest.raises(bd.BdlmError) as err:
                        call(dict(good, **{name: torch.zeros((8, 8), dtype=other)}))
                    assert err.value.status == bd.BDLM_ERR_INVALID, (name, other)
            # the same bits under another name pass
            if t in ("bfloat16", "float8_e4m3fn"):
                call(dict(good, **{name: good[name].view(torch.int16 if t == "bfloat16" else torch.uint8)}))
            # parts of a wider tensor do not
            wide = torch.zeros((8, 16), dtype=getattr(torch, t))
            for bad in (wide[:, ::2], wide[:, :8]):
                with pytest.raises(bd.BdlmError):
                    call(dict(good, **{name: bad}))
    types, call = binding_calls(bd)[1]
    good = {n: torch.zeros((8, 8), dtype=getattr(torch, t)) for n, t in types.items()}
    rows = torch.zeros((4, 6, 128), dtype=torch.bfloat16)
    call(dict(good, q=rows[:, :3], k=rows[:, 3:5]))
    call(dict(good, q=rows[:, :1]))
    for bad in (rows[:, ::2], rows[..., :64], rows[..., ::2], rows.transpose(1, 2), rows[0, 0, ::2]):
        with pytest.raises(bd.BdlmError):
            call(dict(good, q=bad))


def test_empty_calls_succeed_without_a_device(so):
    for call in (tables, rotary, write, attend):
        assert call(so, desc(B=0)) == 0
