"""Page tables, slot maps and rotary positions against plain forms; the operators of a step as they are run
together."""
import numpy as np
import pytest

import step_ref as R
import workloads as W
from gpu_util import bf16_tensor, dev, host

pytestmark = pytest.mark.gpu


def f(t):
    return host(t.float()).astype(np.float64)


def build(lib, old, new, free, table, max_tokens, num_pages, start=0, from_arg=True):
    import torch
    B, cols = table.shape
    d = lib.attn_desc(B, 1, 1, 1, 128, cols, num_pages)
    t = dev(table)
    lens, first = torch.full((B,), -7, dtype=torch.int32, device="cuda"), torch.full((B + 1,), -7, dtype=torch.int32, device="cuda")
    pos, slots = (torch.full((max(1, max_tokens),), -7, dtype=torch.int32, device="cuda") for _ in range(2))
    nxt = torch.full((1,), -7, dtype=torch.int32, device="cuda")
    lib.bdlm_build_tables(d, dev(old), dev(new), dev(free) if len(free) else None, len(free),
                          dev(np.array([start], np.int32)) if from_arg else None, t, lens, first, max_tokens, pos, slots, nxt)
    return host(t), host(lens), host(first), host(pos)[:max_tokens], host(slots)[:max_tokens], int(host(nxt)[0])


def check(lib, old, new, free, table, max_tokens, num_pages, start=0, **kw):
    got = build(lib, old, new, free, table, max_tokens, num_pages, start, **kw)
    want = R.build_tables(old, new, free, start, table, max_tokens, num_pages)
    for name, g, w in zip(("table", "lens", "first", "positions", "slots", "next"), got, want):
        assert np.array_equal(g, w), name
    return got


def batch(rng, B, hi, grow, spare=1.0):
    old = rng.integers(0, hi + 1, B).astype(np.int32)
    new = (old + rng.integers(0, grow + 1, B)).astype(np.int32)
    held = (old + 15) // 16
    need = int(((new + 15) // 16 - held).sum())
    cols = (hi + grow + 15) // 16 + 1
    n_free = int(need * spare)
    ids = rng.permutation(int(held.sum()) + n_free + 5).astype(np.int32)
    table = np.full((B, cols), -1, np.int32)
    at = 0
    for b in range(B):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    return old, new, ids[at:at + n_free], table, len(ids)


@pytest.mark.parametrize("B,hi,grow", [(1, 0, 1), (1, 5, 0), (3, 40, 4), (64, 100, 16), (130, 300, 40), (1024, 64, 4), (1025, 64, 5),
                                       (2500, 20, 3), (40, 0, 700)])
@pytest.mark.parametrize("spare", [1.0, 0.6, 0.0])
def test_tables(lib, B, hi, grow, spare):
    rng = np.random.default_rng(B + grow)
    old, new, free, table, pages = batch(rng, B, hi, grow, spare)
    check(lib, old, new, free, table, B * max(grow, 1), pages)
    assert lib.bdlm_device_error() == 0


@pytest.mark.parametrize("max_tokens", [0, 1, 50, 500, 6000])
def test_tables_of_few_rows(lib, max_tokens):
    """Rows that do not suffice: from the first sequence that does not fit, none with new tokens is served."""
    rng = np.random.default_rng(4)
    old, new, free, table, pages = batch(rng, 40, 90, 30)
    new[7] = old[7]
    new[20] = old[20] // 2                       # shorter: nothing to add
    got = check(lib, old, new, free, table, max_tokens, pages)
    assert got[1][20] == new[20] and got[2][-1] <= max_tokens


def test_tables_from_within_the_list(lib):
    rng = np.random.default_rng(5)
    old, new, free, table, pages = batch(rng, 30, 90, 30, 2.0)
    for start in (0, 3, len(free) // 2, len(free)):
        check(lib, old, new, free, table, 1000, pages, start)
    check(lib, old, new, free, table, 1000, pages, 0, from_arg=False)


def test_tables_of_bad_values(lib):
    """Lengths that do not fit, a start outside the list, page ids outside the pool."""
    rng = np.random.default_rng(6)
    old, new, free, table, pages = batch(rng, 12, 90, 30)
    cap = table.shape[1] * 16
    old[1], new[2], new[3], old[4] = -3, cap + 1, -1, cap + 9
    new[5] = 2 ** 31 - 1
    got = check(lib, old, new, free, table, 1000, pages)
    assert lib.bdlm_device_error() == lib.BDLM_DEVERR_LENGTH
    old, new, free, table, pages = batch(rng, 12, 90, 30)
    for start in (-1, len(free) + 1, 2 ** 31 - 1):
        got = build(lib, old, new, free, table, 1000, pages, start)
        assert lib.bdlm_device_error() == lib.BDLM_DEVERR_ROW
        assert np.array_equal(got[0], table)
    free[0], free[1] = pages, -9
    check(lib, old, new, free, table, 1000, pages)
    assert lib.bdlm_device_error() == lib.BDLM_DEVERR_PAGE


def test_tables_in_place_step_by_step(lib):
    """Lengths and the list's place updated in place, no rows wanted or a wide map, in a captured graph."""
    import torch
    B, cols, pages = 6, 8, 60
    rng = np.random.default_rng(7)
    free = rng.permutation(pages).astype(np.int32)
    d = lib.attn_desc(B, 1, 1, 1, 128, cols, pages)
    grow = np.array([3, 0, 16, 5, 1, 20], np.int32)
    lens, add = dev(np.zeros(B, np.int32)), dev(grow)
    t, fr, at = dev(np.full((B, cols), -1, np.int32)), dev(free), dev(np.zeros(1, np.int32))
    first = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    pos = torch.zeros(5000, dtype=torch.int32, device="cuda")
    slots = torch.zeros(5000, dtype=torch.int32, device="cuda")
    want = torch.zeros(B, dtype=torch.int32, device="cuda")

    def step():
        torch.add(lens, add, out=want)
        lib.bdlm_build_tables(d, lens, want, fr, pages, at, t, lens, first, 5000, pos, slots, at)

    step()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        step()
    for _ in range(2):
        g.replay()
    table, l, a = np.full((B, cols), -1, np.int32), np.zeros(B, np.int32), 0
    for _ in range(3):
        table, l, fi, ps, sl, a = R.build_tables(l, l + grow, free, a, table, 5000, pages)
    for got, w in ((t, table), (lens, l), (first, fi), (pos, ps), (slots, sl)):
        assert np.array_equal(host(got), w)
    assert int(host(at)[0]) == a
    lib.bdlm_build_tables(d, lens, want, fr, pages, None, t, want, first, 5000, None, None, None)
    assert lib.bdlm_device_error() == 0


CASES = [(128, False, 0), (128, True, 0), (64, False, 1), (96, True, 4), (16, True, 2), (32, False, 3), (112, False, 4)]


@pytest.mark.parametrize("rot,inter,scaling", CASES)
@pytest.mark.parametrize("B,n,Hq,Hkv", [(1, 1, 1, 1), (3, 5, 5, 1), (2, 9, 16, 8), (1, 130, 40, 4)])
def test_rotary(lib, rot, inter, scaling, B, n, Hq, Hkv):
    """Against the formula; both directions; slices of a wider tensor; far positions; padding."""
    import torch
    rng = np.random.default_rng(rot + n)
    args = dict(scaling=scaling, factor=6.0, few=1.0, many=8.0 if scaling == 3 else 32.0)
    r = lib.bdlm_rotary_init(rot, inter, 10000.0, original_len=2048.0, **args)
    freq = R.frequencies(rot, 10000.0, original=2048.0, **args)
    amp = float(np.float32(0.1 * np.log(6.0) + 1)) if scaling == 4 else 1.0
    assert abs(r.amplitude - amp) <= 1e-7
    start = rng.integers(0, 10 ** 6, B).astype(np.int32)
    start[-1] = 2 ** 31 - 1 - n if B > 1 else start[-1]
    at = start[:, None].astype(np.int64) + np.arange(n)
    qkv = W._normal_bf16(rng, (B, n, Hq + 2 * Hkv, 128), 1.0)
    t = bf16_tensor(qkv)
    q, k = t[:, :, :Hq], t[:, :, Hq:Hq + Hkv]
    wide = (Hq + 2 * Hkv) * 128
    d = lib.attn_desc(B, 1, Hq, Hkv, 128, 1, 1)
    for inverse in (False, True):
        for given in (False, True):
            pos = at.copy()
            if given:
                pos[rng.random(pos.shape) < 0.3] = -1
                pos[pos >= 0] = rng.integers(0, 2 ** 31, int((pos >= 0).sum()))
            qo, ko = (torch.full((B, n, H, 128), 3.0, dtype=torch.bfloat16, device="cuda") for H in (Hq, Hkv))
            lib.bdlm_rotary(d, r, n, q, wide, k, wide, dev(start), dev(pos.astype(np.int32)) if given else None, inverse, qo, ko)
            for got, x in ((qo, qkv[:, :, :Hq]), (ko, qkv[:, :, Hq:Hq + Hkv])):
                x = R.f64(x)
                want = R.rotary(x, pos, freq, r.amplitude, inter, inverse)
                want = np.where((pos >= 0)[..., None, None], want, 3.0)
                # angles within 2^-32 turns and 2^-24 of the turn kept in float32 (2 pi 2^-25 = 1.9e-7), sine and
                # cosine within a few steps of float32, three roundings of the products: below 2^-20 of the pair;
                # the frequency's own 2^-52 over 2^31 positions and up to a radian each: 5e-7 more
                size = np.abs(x).max(axis=-1, keepdims=True) * r.amplitude
                tol = R.BF16 * np.abs(want) * 1.001 + 2 * (2.0 ** -20 + 1e-6) * size
                assert np.all(np.abs(f(got) - want) <= tol)


def test_rotary_in_place_and_alone(lib):
    """In place; q or k alone; nothing outside the rows is touched."""
    import torch
    rng = np.random.default_rng(2)
    B, n, Hq, Hkv = 2, 7, 6, 2
    r = lib.bdlm_rotary_init(128, False, 500000.0)
    d = lib.attn_desc(B, 1, Hq, Hkv, 128, 1, 1)
    start = dev(np.array([5, 900], np.int32))
    q, k = bf16_tensor(W._normal_bf16(rng, (B, n, Hq, 128), 1.0)), bf16_tensor(W._normal_bf16(rng, (B, n, Hkv, 128), 1.0))
    qo, ko = torch.zeros_like(q), torch.zeros_like(k)
    lib.bdlm_rotary(d, r, n, q, 0, k, 0, start, None, False, qo, ko)
    q1, k1 = q.clone(), k.clone()
    lib.bdlm_rotary(d, r, n, q1, 0, None, 0, start, None, False, q1, None)
    lib.bdlm_rotary(d, r, n, None, 0, k1, 0, start, None, False, None, k1)
    assert torch.equal(q1, qo) and torch.equal(k1, ko)
    neg = dev(np.array([-1, 900], np.int32))
    q2 = torch.full_like(q, 9.0)
    lib.bdlm_rotary(d, r, n, q, 0, None, 0, neg, None, False, q2, None)
    assert torch.equal(q2[1], qo[1]) and bool((q2[0] == 9.0).all())


@pytest.mark.parametrize("inter", [False, True])
def test_rotary_gradient(lib, inter):
    """The inverse call is the gradient's way back: against the formula's transpose and differences."""
    import torch
    rng = np.random.default_rng(3)
    B, n, H, rot = 2, 3, 2, 96
    args = dict(scaling=4, factor=4.0, few=1.0, many=32.0)
    r = lib.bdlm_rotary_init(rot, inter, 10000.0, original_len=1000.0, **args)
    freq = R.frequencies(rot, 10000.0, original=1000.0, **args)
    at = rng.integers(0, 5000, (B, n))
    d = lib.attn_desc(B, 1, H, H, 128, 1, 1)
    g = W._normal_bf16(rng, (B, n, H, 128), 1.0)
    out = torch.empty((B, n, H, 128), dtype=torch.bfloat16, device="cuda")
    lib.bdlm_rotary(d, r, n, bf16_tensor(g), 0, None, 0, None, dev(at.astype(np.int32)), True, out, None)
    # differences of sum(g * y(x)), y linear in x: exact but for 64-bit rounding
    x, got = rng.normal(size=(B, n, H, 128)), f(out)
    for _ in range(40):
        i = tuple(rng.integers(s) for s in x.shape)
        step = np.zeros_like(x)
        step[i] = 1e-3
        hi, lo = (R.rotary(x + s * step, at, freq, r.amplitude, inter, False) for s in (1, -1))
        slope = np.sum(R.f64(g) * (hi - lo)) / 2e-3
        assert abs(got[i] - slope) <= R.BF16 * abs(slope) * 1.001 + 1e-5


@pytest.mark.parametrize("L,Hq,Hkv", [(4, 32, 8), (1, 8, 1), (64, 8, 2)])
def test_a_step_from_lengths_to_attention(lib, L, Hq, Hkv):
    """Prompts of different lengths taken in, then blocks: tables and positions, rotary, the 8-bit write,
    attention; the last step captured into a graph and replayed."""
    import torch
    rng = np.random.default_rng(11)
    B, cols, pages = 3, 24, 80      # 130 + 3 * 64 tokens in the longest
    prompts = np.array([50, 7, 130], np.int32)
    free = rng.permutation(pages).astype(np.int32)
    d = lib.attn_desc(B, L, Hq, Hkv, 128, cols, pages)
    packed = lib.attn_desc(256, 1, Hq, Hkv, 128, cols, pages)       # a row a sequence, for the packed tokens
    r = lib.bdlm_rotary_init(128, False, 10000.0)
    freq = R.frequencies(128, 10000.0)
    i32 = dict(dtype=torch.int32, device="cuda")
    t, at, lens = dev(np.full((B, cols), -1, np.int32)), dev(np.zeros(1, np.int32)), dev(np.zeros(B, np.int32))
    first, pos, slots, grown = torch.zeros(B + 1, **i32), torch.zeros(256, **i32), torch.zeros(256, **i32), torch.zeros(B, **i32)
    k8, v8 = (torch.full((pages, Hkv, 16, 128), 127, dtype=torch.uint8, device="cuda") for _ in range(2))
    sc = torch.ones((pages, Hkv, 2), device="cuda")
    fr = dev(free)
    k_in, v_in = (W._normal_bf16(rng, (256, Hkv, 128), 1.0) for _ in range(2))
    ki, vi = bf16_tensor(k_in), bf16_tensor(v_in)
    ko = torch.zeros_like(ki)
    lib.bdlm_build_tables(d, lens, dev(prompts), fr, pages, at, t, grown, first, 256, pos, slots, at)
    lib.bdlm_rotary(packed, r, 1, None, 0, ki, 0, None, pos, False, None, ko)
    lib.bdlm_write_kv8(d, 256, first, 256, ko, vi, k8, v8, sc, t, lens)
    lens.copy_(grown)
    # the same on the host
    table, hl, fi, ps, _, a = R.build_tables(np.zeros(B, np.int32), prompts, free, 0, np.full((B, cols), -1, np.int32), 256, pages)
    turned = R.rotary(R.f64(k_in)[:, None], ps[:, None], freq, 1.0, False, False)[:, 0]
    got = f(ko)
    n = int(fi[-1])
    assert np.abs(got[:n] - turned[:n]).max() <= 2.0 ** -8 * np.abs(turned[:n]).max() * 1.01 and np.all(got[n:] == 0)
    kb = W.f32_to_bf16_bits(got.astype(np.float32))
    blank = np.full((pages, Hkv, 16, 128), 127, np.uint8)
    wk, wv, ws = R.write_kv8(256, fi, kb, v_in, blank, blank, np.ones((pages, Hkv, 2), np.float32), table, np.zeros(B, np.int32))
    assert np.array_equal(host(t), table) and np.array_equal(host(sc), ws)
    assert R.same_codes(host(k8), wk) and R.same_codes(host(v8), wv)
    # blocks, step by step, in place
    q_in, kb_in, vb_in = (torch.zeros((B, L, H, 128), dtype=torch.bfloat16, device="cuda") for H in (Hq, Hkv, Hkv))
    qr, kr, out = torch.zeros_like(q_in), torch.zeros_like(kb_in), torch.zeros_like(q_in)

    def step():
        torch.add(lens, L, out=grown)
        lib.bdlm_build_tables(d, lens, grown, fr, pages, at, t, grown, first, B * L, None, None, at)
        lib.bdlm_rotary(d, r, L, q_in, 0, kb_in, 0, lens, None, False, qr, kr)
        lib.bdlm_write_kv8(d, L, None, 0, kr, vb_in, k8, v8, sc, t, lens)
        lib.bdlm_attention_kv8(d, qr, k8, v8, sc, t, lens, out)
        lens.copy_(grown)

    graph = None
    for turn in range(3):
        q, kn, vn = (W._normal_bf16(rng, (B, L, H, 128), 1.0) for H in (Hq, Hkv, Hkv))
        for dst, x in ((q_in, q), (kb_in, kn), (vb_in, vn)):
            dst.copy_(bf16_tensor(x))
        if turn == 2 or graph is not None:
            graph.replay()
        else:
            step()
        if turn == 1:
            state = [x.clone() for x in (lens, t, at, k8, v8, sc)]
            graph = torch.cuda.CUDAGraph()
            torch.cuda.synchronize()
            with torch.cuda.graph(graph):
                step()
            for x, s in zip((lens, t, at, k8, v8, sc), state):
                assert torch.equal(x, s)          # (capturing runs nothing)
        table, nl, _, _, _, a = R.build_tables(hl, hl + L, free, a, table, B * L, pages)
        qb, kb = (W.f32_to_bf16_bits(f(x).astype(np.float32)) for x in (qr, kr))
        wk, wv, ws = R.write_kv8(L, None, kb.reshape(B * L, Hkv, 128), vn.reshape(B * L, Hkv, 128), wk, wv, ws, table, hl)
        assert np.array_equal(host(t), table) and R.same_codes(host(k8), wk) and np.array_equal(host(sc), ws)
        R.check_attention(f(out), R.attention_kv8(qb, wk, wv, ws, table, hl, Hkv))
        hl = nl
    assert lib.bdlm_device_error() == 0
