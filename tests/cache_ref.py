"""Plain 64-bit forms of the operators over part of a paged cache, on numpy arrays of bf16 bits.

Written from the definitions in include/bdlm.h, one sequence and head at a time; they share no code
with the library.  Each also returns what its error bound needs.
"""
import numpy as np

import workloads as W

D, P = 128, 16
BF16 = 2.0 ** -8     # half a step of bf16, relative


def f64(bits):
    return W.bf16_bits_to_f32(bits).astype(np.float64)


def tokens(pages, ids, n, head):
    """The first n tokens of a page list, one head, [n, D] float64."""
    x = pages[np.asarray(ids)[:(n + P - 1) // P]][:, :, head].reshape(-1, D)[:n]
    return f64(x)


def attend(q, k, v, seen, scale):
    """q [R, D], k / v [n, D], seen [R, n] -> out, lse, and A = sum p |v|, S1 = largest score sum."""
    k, v = (np.where(np.isfinite(z), z, 0.0) for z in (k, v))     # what is not seen may be anything
    x = q @ k.T * scale
    x = np.where(seen, x, -np.inf)
    top = np.max(x, axis=1, keepdims=True, initial=-np.inf)
    e = np.where(seen, np.exp(x - np.where(np.isinf(top), 0.0, top)), 0.0)
    l = e.sum(1, keepdims=True)
    p = np.divide(e, l, out=np.zeros_like(e), where=l > 0)
    with np.errstate(divide="ignore"):
        lse = np.where(l[:, 0] > 0, np.where(np.isinf(top[:, 0]), 0.0, top[:, 0]) + np.log(l[:, 0]), -np.inf)
    s1 = (np.abs(q) @ np.abs(k).T * scale).max(initial=0.0)
    return p @ v, lse, p @ np.abs(v), s1


def tree_attention(q, k, v, table, lens, mask, Hkv, scale=None):
    """mask [B, L] uint64 or None."""
    B, L, Hq, _ = q.shape
    G = Hq // Hkv
    scale = 1.0 / np.sqrt(D) if scale is None else scale
    out, A = np.zeros((B, L, Hq, D)), np.zeros((B, L, Hq, D))
    lse, s1 = np.zeros((B, L, Hq)), 0.0
    for b in range(B):
        n = int(lens[b]) + L
        seen = np.ones((L, n), bool)
        if mask is not None:
            for i in range(L):
                for t in range(L):
                    seen[i, int(lens[b]) + t] = (int(mask[b, i]) >> t) & 1
        for h in range(Hq):
            kk, vv = tokens(k, table[b], n, h // G), tokens(v, table[b], n, h // G)
            o, s, a, m = attend(f64(q[b, :, h]), kk, vv, seen, scale)
            out[b, :, h], lse[b, :, h], A[b, :, h] = o, s, a
            s1 = max(s1, m)
    return out, lse, A, s1


def score_error(s1):
    """Error of a score in nats: 128 products in 8 MMAs of 16, each at most 17 roundings or
    truncations of 2^-23 of the sum of magnitudes, then the scaling's own rounding."""
    return (8 * 17 * 2.0 ** -23 + 2.0 ** -22) * s1


def check_out(got, out, A, s1):
    """bf16 P (half a step each) and the bf16 output, plus the scores' float32 error on every p."""
    tol = BF16 * 1.01 * (A + np.abs(out)) + 2 * score_error(s1) * A + 1e-5 * A + 1e-30
    assert np.all(np.isfinite(got))
    excess = np.abs(got - out) - tol
    assert excess.max() <= 0, f"{excess.max()} over at {np.unravel_index(excess.argmax(), excess.shape)}"


def check_lse(got, lse, s1):
    """ln of the sum: the scores' error, 2^-22 for the exponentials and the log, and the float32
    sums of up to a few hundred terms in a row (below 2^-15)."""
    empty = np.isneginf(lse)
    assert np.array_equal(np.isneginf(got), empty)
    tol = score_error(s1) + 2.0 ** -15 + np.abs(lse[~empty]) * 2.0 ** -22
    assert np.all(np.abs(got[~empty] - lse[~empty]) <= tol)


def page_bounds(k, table, frm, to, bounds):
    out = bounds.copy()
    for b in range(len(to)):
        for p in range(int(frm[b]) // P, int(to[b]) // P):
            x = f64(k[table[b, p]])
            out[table[b, p], :, 0] = W.f32_to_bf16_bits(x.min(0).astype(np.float32))
            out[table[b, p], :, 1] = W.f32_to_bf16_bits(x.max(0).astype(np.float32))
    return out


def page_scores(q, bounds, ids, head, G):
    """Scores [pages] of one group: q [positions, Hq, D] bits."""
    rows = f64(q[:, head * G:(head + 1) * G]).reshape(-1, D)
    b = f64(bounds[ids][:, head])
    return (np.maximum(rows, 0) @ b[:, 1].T + np.minimum(rows, 0) @ b[:, 0].T).max(0)


def select_pages(q, bounds, table, lens, group, n_select, cols, Hkv):
    B, L, Hq, _ = q.shape
    S, G = L // group, Hq // Hkv
    sel = np.full((B, S, Hkv, cols), -1, np.int32)
    sel_lens = np.zeros((B, S), np.int32)
    for b in range(B):
        n = int(lens[b]) // P
        k = min(n, n_select)
        tail = table[b, n:(int(lens[b]) + L + P - 1) // P]
        for s in range(S):
            sel_lens[b, s] = k * P + int(lens[b]) % P + L - group
            for h in range(Hkv):
                sc = page_scores(q[b, s * group:(s + 1) * group], bounds, table[b, :n], h, G)
                best = np.sort(np.argsort(-sc, kind="stable")[:k])
                sel[b, s, h, :k] = table[b, best]
                sel[b, s, h, k:k + len(tail)] = tail
    return sel, sel_lens


def sparse_attention(q, k, v, sel, sel_lens, group, Hkv, scale=None):
    B, L, Hq, _ = q.shape
    G = Hq // Hkv
    scale = 1.0 / np.sqrt(D) if scale is None else scale
    out, A, s1 = np.zeros((B, L, Hq, D)), np.zeros((B, L, Hq, D)), 0.0
    for b in range(B):
        for s in range(L // group):
            n = int(sel_lens[b, s]) + group
            at = slice(s * group, (s + 1) * group)
            for h in range(Hq):
                kk, vv = (tokens(x, sel[b, s, h // G], n, h // G) for x in (k, v))
                o, _, a, m = attend(f64(q[b, at, h]), kk, vv, np.ones((group, n), bool), scale)
                out[b, at, h], A[b, at, h], s1 = o, a, max(s1, m)
    return out, A, s1


def attention_weights(q, k, table, lens, lse, decay, weights, Hkv, scale=None):
    """-> weights, and the added part alone and S1 for the bound."""
    B, L, Hq, _ = q.shape
    G = Hq // Hkv
    scale = 1.0 / np.sqrt(D) if scale is None else scale
    out, add, s1 = weights.astype(np.float64), np.zeros(weights.shape), 0.0
    for b in range(B):
        n = int(lens[b])
        for h in range(Hkv):
            kk = tokens(k, table[b], n, h)
            qq = f64(q[b, :, h * G:(h + 1) * G]).reshape(-1, D)
            x = qq @ kk.T * scale - lse[b, :, h * G:(h + 1) * G].astype(np.float64).reshape(-1, 1)
            add[b, h, :n] = np.exp(x).sum(0)
            out[b, h, :n] = decay * out[b, h, :n] + add[b, h, :n]
            s1 = max(s1, (np.abs(qq) @ np.abs(kk).T * scale).max(initial=0.0))
    return out, add, s1


def evict(w, n, keep, recent):
    """Kept positions of one row of weights."""
    if n <= keep:
        return np.arange(n)
    key = np.where(np.isnan(w[:n - recent]), -np.inf, w[:n - recent])
    order = sorted(range(n - recent), key=lambda i: (np.isnan(w[i]), -key[i], i))
    return np.concatenate([np.sort(order[:keep - recent]).astype(np.int64), np.arange(n - recent, n)])
