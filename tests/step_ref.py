"""Plain 64-bit forms of the operators on the cache's side of a step, on numpy arrays: tables and slot
maps, rotary positions, the 8-bit cache's writes and the attention over it.

Written from the definitions in include/bdlm.h; they share no code with the library.
"""
import math

import numpy as np

import workloads as W

D, P = 128, 16
TOP = 448.0
BF16 = 2.0 ** -8     # half a step of bf16, relative


def f64(bits):
    return W.bf16_bits_to_f32(bits).astype(np.float64)


def _decode(c):
    e, m = (c >> 3) & 15, c & 7
    if e == 15 and m == 7:
        return math.nan
    v = (1 + m / 8) * 2.0 ** (e - 7) if e else m * 2.0 ** -9
    return -v if c & 128 else v


E4M3 = np.array([_decode(c) for c in range(256)])
_POSITIVE = E4M3[:127]                     # 0 .. 448, rising


def encode(x):
    """float64 -> e4m3 codes, to nearest, ties to the even code, at most +-448; NaN keeps 0x7F."""
    a = np.minimum(np.abs(x), TOP)
    up = np.searchsorted(_POSITIVE, np.where(np.isnan(a), 0, a))          # first not below
    down = np.maximum(up - 1, 0)
    hi, lo = _POSITIVE[up] - a, a - _POSITIVE[down]
    code = np.where((lo < hi) | ((lo == hi) & (down % 2 == 0)), down, up)
    code = np.where(np.isnan(x), 127, code)
    return (code | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def same_codes(got, want):
    """Equal codes; a NaN may have either sign."""
    return np.array_equal(np.where((got & 127) == 127, 127, got), np.where((want & 127) == 127, 127, want))


def exponent(most):
    e = -40
    while e < 40 and most > TOP * 2.0 ** e:
        e += 1
    return e


def write_kv8(n_tokens, first, k_new, v_new, k, v, scales, table, lens):
    """k_new, v_new bf16 bits [rows, Hkv, D]; returns the pools after the call."""
    out = [k.copy(), v.copy()]
    scales = scales.copy()
    for b in range(len(lens)):
        row = b * n_tokens if first is None else int(first[b])
        n = n_tokens if first is None else int(first[b + 1]) - row
        pre = int(lens[b])
        for col in range(pre // P, (pre + n + P - 1) // P if n else 0):
            page = table[b, col]
            held, live = max(0, pre - col * P), min(P, pre + n - col * P)
            for c, new in enumerate((k_new, v_new)):
                for h in range(k.shape[1]):
                    x = np.zeros((live, D))
                    # (a held value is its code times the scale, in float32)
                    x[:held] = (E4M3[out[c][page, h, :held]].astype(np.float32) * scales[page, h, c]).astype(np.float64)
                    at = row + col * P + held - pre
                    x[held:] = f64(new[at:at + live - held, h])
                    a = np.abs(x)
                    e = exponent(a[~np.isnan(a)].max(initial=0.0))
                    out[c][page, h, :live] = encode(x / 2.0 ** e)
                    scales[page, h, c] = 2.0 ** e
    return out[0], out[1], scales


def attention_kv8(q, k, v, scales, table, lens, Hkv, scale=None):
    """q bf16 bits [B, L, Hq, D] -> out, A = sum p |v|, the largest score magnitude sum with each query's
    elements (s1) and with its group's largest element for all of them (s2), and a row's largest p times its
    page's scale, over all tokens' codes of V."""
    B, L, Hq, _ = q.shape
    G = Hq // Hkv
    scale = 1.0 / np.sqrt(D) if scale is None else scale
    out, A, top = (np.zeros((B, L, Hq, D)) for _ in range(3))
    s1 = s2 = 0.0
    for b in range(B):
        n = int(lens[b]) + L
        ids = table[b, :(n + P - 1) // P]
        for g in range(Hkv):
            real = ((ids >= 0) & (ids < len(k)))[:, None, None]
            at = np.where(real[:, 0, 0], ids, 0)
            kk, vv = (np.where(real, E4M3[x[at, g]] * scales[at, g, c, None, None].astype(np.float64), 0.0).reshape(-1, D)[:n]
                      for c, x in enumerate((k, v)))
            sv = np.repeat(scales[at, g, 1].astype(np.float64), P)[:n]
            qq = f64(q[b, :, g * G:(g + 1) * G])
            for i in range(L):
                x = qq[i] @ kk.T * scale
                e = np.exp(x - x.max(1, keepdims=True))
                p = e / e.sum(1, keepdims=True)
                out[b, i, g * G:(g + 1) * G] = p @ vv
                A[b, i, g * G:(g + 1) * G] = p @ np.abs(vv)
                s1 = max(s1, (np.abs(qq[i]) @ np.abs(kk).T * scale).max())
                top[b, i, g * G:(g + 1) * G] = (p * sv).max(1, keepdims=True) * np.abs(vv / sv[:, None]).sum(0)
            s2 = max(s2, np.abs(qq).max() * np.abs(kk).sum(1).max() * scale)
    return out, A, s1, s2, top


def check_attention(got, ref):
    """Derived from what the kernel rounds:
    - q is held as two e4m3 parts, a power of two taking its group's largest element to (224, 448]: an
      element is off by at most 2^-8 of itself / 2^4 where both parts are normal, and by half the smallest
      step, 2^-10 / 224 of the largest, elsewhere: 2^-17 of it, in s2;
    - a score is 128 products in 8 MMAs of 32 and at most 33 truncations of 2^-23 of the magnitudes each;
    - p times its page's scale is held as two e4m3 parts as well: within 2^-8 of itself, or half the
      smallest step, 2^-10 / 128 of the row's largest such weight (its power of two is 2^7), per token;
    - sums are float32 (2^-15 for up to a few hundred truncations in a row), the output is bf16."""
    out, A, s1, s2, top = ref
    ds = 2.0 ** -17 * s2 + (8 * 33 * 2.0 ** -23 + 2.0 ** -21) * s1
    tol = BF16 * 1.01 * (A + np.abs(out)) + (np.expm1(2 * ds) + 2.0 ** -14) * A + 2.0 ** -17 * top + 1e-30
    assert np.all(np.isfinite(got))
    excess = np.abs(got - out) - tol
    assert excess.max() <= 0, f"{excess.max()} over at {np.unravel_index(excess.argmax(), excess.shape)}"


def frequencies(rot, base, scaling=0, factor=1.0, original=0.0, few=0.0, many=0.0):
    """Radians per position of each pair."""
    if scaling == 2:
        base = base * factor ** (rot / (rot - 2))
    f = [base ** (-2 * i / rot) for i in range(rot // 2)]
    if scaling == 1:
        f = [x / factor for x in f]
    if scaling == 3:
        keep = [min(1.0, max(0.0, (original * x / (2 * math.pi) - few) / (many - few))) for x in f]
        f = [x * s + x / factor * (1 - s) for x, s in zip(f, keep)]
    if scaling == 4:
        at = [rot * math.log(original / (t * 2 * math.pi)) / (2 * math.log(base)) for t in (many, few)]
        low, high = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot // 2 - 1)
        keep = [1 - min(1.0, max(0.0, (i - low) / max(high - low, 0.001))) for i in range(rot // 2)]
        f = [x * s + x / factor * (1 - s) for x, s in zip(f, keep)]
    return np.array(f)


def rotary(x, at, f, amplitude, interleaved, inverse):
    """x float64 [B, n, H, D], at [B, n] -> the turned x (rows of at < 0 as they are)."""
    rot = 2 * len(f)
    a = (np.maximum(at, 0)[..., None] * f)[:, :, None]
    cos, sin = np.cos(a) * amplitude, np.sin(a) * amplitude * (-1 if inverse else 1)
    y = x.copy()
    i = np.arange(rot // 2)
    u, v = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    y[..., u] = x[..., u] * cos - x[..., v] * sin
    y[..., v] = x[..., u] * sin + x[..., v] * cos
    return np.where((at >= 0)[..., None, None], y, x)


def build_tables(old, new, free, start, table, max_tokens, num_pages):
    """-> table, lens, first, positions, slots, next."""
    table = table.copy()
    B, cols = table.shape
    lens, first = old.copy(), [0]
    positions, slots = np.full(max_tokens, -1, np.int32), np.full(max_tokens, -1, np.int32)
    need_so_far = tokens_so_far = 0
    taken = start
    for b in range(B):
        o, n = int(old[b]), int(new[b])
        if o < 0 or n < 0 or o > cols * P or n > cols * P:
            n = o
        need = max(0, -(-n // P) - -(-o // P)) if n > o else 0
        need_so_far += need
        pages = need == 0 or need_so_far <= len(free) - start
        grow = max(0, n - o) if pages else 0
        tokens_so_far += grow
        if not pages or (grow and tokens_so_far > max_tokens):
            first.append(first[-1])
            continue
        lens[b] = n
        for j in range(need):
            table[b, -(-o // P) + j] = free[taken]
            taken += 1
        for t in range(o, o + grow):
            r = first[-1] + t - o
            page = table[b, t // P]
            positions[r] = t
            slots[r] = page * P + t % P if 0 <= page < num_pages else -1
        first.append(first[-1] + grow)
    return table, lens, np.array(first, np.int32), positions, slots, taken
