"""Cases of the operators on the cache's side of a step: page tables and slot maps built from request
lengths, rotary positions, K/V written into a cache of 8 bits and attention over it.

The 8-bit cache: K and V in pages of 16 tokens, ``[num_pages, Hkv, 16, 128]`` e4m3, and for each page and
head a scale of K and one of V, ``[num_pages, Hkv, 2]``; a value is its code times its scale.  ``run``
either makes the library's calls (``own``) or computes the same thing from elementary torch operations.
"""
import math

import torch

own = False

D = 128
PAGE = 16
SCALE = 1.0 / math.sqrt(D)
TOP = 448.0                       # largest e4m3
HEADS = [(16, 8), (32, 8), (8, 8), (16, 2), (24, 8), (16, 1), (32, 4)]


def listed():
    return [
        # one request, a block of four over a prompt of two thousand tokens: latency
        dict(name="attend_one_request", op="attend", B=1, L=4, Hq=16, Hkv=8, lo=2000, hi=2000),
        # a serving batch: blocks of four over prefixes of mixed lengths
        dict(name="attend_batch", op="attend", B=128, L=4, Hq=32, Hkv=8, lo=512, hi=4096),
        # single tokens over long documents
        dict(name="attend_single_tokens", op="attend", B=32, L=1, Hq=32, Hkv=4, lo=16384, hi=32768),
        # wide blocks over long prefixes
        dict(name="attend_wide", op="attend", B=16, L=64, Hq=32, Hkv=8, lo=8192, hi=16384),
        # a batch's blocks of four into pages that are partly full
        dict(name="write_block", op="write", B=128, L=4, Hq=32, Hkv=8, lo=512, hi=4096, ragged=False),
        # prompts of mixed lengths, packed one after another
        dict(name="write_prompts", op="write", B=32, L=4096, Hq=32, Hkv=8, lo=0, hi=0, ragged=True),
        # a batch's blocks of four: all of the head, halves
        dict(name="rotary_block", op="rotary", B=128, L=4, Hq=32, Hkv=8, lo=512, hi=4096, rot=128, inter=False,
             scaling="none", given=False),
        # prompts at far positions: three quarters of the head, pairs side by side, frequencies scaled for long contexts
        dict(name="rotary_prompts", op="rotary", B=8, L=4096, Hq=32, Hkv=8, lo=0, hi=500000, rot=96, inter=True,
             scaling="yarn", given=True),
        # a step of a batch: every request grows by a block of four
        dict(name="tables_step", op="tables", B=128, Hq=32, Hkv=8, lo=0, hi=4096, grow=4, spare=1.25),
        # prompts taken in, more than there are pages for
        dict(name="tables_prompts", op="tables", B=256, Hq=32, Hkv=8, lo=0, hi=0, grow=4096, spare=0.9),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], even over its logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "write", "rotary", "tables"])
    Hq, Hkv = rng.choice(HEADS)
    case = dict(op=op, Hq=Hq, Hkv=Hkv)
    if op == "attend":
        L, hi, B = _log(rng, 1, 64), _log(rng, 1, 32768), _log(rng, 1, 128)
        L = min(L, 256 // (Hq // Hkv))
        B = max(1, min(B, 160000 * 8 * 256 // ((hi + L) * Hkv * max(64, L * Hq // Hkv))))
        case.update(B=B, L=L, lo=rng.randrange(0, hi + 1), hi=hi)
    elif op == "write":
        L, hi, B = _log(rng, 1, 4096), rng.randrange(0, 4097), _log(rng, 1, 128)
        B = max(1, min(B, 32 * 4096 * 8 // (L * Hkv)))
        case.update(B=B, L=L, lo=rng.randrange(0, hi + 1), hi=hi, ragged=rng.random() < 0.5)
    elif op == "rotary":
        L, hi, B = _log(rng, 1, 4096), _log(rng, 1, 1000000), _log(rng, 1, 128)
        B = max(1, min(B, 8 * 4096 * 40 // (L * (Hq + Hkv))))
        case.update(B=B, L=L, lo=rng.randrange(0, hi + 1), hi=hi, rot=16 * rng.randrange(1, 9), inter=rng.random() < 0.5,
                    scaling=rng.choice(["none", "linear", "base", "bands", "yarn"]), given=rng.random() < 0.5)
    else:
        B, hi, grow = _log(rng, 1, 1024), rng.randrange(0, 8193), _log(rng, 1, 4096)
        B = max(1, min(B, 256 * 4096 // grow))
        case.update(B=B, lo=rng.randrange(0, hi + 1), hi=hi, grow=grow, spare=rng.choice([0.5, 0.9, 1.0, 1.25]))
    return case


def _lens(case):
    """The sequences' lengths: evenly spread from lo to hi."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    return [hi if B == 1 else lo + (hi - lo) * b // (B - 1) for b in range(B)]


def _counts(case):
    """New tokens of each sequence: evenly spread up to L where they are ragged."""
    B, L = case["B"], case["L"]
    return [L if not case["ragged"] or B == 1 else max(1, L * (b + 1) // B) for b in range(B)]


def _bf16(shape, std, gen):
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(0.0, std, generator=gen)


def _codes(shape, gen):
    """e4m3 codes of normal values whose largest of some thousand is about 448."""
    x = torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(0.0, 110.0, generator=gen)
    return x.clamp_(-TOP, TOP).to(torch.float8_e4m3fn)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, B, Hq, Hkv = (case[k] for k in ("op", "B", "Hq", "Hkv"))
    lens = torch.tensor(_lens(case), dtype=torch.int32, device="cuda")
    order = torch.randperm(B, generator=gen, device="cuda")
    lens = lens[order]
    s = dict(case, lens=lens)
    if op == "rotary":
        L = case["L"]
        # a projection's output: q, k and v of a token side by side
        qkv = _bf16((B * L, (Hq + 2 * Hkv) * D), 1.0, gen)
        s["q"], s["k"] = qkv[:, :Hq * D].view(B, L, Hq, D), qkv[:, Hq * D:(Hq + Hkv) * D].view(B, L, Hkv, D)
        s["stride"] = qkv.stride(0)
        s["positions"] = None
        if case["given"]:
            # positions of a packed batch, its last rows padding
            at = lens[:, None] + torch.arange(L, dtype=torch.int32, device="cuda")
            at.view(-1)[B * L - B * L // 16:] = -1
            s["positions"] = at
        s["q_out"] = torch.zeros((B, L, Hq, D), dtype=torch.bfloat16, device="cuda")
        s["k_out"] = torch.zeros((B, L, Hkv, D), dtype=torch.bfloat16, device="cuda")
        return s
    if op == "tables":
        # every request grows by 1 to `grow` tokens
        new = lens + 1 + (torch.rand(B, generator=gen, device="cuda") * case["grow"]).int().clamp(max=case["grow"] - 1)
        cols = (case["hi"] + case["grow"] + PAGE - 1) // PAGE
        held = (lens + PAGE - 1) // PAGE
        need = B * ((case["grow"] + PAGE - 1) // PAGE)          # pages, at most
        n_free = max(1, int(need * 0.6 * case["spare"])) if case["grow"] >= PAGE else max(1, int(need * case["spare"]))
        n_pool = sum((n + PAGE - 1) // PAGE for n in _lens(case)) + n_free
        ids = torch.randperm(n_pool, generator=gen, device="cuda").int()
        first = torch.cumsum(held, 0) - held
        at = torch.arange(cols, device="cuda")
        table = torch.where(at < held[:, None], ids[(first[:, None] + at).clamp(max=n_pool - 1)], -1).int()
        rows = B * case["grow"]
        s.update(table=table, cols=cols, n_pool=n_pool, new=new.int(), free=ids[n_pool - n_free:].contiguous(), n_free=n_free, rows=rows,
                 out_lens=torch.empty_like(lens), first=torch.empty(B + 1, dtype=torch.int32, device="cuda"),
                 positions=torch.empty(rows, dtype=torch.int32, device="cuda"),
                 slots=torch.empty(rows, dtype=torch.int32, device="cuda"),
                 next=torch.empty(1, dtype=torch.int32, device="cuda"), start=torch.zeros(1, dtype=torch.int32, device="cuda"))
        return s
    L = case["L"]
    counts = [L] * B if op == "attend" else _counts(case)
    total = lens + torch.tensor(counts, dtype=torch.int32, device="cuda")[order]    # tokens of each sequence in the cache
    cols = (case["hi"] + L + PAGE - 1) // PAGE
    count = (total.long() + PAGE - 1) // PAGE
    first = torch.cumsum(count, 0) - count
    n_pages = sum((n + m + PAGE - 1) // PAGE for n, m in zip(_lens(case), counts))
    n_pool = n_pages + n_pages // 4 + 1                         # a pool with free pages in it
    shuffle = torch.randperm(n_pool, generator=gen, device="cuda")
    at = torch.arange(cols, device="cuda")
    table = torch.where(at < count[:, None], shuffle[(first[:, None] + at).clamp(max=n_pool - 1)], -1).int()
    s.update(table=table, cols=cols, n_pool=n_pool)
    s["k8"], s["v8"] = _codes((n_pool, Hkv, PAGE, D), gen), _codes((n_pool, Hkv, PAGE, D), gen)
    # a page's scale: its largest value over 448, about 4 / 448, differing from page to page
    s["scales"] = torch.exp2(torch.rand((n_pool, Hkv, 2), generator=gen, device="cuda") * 2 - 1) / 110
    if op == "attend":
        s["q"] = _bf16((B, L, Hq, D), 1.0, gen)
        s["out"] = torch.empty((B, L, Hq, D), dtype=torch.bfloat16, device="cuda")
        return s
    s["total"] = total
    s["first"] = None
    rows = B * L
    if case["ragged"]:
        n = total - lens
        s["first"] = torch.cat((n.new_zeros(1), torch.cumsum(n, 0).int())).int()
        rows = sum(counts)
    # heads have their own magnitudes
    size = torch.exp2(torch.randint(-3, 4, (Hkv, 1), generator=gen, device="cuda").float()).bfloat16()
    s["k_new"], s["v_new"] = _bf16((rows, Hkv, D), 1.0, gen).mul_(size), _bf16((rows, Hkv, D), 1.0, gen).mul_(size)
    return s


# ---------------------------------------------------------------- rotary frequencies

BASE = 10000.0
SCALINGS = {"none": 0, "linear": 1, "base": 2, "bands": 3, "yarn": 4}
FACTOR, ORIGINAL = 8.0, 4096.0
EDGES = {"bands": (1.0, 4.0), "yarn": (1.0, 32.0)}            # turns over the original length: few, many


def _frequencies(rot, scaling):
    """Radians per position of each pair, in 64 bits, and what cos and sin are multiplied by."""
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    if scaling == "base":
        # the base that leaves the first pair and divides the last pair's frequency by the factor
        return (BASE * FACTOR ** (rot / max(1, rot - 2))) ** (-2 * i / rot), 1.0
    f = BASE ** (-2 * i / rot)
    if scaling == "none":
        return f, 1.0
    if scaling == "linear":
        return f / FACTOR, 1.0
    few, many = EDGES[scaling]
    if scaling == "bands":
        # pairs of many turns keep their frequency, those of few take the factor, between them by their turns
        keep = ((ORIGINAL * f / (2 * math.pi) - few) / (many - few)).clamp(0, 1)
        return f * keep + f / FACTOR * (1 - keep), 1.0
    # the same, between them by the pair's number
    at = [rot * math.log(ORIGINAL / (t * 2 * math.pi)) / (2 * math.log(BASE)) for t in (many, few)]
    low, high = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot // 2 - 1)
    keep = 1 - ((i - low) / max(high - low, 0.001)).clamp(0, 1)
    return f * keep + f / FACTOR * (1 - keep), 0.1 * math.log(FACTOR) + 1


def _positions(s):
    if s["positions"] is not None:
        return s["positions"].long()
    return s["lens"].long()[:, None] + torch.arange(s["L"], device="cuda")


def _rotary(s):
    rot, half = s["rot"], s["rot"] // 2
    f, size = _frequencies(rot, s["scaling"])
    at = _positions(s)
    angle = (at.double()[..., None] * f)[:, :, None]           # [B, L, 1, pairs], in 64 bits: positions are far
    cos, sin = (torch.cos(angle) * size).float(), (torch.sin(angle) * size).float()
    for x, out in ((s["q"], s["q_out"]), (s["k"], s["k_out"])):
        y = x.float()
        a, b = (y[..., :rot:2], y[..., 1:rot:2]) if s["inter"] else (y[..., :half], y[..., half:rot])
        u, v = a * cos - b * sin, a * sin + b * cos
        y = torch.cat((torch.stack((u, v), -1).flatten(-2) if s["inter"] else torch.cat((u, v), -1), y[..., rot:]), -1)
        out.copy_(torch.where((at >= 0)[:, :, None, None], y.bfloat16(), out))
    return s["q_out"], s["k_out"]


# ---------------------------------------------------------------- tables and slots

def _tables(s):
    old, new, cols = s["lens"].long(), s["new"].long(), s["cols"]
    held, want = (old + PAGE - 1) // PAGE, (new + PAGE - 1) // PAGE
    need = want - held
    upto = torch.cumsum(need, 0)
    served = (need == 0) | (upto <= s["n_free"] - s["start"])
    s["out_lens"].copy_(torch.where(served, new, old))
    col = torch.arange(cols, device="cuda")
    take = served[:, None] & (col >= held[:, None]) & (col < want[:, None])
    source = s["start"] + (upto - need)[:, None] + col - held[:, None]
    s["table"].copy_(torch.where(take, s["free"][source.clamp(0, s["n_free"] - 1)], s["table"]))
    s["next"].copy_(s["start"] + torch.where(served, need, 0).sum())
    n = torch.where(served, new - old, 0)
    s["first"][0] = 0
    s["first"][1:] = torch.cumsum(n, 0)
    row = torch.arange(s["rows"], device="cuda")
    b = (torch.searchsorted(s["first"].long(), row, right=True) - 1).clamp(max=s["B"] - 1)
    live = row < s["first"][-1]
    at = old[b] + row - s["first"][b]
    page = s["table"][b, (at // PAGE).clamp(0, cols - 1)]
    s["positions"].copy_(torch.where(live, at, -1))
    s["slots"].copy_(torch.where(live, page * PAGE + at % PAGE, -1))
    return s["table"], s["out_lens"], s["first"], s["positions"], s["slots"], s["next"]


# ---------------------------------------------------------------- the 8-bit cache

def _write(s):
    """The pages that hold new tokens, whole: [B, pages, Hkv, 16, D]."""
    B, L, Hkv = s["B"], s["L"], s["Hkv"]
    start, total = s["lens"].long(), s["total"].long()
    col = (start // PAGE)[:, None] + torch.arange((L + 2 * PAGE - 2) // PAGE, device="cuda")
    ids = torch.where(col < ((total + PAGE - 1) // PAGE)[:, None], s["table"].long().gather(1, col.clamp(max=s["cols"] - 1)), -1)
    at = col[:, :, None] * PAGE + torch.arange(PAGE, device="cuda")             # [B, pages, 16]
    first = s["first"].long()[:-1] if s["first"] is not None else torch.arange(B, device="cuda") * L
    fresh = (at >= start[:, None, None]) & (at < total[:, None, None])
    held = at < start[:, None, None]
    row = torch.where(fresh, first[:, None, None] + at - start[:, None, None], 0)
    b, p = torch.nonzero(ids >= 0, as_tuple=True)
    page, fresh, held, row = ids[b, p], fresh[b, p], held[b, p], row[b, p]
    live = (fresh | held)[:, None, :, None]
    for c, (x, codes) in enumerate(((s["k_new"], s["k8"]), (s["v_new"], s["v8"]))):
        raw = codes.view(torch.uint8)
        was = raw[page]
        old = was.view(torch.float8_e4m3fn).float() * s["scales"][page, :, c][:, :, None, None]
        value = torch.where(fresh[:, None, :, None], x[row].float().transpose(1, 2), torch.where(held[:, None, :, None], old, 0.0))
        most = value.abs().amax((2, 3))
        # the least power of two that takes the page's largest value to 448 or less
        m, e = torch.frexp(most.double() / TOP)
        e = torch.where(m == 0.5, e - 1, e).clamp(-40, 40)
        e = torch.where(most > 0, e, -40)
        scale = ((e + 127).int() << 23).view(torch.float32)
        code = (value / scale[:, :, None, None]).clamp(-TOP, TOP).to(torch.float8_e4m3fn).view(torch.uint8)
        raw[page] = torch.where(live, code, was)
        s["scales"][page, :, c] = scale
    return s["k8"], s["v8"], s["scales"]


def _tokens(s, name, c):
    """Every sequence's tokens, [B, Hkv, tokens, D], in 32 bits."""
    ids = s["table"].clamp(min=0).long()
    x = s[name].view(torch.uint8)[ids].view(torch.float8_e4m3fn).float() * s["scales"][ids][..., c, None, None]
    return x.transpose(1, 2).reshape(ids.shape[0], s["Hkv"], -1, D)


def _attend(s):
    B, L, Hq, Hkv = (s[k] for k in ("B", "L", "Hq", "Hkv"))
    k, v = _tokens(s, "k8", 0), _tokens(s, "v8", 1)
    q = s["q"].float().reshape(B, L, Hkv, Hq // Hkv, D).transpose(1, 2).reshape(B, Hkv, -1, D)
    seen = (torch.arange(k.shape[2], device="cuda") < (s["lens"] + L)[:, None])[:, None, None]
    x = ((q @ k.transpose(2, 3)) * SCALE).masked_fill(~seen, -math.inf)
    e = torch.exp(x - x.amax(-1, keepdim=True))
    out = (e @ v.masked_fill(~seen.transpose(2, 3), 0.0)) / e.sum(-1, keepdim=True)
    out = out.reshape(B, Hkv, L, Hq // Hkv, D).transpose(1, 2).reshape(B, L, Hq, D)
    s["out"].copy_(out)
    return s["out"]


def _own(s):
    import block_diffusion_gb300 as bd

    op = s["op"]
    if "desc" not in s:
        s["desc"] = bd.attn_desc(s["B"], min(s.get("L", 1), 64), s["Hq"], s["Hkv"], D, s.get("cols", 1), s.get("n_pool", 1))
        if op == "rotary":
            few, many = EDGES.get(s["scaling"], (0.0, 0.0))
            s["rotary"] = bd.bdlm_rotary_init(s["rot"], s["inter"], BASE, SCALINGS[s["scaling"]], FACTOR, ORIGINAL, few, many)
    d = s["desc"]
    if op == "attend":
        bd.bdlm_attention_kv8(d, s["q"], s["k8"], s["v8"], s["scales"], s["table"], s["lens"], s["out"])
        return s["out"]
    if op == "write":
        bd.bdlm_write_kv8(d, s["L"], s["first"], s["k_new"].shape[0], s["k_new"], s["v_new"], s["k8"], s["v8"],
                          s["scales"], s["table"], s["lens"])
        return s["k8"], s["v8"], s["scales"]
    if op == "rotary":
        bd.bdlm_rotary(d, s["rotary"], s["L"], s["q"], s["stride"], s["k"], s["stride"], s["lens"], s["positions"], False,
                       s["q_out"], s["k_out"])
        return s["q_out"], s["k_out"]
    bd.bdlm_build_tables(d, s["lens"], s["new"], s["free"], s["n_free"], s["start"], s["table"], s["out_lens"], s["first"],
                         s["rows"], s["positions"], s["slots"], s["next"])
    return s["table"], s["out_lens"], s["first"], s["positions"], s["slots"], s["next"]


def run(s):
    if own:
        return _own(s)
    return {"attend": _attend, "write": _write, "rotary": _rotary, "tables": _tables}[s["op"]](s)


def work(case):
    op, B, Hq, Hkv = (case[k] for k in ("op", "B", "Hq", "Hkv"))
    lens = _lens(case)
    if op == "attend":
        L = case["L"]
        kv, pages = sum(lens) + B * L, sum((n + L + PAGE - 1) // PAGE for n in lens)
        return dict(bytes=2 * kv * Hkv * D + pages * (8 * Hkv + 4) + 4 * B * L * Hq * D + 4 * B, flops=4 * kv * L * Hq * D)
    if op == "write":
        counts = _counts(case)
        new, held = sum(counts), sum(n % PAGE for n in lens)
        pages = sum((n + m + PAGE - 1) // PAGE - n // PAGE for n, m in zip(lens, counts))
        return dict(bytes=2 * Hkv * D * (3 * new + 2 * held) + pages * (8 * Hkv + 4) + 4 * B, flops=4 * new * Hkv * D)
    if op == "rotary":
        rows = B * case["L"] - (B * case["L"] // 16 if case["given"] else 0)
        return dict(bytes=rows * (Hq + Hkv) * D * 4 + 4 * B * case["L"] * case["given"] + 4 * B, flops=3 * rows * (Hq + Hkv) * case["rot"])
    tokens = B * (case["grow"] + 1) // 2                        # on average
    return dict(bytes=16 * B + 8 * B * case["grow"] + 8 * (tokens // PAGE), flops=B + tokens)


def exact(case, seed):
    """What run() returns, from the definitions in 64 bits, one sequence or head at a time."""
    s = prepare(case, seed)
    op, B, Hq, Hkv = (case[k] for k in ("op", "B", "Hq", "Hkv"))
    if op == "tables":
        return None                                             # whole numbers only
    if op == "attend":
        L, G = case["L"], Hq // Hkv
        out = torch.empty((B, L, Hq, D), dtype=torch.float64, device="cuda")
        for i, n in enumerate(s["lens"].tolist()):
            n += L
            ids = s["table"][i, :(n + PAGE - 1) // PAGE].long()
            for g in range(Hkv):
                k, v = (s[x].view(torch.uint8)[ids, g].view(torch.float8_e4m3fn).double() * s["scales"][ids, g, c].double()[:, None, None]
                        for c, x in enumerate(("k8", "v8")))
                q = s["q"][i, :, g * G:(g + 1) * G].double()
                out[i, :, g * G:(g + 1) * G] = (q @ k.flatten(0, 1)[:n].T * SCALE).softmax(-1) @ v.flatten(0, 1)[:n]
        return out
    if op == "write":
        got = [s["k8"].double(), s["v8"].double()]
        scales = s["scales"].double()
        powers = torch.tensor([2.0 ** e for e in range(-40, 41)], dtype=torch.float64, device="cuda")
        for i, (n, m) in enumerate(zip(s["lens"].tolist(), s["total"].tolist())):
            row = int(s["first"][i]) if s["first"] is not None else i * case["L"]
            p0, p1 = n // PAGE, (m + PAGE - 1) // PAGE
            ids = s["table"][i, p0:p1].long()
            for c, x in enumerate((s["k_new"], s["v_new"])):
                # head by head, the pages' tokens in a row
                w = (got[c][ids] * scales[ids, :, c][:, :, None, None]).transpose(0, 1).reshape(Hkv, -1, D)
                w[:, n - p0 * PAGE:m - p0 * PAGE] = x[row:row + m - n].double().transpose(0, 1)
                most = w.abs().clone()
                most[:, m - p0 * PAGE:] = 0
                power = powers[torch.searchsorted(TOP * powers, most.reshape(Hkv, -1, PAGE * D).amax(2)).clamp(max=80)]
                w = (w.reshape(Hkv, -1, PAGE, D) / power[:, :, None, None]).clamp(-TOP, TOP)
                # e4m3: steps of an eighth of the power of two below, of 2^-9 at the smallest
                step = torch.exp2(torch.floor(torch.log2(w.abs().clamp(min=2.0 ** -6))) - 3)
                w = torch.round(w / step) * step
                live = (torch.arange((p1 - p0) * PAGE, device="cuda") < m - p0 * PAGE).reshape(1, -1, PAGE, 1)
                got[c][ids] = torch.where(live, w, got[c][ids].transpose(0, 1)).transpose(0, 1)
                scales[ids, :, c] = power.T
        return got[0], got[1], scales
    rot = case["rot"]
    f, size = _frequencies(rot, case["scaling"])
    at = _positions(s)
    result = []
    for x, out in ((s["q"], s["q_out"]), (s["k"], s["k_out"])):
        y = out.double()
        for h in range(x.shape[2]):
            w = x[:, :, h].double()
            pair = w[..., :rot].unflatten(-1, (-1, 2) if case["inter"] else (2, -1))
            pair = pair if case["inter"] else pair.transpose(-1, -2)
            turned = torch.view_as_complex(pair.contiguous()) * torch.polar(torch.full_like(f, size), at.double()[..., None] * f)
            turned = torch.view_as_real(turned)
            w = torch.cat(((turned if case["inter"] else turned.transpose(-1, -2)).flatten(-2), w[..., rot:]), -1)
            y[:, :, h] = torch.where((at >= 0)[..., None], w, y[:, :, h])
        result.append(y)
    return tuple(result)
