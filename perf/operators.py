"""Cases of the operators over part of a paged K/V cache: drafted-token trees, page selection and the
sparse attention it feeds, attention-weight accumulation and eviction.

Tokens live in pages of 16, heads are 128 wide, data are bf16.  ``run`` either makes the library's calls
(``own``) or computes the same thing from elementary torch operations.
"""
import math

import torch

own = False

D = 128
PAGE = 16
SCALE = 1.0 / math.sqrt(D)
HEADS = [(16, 8), (32, 8), (8, 8), (16, 2), (24, 8), (16, 1), (32, 4)]


def listed():
    return [
        # one request whose eight drafted tokens are verified after a short prompt: latency
        dict(name="tree_one_request", op="tree", B=1, L=8, Hq=16, Hkv=8, lo=60, hi=60),
        # a serving batch verifying sixteen drafted tokens each over prefixes of mixed lengths
        dict(name="tree_batch", op="tree", B=64, L=16, Hq=32, Hkv=8, lo=1024, hi=8192),
        # a finished block of sixteen positions in each sequence of a batch: its page gets its bounds
        dict(name="bounds_block", op="bounds", B=128, L=16, Hq=32, Hkv=8, lo=512, hi=4096),
        # prompts just written into the cache: bounds of all their pages
        dict(name="bounds_prompts", op="bounds", B=32, L=4096, Hq=32, Hkv=8, lo=0, hi=0),
        # one request, a block of four, a prompt of two thousand tokens: latency
        dict(name="select_one_request", op="select", B=1, L=4, Hq=16, Hkv=8, lo=2000, hi=2000, group=4, n=32),
        # long documents, 256 pages kept for each block
        dict(name="select_long", op="select", B=16, L=4, Hq=32, Hkv=8, lo=30000, hi=60000, group=4, n=256),
        # one request whose four queries each have pages of their own
        dict(name="sparse_one_request", op="sparse", B=1, L=4, Hq=16, Hkv=8, lo=2000, hi=2000, group=1, n=32),
        # a batch of long documents, a block's queries sharing 256 pages
        dict(name="sparse_long", op="sparse", B=32, L=4, Hq=32, Hkv=8, lo=10000, hi=20000, group=4, n=256),
        # one request, one block of four over a short prefix: latency
        dict(name="weights_one_request", op="weights", B=1, L=4, Hq=16, Hkv=8, lo=500, hi=500),
        # wide blocks over long prefixes
        dict(name="weights_wide", op="weights", B=16, L=64, Hq=32, Hkv=8, lo=8192, hi=16384),
        # one request cut back to a small budget
        dict(name="evict_one_request", op="evict", B=1, L=1, Hq=16, Hkv=8, lo=600, hi=600, keep=256, recent=32),
        # a batch of long sequences cut back to 4096 tokens
        dict(name="evict_batch", op="evict", B=32, L=1, Hq=32, Hkv=8, lo=8192, hi=16384, keep=4096, recent=64),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], even over its logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["tree", "bounds", "select", "sparse", "weights", "evict"])
    Hq, Hkv = rng.choice(HEADS)
    G = Hq // Hkv
    case = dict(op=op, L=1, Hq=Hq, Hkv=Hkv)
    if op in ("tree", "weights"):
        L, hi, B = _log(rng, 1, 64), _log(rng, 1, 16384), _log(rng, 1, 128)
        L = min(L, 256 // G)
        B = max(1, min(B, 160000 * 8 // (Hkv * (hi + L))))
        case.update(B=B, L=L, lo=rng.randrange(0, hi + 1), hi=hi)
    elif op == "bounds":
        L, hi, B = _log(rng, 1, 4096), rng.randrange(0, 4097), _log(rng, 1, 128)
        B = max(1, min(B, 32 * 4096 // L))
        case.update(B=B, L=L, lo=rng.randrange(0, hi + 1), hi=hi)
    elif op in ("select", "sparse"):
        group = rng.choice([1, 2, 3, 4, 5, 8])
        L = group * rng.choice([1, 2, 4])
        hi, n, B = _log(rng, 1, 60000), _log(rng, 1, 256), _log(rng, 1, 64)
        B = max(1, min(B, 480000 // (hi + L)))
        if op == "sparse":
            B = max(1, min(B, 32 * 256 * 8 // (n * Hkv * (L // group))))
        case.update(B=B, L=L, lo=rng.randrange(0, hi + 1), hi=hi, group=group, n=n)
    else:
        hi, B = _log(rng, 1, 16384), _log(rng, 1, 64)
        B = max(1, min(B, 32 * 12288 // hi))
        keep = min(_log(rng, 1, 4096), hi)
        case.update(B=B, lo=rng.randrange(0, hi + 1), hi=hi, keep=keep, recent=rng.randrange(0, keep + 1))
    return case


def _lens(case):
    """The sequences' lengths: evenly spread from lo to hi."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    return [hi if B == 1 else lo + (hi - lo) * b // (B - 1) for b in range(B)]


def _bf16(shape, std, gen):
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(0.0, std, generator=gen)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, B, L, Hq, Hkv = (case[k] for k in ("op", "B", "L", "Hq", "Hkv"))
    lens = torch.tensor(_lens(case), dtype=torch.int32, device="cuda")
    lens = lens[torch.randperm(B, generator=gen, device="cuda")]
    tail = L if op != "evict" else 0
    total = lens + tail                                       # tokens of each sequence in the cache
    cols = (case["hi"] + tail + PAGE - 1) // PAGE
    used = torch.arange(cols, device="cuda") < ((total + PAGE - 1) // PAGE)[:, None]
    count = (lens.long() + tail + PAGE - 1) // PAGE
    first = torch.cumsum(count, 0) - count
    n_pages = sum((n + tail + PAGE - 1) // PAGE for n in _lens(case))
    n_pool = n_pages + n_pages // 4 + 1                       # a pool with free pages in it
    shuffle = torch.randperm(n_pool, generator=gen, device="cuda")
    slot = (first[:, None] + torch.arange(cols, device="cuda")).clamp(max=n_pool - 1)
    table = torch.where(used, shuffle[slot], -1).int()
    s = dict(case, lens=lens, table=table, cols=cols, n_pool=n_pool)
    if op in ("tree", "weights", "select", "sparse"):
        s["q"] = _bf16((B, L, Hq, D), 1.0, gen)
    if op in ("tree", "weights", "bounds", "sparse"):
        s["k"] = _bf16((n_pool, PAGE, Hkv, D), 1.0, gen)
    if op in ("tree", "sparse"):
        s["v"] = _bf16((n_pool, PAGE, Hkv, D), 1.0, gen)
    if op in ("tree", "sparse"):
        s["out"] = torch.empty((B, L, Hq, D), dtype=torch.bfloat16, device="cuda")
    if op == "tree":
        # each drafted token has an earlier one (or the prefix) as its parent and sees its ancestors
        parent = torch.rand((B, L), generator=gen, device="cuda") * torch.arange(1, L + 1, device="cuda")
        parent = parent.long().clamp(max=L - 1) - 1
        mask = torch.zeros((B, L), dtype=torch.int64, device="cuda")
        rows = torch.arange(B, device="cuda")
        for i in range(L):
            above = torch.where(parent[:, i] >= 0, mask[rows, parent[:, i].clamp(min=0)], 0)
            mask[:, i] = above | (1 << i if i < 63 else -(1 << 63))
        s["mask"] = mask
        s["lse"] = torch.empty((B, L, Hq), dtype=torch.float32, device="cuda")
    if op == "weights":
        s["lse"] = _lse(s)
        s["weights"] = torch.rand((B, Hkv, cols * PAGE), generator=gen, device="cuda")
        s["decay"] = 0.9
    if op == "bounds":
        s["to"] = total
        s["bounds"] = torch.zeros((n_pool, Hkv, 2, D), dtype=torch.bfloat16, device="cuda")
    if op == "select":
        # keys of a page lie around a centre of its own
        centre, spread = _bf16((n_pool, Hkv, D), 0.7, gen), _bf16((n_pool, Hkv, 2, D), 0.3, gen).abs() + 1.0
        s["bounds"] = torch.stack((centre - spread[:, :, 0], centre + spread[:, :, 1]), 2)
    if op in ("select", "sparse"):
        s["sel_cols"] = case["n"] + (L + 30) // PAGE
        lists = B * (L // case["group"])
        s["sel"] = torch.empty((lists, Hkv, s["sel_cols"]), dtype=torch.int32, device="cuda")
        s["sel_lens"] = torch.empty((lists,), dtype=torch.int32, device="cuda")
    if op == "sparse":
        # the selection of an earlier step of the block
        score = torch.rand((lists, Hkv, cols), generator=gen, device="cuda")
        s["sel"], s["sel_lens"] = _selection(s, score)
    if op == "evict":
        extra = B * ((case["keep"] + PAGE - 1) // PAGE)       # fresh pages for what is kept
        s["n_src"] = n_pool
        s["k"] = _bf16((n_pool + extra, PAGE, Hkv, D), 1.0, gen)
        s["v"] = _bf16((n_pool + extra, PAGE, Hkv, D), 1.0, gen)
        s["k"][n_pool:], s["v"][n_pool:] = 0, 0
        to = n_pool + torch.randperm(extra, generator=gen, device="cuda").int().view(B, -1)
        s["to_table"] = torch.cat((to, to.new_full((B, cols), -1)), 1)[:, :cols].contiguous()
        # attention weight is heavy tailed: a few tokens gather most of it
        s["weights"] = torch.empty((B, Hkv, cols * PAGE), device="cuda").exponential_(1.0, generator=gen) ** 2
        s["to_weights"] = torch.zeros_like(s["weights"])
        s["kept"] = torch.empty((B, Hkv, case["keep"]), dtype=torch.int32, device="cuda")
        s["new_lens"] = torch.empty_like(lens)
    return s


def _tokens(pages, table):
    """Every sequence's tokens, [B, Hkv, tokens, D], in 32 bits."""
    B, cols = table.shape
    x = pages[table.clamp(min=0).long()].float()
    return x.reshape(B, cols * PAGE, -1, D).transpose(1, 2)


def _rows(x, Hkv):
    """Query rows by KV head: [B, L, Hq, ...] -> [B, Hkv, L * G, ...]."""
    B, L, Hq = x.shape[:3]
    return x.reshape(B, L, Hkv, Hq // Hkv, *x.shape[3:]).transpose(1, 2).reshape(B, Hkv, L * (Hq // Hkv), *x.shape[3:])


def _heads(x, L):
    """The other way round: [B, Hkv, L * G, ...] -> [B, L, Hq, ...]."""
    B, Hkv, R = x.shape[:3]
    return x.reshape(B, Hkv, L, R // L, *x.shape[3:]).transpose(1, 2).reshape(B, L, Hkv * (R // L), *x.shape[3:])


def _lse(s):
    """ln sum exp of the block attention's scores, [B, L, Hq]: every query sees prefix and block."""
    q = _rows(s["q"], s["Hkv"]).float()
    k = _tokens(s["k"], s["table"])
    at = torch.arange(k.shape[2], device="cuda")
    x = (q @ k.transpose(2, 3)) * SCALE
    x = x.masked_fill((at >= (s["lens"] + s["L"])[:, None])[:, None, None, :], -math.inf)
    return _heads(torch.logsumexp(x, 3), s["L"])


def _attend(q, k, v, seen):
    """Softmax attention of query rows over tokens; rows that see nothing give 0 and -inf."""
    x = ((q @ k.transpose(-1, -2)) * SCALE).masked_fill(~seen, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    e = torch.exp(x - top)
    total = e.sum(-1, keepdim=True)
    out = torch.where(total > 0, (e @ v) / total, torch.zeros_like(total))
    return out, (top + torch.log(total))[..., 0]


def _tree(s):
    L, Hkv = s["L"], s["Hkv"]
    k, v = _tokens(s["k"], s["table"]), _tokens(s["v"], s["table"])
    at = torch.arange(k.shape[2], device="cuda") - s["lens"][:, None]            # position in the block
    bits = (s["mask"][:, :, None] >> at.clamp(0, L - 1)[:, None, :]) & 1         # [B, L, tokens]
    seen = (at < 0)[:, None, :] | ((bits == 1) & (at < L)[:, None, :])
    v = v.masked_fill((at >= L)[:, None, :, None], 0.0)
    seen = seen.repeat_interleave(s["Hq"] // Hkv, 1)[:, None]
    out, lse = _attend(_rows(s["q"], Hkv).float(), k, v, seen)
    return _heads(out, L).bfloat16(), _heads(lse, L)


def _bounds(s):
    at = torch.arange(s["cols"], device="cuda")
    whole = (at >= (s["lens"] // PAGE)[:, None]) & (at < (s["to"] // PAGE)[:, None])
    ids = s["table"][whole].long()
    k = s["k"][ids].float()
    s["bounds"][ids] = torch.stack((k.amin(1), k.amax(1)), 2).bfloat16()
    return s["bounds"]


def _selection(s, score):
    """The pages of the best scores ([lists, Hkv, cols]) as a table of page ids, and the lists' lengths."""
    B, L, group, n = s["B"], s["L"], s["group"], s["n"]
    S = L // group
    full = (s["lens"] // PAGE).long().repeat_interleave(S)[:, None, None]
    table = s["table"].long().repeat_interleave(S, 0)[:, None].expand(-1, s["Hkv"], -1)
    at = torch.arange(s["cols"], device="cuda")
    score = score.masked_fill(at >= full, -math.inf)
    best = torch.sort(score, dim=-1, descending=True, stable=True)[1][..., :n]
    best = torch.sort(best.masked_fill(torch.arange(best.shape[-1], device="cuda") >= full, s["cols"]), dim=-1)[0]
    take = full.clamp(max=n)
    col = torch.arange(s["sel_cols"], device="cuda")
    rest = (((s["lens"] + L + PAGE - 1) // PAGE).long().repeat_interleave(S)[:, None, None] - full)
    where = torch.where(col < take, torch.nn.functional.pad(best, (0, s["sel_cols"] - best.shape[-1])), full + col - take)
    ids = table.gather(2, where.clamp(max=s["cols"] - 1).contiguous())
    lens = take[:, 0, 0] * PAGE + (s["lens"] % PAGE).long().repeat_interleave(S) + L - group
    return torch.where(col < take + rest, ids, -1).int(), lens.int()


def _scores(s):
    """max over a group's rows of sum_d max(q_d lo_d, q_d hi_d), in 64 bits: neighbours in rank lie close."""
    S = s["L"] // s["group"]
    lo, hi = s["bounds"][s["table"].clamp(min=0).long()].double().permute(3, 0, 2, 1, 4)
    q = _rows(s["q"], s["Hkv"]).double()
    x = q.clamp(min=0) @ hi.transpose(2, 3) + q.clamp(max=0) @ lo.transpose(2, 3)
    x = x.reshape(s["B"], s["Hkv"], S, -1, s["cols"]).amax(3)
    return x.transpose(1, 2).reshape(s["B"] * S, s["Hkv"], s["cols"])


def _sparse(s):
    L, Hkv, group = s["L"], s["Hkv"], s["group"]
    S, c = L // group, s["sel_cols"]
    sel = s["sel"].clamp(min=0).long()
    heads = torch.arange(Hkv, device="cuda")[None, :, None]
    k = s["k"].transpose(1, 2)[sel, heads].float().reshape(-1, Hkv, c * PAGE, D)
    v = s["v"].transpose(1, 2)[sel, heads].float().reshape(-1, Hkv, c * PAGE, D)
    seen = torch.arange(c * PAGE, device="cuda") < (s["sel_lens"] + group)[:, None]
    v = v.masked_fill(~seen[:, None, :, None], 0.0)
    q = s["q"].reshape(s["B"] * S, group, s["Hq"], D)
    out, _ = _attend(_rows(q, Hkv).float(), k, v, seen[:, None, None, :])
    return _heads(out, group).bfloat16().reshape(s["B"], L, s["Hq"], D)


def _weights(s):
    q, k = _rows(s["q"], s["Hkv"]).float(), _tokens(s["k"], s["table"])
    p = torch.exp((q @ k.transpose(2, 3)) * SCALE - _rows(s["lse"], s["Hkv"])[..., None]).sum(2)
    prefix = (torch.arange(k.shape[2], device="cuda") < s["lens"][:, None])[:, None]
    s["weights"] = torch.where(prefix, s["decay"] * s["weights"] + p, s["weights"])
    return s["weights"]


def _evict(s):
    B, Hkv, keep = s["B"], s["Hkv"], s["keep"]
    w, n = s["weights"], s["lens"][:, None, None]
    at = torch.arange(w.shape[2], device="cuda")
    key = w.masked_fill(at >= n - s["recent"], math.inf).masked_fill(at >= n, -math.inf)
    best = torch.sort(key, dim=-1, descending=True, stable=True)[1][..., :keep]
    col = torch.arange(keep, device="cuda")
    new = s["lens"].clamp(max=keep)
    if best.shape[2] < keep:
        best = torch.nn.functional.pad(best, (0, keep - best.shape[2]))
    live = (col < new[:, None])[:, None].expand(B, Hkv, keep)
    kept = torch.sort(best.masked_fill(~live, w.shape[2]), dim=-1)[0]
    b, h, j = torch.nonzero(live, as_tuple=True)
    old = kept[live]
    source, target = s["table"][b, old // PAGE].long(), s["to_table"][b, j // PAGE].long()
    s["k"][target, j % PAGE, h] = s["k"][source, old % PAGE, h]
    s["v"][target, j % PAGE, h] = s["v"][source, old % PAGE, h]
    s["to_weights"][b, h, j] = w[b, h, old]
    return kept.masked_fill(~live, -1).int(), new, s["k"][s["n_src"]:], s["v"][s["n_src"]:], s["to_weights"]


def _own(s):
    import block_diffusion_gb300 as bd

    op, L = s["op"], s["L"]
    if "desc" not in s:
        s["desc"] = bd.attn_desc(s["B"], L, s["Hq"], s["Hkv"], D, s["cols"], s["k"].shape[0] if "k" in s else s["n_pool"])
    d = s["desc"]
    if op == "tree":
        bd.bdlm_tree_attention(d, s["q"], s["k"], s["v"], s["table"], s["lens"], s["mask"], s["out"], s["lse"])
        return s["out"], s["lse"]
    if op == "bounds":
        bd.bdlm_page_bounds(d, s["k"], s["table"], s["lens"], s["to"], s["bounds"])
        return s["bounds"]
    if op == "select":
        bd.bdlm_select_pages(d, s["q"], s["bounds"], s["table"], s["lens"], s["group"], s["n"], s["sel_cols"], s["sel"], s["sel_lens"])
        return s["sel"], s["sel_lens"]
    if op == "sparse":
        bd.bdlm_sparse_attention(d, s["q"], s["k"], s["v"], s["group"], s["sel_cols"], s["sel"], s["sel_lens"], s["out"])
        return s["out"]
    if op == "weights":
        # (the library takes lse densely laid out; one that is passes as it is)
        bd.bdlm_attention_weights(d, s["q"], s["k"], s["table"], s["lens"], s["lse"].contiguous(), s["decay"], s["weights"])
        return s["weights"]
    bd.bdlm_evict_kv(d, s["k"], s["v"], s["table"], s["lens"], s["weights"], s["keep"], s["recent"], s["to_table"],
                     s["to_weights"], s["kept"], s["new_lens"])
    return s["kept"], s["new_lens"], s["k"][s["n_src"]:], s["v"][s["n_src"]:], s["to_weights"]


def run(s):
    if own:
        return _own(s)
    op = s["op"]
    if op == "tree":
        return _tree(s)
    if op == "bounds":
        return _bounds(s)
    if op == "select":
        return _selection(s, _scores(s))
    if op == "sparse":
        return _sparse(s)
    if op == "weights":
        return _weights(s)
    return _evict(s)


def work(case):
    op, B, L, Hq, Hkv = (case[k] for k in ("op", "B", "L", "Hq", "Hkv"))
    lens = _lens(case)
    row = 2 * D                                               # bytes of one token's K of one head
    table = 4 * sum(n // PAGE + 1 for n in lens)
    io = B * L * Hq * row                                     # queries, or outputs
    if op == "tree":
        kv = sum(lens) + B * L
        return dict(bytes=2 * kv * Hkv * row + 2 * io + table + 8 * B * L + 4 * B * L * Hq, flops=4 * kv * L * Hq * D)
    if op == "bounds":
        pages = sum((n + L) // PAGE - n // PAGE for n in lens)
        return dict(bytes=pages * Hkv * (PAGE + 2) * row + 4 * pages + 8 * B, flops=2 * pages * PAGE * Hkv * D)
    if op == "select":
        pages = sum(n // PAGE for n in lens)
        lists = B * (L // case["group"]) * Hkv
        return dict(bytes=pages * Hkv * 2 * row + io + table + 4 * lists * (case["n"] + (L + 30) // PAGE), flops=2 * pages * L * Hq * D)
    if op == "sparse":
        kv = sum(min(n // PAGE, case["n"]) * PAGE + n % PAGE + L for n in lens) * (L // case["group"])
        return dict(bytes=2 * kv * Hkv * row + 2 * io + kv * Hkv // PAGE * 4, flops=4 * kv * case["group"] * Hq * D)
    if op == "weights":
        return dict(bytes=sum(lens) * Hkv * (row + 8) + io + table + 4 * B * L * Hq, flops=2 * sum(lens) * L * Hq * D)
    kept = sum(min(n, case["keep"]) for n in lens)
    return dict(bytes=4 * sum(lens) * Hkv + kept * Hkv * (4 * row + 8) + table, flops=sum(lens) * Hkv)


def exact(case, seed):
    """The floating outputs from their definitions in 64 bits, one sequence at a time."""
    s = prepare(case, seed)
    op, B, L, Hq, Hkv = (case[k] for k in ("op", "B", "L", "Hq", "Hkv"))
    G = Hq // Hkv
    if op == "select":
        return None                                           # whole numbers only
    if op == "bounds":
        b = s["bounds"].double()
        for i, (start, end) in enumerate(zip(s["lens"].tolist(), s["to"].tolist())):
            for p in s["table"][i, start // PAGE:end // PAGE].tolist():
                b[p, :, 0], b[p, :, 1] = s["k"][p].double().min(0)[0], s["k"][p].double().max(0)[0]
        return b
    if op == "evict":
        keep, recent = case["keep"], case["recent"]
        k, v, w = (s[x].double() for x in ("k", "v", "to_weights"))
        for i, n in enumerate(s["lens"].tolist()):
            m = min(n, keep)
            for h in range(Hkv):
                old = torch.arange(n, device="cuda")
                if n > keep:
                    rank = torch.sort(s["weights"][i, h, :n - recent], descending=True, stable=True)[1][:keep - recent]
                    old = torch.cat((rank.sort()[0], old[n - recent:]))
                new = torch.arange(m, device="cuda")
                source, target = s["table"][i, old // PAGE].long(), s["to_table"][i, new // PAGE].long()
                k[target, new % PAGE, h] = s["k"][source, old % PAGE, h].double()
                v[target, new % PAGE, h] = s["v"][source, old % PAGE, h].double()
                w[i, h, :m] = s["weights"][i, h, old].double()
        return None, None, k[s["n_src"]:], v[s["n_src"]:], w

    def sequence(pages, ids, n):
        return pages[ids[:(n + PAGE - 1) // PAGE].long()].flatten(0, 1)[:n].double()

    if op == "weights":
        w = s["weights"].double()
        for i, n in enumerate(s["lens"].tolist()):
            k = sequence(s["k"], s["table"][i], n)
            for h in range(Hq):
                x = k[:, h // G] @ s["q"][i, :, h].double().T * SCALE - s["lse"][i, :, h].double()
                w[i, h // G, :n] = (0.9 * w[i, h // G, :n] if h % G == 0 else w[i, h // G, :n]) + x.exp().sum(1)
        return w
    out = torch.empty((B, L, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.empty((B, L, Hq), dtype=torch.float64, device="cuda")
    if op == "tree":
        for i, n in enumerate(s["lens"].tolist()):
            k, v = sequence(s["k"], s["table"][i], n + L), sequence(s["v"], s["table"][i], n + L)
            m = s["mask"][i].tolist()
            hidden = torch.tensor([[not (m[r] >> t) & 1 for t in range(L)] for r in range(L)], device="cuda")
            for h in range(Hq):
                x = s["q"][i, :, h].double() @ k[:, h // G].T * SCALE
                x[:, n:][hidden] = -math.inf
                lse[i, :, h] = x.logsumexp(1)
                out[i, :, h] = x.softmax(1) @ v[:, h // G]
        return out, lse
    group = case["group"]
    for i in range(B):
        for r in range(L // group):
            a = i * (L // group) + r
            n = int(s["sel_lens"][a]) + group
            for g in range(Hkv):
                ids = s["sel"][a, g]
                k, v = (sequence(s[c][:, :, g], ids, n) for c in "kv")
                q = s["q"][i, r * group:(r + 1) * group, g * G:(g + 1) * G].double()
                out[i, r * group:(r + 1) * group, g * G:(g + 1) * G] = (q @ k.T * SCALE).softmax(-1) @ v
    return out
