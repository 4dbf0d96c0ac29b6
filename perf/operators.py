"""Cases of the serving operators around the paged cache: page tables and slot maps built on the
GPU (update_page_table), new K/V rows written by slot with their quantised keys and page min / max
(write_rows), and attention for a batch that shares a long prefix (prefix_decode).

The plain forms are elementary torch operations in 32 bits; where `own` is set, `run` makes the
package's calls instead.
"""
import math

import torch

own = False

D = 128       # head_dim
PAGE = 16     # tokens per page
GROUP = 32    # channels per quantisation group


# ------------------------------------------------------------------------------------- the cases
def listed():
    return [
        # a handful of interactive requests behind one short system prompt: latency
        dict(name="prefix_small_b3", op="prefix", B=3, Hq=32, Hk=8, P=512, lo=1, hi=96, short=0,
             paged=True),
        # multi-head attention, a medium batch behind a document
        dict(name="prefix_mha_b16", op="prefix", B=16, Hq=32, Hk=32, P=4096, lo=1, hi=1024,
             short=0, paged=True),
        # a grouped-query batch behind a 32k prompt: memory and tensor time about equal
        dict(name="prefix_gqa_b64_32k", op="prefix", B=64, Hq=32, Hk=8, P=32768, lo=16, hi=1024,
             short=0, paged=True),
        # the largest: many samples of one 128k context, bound by the tensor cores
        dict(name="prefix_gqa_b128_128k", op="prefix", B=128, Hq=32, Hk=8, P=131072, lo=1, hi=256,
             short=0, paged=True),
        # a contiguous cache of odd length, finished rows and rows shorter than the prefix
        dict(name="prefix_contig_ragged", op="prefix", B=21, Hq=8, Hk=1, P=2000, lo=1, hi=777,
             short=4, paged=False),
        # nothing shared: plain dense decode of a ragged batch
        dict(name="dense_b16", op="prefix", B=16, Hq=32, Hk=8, P=0, lo=1000, hi=9000, short=1,
             paged=True),
        # one decode step of a batch: a token each, now and then a new page
        dict(name="pages_decode_b256", op="pages", B=256, width=512, grow_lo=1, grow_hi=1,
             finish=0, prefix_pages=0, scarce=False),
        # prompts admitted together, some requests finished
        dict(name="pages_prefill_b48", op="pages", B=48, width=256, grow_lo=1, grow_hi=2000,
             finish=8, prefix_pages=32, scarce=False),
        # a large mixed batch that runs out of pages
        dict(name="pages_mixed_b2999", op="pages", B=2999, width=128, grow_lo=0, grow_hi=63,
             finish=200, prefix_pages=0, scarce=True),
        # the rows of one decode step
        dict(name="write_decode_t64", op="write", T=64, run=1, Hk=8, bits=4, paged=True, pad=0),
        # prompts of a grouped-query layer, with padded rows at the end
        dict(name="write_prefill_t8191", op="write", T=8191, run=1000, Hk=8, bits=4, paged=True,
             pad=100),
        # prompts of a multi-head layer on the 2-bit cache
        dict(name="write_mha_t20000", op="write", T=20000, run=4000, Hk=32, bits=2, paged=True,
             pad=0),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prefix", "prefix", "pages", "write"])
    if op == "prefix":
        while True:
            G, Hk = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 8, 32])
            B = _log(rng, 1, 256)
            P = PAGE * (_log(rng, 1, 8192) if rng.random() < 0.85 else 0)
            lo = _log(rng, 1, 64)
            hi = lo + _log(rng, 1, 4000)
            short = rng.randint(0, min(4, B - 1)) if rng.random() < 0.4 else 0
            paged = rng.random() < 0.75
            rows = B * (hi if paged else P + hi) + P
            if B * Hk * G * (P + hi) <= 400e6 and rows * Hk * 512 <= 1.2e9 and hi <= 4000:
                return dict(op=op, B=B, Hq=Hk * G, Hk=Hk, P=P, lo=lo, hi=hi, short=short,
                            paged=paged)
    if op == "pages":
        B = _log(rng, 1, 4000)
        width = _log(rng, 16, 512)
        lo = rng.randint(0, 2)
        hi = lo + rng.randint(0, min(PAGE * width // 2, 400000 // B))
        return dict(op=op, B=B, width=width, grow_lo=lo, grow_hi=hi,
                    finish=rng.randint(0, B // 4), prefix_pages=rng.choice([0, 0, width // 8]),
                    scarce=rng.random() < 0.3)
    while True:
        T, Hk = _log(rng, 1, 40000), rng.choice([1, 2, 4, 8, 32])
        if T * Hk <= 640000:
            return dict(op=op, T=T, run=_log(rng, 1, min(T, 4000)), Hk=Hk, bits=rng.choice([2, 4]),
                        paged=rng.random() < 0.75, pad=rng.randint(0, T // 8))


def _spread(n, lo, hi):
    """n whole numbers of [lo, hi], evenly spread: their sum does not depend on a seed."""
    return [lo + (hi - lo) * i // max(1, n - 1) for i in range(n)]


def _lengths(c):
    """Lengths of the batch: `short` rows within the prefix (the first of them empty), the rest
    prefix + [lo, hi]."""
    s = c["short"]
    return [c["P"] * i // max(1, s) for i in range(s)] + \
        [c["P"] + x for x in _spread(c["B"] - s, c["lo"], c["hi"])]


def work(c):
    if c["op"] == "prefix":
        lens = _lengths(c)
        rows = min(c["P"], max(lens)) + sum(max(0, n - c["P"]) for n in lens)
        heads = c["B"] * c["Hq"]
        return {"bytes": 512.0 * c["Hk"] * rows + heads * (2 * D * 2 + 4),
                "flops": 512.0 * c["Hq"] * sum(lens)}
    if c["op"] == "pages":
        grow = sum(_spread(c["B"], c["grow_lo"], c["grow_hi"]))
        slots = max(1, grow)
        # lengths in and out, offsets, a slot per token, a page id in and out per new or freed page
        return {"bytes": 16.0 * c["B"] + 4.0 * slots + 8.0 * (slots / PAGE), "flops": 0.0}
    rows = (c["T"] - c["pad"]) * c["Hk"]
    pages = -(-rows // min(PAGE, c["run"]))
    return {"bytes": rows * (1024.0 + D * c["bits"] / 8 + 16) + pages * 512.0 + 4.0 * c["T"],
            "flops": 0.0}


# ------------------------------------------------------------------------------------ the inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float16)


def _perm(g, n):
    return torch.randperm(n, generator=g, device="cuda")


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def prepare(c, seed):
    g = _gen(seed)
    state = {"prefix": _prepare_prefix, "pages": _prepare_pages, "write": _prepare_write}[c["op"]](
        c, g)
    state["c"] = c
    if own:
        _prepare_own(c, state)
    return state


def _prepare_prefix(c, g):
    B, Hq, Hk, P = c["B"], c["Hq"], c["Hk"], c["P"]
    lens = _i32(_lengths(c))[_perm(g, B)]
    longest = P + c["hi"]
    width = -(-longest // PAGE)
    q = _randn(g, B, Hq, D)
    if c["paged"]:
        own_pages = width - P // PAGE   # every sequence's own pages, as a server reserves them
        total = P // PAGE + B * own_pages
        ids = _perm(g, total).to(torch.int32)
        table = torch.empty(B, width, dtype=torch.int32, device="cuda")
        table[:, :P // PAGE] = ids[:P // PAGE]
        table[:, P // PAGE:] = ids[P // PAGE:].view(B, own_pages)
        k, v = _randn(g, total, Hk, PAGE, D), _randn(g, total, Hk, PAGE, D)
    else:
        table = None
        k, v = _randn(g, B, Hk, longest, D), _randn(g, B, Hk, longest, D)
        k[:, :, :P] = k[:1, :, :P].clone()
        v[:, :, :P] = v[:1, :, :P].clone()
    # a few keys that many queries look at
    heavy = _randn(g, Hk, D) * 0.5 + q[0].view(Hk, Hq // Hk, D).float().mean(1) * 0.35
    for t in (range(0, P, max(1, P // 5)) if P else ()):
        if c["paged"]:
            k[table[0, t // PAGE].long(), :, t % PAGE] = heavy.half()
        else:
            k[:, :, t] = heavy.half()
    return dict(q=q, k=k, v=v, lens=lens, table=table)


def _prepare_pages(c, g):
    B, width, keep = c["B"], c["width"], c["prefix_pages"]
    grow = _i32(_spread(B, c["grow_lo"], c["grow_hi"]))[_perm(g, B)]
    room = PAGE * (width - keep) - grow
    old = PAGE * keep + (torch.rand(B, generator=g, device="cuda") * (room + 1)).to(torch.int32)
    old = torch.minimum(old, torch.full_like(old, PAGE * width)).clamp_min_(0)
    new = old + grow
    if c["finish"]:
        new[_perm(g, B)[:c["finish"]]] = 0
    have = (old + PAGE - 1) // PAGE
    # page 0 is nobody's; each row holds its own pages, the shared ones first
    pool = 1 + keep + B * (width - keep)
    ids = 1 + _perm(g, pool - 1).to(torch.int32)
    full = ids[keep:].view(B, width - keep)
    table = torch.cat([ids[:keep].expand(B, keep), full], 1).contiguous()
    used = torch.arange(keep, width, device="cuda")[None] < have[:, None]
    # the stack: ids that no row uses, packed to the front
    rank = torch.argsort(used.reshape(-1).to(torch.int32), stable=True)
    free_pages = torch.zeros(pool, dtype=torch.int32, device="cuda")
    free_pages[:rank.numel()] = full.reshape(-1)[rank]
    num_free = (~used).sum().to(torch.int32).view(1)
    take = ((new + PAGE - 1) // PAGE - have.clamp_min(keep)).clamp_min(0).sum()
    if c["scarce"]:
        num_free = torch.minimum(num_free, (take * 3 // 4).to(torch.int32).view(1))
    table = torch.where(torch.arange(width, device="cuda")[None] < have.clamp_min(keep)[:, None],
                        table, torch.zeros_like(table)).contiguous()
    slots = max(1, sum(_spread(B, c["grow_lo"], c["grow_hi"])))
    return dict(lens=old, new=new, table=table, free=free_pages, num_free=num_free, keep=keep,
                num_slots=slots)


def _prepare_write(c, g):
    T, Hk, bits = c["T"], c["Hk"], c["bits"]
    real = max(1, T - c["pad"])
    runs = [min(c["run"], real - s) for s in range(0, real, c["run"])]
    B = len(runs)
    start = torch.randint(0, 37, (B,), generator=g, device="cuda")
    count = torch.tensor(runs, device="cuda")
    width = -(-(40 + c["run"]) // PAGE)
    seq = torch.arange(real, device="cuda") // c["run"]
    pos = start[seq] + torch.arange(real, device="cuda") - seq * c["run"]
    slots = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    if c["paged"]:
        pool = 1 + B * width   # page 0 is nobody's
        table = 1 + _perm(g, pool - 1).view(B, width)
        slots[:real] = (table[seq, pos // PAGE] * PAGE + pos % PAGE).to(torch.int32)
        shape = (pool, Hk, PAGE)
        meta_shape = (pool, Hk, 2, D)
        table = table.to(torch.int32).contiguous()
    else:
        N = PAGE * width - 3
        B += 1                 # sequence 0 is nobody's
        slots[:real] = ((seq + 1) * N + pos).to(torch.int32)
        shape = (B, Hk, N)
        meta_shape = (B, Hk, width, 2, D)
        table = None
        start = torch.cat([start[:1] * 0, start])
        count = torch.cat([count[:1] * 0, count])
    # rows as they come out of a fused projection: q, k and v side by side
    qkv = _randn(g, T, 3 * Hk * D)
    k_new = qkv[:, Hk * D:2 * Hk * D].view(T, Hk, D)
    v_new = qkv[:, 2 * Hk * D:].view(T, Hk, D)
    meta = torch.sort(_randn(g, *meta_shape), dim=-2).values
    lens = (start + count).to(torch.int32)
    return dict(k=_randn(g, *shape, D), v=_randn(g, *shape, D),
                codes=torch.zeros(*shape, D * bits // 8, dtype=torch.uint8, device="cuda"),
                scales=torch.zeros(*shape, D // GROUP, dtype=torch.float16, device="cuda"),
                zeros=torch.zeros(*shape, D // GROUP, dtype=torch.float16, device="cuda"),
                meta=meta, k_new=k_new, v_new=v_new, slots=slots, table=table, lens=lens)


def _prepare_own(c, s):
    """What a program keeps from step to step: cache handles, output buffers, a workspace."""
    import adaptive_top_sparse_quest_b200 as tw
    s["tw"] = tw
    if c["op"] == "prefix":
        kv = tw.KVCache(s["k"], s["v"], s["lens"], s["table"])
        s["step"] = tw.PrefixDecodeStep(kv, c["Hq"], c["P"])
    elif c["op"] == "pages":
        # the table serves every layer's cache, so it comes by itself
        s["update"] = tw.PageTableUpdate(s["lens"], s["table"], s["free"], s["num_slots"],
                                         PAGE * s["keep"])
    else:
        s["kv"] = tw.KVCache(s["k"], s["v"], s["lens"], s["table"], key_bits=c["bits"])
        s["keys"] = tw.Int4Keys(s["codes"], s["scales"], s["zeros"])


# -------------------------------------------------------------------------------------- one pass
def run(s):
    if own:
        return _run_own(s)
    return {"prefix": _plain_prefix, "pages": _plain_pages, "write": _plain_write}[s["c"]["op"]](s)


def _run_own(s):
    op = s["c"]["op"]
    if op == "prefix":
        step = s["step"]
        step(s["q"])
        return {"out": step.out, "lse": step.lse}
    if op == "pages":
        u = s["update"]
        u(s["new"], s["num_free"])
        return {"lens": u.seq_lens_out, "num_free": u.num_free_out, "table": s["table"],
                "free": s["free"], "slots": u.slots, "offsets": u.offsets}
    s["tw"].write_rows(s["kv"], s["k_new"], s["v_new"], s["slots"], s["keys"], s["meta"])
    return {n: s[n] for n in ("k", "v", "codes", "scales", "zeros", "meta")}


def _plain_prefix(s):
    """Scores of the shared prefix once for all rows, of each sequence's own tokens by itself,
    one softmax over both."""
    c = s["c"]
    B, Hq, Hk, P, lens = c["B"], c["Hq"], c["Hk"], c["P"], s["lens"]
    G = Hq // Hk
    if c["paged"]:
        n = P // PAGE
        first, rest = s["table"][0, :n].long(), s["table"][:, n:].long()
        kp, vp = (x[first].transpose(0, 1).reshape(Hk, P, D).float() for x in (s["k"], s["v"]))
        ks, vs = (x[rest].transpose(1, 2).reshape(B, Hk, -1, D).float() for x in (s["k"], s["v"]))
    else:
        kp, vp = (x[0, :, :P].float() for x in (s["k"], s["v"]))
        ks, vs = (x[:, :, P:].float() for x in (s["k"], s["v"]))
    q = s["q"].float().view(B, Hk, G, D) / math.sqrt(D)
    low = float("-inf")
    own_len = (lens - P)[:, None, None, None]
    s2 = (q @ ks.transpose(-1, -2)).masked_fill_(
        torch.arange(ks.shape[2], device="cuda") >= own_len, low)          # [B][Hk][G][S]
    top = s2.amax(-1)
    if P:
        s1 = q.transpose(0, 1).reshape(Hk, B * G, D) @ kp.transpose(-1, -2)   # [Hk][B G][P]
        s1 = s1.view(Hk, B, G, P).masked_fill_(
            torch.arange(P, device="cuda") >= lens[:, None, None], low)
        top = torch.maximum(top, s1.amax(-1).transpose(0, 1))
    base = top.masked_fill(top == low, 0.0)
    p2 = (s2 - base[..., None]).exp_()
    total = p2.sum(-1)
    acc = p2 @ vs
    if P:
        p1 = (s1 - base.transpose(0, 1)[..., None]).exp_()
        total = total + p1.sum(-1).transpose(0, 1)
        acc = acc + (p1.view(Hk, B * G, P) @ vp).view(Hk, B, G, D).transpose(0, 1)
    out = acc / total.masked_fill(total == 0, 1.0)[..., None]
    return {"out": out.reshape(B, Hq, D).half(), "lse": (base + total.log()).reshape(B, Hq)}


def _plain_pages(s):
    """Sums over the batch, then every table entry and every slot by its own formula."""
    old, new, table, free, keep = (s[n] for n in ("lens", "new", "table", "free", "keep"))
    B, width = table.shape
    n_slots = s["num_slots"]
    have, want = (torch.clamp((x + PAGE - 1) // PAGE, min=keep) for x in (old, new))
    grow = (new - old).clamp_min(0).long()
    ends = grow.cumsum(0)
    offsets = torch.cat([ends.new_zeros(1), ends])
    give = (have - want).clamp_min(0).long()
    give_at = give.cumsum(0) - give
    fits = (new <= width * PAGE) & (ends <= n_slots)
    take = torch.where(fits, (want - have).clamp_min(0), 0).long()
    take_end = take.cumsum(0)
    avail = s["num_free"].long() + give.sum()
    granted = fits & ((take == 0) | (take_end <= avail)) & (new > old)
    out_lens = torch.where((new < old) | granted, new, old)
    left = avail - torch.where(granted, take, 0).sum()
    # pages given back go onto the stack
    col = torch.arange(width, device="cuda")[None]
    back = (col >= want[:, None]) & (col < have[:, None])
    at = torch.where(back, s["num_free"] + give_at[:, None] + col - want[:, None], free.numel())
    stack = torch.cat([free, free.new_zeros(1)])
    stack = stack.scatter(0, at.reshape(-1), table.reshape(-1))[:-1]
    free.copy_(stack)
    # pages taken come off its top
    fresh = granted[:, None] & (col >= have[:, None]) & (col < want[:, None])
    pick = avail - 1 - ((take_end - take)[:, None] + col - have[:, None])
    table.copy_(torch.where(fresh, stack[pick.clamp(0, free.numel() - 1)], table))
    # a slot for each token that grew
    i = torch.arange(n_slots, device="cuda")
    b = torch.searchsorted(ends, i, right=True)
    inside = b < B
    b = b.clamp_max(B - 1)
    pos = old[b] + i - offsets[b]
    page = table[b, (pos // PAGE).clamp(0, width - 1)]
    ok = inside & granted[b] & (pos >= keep * PAGE)
    slots = torch.where(ok, page * PAGE + pos % PAGE, -1).to(torch.int32)
    return {"lens": out_lens.to(torch.int32), "num_free": left.to(torch.int32).view(1),
            "table": table, "free": free, "slots": slots, "offsets": offsets.to(torch.int32)}


def _plain_write(s):
    """Rows by index; the quantised keys of the new rows; page min / max by an indexed reduction.
    A slot below zero goes to row 0, which nobody uses, with what is there already."""
    c = s["c"]
    bits, levels = c["bits"], 2 ** c["bits"] - 1
    slots, kn, vn = s["slots"].long(), s["k_new"], s["v_new"]
    live = slots >= 0
    slots = slots.clamp_min(0)
    if c["paged"]:
        first, off = slots // PAGE, slots % PAGE
    else:
        N = s["k"].shape[2]
        first, off = slots // N, slots % N
    ix = (first[:, None], torch.arange(c["Hk"], device="cuda")[None], off[:, None])
    lv = live[:, None, None]
    x = kn.float().view(c["T"], c["Hk"], D // GROUP, GROUP)
    lo, hi = x.amin(-1), x.amax(-1)
    scale = ((hi - lo) / levels).half()
    sc = scale.float()[..., None]
    code = torch.round((x - lo[..., None]) / sc.masked_fill(sc == 0, 1.0))
    code = code.clamp_(0, levels).masked_fill_(sc == 0, 0).to(torch.uint8)
    per = 8 // bits
    code = code.view(c["T"], c["Hk"], D // per, per)
    shift = torch.arange(per, device="cuda", dtype=torch.uint8) * bits
    packed = (code << shift).sum(-1, dtype=torch.uint8)
    for name, new in (("k", kn), ("v", vn), ("codes", packed), ("scales", scale),
                      ("zeros", lo.half())):
        t = s[name]
        t[ix] = torch.where(lv, new, t[ix])
    # the page of each row, and whether these rows begin it
    meta = s["meta"]
    flat = meta.view(-1, c["Hk"], 2, D) if c["paged"] else meta.transpose(1, 2)
    flat = flat.reshape(-1, c["Hk"], 2, D)
    pg = first if c["paged"] else first * meta.shape[2] + off // PAGE
    begins = live & (off % PAGE == 0)
    fresh = torch.zeros(flat.shape[0], dtype=torch.int32, device="cuda")
    fresh = fresh.scatter_reduce(0, pg, begins.to(torch.int32), "amax")
    fresh = fresh.bool()[:, None, None]
    inf = float("inf")
    low = torch.where(fresh, inf, flat[:, :, 0].float())
    high = torch.where(fresh, -inf, flat[:, :, 1].float())
    at = pg[:, None, None].expand(c["T"], c["Hk"], D)
    low = low.scatter_reduce(0, at, torch.where(lv, kn.float(), inf), "amin")
    high = high.scatter_reduce(0, at, torch.where(lv, kn.float(), -inf), "amax")
    both = torch.stack([low, high], 2).half()
    if not c["paged"]:
        both = both.view(meta.shape[0], meta.shape[2], c["Hk"], 2, D).transpose(1, 2)
    meta.copy_(both)
    return {n: s[n] for n in ("k", "v", "codes", "scales", "zeros", "meta")}


# --------------------------------------------------------------------- the definitions, in 64 bits
def exact(c, seed):
    if c["op"] == "pages":
        return None   # whole numbers
    g = _gen(seed)
    if c["op"] == "prefix":
        return _exact_prefix(c, _prepare_prefix(c, g))
    return _exact_write(c, _prepare_write(c, g))


def _exact_prefix(c, s):
    """Each sequence by itself: its own list of rows, the softmax of its scores, their mean of V."""
    B, Hq, Hk = c["B"], c["Hq"], c["Hk"]
    out = torch.zeros(B, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq), float("-inf"), dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["lens"].tolist()):
        if n == 0:
            continue
        for h in range(Hk):
            if c["paged"]:
                t = torch.arange(n, device="cuda")
                page = s["table"][b].long()[t // PAGE]
                k, v = s["k"][page, h, t % PAGE].double(), s["v"][page, h, t % PAGE].double()
            else:
                k, v = s["k"][b, h, :n].double(), s["v"][b, h, :n].double()
            r = slice(h * Hq // Hk, (h + 1) * Hq // Hk)
            z = s["q"][b, r].double() @ k.t() / D ** 0.5
            lse[b, r] = torch.logsumexp(z, -1)
            out[b, r] = (z - lse[b, r][:, None]).exp() @ v
    return {"out": out, "lse": lse}


def _exact_write(c, s):
    """Token by token in runs of one page: what each row and each page holds afterwards."""
    T, Hk = c["T"], c["Hk"]
    res = {n: s[n].double() for n in ("k", "v", "scales", "zeros", "meta")}
    N = PAGE if c["paged"] else s["k"].shape[2]
    slot = s["slots"].tolist()
    levels = 2 ** c["bits"] - 1
    group = s["k_new"].double().reshape(T, Hk, D // GROUP, GROUP)
    low, high = group.min(-1).values, group.max(-1).values
    step = (high - low) / levels
    i = 0
    while i < T:
        if slot[i] < 0:
            i += 1
            continue
        a, o = divmod(slot[i], N)
        j = i + 1
        while j < T and slot[j] == slot[j - 1] + 1 and (slot[j] % N) // PAGE == o // PAGE and \
                slot[j] // N == a:
            j += 1
        rows = slice(o, o + j - i)
        res["k"][a, :, rows] = s["k_new"][i:j].transpose(0, 1).double()
        res["v"][a, :, rows] = s["v_new"][i:j].transpose(0, 1).double()
        res["scales"][a, :, rows] = step[i:j].transpose(0, 1)
        res["zeros"][a, :, rows] = low[i:j].transpose(0, 1)
        m = res["meta"][a] if c["paged"] else res["meta"][a, :, o // PAGE]
        k = s["k_new"][i:j].double()
        k_lo, k_hi = k.min(0).values, k.max(0).values
        if o % PAGE:
            k_lo, k_hi = torch.minimum(k_lo, m[:, 0]), torch.maximum(k_hi, m[:, 1])
        m[:, 0], m[:, 1] = k_lo, k_hi
        i = j
    return {"k": res["k"], "v": res["v"], "codes": None, "scales": res["scales"],
            "zeros": res["zeros"], "meta": res["meta"]}
