"""Plain models of the serving operators (page tables, row writes, dense
attention behind a shared prefix), in Python integers and 64-bit floats."""
from __future__ import annotations

import math

import torch

PAGE = 16
D = 128


def model_page_table(old, new, table, free_pages, num_free, num_slots, prefix_len):
    """The update as a list program.  table (list of lists) and free_pages (list
    of pool-page count entries) are changed in place.  num_slots None: no slots.
    Returns (lens, num_free, slots, offsets)."""
    W, cap, keep = len(table[0]), len(free_pages), prefix_len // PAGE

    def pages(n):
        return max(-(-n // PAGE), keep)

    old = [max(0, min(o, W * PAGE)) for o in old]
    new = [max(0, n) for n in new]
    F = max(0, min(num_free, cap))
    for b in range(len(old)):
        for j in range(pages(new[b]), pages(old[b])):
            if new[b] < old[b]:
                if F < cap:
                    free_pages[F] = table[b][j]
                F = min(F + 1, cap)
    stack = free_pages[:F]
    lens, slots, offsets = [], [], [0]
    out_of_pages = False
    for b in range(len(old)):
        o, n = old[b], new[b]
        grow = max(0, n - o)
        end = offsets[-1] + grow
        fits = n <= W * PAGE and (num_slots is None or end <= num_slots)
        take = pages(n) - pages(o) if grow and fits else 0
        if take > len(stack):
            out_of_pages = True
        ok = grow and fits and (take == 0 or not out_of_pages)
        if ok:
            assert len(slots) == offsets[-1]
            for j in range(take):
                table[b][pages(o) + j] = stack.pop()
            for t in range(o, n):
                p = table[b][t // PAGE]
                slots.append(-1 if t < prefix_len or not 0 <= p < cap
                             else p * PAGE + t % PAGE)
        else:
            slots += [-1] * (grow if num_slots is None else min(grow, num_slots))
        lens.append(n if ok or n < o else o)
        offsets.append(min(end, 2 ** 31 - 1))
    if num_slots is not None:
        slots = (slots + [-1] * num_slots)[:num_slots]
    return lens, len(stack), slots, offsets


def gather(x, table, b, h, n):
    """Rows [0, n) of (b, h) in float64."""
    if table is None:
        return x[b, h, :n].double()
    t = torch.arange(n, device=x.device)
    return x[table[b].long()[t // PAGE], h, t % PAGE].double()


def check_attention(q, k, v, table, lens, out, lse):
    """Compare with softmax(q K^T / sqrt(128)) V of every sequence by itself.

    Bounds, per output channel, with w the exact weights, A = sum_t w_t |v_t|:
      - a weight rounded to fp16 is off by 2^-11 of itself: 2^-11 A; weights
        below fp16's normal range by 2^-32 of the largest: N 2^-32 max |v|;
      - a score is a sum of 128 exact products; in 32 bits, whatever the order
        and with a truncating adder, it is off by less than 128 * 2^-24 =
        2^-17 of s = sum |q k| / sqrt(128); a weight by twice that, as is the sum;
      - 32-bit exponentials, sums and merges: 2^-18 A for up to 2^18 terms in
        the orders used (blocked sums), 2^-11 |out| for the fp16 result."""
    B, Hq, _ = q.shape
    Hk = k.shape[1]
    G = Hq // Hk
    worst = 0.0
    for b in range(B):
        n = int(lens[b])
        if n == 0:
            assert bool((out[b] == 0).all()), b
            if lse is not None:
                assert bool((lse[b] == float("-inf")).all()), b
            continue
        for h in range(Hk):
            K, V = gather(k, table, b, h, n), gather(v, table, b, h, n)
            r = slice(h * G, (h + 1) * G)
            Q = q[b, r].double()
            z = Q @ K.t() / math.sqrt(D)
            s = float((Q.abs() @ K.abs().t()).max()) / math.sqrt(D)
            ref_lse = torch.logsumexp(z, -1)
            w = (z - ref_lse[:, None]).exp()
            ref, A = w @ V, w @ V.abs()
            tol = 2.0 ** -11 * (A + ref.abs()) * 1.001 + (4 * 2.0 ** -17 * s + 2.0 ** -18) * A \
                + n * 2.0 ** -32 * float(V.abs().max()) + 2.0 ** -25
            err = (out[b, r].double() - ref).abs()
            bad = bool((err > tol).any()) or not bool(torch.isfinite(out[b, r]).all())
            assert not bad, (b, h, n, float((err / tol).max()))
            worst = max(worst, float((err / tol).max()))
            if lse is not None:
                lt = 2.0 ** -17 * s + 2.0 ** -18 + 2.0 ** -23 * float(ref_lse.abs().max())
                e = float((lse[b, r].double() - ref_lse).abs().max())
                assert e <= lt, (b, h, n, e, lt)
    return worst


def make_prefix_case(seed, Hq, Hk, P, lens, paged, N=None, device="cuda", spread=1.0):
    """q, K, V, table, lens: every sequence's first P tokens are the same rows.
    Whatever the call may not use is NaN: rows at and past each sequence's end
    (beyond the prefix), pages that no sequence holds; table entries past the
    end are no page's id."""
    g = torch.Generator(device=device).manual_seed(seed)
    B = len(lens)
    longest = max([P] + list(lens)) if N is None else N
    W = max(1, -(-longest // PAGE))
    N = W * PAGE if paged else longest

    def rnd(*shape):
        return torch.randn(shape, generator=g, device=device, dtype=torch.float16)

    q = rnd(B, Hq, D) * spread
    nan = float("nan")
    if paged:
        own = [max(0, -(-n // PAGE) - P // PAGE) for n in lens]
        total = P // PAGE + sum(own) + 2
        ids = torch.randperm(total, generator=g, device=device).tolist()
        table = [[2 ** 30 + 7] * W for _ in range(B)]
        k = torch.full((total, Hk, PAGE, D), nan, dtype=torch.float16, device=device)
        v = k.clone()
        for j in range(P // PAGE):
            page = ids.pop()
            k[page], v[page] = rnd(Hk, PAGE, D), rnd(Hk, PAGE, D)
            table[0][j] = page
            for b in range(B):
                if j * PAGE < lens[b]:
                    table[b][j] = page
        for b in range(B):
            for j in range(P // PAGE, P // PAGE + own[b]):
                page = ids.pop()
                n = min(PAGE, lens[b] - j * PAGE)
                k[page, :, :n], v[page, :, :n] = rnd(Hk, n, D), rnd(Hk, n, D)
                table[b][j] = page
        table = torch.tensor(table, dtype=torch.int32, device=device)
    else:
        table = None
        k = torch.full((B, Hk, N, D), nan, dtype=torch.float16, device=device)
        v = k.clone()
        pk, pv = rnd(Hk, P, D), rnd(Hk, P, D)
        for b in range(B):
            n, m = lens[b], min(lens[b], P)
            k[b, :, :m], v[b, :, :m] = pk[:, :m], pv[:, :m]
            if n > P:
                k[b, :, P:n], v[b, :, P:n] = rnd(Hk, n - P, D), rnd(Hk, n - P, D)
        k[0, :, :P], v[0, :, :P] = pk, pv
    return q, k, v, table, torch.tensor(lens, dtype=torch.int32, device=device)
