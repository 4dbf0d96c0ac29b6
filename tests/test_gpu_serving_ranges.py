"""The serving operators at ends of their ranges that the other tests pass over:
lists of so many short runs that a warp takes sixteen, several tiles of query
rows behind a long prefix, and page bounds of pages that changed hands."""
import random

import pytest
import torch

import oracle as O
from _parity import gpu_meta, np16
from _serving import D, PAGE, check_attention, make_prefix_case, model_page_table

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from adaptive_top_sparse_quest_b200 import _capi, build
    build.build()
    _capi.load()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("paged", [True, False])
@pytest.mark.parametrize("run,T,Hk,bits", [(1, 16384, 8, 4), (2, 20000, 8, 2), (3, 9001, 16, 4),
                                           (1, 4736, 8, 4), (17, 40000, 1, 4)])
def test_write_rows_of_many_short_runs(run, T, Hk, bits, paged):
    """`run` tokens for each of T / run sequences, whose earlier rows are current,
    some places of the list empty: the rows, and the quantised keys and bounds as
    rebuilt from them."""
    from adaptive_top_sparse_quest_b200 import KVCache, page_meta, quantize_keys, write_rows
    g = torch.Generator(device="cuda").manual_seed(run * T)
    B, W = T // run, 3
    N = W * PAGE if paged else W * PAGE - 5

    def rnd(*s):
        return torch.randn(s, generator=g, device="cuda", dtype=torch.float16)

    if paged:
        table = torch.randperm(B * W, generator=g, device="cuda").to(torch.int32).view(B, W)
        k, v = rnd(B * W, Hk, PAGE, D), rnd(B * W, Hk, PAGE, D)
    else:
        table, k, v = None, rnd(B, Hk, N, D), rnd(B, Hk, N, D)
    old = torch.randint(0, 20, (B,), generator=g, device="cuda").to(torch.int32)
    kv = KVCache(k, v, old, table, bits)
    keys, meta = quantize_keys(kv), page_meta(kv)
    before = k.clone(), v.clone()
    grow = torch.full_like(old, run)
    grow[::7] = 0                       # sequences that do not grow: -1 in their places
    pos = old[:, None] + torch.arange(run, device="cuda", dtype=torch.int32)
    b = torch.arange(B, device="cuda")[:, None].expand(B, run)
    if paged:
        slots = table[b, (pos // PAGE).long()] * PAGE + pos % PAGE
    else:
        slots = (b * N + pos).to(torch.int32)
    slots = torch.where(grow[:, None] > 0, slots, -1).reshape(-1).contiguous()
    new = rnd(B * run, 2, Hk, D)
    write_rows(kv, new[:, 0], new[:, 1], slots, keys, meta)
    live = slots >= 0
    s, rows = slots[live].long(), PAGE if paged else N
    for x, was, i in ((k, before[0], 0), (v, before[1], 1)):
        was[s // rows, :, s % rows] = new[live, i]
        assert torch.equal(x, was)
    kv.seq_lens = old + grow
    again, bounds = quantize_keys(kv), page_meta(kv)
    # (both start from zeros, and rows past the lengths stay so)
    assert torch.equal(keys.codes, again.codes)
    for x, y in ((keys.scales, again.scales), (keys.zeros, again.zeros), (meta, bounds)):
        assert torch.equal(x.view(torch.int16), y.view(torch.int16))


@pytest.mark.parametrize("c", [
    # 300 and 520 rows per KV head: two and three tiles of 256, the last one ragged
    dict(Hq=4, Hk=2, P=20000, lens=[20000 + (29 * i) % 170 for i in range(150)], paged=True),
    dict(Hq=8, Hk=1, P=12816, lens=[12816 * (i % 9 > 0) + (401 * i) % 333 for i in range(65)],
         paged=True),
    dict(Hq=32, Hk=4, P=8208, lens=[8208 - 131 * (i % 5) for i in range(64)], paged=False),
], ids=["2tiles", "3tiles", "short"])
def test_prefix_decode_row_tiles_behind_a_long_prefix(c):
    from adaptive_top_sparse_quest_b200 import KVCache, PrefixDecodeStep, device_status
    q, k, v, table, lens = make_prefix_case(21, c["Hq"], c["Hk"], c["P"], c["lens"], c["paged"])
    step = PrefixDecodeStep(KVCache(k, v, lens, table), c["Hq"], c["P"])
    step(q)
    assert device_status(step.ws) == 0
    check_attention(q, k, v, table, lens.tolist(), step.out, step.lse)


def test_page_bounds_of_pages_that_change_hands():
    """Requests grow, finish and shrink on few pages, so that pages return to the
    stack and serve others.  Bounds are exact, bit for bit, but for pages cut short
    inside, which keep bounds that hold the rows cut off as well, until they are
    given back."""
    from adaptive_top_sparse_quest_b200 import (KVCache, PageTableUpdate, page_meta, quantize_keys,
                                                write_rows)
    rng = random.Random(17)
    B, Hk, W, P, T = 6, 2, 12, 32, 200
    keep = P // PAGE
    pool = keep + 14
    g = torch.Generator(device="cuda").manual_seed(6)

    def rnd(*s):
        return torch.randn(s, generator=g, device="cuda", dtype=torch.float16)

    k = rnd(pool, Hk, PAGE, D) * 50     # what pages held before must not reach their bounds
    table = i32([list(range(keep)) + [0] * (W - keep) for _ in range(B)])
    lens = i32([P] * B)
    free, nf, new = i32(list(range(keep, pool)) + [0] * keep), i32([pool - keep]), i32([P] * B)
    kv = KVCache(k, k.clone(), lens, table)
    keys, meta = quantize_keys(kv), page_meta(kv)
    update = PageTableUpdate(lens, table, free, T, P, in_place=True)
    m = dict(lens=[P] * B, table=table.tolist(), free=free.tolist(), nf=pool - keep)
    cut, owner, moved, exact, wide = set(), {}, 0, 0, 0
    for step in range(40):
        want = [rng.choice([n + 1, n + 1, n + rng.randint(0, 40), P, max(P, n - 3)])
                for n in m["lens"]]
        new.copy_(i32(want))
        update(new, nf)
        before = m["lens"]
        held = {m["table"][b][j] for b in range(B) for j in range(keep, -(-before[b] // PAGE))}
        cut |= {m["table"][b][n // PAGE] for b, n in enumerate(want)
                if n < before[b] and n % PAGE}
        ml, mnf, mslots, _ = model_page_table(before, want, m["table"], m["free"], m["nf"], T, P)
        m.update(lens=ml, nf=mnf)
        assert lens.tolist() == ml and update.slots.tolist() == mslots
        now = {m["table"][b][j]: b for b in range(B) for j in range(keep, -(-ml[b] // PAGE))}
        # a page that is no row's any more, or another's, began anew
        cut = {p for p in cut if p in held and now.get(p) == owner.get(p, now.get(p))}
        moved += sum(p in owner and owner[p] != b for p, b in now.items())
        owner.update(now)
        write_rows(kv, rnd(T, Hk, D), rnd(T, Hk, D), update.slots, keys, meta)
        K, M, tb = np16(k), np16(meta), table.cpu().numpy()
        for b in range(B):
            for h in range(Hk):
                got = gpu_meta(M, tb, b, h, ml[b])
                full = O.page_meta(O.sequence_rows(K, tb, b, h, ml[b]), ml[b])
                for j in range(len(got)):
                    if m["table"][b][j] in cut:
                        assert (got[j, 0] <= full[j, 0]).all() and (got[j, 1] >= full[j, 1]).all()
                        wide += 1
                    else:
                        assert (got[j].view("u2") == full[j].view("u2")).all(), (step, b, h, j)
                        exact += 1
    assert moved > 20 and exact > 500 and wide > 20, (moved, exact, wide)


def test_sizes_past_32_bits_and_bad_prefixes_are_refused():
    """Not cut to their low 32 bits on the way into the library."""
    from adaptive_top_sparse_quest_b200 import PageTableUpdate, update_page_table
    lens, table, free = i32([0, 3]), i32([[0, 0], [1, 0]]), i32([2, 3, 4, 0, 0])
    for bad in (dict(num_slots=-1), dict(num_slots=2 ** 32 + 8), dict(prefix_len=2 ** 32),
                dict(prefix_len=-16), dict(prefix_len=8), dict(prefix_len=48)):
        with pytest.raises(ValueError):
            PageTableUpdate(lens, table, free, **bad)
        with pytest.raises(ValueError):
            update_page_table(lens, lens, table, free, i32([3]), **bad)
    PageTableUpdate(lens, table, free, 8, 32)(lens, i32([3]))


def test_prefix_decode_of_nothing():
    """No sequences; a cache without rows (refused where it has no address, as all
    calls do); sequences that are all empty."""
    import ctypes
    from adaptive_top_sparse_quest_b200 import KVCache, PrefixDecodeStep, TwError, _capi, prefix_decode
    k = torch.zeros(4, 2, PAGE, D, dtype=torch.float16, device="cuda")
    kv = KVCache(k, k, i32([]), torch.zeros(0, 4, dtype=torch.int32, device="cuda"))
    out, lse = prefix_decode(k.new_zeros(0, 8, D), kv, 16)
    assert out.shape == (0, 8, D) and lse.shape == (0, 8)
    none, q = k.new_zeros(3, 2, 0, D), torch.randn(3, 4, D, device="cuda").half()
    with pytest.raises(TwError):
        PrefixDecodeStep(KVCache(none, none, i32([0, 5, -1])), 4, 0)(q)
    kv = KVCache(k[:3], k[:3], i32([0, 0, -7]))
    step = PrefixDecodeStep(kv, 4, 0)
    for rows in (PAGE, 0):
        step.out.fill_(7)
        st = kv.struct()
        st.max_seq_len = rows
        assert _capi.load().tw_prefix_decode(
            q.data_ptr(), 4, ctypes.byref(st), 0, step.out.data_ptr(), step.lse.data_ptr(),
            step.ws.data_ptr(), step.ws.numel(), torch.cuda.current_stream().cuda_stream) == 0
        assert bool((step.out == 0).all()) and bool((step.lse == float("-inf")).all())


@pytest.mark.parametrize("c", [
    dict(Hq=8, Hk=1, P=16, lens=[16 + i % 5 for i in range(5000)], paged=True),
    dict(Hq=256, Hk=128, P=48, lens=[50, 47, 300], paged=True),
    dict(Hq=4, Hk=1, P=0, lens=[262144], paged=False),
    dict(Hq=2, Hk=2, P=4096, lens=[4096, 4096, 1], paged=True),
], ids=["5000", "128heads", "256k", "no_own"])
def test_prefix_decode_at_the_ends_of_the_range(c):
    from adaptive_top_sparse_quest_b200 import KVCache, PrefixDecodeStep, device_status
    q, k, v, table, lens = make_prefix_case(31, c["Hq"], c["Hk"], c["P"], c["lens"], c["paged"])
    step = PrefixDecodeStep(KVCache(k, v, lens, table), c["Hq"], c["P"])
    step(q)
    assert device_status(step.ws) == 0
    check_attention(q, k, v, table, lens.tolist(), step.out, step.lse)


def test_serving_step_captured_across_streams():
    """A graph that forks: lengths come by a copy, the table is updated on one
    branch while q is copied on another, rows are written and attended to after
    both; replayed with other inputs."""
    from adaptive_top_sparse_quest_b200 import (KVCache, PageTableUpdate, PrefixDecodeStep,
                                                device_status, page_meta, quantize_keys, write_rows)
    g = torch.Generator(device="cuda").manual_seed(3)
    B, Hq, Hk, W, P, T = 5, 16, 2, 10, 32, 60
    pool = 2 + B * (W - 2)

    def rnd(*s):
        return torch.randn(s, generator=g, device="cuda", dtype=torch.float16)

    k, v = rnd(pool, Hk, PAGE, D), rnd(pool, Hk, PAGE, D)
    table = i32([[0, 1] + [0] * (W - 2) for _ in range(B)])
    lens, free, nf = i32([P] * B), i32(list(range(2, pool)) + [0, 0]), i32([pool - 2])
    kv = KVCache(k, v, lens, table)
    keys, meta = quantize_keys(kv), page_meta(kv)
    update = PageTableUpdate(lens, table, free, T, P, in_place=True)
    step = PrefixDecodeStep(kv, Hq, P)
    new, q, kn, vn = i32([P] * B), rnd(B, Hq, D), rnd(T, Hk, D), rnd(T, Hk, D)
    h_new, h_q = new.cpu().pin_memory(), q.cpu().pin_memory()

    def once(side):
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        with torch.cuda.stream(side):
            new.copy_(h_new, non_blocking=True)
            update(new, nf)
        q.copy_(h_q, non_blocking=True)
        here.wait_stream(side)
        write_rows(kv, kn, vn, update.slots, keys, meta)
        side.wait_stream(here)
        step(q, stream=side)
        here.wait_stream(side)

    side = torch.cuda.Stream()
    once(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        once(side)
    m = dict(lens=[P] * B, table=table.tolist(), free=free.tolist(), nf=int(nf))
    for want in ([33, 40, 32, 50, 32], [34, 41, 32, 32, 60], [90, 42, 45, 33, 61], [32] * 5):
        h_new.copy_(torch.tensor(want, dtype=torch.int32))
        h_q.copy_(rnd(B, Hq, D).cpu())
        kn.copy_(rnd(T, Hk, D))
        vn.copy_(rnd(T, Hk, D))
        graph.replay()
        torch.cuda.synchronize()
        ml, mnf, slots, _ = model_page_table(m["lens"], want, m["table"], m["free"], m["nf"], T, P)
        m.update(lens=ml, nf=mnf)
        # (the third asks for 56 + 1 + 13 + 1 + 1 of 60 places: two are served)
        assert lens.tolist() == ml and update.slots.tolist() == slots
        assert table.tolist() == m["table"] and device_status(step.ws) == 0
        for i, s in enumerate(slots):
            if s >= 0:
                assert torch.equal(k[s // PAGE, :, s % PAGE], kn[i])
        check_attention(h_q.cuda(), k, v, table, ml, step.out, step.lse)
