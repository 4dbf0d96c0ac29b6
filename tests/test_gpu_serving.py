"""The serving operators on the GPU against plain models: page tables and slot
maps from lengths (exact), rows written by slot with their quantised keys and
page metadata (bit for bit a rebuild), dense attention behind a shared prefix
(64-bit reference), each alone, captured, on other streams, and together as a
serving loop uses them."""
import random

import pytest
import torch

import oracle as O
from _parity import gpu_meta, gpu_rows, np16
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


# ------------------------------------------------------------------------------ page tables
def _pages_case(seed, B, W, keep, grow, fill, num_slots=None):
    """Rows that hold distinct pages for their lengths, a stack of the rest."""
    rng = random.Random(seed)
    pool = keep + B * (W - keep) + 3
    ids = list(range(pool))
    rng.shuffle(ids)
    prefix, ids = ids[:keep], ids[keep:]
    old, new, table = [], [], []
    for b in range(B):
        o = rng.choice([0, keep * PAGE, rng.randint(0, int(W * PAGE * fill)), W * PAGE,
                        PAGE * rng.randint(0, W)])
        n = rng.choice([o + rng.randint(0, grow), o + 1, o, 0, rng.randint(0, o), o - 1, o + grow])
        have = max(-(-o // PAGE), keep)
        table.append(prefix + [ids.pop() for _ in range(have - keep)] + [-5] * (W - have))
        old.append(o)
        new.append(n)
    free = ids + [0] * (pool - len(ids))
    slots = sum(max(0, n - o) for o, n in zip(old, new))
    return old, new, table, free, len(ids), slots if num_slots is None else num_slots(slots)


PAGE_CASES = [
    dict(seed=1, B=1, W=1, keep=0, grow=5, fill=1.0),
    dict(seed=2, B=7, W=9, keep=2, grow=40, fill=0.8),
    dict(seed=3, B=33, W=20, keep=0, grow=1, fill=0.5),
    dict(seed=4, B=256, W=64, keep=5, grow=300, fill=0.6),
    dict(seed=5, B=1025, W=12, keep=0, grow=50, fill=0.7),
    dict(seed=6, B=8192, W=8, keep=1, grow=30, fill=0.5),
    dict(seed=7, B=60, W=200, keep=0, grow=2000, fill=0.3, num_slots=lambda s: s // 2),
    dict(seed=8, B=60, W=200, keep=0, grow=2000, fill=0.3, num_slots=lambda s: s + 777),
    dict(seed=9, B=12, W=30, keep=0, grow=100, fill=0.3, scarce=0.4),
    dict(seed=10, B=900, W=30, keep=3, grow=100, fill=0.3, scarce=0.5),
    dict(seed=11, B=20, W=30, keep=30, grow=100, fill=0.3),
    dict(seed=12, B=50, W=16, keep=0, grow=90, fill=0.9, scarce=0.0),
]


@pytest.mark.parametrize("c", PAGE_CASES, ids=lambda c: f"s{c['seed']}")
@pytest.mark.parametrize("in_place", [False, True])
def test_page_table_update(c, in_place):
    from adaptive_top_sparse_quest_b200 import PageTableUpdate
    c = dict(c)
    scarce = c.pop("scarce", None)
    old, new, table, free, nf, ns = _pages_case(**c)
    if scarce is not None:
        nf = int(nf * scarce)
    lens_t, table_t, free_t, nf_t = i32(old), i32(table), i32(free), i32([nf])
    u = PageTableUpdate(lens_t, table_t, free_t, ns, PAGE * c["keep"], in_place=in_place)
    u(i32(new), nf_t)
    got = (u.seq_lens_out.tolist(), int(u.num_free_out), u.slots.tolist(), u.offsets.tolist())
    want = model_page_table(old, new, table, free, nf, ns if ns else None, PAGE * c["keep"])
    if not ns:
        want = (want[0], want[1], [], want[3])
    assert got == want
    assert table_t.tolist() == table and free_t.tolist() == free
    if in_place:
        assert lens_t.tolist() == want[0] and int(nf_t) == want[1]
    else:
        assert lens_t.tolist() == old and int(nf_t) == nf


def test_page_table_without_slots_and_empty_batch():
    from adaptive_top_sparse_quest_b200 import update_page_table
    old, new, table, free, nf, _ = _pages_case(21, 40, 10, 0, 60, 0.5)
    table_t, free_t = i32(table), i32(free)
    u = update_page_table(i32(old), i32(new), table_t, free_t, i32([nf]))
    want = model_page_table(old, new, table, free, nf, None, 0)
    assert u.seq_lens_out.tolist() == want[0] and int(u.num_free_out) == want[1]
    assert u.offsets.tolist() == want[3] and table_t.tolist() == table
    u = update_page_table(i32([]), i32([]), torch.zeros(0, 4, dtype=torch.int32, device="cuda"),
                          free_t, i32([3]), num_slots=5)
    assert u.slots.tolist() == [-1] * 5 and u.offsets.tolist() == [0] and int(u.num_free_out) == 3


def test_page_table_hostile_values():
    """Lengths, heights and ids that no server should pass: clamped, nothing
    outside the arrays is touched."""
    from adaptive_top_sparse_quest_b200 import update_page_table
    big = 2 ** 31 - 1
    old = [-4, big, 10, 20, 0, 5]
    new = [3, 5, big, -7, big, 40]
    table = [[-1] * 4, [1, 2, 99, -8], [3, 0, 0, 0], [4, 77, 0, 0], [0] * 4, [2 ** 30, 0, 0, 0]]
    for nf in (-3, 0, 5, 99):
        free = [9, 8, 7, 6, 5, 4, 3, 2]
        t, f = [r[:] for r in table], free[:]
        table_t, free_t = i32(t), i32(f)
        u = update_page_table(i32(old), i32(new), table_t, free_t, i32([nf]), num_slots=64)
        want = model_page_table(old, new, t, f, nf, 64, 0)
        assert (u.seq_lens_out.tolist(), int(u.num_free_out), u.slots.tolist(),
                u.offsets.tolist()) == want
        assert table_t.tolist() == t and free_t.tolist() == f


def test_page_table_captured_in_place():
    """A captured in-place update replayed step by step is the model's loop."""
    from adaptive_top_sparse_quest_b200 import PageTableUpdate
    rng = random.Random(3)
    B, W, pool = 50, 20, 400
    lens_t, table_t = i32([0] * B), i32([[0] * W for _ in range(B)])
    free_t, nf_t, new_t = i32(list(range(pool))), i32([pool]), i32([0] * B)
    u = PageTableUpdate(lens_t, table_t, free_t, 900, in_place=True)
    u(new_t, nf_t)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        u(new_t, nf_t)
    lens, table, free, nf = [0] * B, [[0] * W for _ in range(B)], list(range(pool)), pool
    for _ in range(15):
        new = [rng.choice([n + 1, n + rng.randint(0, 33), 0, n]) for n in lens]
        new_t.copy_(i32(new))
        g.replay()
        lens, nf, slots, offs = model_page_table(lens, new, table, free, nf, 900, 0)
        assert lens_t.tolist() == lens and int(nf_t) == nf
        assert u.slots.tolist() == slots and u.offsets.tolist() == offs
        assert table_t.tolist() == table and free_t.tolist() == free


# -------------------------------------------------------------------------------- row writes
def _cache(B, Hk, W, paged, N, bits):
    from adaptive_top_sparse_quest_b200 import Int4Keys, KVCache, page_meta, quantize_keys
    g = torch.Generator(device="cuda").manual_seed(77)
    if paged:
        pool = B * W + 1
        ids = (torch.randperm(pool - 1, generator=g, device="cuda") + 1).to(torch.int32)
        table = ids.view(B, W).contiguous()
        shape = (pool, Hk, PAGE, D)
    else:
        table, shape = None, (B, Hk, N, D)
    k = torch.randn(shape, generator=g, device="cuda", dtype=torch.float16)
    v = torch.randn(shape, generator=g, device="cuda", dtype=torch.float16)
    kv = KVCache(k, v, torch.zeros(B, dtype=torch.int32, device="cuda"), table, bits)
    return kv


WRITE_CASES = [
    dict(old=[0], new=[1], Hk=1, paged=True, bits=4),
    dict(old=[0, 15, 16, 31, 5], new=[1, 16, 17, 33, 5], Hk=2, paged=True, bits=4),
    dict(old=[0, 3, 40, 16], new=[90, 50, 41, 64], Hk=8, paged=True, bits=2),
    dict(old=[0, 0, 100], new=[300, 17, 333], Hk=3, paged=False, bits=4),
    dict(old=[7, 8], new=[77, 9], Hk=32, paged=False, bits=2),
    dict(old=[0] * 40, new=list(range(0, 400, 10)), Hk=20, paged=True, bits=4),
    dict(old=[0, 1], new=[3000, 2000], Hk=4, paged=True, bits=4),
]


@pytest.mark.parametrize("c", WRITE_CASES, ids=lambda c: f"B{len(c['old'])}Hk{c['Hk']}b{c['bits']}")
def test_write_rows_equals_rebuild(c):
    """After the write, K / V hold the new rows, nothing else changed, and the
    quantised cache and metadata equal the oracle's rebuild for the new lengths."""
    from adaptive_top_sparse_quest_b200 import page_meta, quantize_keys, write_rows
    B, Hk = len(c["old"]), c["Hk"]
    W = -(-max(c["new"]) // PAGE) + 1
    N = max(c["new"]) + 3
    kv = _cache(B, Hk, W, c["paged"], N, c["bits"])
    kv.seq_lens.copy_(i32(c["old"]))
    keys, meta = quantize_keys(kv), page_meta(kv)
    before = [t.clone() for t in (kv.k, kv.v, keys.codes, keys.scales, keys.zeros, meta)]
    slots, where = [], []
    pages = kv.page_table.tolist() if c["paged"] else None
    for b in range(B):
        for t in range(c["old"][b], c["new"][b]):
            if c["paged"]:
                slots.append(pages[b][t // PAGE] * PAGE + t % PAGE)
            else:
                slots.append(b * N + t)
            where.append((b, t))
    slots = slots + [-1] * 5 if len(slots) % 2 else slots
    T = len(slots)
    g = torch.Generator(device="cuda").manual_seed(5)
    qkv = torch.randn(T, 3, Hk, D, generator=g, device="cuda", dtype=torch.float16)
    qkv[::7, 1, :, 5:40] = 0.25          # groups of one value: scale 0
    qkv[1::5, 1, :, 3] = -0.0
    k_new, v_new = qkv[:, 1], qkv[:, 2]
    write_rows(kv, k_new, v_new, i32(slots), keys, meta)
    kv.seq_lens.copy_(i32(c["new"]))
    torch.cuda.synchronize()
    want = [t.clone() for t in before[:2]]
    n = len(where)
    s_idx = torch.tensor(slots[:n], device="cuda")
    rows = PAGE if c["paged"] else N
    for w, x in zip(want, (k_new, v_new)):
        w[s_idx // rows, :, s_idx % rows] = x[:n]
    assert torch.equal(kv.k.view(torch.int16), want[0].view(torch.int16))
    assert torch.equal(kv.v.view(torch.int16), want[1].view(torch.int16))
    table = None if kv.page_table is None else kv.page_table.cpu().numpy()
    K = np16(kv.k)
    codes, scales, zeros, m = np16(keys.codes), np16(keys.scales), np16(keys.zeros), np16(meta)
    for b in range(B):
        L = c["new"][b]
        for h in range(0, Hk if L else 0, max(1, Hk // 2)):
            ks = O.sequence_rows(K, table, b, h, L)
            rc, rs, rz = O.quantize_keys(ks, c["bits"])
            assert (gpu_rows(codes, table, b, h, L) == rc).all(), (b, h)
            assert (gpu_rows(scales, table, b, h, L).view("u2") == rs.view("u2")).all(), (b, h)
            assert (gpu_rows(zeros, table, b, h, L).view("u2") == rz.view("u2")).all(), (b, h)
            assert (gpu_meta(m, table, b, h, L).view("u2") == O.page_meta(ks, L).view("u2")).all()
    # nothing but the written rows and pages moved
    if c["paged"]:
        touched = torch.zeros(kv.k.shape[0], PAGE, dtype=torch.bool, device="cuda")
        touched.view(-1)[s_idx] = True
        still = ~touched[:, None, :].expand(-1, Hk, -1)
        pages_still = ~touched.any(1)
        assert torch.equal(meta[pages_still], before[5][pages_still])
    else:
        still = torch.ones(B, N, dtype=torch.bool, device="cuda")
        still.view(-1)[s_idx] = False
        still = still[:, None, :].expand(-1, Hk, -1)
    for t, old in ((keys.codes, before[2]), (keys.scales, before[3]), (keys.zeros, before[4])):
        assert torch.equal(t[still], old[still])


@pytest.mark.parametrize("bits", [2, 4])
def test_quantised_keys_of_infinities_and_nan(bits):
    """A group of 32 channels that holds an infinity or a NaN has codes of zero
    (and says so by its scale); every other group is as without it.  Rebuilt and
    written by slot alike."""
    from adaptive_top_sparse_quest_b200 import quantize_keys, write_rows
    kv = _cache(1, 2, 3, False, 40, bits)
    inf = float("inf")
    for t, (ch, x) in enumerate([(0, inf), (31, -inf), (40, float("nan")), (64, inf), (65, -inf),
                                 (127, 65504.0)]):
        kv.k[0, :, t, ch] = x
    kv.k[0, 1, 6] = inf
    kv.seq_lens.fill_(40)
    keys = quantize_keys(kv)
    rc, rs, _ = O.quantize_keys(np16(kv.k), bits)
    bad = ~torch.from_numpy(rs).isfinite()
    assert bad.sum() == 2 * 5 + 4
    rc = torch.from_numpy(rc).view(1, 2, 40, 4, -1)
    rc[bad] = 0
    assert torch.equal(keys.codes.cpu().view(rc.shape), rc)
    again = quantize_keys(_cache(1, 2, 3, False, 40, bits))
    rows = kv.k[0].transpose(0, 1).contiguous()
    write_rows(kv, rows, rows, torch.arange(40, device="cuda", dtype=torch.int32), again)
    assert torch.equal(again.codes, keys.codes)
    assert torch.equal(again.scales.view(torch.int16), keys.scales.view(torch.int16))


@pytest.mark.parametrize("bits", [2, 4])
def test_quantised_keys_of_all_ranges_and_ties(bits):
    """Codes, scales and zeros equal the definition's for groups whose ranges run
    from fp16's smallest values to its largest, and for keys half-way between two
    levels."""
    from adaptive_top_sparse_quest_b200 import KVCache, quantize_keys
    N, n = 6000, 2 ** bits - 1
    g = torch.Generator(device="cuda").manual_seed(3 + bits)

    def uni(*s):
        return torch.rand(s, generator=g, device="cuda")

    k = torch.randn(N, 4, 32, generator=g, device="cuda") * torch.exp2(15 - 41 * uni(N, 4, 1))
    step = torch.exp2(torch.floor(-24 + 30 * uni(2000, 4, 1))) * torch.floor(1 + 7 * uni(2000, 4, 1))
    half = torch.floor(uni(2000, 4, 32) * (2 * n + 1))       # halves of a level
    half[..., 0], half[..., 1] = 0, 2 * n
    k[:2000] = half * step / 2 - step * torch.floor(9 * uni(2000, 4, 1))
    k[4000:4100, 1] = k[4000:4100, 1, :1]                    # all alike
    k = k.clamp(-65504, 65504).half().view(1, 1, N, D)
    kv = KVCache(k, None, i32([N]), None, bits)
    keys = quantize_keys(kv)
    rc, rs, rz = O.quantize_keys(np16(k), bits)
    assert (np16(keys.scales).view("u2") == rs.view("u2")).all()
    assert (np16(keys.zeros).view("u2") == rz.view("u2")).all()
    assert (np16(keys.codes) == rc).all()


def test_write_rows_without_keys_or_meta_and_bad_slots():
    from adaptive_top_sparse_quest_b200 import write_rows
    kv = _cache(2, 2, 4, True, 0, 4)
    before = kv.k.clone()
    slots = i32([-1, 2 ** 31 - 1, -2 ** 31, kv.k.shape[0] * PAGE, 18])
    new = torch.randn(5, 2, D, device="cuda").half()
    write_rows(kv, new, new, slots)
    want = before.clone()
    want[1, :, 2] = new[4]
    assert torch.equal(kv.k, want)
    assert torch.equal(kv.v[1, :, 2], new[4])
    write_rows(kv, new[:0], new[:0], slots[:0])      # no tokens


def test_write_rows_refusals():
    from adaptive_top_sparse_quest_b200 import KVCache, write_rows
    kv = _cache(2, 2, 4, True, 0, 4)
    new = torch.zeros(3, 2, D, device="cuda", dtype=torch.float16)
    s = i32([1, 2, 3])
    for bad in (new[:2], new.float(), new[:, :1], new.cpu(), new.transpose(0, 1),
                torch.zeros(3, 2, 2 * D, device="cuda", dtype=torch.float16)[..., ::2],
                torch.zeros(3 * 260, device="cuda", dtype=torch.float16).as_strided(
                    (3, 2, D), (260, D, 1)),
                torch.zeros(1, 2, D, device="cuda", dtype=torch.float16).expand(3, 2, D)):
        with pytest.raises(ValueError):
            write_rows(kv, bad, new, s)
    with pytest.raises((ValueError, TypeError)):
        write_rows(kv, new, new, s.long())
    with pytest.raises(ValueError):
        write_rows(KVCache(kv.k, None, kv.seq_lens, kv.page_table), new, new, s)


# -------------------------------------------------------------------------- prefix attention
PREFIX_CASES = [
    # one sequence, nothing shared, one token / a page and a bit / several tiles
    dict(Hq=1, Hk=1, P=0, lens=[1], paged=True),
    dict(Hq=4, Hk=4, P=0, lens=[17, 0, 128, 129, 300], paged=False),
    dict(Hq=8, Hk=2, P=0, lens=[2500, 1, 700, 16, 15], paged=True),
    # all lengths at the prefix's edges
    dict(Hq=8, Hk=2, P=16, lens=[16, 0, 15, 1, 17, 40], paged=True),
    dict(Hq=8, Hk=1, P=128, lens=[128, 129, 127, 0, 256], paged=False),
    dict(Hq=16, Hk=2, P=144, lens=[0, 160, 144, 145, 300, 5], paged=True),
    # rows of a tile: 128 exactly, just above, 256, above, several tiles
    dict(Hq=8, Hk=1, P=1040, lens=[1040 + 13 * i for i in range(16)], paged=True),
    dict(Hq=8, Hk=1, P=1040, lens=[1040 + 11 * i for i in range(17)], paged=True),
    dict(Hq=16, Hk=2, P=2064, lens=[2064 + (7 * i) % 300 for i in range(32)], paged=True),
    dict(Hq=8, Hk=2, P=528, lens=[528 + (37 * i) % 150 for i in range(70)], paged=False),
    dict(Hq=8, Hk=1, P=400, lens=[400 * (i % 5 > 0) + (53 * i) % 257 for i in range(100)],
         paged=True),
    # many heads, long prefix, one sequence: the split over keys
    dict(Hq=32, Hk=32, P=4096, lens=[4100], paged=True),
    dict(Hq=32, Hk=8, P=16384, lens=[16384, 16500, 9000], paged=True),
    dict(Hq=4, Hk=1, P=20000, lens=[20001] * 66, paged=False),
    # many sequences with short own parts, empty ones among them
    dict(Hq=4, Hk=2, P=64, lens=[(0 if i % 7 == 3 else 64 + i % 50) for i in range(600)],
         paged=True),
]


def _run_prefix(c, seed=11, spread=1.0, **kw):
    from adaptive_top_sparse_quest_b200 import KVCache, PrefixDecodeStep
    q, k, v, table, lens = make_prefix_case(seed, c["Hq"], c["Hk"], c["P"], c["lens"], c["paged"],
                                            spread=spread)
    step = PrefixDecodeStep(KVCache(k, v, lens, table), c["Hq"], c["P"], **kw)
    return step, (q, k, v, table, lens)


def _check_status(step):
    from adaptive_top_sparse_quest_b200 import device_status
    assert device_status(step.ws) == 0


@pytest.mark.parametrize("c", PREFIX_CASES,
                         ids=lambda c: f"h{c['Hq']}_{c['Hk']}P{c['P']}B{len(c['lens'])}")
def test_prefix_decode(c):
    step, (q, k, v, table, lens) = _run_prefix(c)
    out = step(q)
    _check_status(step)
    check_attention(q, k, v, table, lens.tolist(), out, step.lse)
    again = out.clone(), step.lse.clone()
    step(q)
    assert torch.equal(step.out, again[0]) and torch.equal(step.lse, again[1])


@pytest.mark.parametrize("spread", [0.0, 4.0, 30.0])
def test_prefix_decode_score_ranges(spread):
    """Uniform weights, peaked ones, and scores of hundreds that rise late."""
    c = dict(Hq=8, Hk=2, P=1008, lens=[1008 + 70 * i for i in range(9)], paged=True)
    step, (q, k, v, table, lens) = _run_prefix(c, seed=5, spread=spread)
    t = table[0].long()
    k[t[60]] = k[t[60]] * 3         # the largest scores come late in the prefix
    step(q)
    _check_status(step)
    check_attention(q, k, v, table, lens.tolist(), step.out, step.lse)


def test_prefix_decode_no_lse_and_function_form():
    from adaptive_top_sparse_quest_b200 import KVCache, prefix_decode
    c = dict(Hq=8, Hk=2, P=32, lens=[50, 32, 0], paged=True)
    step, (q, k, v, table, lens) = _run_prefix(c, with_lse=False)
    assert step.lse is None
    out, lse = prefix_decode(q, KVCache(k, v, lens, table), 32)
    step(q)
    assert torch.equal(out, step.out)
    check_attention(q, k, v, table, lens.tolist(), out, lse)


def test_prefix_decode_capture_two_graphs_one_workspace_other_lengths():
    """Two graphs that share a step's buffers, replayed in turn on one stream,
    with lengths that change between replays."""
    c = dict(Hq=8, Hk=2, P=256, lens=[304, 512, 704, 100], paged=True)
    step, (q, k, v, table, lens) = _run_prefix(c)
    step(q)
    q2 = q.flip(0).contiguous()
    graphs = []
    for x in (q, q2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(x)
        graphs.append(g)
    for new in ([304, 512, 704, 100], [1, 290, 512, 0], [0, 0, 0, 0], [300, 256, 700, 1]):
        lens.copy_(i32(new))
        for g, x in zip(graphs, (q, q2)):
            g.replay()
            _check_status(step)
            check_attention(x, k, v, table, new, step.out, step.lse)


def test_prefix_decode_two_streams():
    """Two steps at once on two streams, neither the current one."""
    c = dict(Hq=32, Hk=8, P=2048, lens=[2100 + 3 * i for i in range(8)], paged=True)
    runs = [_run_prefix(c, seed=s) for s in (1, 2)]
    streams = [torch.cuda.Stream() for _ in runs]
    torch.cuda.synchronize()
    for _ in range(20):
        for (step, data), st in zip(runs, streams):
            step(data[0], stream=st)
    torch.cuda.synchronize()
    for step, (q, k, v, table, lens) in runs:
        _check_status(step)
        check_attention(q, k, v, table, lens.tolist(), step.out, step.lse)


def test_prefix_decode_refusals():
    from adaptive_top_sparse_quest_b200 import KVCache, PrefixDecodeStep, TwError
    q, k, v, table, lens = make_prefix_case(3, 8, 2, 32, [40, 33], True)
    kv = KVCache(k, v, lens, table)
    for bad in (-16, 8, 17, 64 + kv.N):
        with pytest.raises(ValueError):
            PrefixDecodeStep(kv, 8, bad)
    with pytest.raises(TwError):
        PrefixDecodeStep(kv, 6, 32)
    with pytest.raises(ValueError):
        PrefixDecodeStep(KVCache(k, None, lens, table), 8, 32)
    with pytest.raises(ValueError):
        PrefixDecodeStep(KVCache(k, v, lens[:1].contiguous(), table), 8, 32)
    step = PrefixDecodeStep(kv, 8, 32)
    for bad in (q[:1], q[:, :4].contiguous(), q.cpu(), q[..., :64]):
        with pytest.raises(ValueError):
            step(bad)
    with pytest.raises(TypeError):
        step(q.float())


@pytest.mark.parametrize("seed", range(12))
def test_prefix_decode_random_shapes(seed):
    """Shapes drawn over the whole range: heads, batch, prefix, ragged own parts."""
    rng = random.Random(100 + seed)
    G, Hk = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 8])
    B = rng.choice([1, 2, 7, 16, 33, 65, 130])
    P = 16 * rng.choice([0, 1, 7, 8, 9, 40, 130])
    top = rng.choice([1, 20, 130, 600])
    lens = [rng.choice([P + rng.randint(0, top), P + rng.randint(0, top), rng.randint(0, P)])
            for _ in range(B)]
    c = dict(Hq=G * Hk, Hk=Hk, P=P, lens=lens, paged=rng.random() < 0.6)
    step, (q, k, v, table, lens) = _run_prefix(c, seed=seed)
    step(q)
    _check_status(step)
    check_attention(q, k, v, table, lens.tolist(), step.out, step.lse)


def test_prefix_decode_many_row_tiles():
    """2048 query rows per KV head: eight row tiles of 256."""
    c = dict(Hq=64, Hk=8, P=528, lens=[528 + (i * 7) % 40 for i in range(256)], paged=True)
    step, (q, k, v, table, lens) = _run_prefix(c)
    step(q)
    _check_status(step)
    check_attention(q, k, v, table, lens.tolist(), step.out, step.lse)


def test_prefix_decode_back_to_back_with_changing_inputs():
    """Calls without a wait between them, queries and lengths written by kernels
    of the same stream just before each: every call sees its own inputs."""
    c = dict(Hq=8, Hk=2, P=128, lens=[704, 512, 304, 128, 256, 640], paged=True)
    step, (q, k, v, table, lens) = _run_prefix(c)
    g = torch.Generator(device="cuda").manual_seed(9)
    qs = torch.randn(40, *q.shape, generator=g, device="cuda", dtype=torch.float16)
    full = torch.tensor(c["lens"], device="cuda")
    all_lens = (full * torch.rand(40, len(full), generator=g, device="cuda")).to(torch.int32)
    x, a = torch.empty_like(q), torch.randn(512, 512, device="cuda", dtype=torch.float16)
    outs, lses = [], []
    for i in range(40):
        if i % 3 == 1:
            a = a @ a * 1e-2              # a library product between two calls
        x.copy_(qs[i])
        lens.copy_(all_lens[i])
        step(x)
        outs.append(step.out.clone())
        lses.append(step.lse.clone())
    torch.cuda.synchronize()
    _check_status(step)
    # rows past a shorter length hold other rows, not NaN: the reference takes the length
    for i in range(0, 40, 3):
        check_attention(qs[i], k, v, table, all_lens[i].tolist(), outs[i], lses[i])


@pytest.mark.parametrize("B", [2, 3, 40])
@pytest.mark.parametrize("paged", [False, True])
def test_prefix_decode_non_finite_rows(B, paged):
    """A NaN in a key that a row sees makes that row NaN; a key whose score is
    minus infinity does not count, plus infinity is NaN; rows of V past the end
    of a sequence inside the prefix do not reach it, whatever they hold.  On
    two of four KV heads; the others are as without it."""
    Hq, Hk, P, G = 16, 4, 400, 4
    lens = [(500, 90, 300, 420, 0, 399)[i % 6] + i // 6 for i in range(B)]
    c = dict(Hq=Hq, Hk=Hk, P=P, lens=lens, paged=paged)
    step, (q, k, v, table, dl) = _run_prefix(c)
    q[..., 7] = torch.where(q[..., 7] < 0, -1.0, 1.0)
    def row(x, b, t):     # [Hk][128] of token t
        return x[table[b, t // PAGE].long(), :, t % PAGE] if paged else x[b, :, t]
    nan, inf = float("nan"), float("inf")
    row(v, 0, 310)[0, 5:9] = inf       # head 0: values in the prefix that shorter ones do not see
    row(v, 0, 399)[0, 100] = nan
    row(k, 0, 350)[1, 3] = nan         # head 1: a key of the prefix, and one of sequence 0's own
    row(k, 0, 450)[1, 9] = nan
    for t in range(128, 256):          # head 2: a whole tile of infinite scores
        row(k, 0, t)[2, 7] = inf
    if not paged:                      # the prefix is the same rows for all
        k[:, :, :P], v[:, :, :P] = k[:1, :, :P].clone(), v[:1, :, :P].clone()
    step(q)
    _check_status(step)
    out, lse = step.out.view(B, Hk, G, D), step.lse.view(B, Hk, G)
    sees = torch.tensor(lens, device="cuda")
    bad = torch.zeros(B, Hk, G, dtype=torch.bool, device="cuda")
    bad[:, 1] = (sees > 350)[:, None]
    up = q.view(B, Hk, G, D)[:, 2, :, 7] > 0
    bad[:, 2] = up & (sees > 128)[:, None]
    assert bool(out[bad].isnan().all()) and bool(lse[bad].isnan().all())
    for b in range(B):
        n = lens[b]
        z0 = out[b, 0]
        if n > 310:
            assert not bool(z0[:, 5:9].isfinite().any())
        if n > 399:
            assert bool(z0[:, 100].isnan().all())
        seen = [x for t, x in ((310, [5, 6, 7, 8]), (399, [100])) if n > t for x in x]
        rest = [x for x in range(D) if x not in seen]
        assert bool(z0[:, rest].isfinite().all()), (b, n)
    # the other rows against the reference, head 2's without the tile that does not count
    for b in range(B):
        n = lens[b]
        for h in range(Hk):
            kb, vb = k[:, h:h + 1], v[:, h:h + 1]
            tb = table[b:b + 1] if paged else None
            if not paged:
                kb, vb = kb[b:b + 1], vb[b:b + 1]
            if h == 0 and n > 310:
                continue
            if h == 2 and n >= 256:
                n -= 128
                if paged:
                    tb = torch.cat([tb[:, :8], tb[:, 16:]], 1)
                else:
                    kb, vb = (torch.cat([x[:, :, :128], x[:, :, 256:]], 2) for x in (kb, vb))
            good = ~bad[b, h]
            if bool(good.any()):
                check_attention(q.view(B, Hk, G, D)[b:b + 1, h][:, good], kb, vb, tb, [n],
                                out[b:b + 1, h][:, good], lse[b:b + 1, h][:, good])
            n = lens[b]


def test_prefix_decode_hostile_table_and_lengths():
    """Lengths outside [0, N] are clamped; page ids outside the pool read some
    page of it, which spoils that sequence and no other."""
    from adaptive_top_sparse_quest_b200 import KVCache, PrefixDecodeStep
    q, k, v, table, lens = make_prefix_case(6, 8, 2, 32, [100, 90, 112, 64], True)
    k.nan_to_num_()
    v.nan_to_num_()
    table[1, 3] = -7
    table[1, 5] = 2 ** 31 - 1
    bad = i32([100, 90, 2 ** 31 - 1, -5])
    step = PrefixDecodeStep(KVCache(k, v, bad, table), 8, 32)
    step(q)
    _check_status(step)
    N = table.shape[1] * PAGE
    assert bool(torch.isfinite(step.out).all())
    good = [0, 2, 3]
    check_attention(q[good], k, v, table[good], [100, N, 0], step.out[good], step.lse[good])


def test_long_pool_offsets():
    """Rows past 2^31 elements of the pool: written by slot, quantised, attended to."""
    from adaptive_top_sparse_quest_b200 import KVCache, PrefixDecodeStep, write_rows
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("needs 30 GB")
    Hk, pool, W = 32, 40000, 6
    k = torch.empty(pool, Hk, PAGE, D, dtype=torch.float16, device="cuda")
    v = torch.empty_like(k)
    table = i32([[pool - 1 - j for j in range(W)], [pool - 50 - 3 * j for j in range(W)]])
    lens = i32([90, 77])
    kv = KVCache(k, v, lens, table)
    slots = i32([int(table[b, t // PAGE]) * PAGE + t % PAGE
                 for b, n in enumerate((90, 77)) for t in range(n)])
    g = torch.Generator(device="cuda").manual_seed(2)
    new = torch.randn(2, 167, Hk, D, generator=g, device="cuda", dtype=torch.float16)
    meta = torch.empty(kv.meta_shape(), dtype=torch.float16, device="cuda")
    write_rows(kv, new[0], new[1], slots, None, meta)
    s = slots.long()
    assert torch.equal(k[s // PAGE, :, s % PAGE], new[0])
    assert torch.equal(v[s // PAGE, :, s % PAGE], new[1])
    want = k[pool - 1].amin(1), k[pool - 1].amax(1)
    assert torch.equal(meta[pool - 1, :, 0], want[0]) and torch.equal(meta[pool - 1, :, 1], want[1])
    q = torch.randn(2, Hk, D, generator=g, device="cuda", dtype=torch.float16)
    step = PrefixDecodeStep(kv, Hk, 0)
    step(q)
    _check_status(step)
    check_attention(q, k, v, table, [90, 77], step.out, step.lse)


def test_write_rows_captured_and_slot_listed_twice():
    """A captured write replayed with other rows and slots; of a slot that is listed
    twice the contents are unspecified (two warps store the row, 16 bytes a lane, in
    any order: each value is one of the two tokens'), and nothing else changes."""
    from adaptive_top_sparse_quest_b200 import write_rows
    kv = _cache(2, 2, 4, True, 0, 4)
    new = torch.randn(4, 2, D, device="cuda").half()
    slots = i32([-1, -1, -1, -1])
    write_rows(kv, new, new, slots)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        write_rows(kv, new, new, slots)
    want = kv.k.clone()
    for s in ([17, 18, 40, -1], [33, 3, 4, 5], [-1, 20, 20, -1]):
        new.copy_(torch.randn(4, 2, D, device="cuda"))
        slots.copy_(i32(s))
        g.replay()
        for i, x in enumerate(s):
            if x >= 0:
                want[x // PAGE, :, x % PAGE] = new[i]
        if s[1] == s[2]:
            got = kv.k[1, :, 4]
            assert bool(((got == new[1]) | (got == new[2])).all())
            want[1, :, 4] = got
        assert torch.equal(kv.k, want)


def test_serving_calls_on_a_side_stream():
    from adaptive_top_sparse_quest_b200 import prefix_decode, update_page_table, write_rows
    old, new, table, free, nf, ns = _pages_case(31, 20, 10, 0, 60, 0.5)
    st = torch.cuda.Stream()
    table_t, free_t, o, n, f = i32(table), i32(free), i32(old), i32(new), i32([nf])
    kv = _cache(2, 2, 4, True, 0, 4)
    rows = torch.randn(3, 2, D, device="cuda").half()
    slots = i32([20, 21, 22])
    q, k, v, tb, lens = make_prefix_case(8, 8, 2, 32, [50, 32, 0], True)
    torch.cuda.synchronize()
    u = update_page_table(o, n, table_t, free_t, f, num_slots=ns, stream=st)
    write_rows(kv, rows, rows, slots, stream=st)
    from adaptive_top_sparse_quest_b200 import KVCache
    out, lse = prefix_decode(q, KVCache(k, v, lens, tb), 32, stream=st)
    st.synchronize()
    want = model_page_table(old, new, table, free, nf, ns, 0)
    assert u.seq_lens_out.tolist() == want[0] and u.slots.tolist() == want[2]
    assert torch.equal(kv.k[1, :, 4:7], rows.transpose(0, 1))
    check_attention(q, k, v, tb, lens.tolist(), out, lse)


# ------------------------------------------------------------------------------- all together
def test_serving_loop():
    """Requests come, grow, are refused and finish behind a shared prefix: table
    and slots from the lengths, rows written by slot, dense attention, and the
    pruned step on the same cache with p = 1, which keeps every token."""
    from adaptive_top_sparse_quest_b200 import (DecodeStep, KVCache, PageTableUpdate,
                                                PrefixDecodeStep, page_meta, quantize_keys,
                                                write_rows)
    rng = random.Random(8)
    B, Hq, Hk, W, P = 6, 8, 2, 24, 64
    keep = P // PAGE
    pool = keep + 9
    g = torch.Generator(device="cuda").manual_seed(4)

    def rnd(*s):
        return torch.randn(s, generator=g, device="cuda", dtype=torch.float16)

    k, v = torch.zeros(pool, Hk, PAGE, D, dtype=torch.float16, device="cuda"), rnd(pool, Hk, PAGE, D)
    k[:keep] = rnd(keep, Hk, PAGE, D)
    table = i32([list(range(keep)) + [0] * (W - keep) for _ in range(B)])
    lens = i32([P] * B)
    free, nf, new = i32(list(range(keep, pool)) + [0] * keep), i32([pool - keep]), i32([P] * B)
    kv = KVCache(k, v, lens, table)
    keys, meta = quantize_keys(kv), page_meta(kv)
    T = 200
    update = PageTableUpdate(lens, table, free, T, P, in_place=True)
    dense = PrefixDecodeStep(kv, Hq, P)
    pruned = DecodeStep(kv, keys, meta, Hq, None, 1.0, 1)
    model = dict(lens=[P] * B, table=table.tolist(), free=free.tolist(), nf=pool - keep)
    refused = 0
    for step in range(14):
        want = [rng.choice([n + 1, n + 1, n + rng.randint(0, 60), P, max(P, n - 3)])
                for n in model["lens"]]
        new.copy_(i32(want))
        update(new, nf)
        ml, mnf, mslots, _ = model_page_table(model["lens"], want, model["table"], model["free"],
                                              model["nf"], T, P)
        refused += ml != want
        model.update(lens=ml, nf=mnf)
        assert lens.tolist() == ml and int(nf) == mnf and update.slots.tolist() == mslots
        kn, vn = rnd(T, Hk, D), rnd(T, Hk, D)
        write_rows(kv, kn, vn, update.slots, keys, meta)
        q = rnd(B, Hq, D)
        dense(q)
        _check_status(dense)
        check_attention(q, k, v, table, ml, dense.out, dense.lse)
        pruned(q)
        torch.cuda.synchronize()
        # both are the same attention; each within the fp16 result's rounding
        # and the bounds that check_attention derives
        assert float((pruned.out.float() - dense.out.float()).abs().max()) < 4e-3
        K, tb = np16(k), table.cpu().numpy()
        for b in range(B):
            for h in range(Hk):
                ks = O.sequence_rows(K, tb, b, h, ml[b])
                rc, rs, rz = O.quantize_keys(ks, 4)
                assert (gpu_rows(np16(keys.codes), tb, b, h, ml[b]) == rc).all()
                m = gpu_meta(np16(meta), tb, b, h, ml[b])
                # a page cut short by a shrink keeps its wider bounds; pages that
                # were only ever grown are exact
                full = O.page_meta(ks, ml[b])
                assert (m[:, 0] <= full[:, 0]).all() and (m[:, 1] >= full[:, 1]).all()
    assert refused > 0
