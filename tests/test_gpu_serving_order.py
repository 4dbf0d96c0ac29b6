"""The serving operators' handles on streams other than the one they were made
on: what that stream still holds when a handle is made (its buffers' fills, and
work on memory that the buffers were given) comes before the calls."""
import pytest
import torch

from _serving import PAGE, check_attention, make_prefix_case, model_page_table

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from adaptive_top_sparse_quest_b200 import _capi, build
    build.build()
    _capi.load()
    # kernels are loaded at their first use, which may wait for the device: here
    _backlog(1024)
    x = torch.zeros(64, dtype=torch.float16, device="cuda")
    for t in (x, x.float(), x.int()):
        t.clone()
    torch.cuda.synchronize()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _backlog(words):
    """Some 50 ms of work on the current stream, then a fill of memory that is
    free for the next allocation of `words` 32-bit words."""
    torch.cuda._sleep(100_000_000)
    t = torch.full((words,), 0x5A5A5A5A, dtype=torch.int32, device="cuda")
    del t


@pytest.mark.parametrize("passed", [True, False])
def test_prefix_decode_made_on_a_busy_stream(passed):
    """`passed`: the other stream is given to the call; else it is current."""
    from adaptive_top_sparse_quest_b200 import KVCache, PrefixDecodeStep, device_status
    q, k, v, table, lens = make_prefix_case(12, 8, 2, 32, [50, 32, 0, 300], True)
    kv = KVCache(k, v, lens, table)
    PrefixDecodeStep(kv, 8, 32)(q)      # the library is loaded, the memory cached
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    _backlog(4 * 8 * 64)                # as large as out
    step = PrefixDecodeStep(kv, 8, 32)
    if passed:
        step(q, stream=side)
    else:
        with torch.cuda.stream(side):
            step(q)
    with torch.cuda.stream(side):
        first = step.out.clone(), step.lse.clone()
    torch.cuda.synchronize()
    check_attention(q, k, v, table, lens.tolist(), *first)
    assert device_status(step.ws) == 0
    assert torch.equal(step.out, first[0]) and torch.equal(step.lse, first[1])


@pytest.mark.parametrize("in_place", [False, True])
def test_page_table_made_on_a_busy_stream(in_place):
    from adaptive_top_sparse_quest_b200 import PageTableUpdate
    old, new = [0, 20, 33, 5], [40, 21, 0, 5]
    table = [[-1] * 4, [3, 4, -1, -1], [5, 6, 7, -1], [8, -1, -1, -1]]
    free = [0, 1, 2] + [9] * 9
    lens_t, new_t, table_t, free_t, nf_t = i32(old), i32(new), i32(table), i32(free), i32([3])
    args = (lens_t.clone(), table_t.clone(), free_t.clone(), 50)
    PageTableUpdate(*args)(new_t, nf_t.clone())
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    _backlog(50)                        # as large as slots
    u = PageTableUpdate(lens_t, table_t, free_t, 50, in_place=in_place)
    u(new_t, nf_t, stream=side)
    with torch.cuda.stream(side):
        slots, offsets = u.slots.clone(), u.offsets.clone()
    torch.cuda.synchronize()
    want = model_page_table(old, new, table, free, 3, 50, 0)
    for s, o in ((slots, offsets), (u.slots, u.offsets)):
        assert s.tolist() == want[2] and o.tolist() == want[3]
    assert u.seq_lens_out.tolist() == want[0] and int(u.num_free_out) == want[1]
    assert table_t.tolist() == table and free_t.tolist() == free


def test_handles_made_before_or_inside_a_capture():
    """A step made outside is captured on the graph's own stream; one made inside
    belongs to the graph."""
    from adaptive_top_sparse_quest_b200 import (KVCache, PageTableUpdate, PrefixDecodeStep,
                                                prefix_decode)
    q, k, v, table, lens = make_prefix_case(13, 8, 2, 32, [70, 33, 100], True)
    kv = KVCache(k, v, lens, table)
    step = PrefixDecodeStep(kv, 8, 32)
    old, new, nf = i32([0, 3]), i32([17, 4]), i32([5])
    pt, free = i32([[-1] * 2, [6, -1]]), i32([0, 1, 2, 3, 4, 0, 0])
    u = PageTableUpdate(old, pt, free, 20)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(q)
        out, lse = prefix_decode(q, kv, 32)
        u(new, nf)
    g.replay()
    torch.cuda.synchronize()
    check_attention(q, k, v, table, lens.tolist(), step.out, step.lse)
    assert torch.equal(out, step.out) and torch.equal(lse, step.lse)
    want = model_page_table([0, 3], [17, 4], [[-1] * 2, [6, -1]], [0, 1, 2, 3, 4, 0, 0], 5, 20, 0)
    assert u.slots.tolist() == want[2] and u.seq_lens_out.tolist() == want[0]
    assert PAGE * (pt.shape[1]) >= max(want[0])


def test_prefix_decode_after_the_cache_changed_its_tensors():
    """A step reads the tensors that its cache names at the call: lengths that an
    update returned in a tensor of its own, a wider table, a pool that moved.
    Tensors that do not fit the step are refused."""
    from adaptive_top_sparse_quest_b200 import KVCache, PrefixDecodeStep, device_status
    q, k, v, table, lens = make_prefix_case(14, 8, 2, 32, [200, 140, 90], True)
    kv = KVCache(k, v, lens, table)
    step = PrefixDecodeStep(kv, 8, 32)
    step(q)
    check_attention(q, k, v, table, [200, 140, 90], step.out, step.lse)
    kv.seq_lens = i32([33, 0, 88])
    step(q)
    check_attention(q, k, v, table, [33, 0, 88], step.out, step.lse)
    kv.page_table = torch.cat([table, table.new_full((3, 3), -1)], 1)
    kv.k, kv.v = (torch.cat([x[:1], x]) for x in (k, v))
    kv.page_table = kv.page_table + 1
    kv.seq_lens = i32([199, 1, 60])
    step(q)
    check_attention(q, kv.k, kv.v, kv.page_table, [199, 1, 60], step.out, step.lse)
    assert device_status(step.ws) == 0
    good = kv.k, kv.v, kv.seq_lens, kv.page_table
    for change in (dict(seq_lens=lens[:2].contiguous()), dict(v=None), dict(v=kv.v[1:]),
                   dict(page_table=table[:2].contiguous()), dict(seq_lens=lens.cpu()),
                   dict(page_table=table[:, :1].contiguous()), dict(k=kv.k[:, :1].contiguous())):
        kv.k, kv.v, kv.seq_lens, kv.page_table = good
        for name, t in change.items():
            setattr(kv, name, t)
        with pytest.raises(ValueError):
            step(q)
    kv.k, kv.v, kv.seq_lens, kv.page_table = good
    step(q)
    check_attention(q, kv.k, kv.v, kv.page_table, [199, 1, 60], step.out, step.lse)


def test_write_rows_after_the_cache_changed_its_tensors():
    """A call writes to the tensors that the cache names then, and refuses those
    that do not go together."""
    from adaptive_top_sparse_quest_b200 import KVCache, write_rows
    k = torch.zeros(6, 2, PAGE, 128, dtype=torch.float16, device="cuda")
    kv = KVCache(k, k.clone(), i32([0]), i32([[1, 2]]))
    new, slots = torch.randn(2, 2, 128, device="cuda").half(), i32([18, 100])
    for bad in (k[:3], k.float(), k[..., :64], k.transpose(0, 1), None):
        kv.v = bad
        with pytest.raises((ValueError, TypeError)):
            write_rows(kv, new, new, slots)
    kv.k, kv.v = torch.zeros_like(k), torch.zeros_like(k)
    write_rows(kv, new, new, slots)
    want = torch.zeros_like(k)
    want[1, :, 2] = new[0]              # slot 100 lies outside this pool of 96
    assert torch.equal(kv.k, want) and torch.equal(kv.v, want)
    kv.k, kv.v = torch.zeros_like(k).repeat(2, 1, 1, 1), torch.zeros_like(k).repeat(2, 1, 1, 1)
    write_rows(kv, new, new, slots)
    assert torch.equal(kv.k[1, :, 2], new[0]) and torch.equal(kv.v[6, :, 4], new[1])
    assert not bool(k.any())


def test_page_table_sums_past_32_bits():
    """Lengths far above the real ones in the largest table: what is given back and
    the stack's height together pass 2^31, and the stack takes what it has room for."""
    from adaptive_top_sparse_quest_b200 import update_page_table
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GB")
    B, W, pool, height = 8192, 262143, 400000, 300000
    table = torch.full((B, W), -1, dtype=torch.int32, device="cuda")
    table[0] = torch.arange(W, dtype=torch.int32, device="cuda")
    free = torch.arange(pool, dtype=torch.int32, device="cuda").flip(0).contiguous()
    before = free.clone()
    old, new = i32([2 ** 31 - 1] * (B - 1) + [0]), i32([0] * (B - 1) + [20])
    u = update_page_table(old, new, table, free, i32([height]), num_slots=24)
    n = pool - height
    assert int(u.num_free_out) == pool - 2
    assert torch.equal(free[:height], before[:height])
    assert torch.equal(free[height:], table[0, :n])
    assert table[-1, :3].tolist() == [n - 1, n - 2, -1]
    slots = [(n - 1 - t // PAGE) * PAGE + t % PAGE for t in range(20)]
    assert u.slots.tolist() == slots + [-1] * 4
    assert u.seq_lens_out.tolist() == new.tolist() and u.offsets.tolist() == [0] * B + [20]
