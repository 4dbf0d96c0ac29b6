"""Host checks of the serving operators: every refusal happens before a launch
(these calls run without a GPU), and the list model of the page-table update
keeps its own invariants."""
import ctypes
import random

import pytest

from _serving import PAGE, model_page_table
from adaptive_top_sparse_quest_b200 import _capi, build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _capi.load()


def _kv(**kw):
    s = _capi.TwKv()
    s.k, s.v = 4096, 8192
    s.batch, s.num_kv_heads, s.max_seq_len = 1, 2, 64
    s.page_size, s.head_dim = 16, 128
    for k, v in kw.items():
        setattr(s, k, v)
    return s


P = 1 << 20
INV, UNS, CAP = _capi.TW_ERR_INVALID_ARG, _capi.TW_ERR_UNSUPPORTED, _capi.TW_ERR_CAPACITY

PT = dict(B=2, lens=P, new=P, table=P, W=4, prefix=0, free=P, pool=9, nf=P, nfo=P, out=P, slots=P,
          ns=8, offs=P)


@pytest.mark.parametrize("change,want", [
    (dict(B=-1), INV), (dict(lens=None), INV), (dict(new=None), INV), (dict(table=None), INV),
    (dict(W=0), INV), (dict(prefix=8), INV), (dict(prefix=-16), INV), (dict(prefix=80), INV),
    (dict(free=None), INV), (dict(pool=0), INV), (dict(nf=None), INV), (dict(nfo=None), INV),
    (dict(out=P + 2), INV), (dict(slots=P + 1), INV), (dict(slots=None), INV), (dict(ns=-1), INV),
    (dict(offs=None), INV), (dict(B=8193), UNS), (dict(W=2 ** 28), UNS),
    (dict(pool=2 ** 27), UNS), (dict(B=8192, W=2 ** 18), UNS),
])
def test_page_table_refusals(lib, change, want):
    a = dict(PT, **change)
    r = lib.tw_update_page_table(a["B"], a["lens"], a["new"], a["table"], a["W"], a["prefix"],
                                 a["free"], a["pool"], a["nf"], a["nfo"], a["out"], a["slots"],
                                 a["ns"], a["offs"], None)
    assert r == want


WR = dict(kv={}, k=P, ks=256, v=P, vs=256, slots=P, T=3, codes=P, scales=P, zeros=P, meta=P)


@pytest.mark.parametrize("change,want", [
    (dict(k=None), INV), (dict(v=None), INV), (dict(k=P + 8), INV), (dict(ks=248), INV),
    (dict(vs=260), INV), (dict(slots=None), INV), (dict(slots=P + 2), INV), (dict(T=-1), INV),
    (dict(codes=None), INV), (dict(zeros=None), INV), (dict(meta=P + 4), INV),
    (dict(kv=dict(v=None)), INV), (dict(kv=dict(head_dim=64)), UNS),
    (dict(kv=dict(key_bits=3)), UNS),
    (dict(kv=dict(page_table=P, max_pages_per_seq=4, num_pool_pages=2 ** 27, num_kv_heads=1),
          ks=256), UNS),
    (dict(T=2 ** 30), UNS), (dict(T=0), _capi.TW_OK), (dict(kv=dict(batch=0)), _capi.TW_OK),
])
def test_write_rows_refusals(lib, change, want):
    a = dict(WR, **change)
    r = lib.tw_write_rows(ctypes.byref(_kv(**a["kv"])), a["k"], a["ks"], a["v"], a["vs"],
                          a["slots"], a["T"], a["codes"], a["scales"], a["zeros"], a["meta"],
                          None)
    assert r == want


PD = dict(kv={}, q=P, Hq=4, prefix=16, out=P, lse=P, ws=P, n=1 << 40)


@pytest.mark.parametrize("change,want", [
    (dict(q=None), INV), (dict(q=P + 8), INV), (dict(out=None), INV), (dict(lse=P + 2), INV),
    (dict(Hq=3), INV), (dict(Hq=32), UNS), (dict(prefix=8), INV), (dict(prefix=-16), INV),
    (dict(prefix=80), INV), (dict(ws=None), INV), (dict(ws=P + 16), INV), (dict(n=255), CAP),
    (dict(kv=dict(v=None)), INV), (dict(kv=dict(page_size=32)), UNS),
    (dict(kv=dict(max_seq_len=2 ** 30)), UNS),
    (dict(kv=dict(batch=0)), _capi.TW_OK),
])
def test_prefix_decode_refusals(lib, change, want):
    a = dict(PD, **change)
    r = lib.tw_prefix_decode(a["q"], a["Hq"], ctypes.byref(_kv(**a["kv"])), a["prefix"], a["out"],
                             a["lse"], a["ws"], a["n"], None)
    assert r == want


def test_prefix_workspace_size(lib):
    n = ctypes.c_size_t(0)
    for B, Hq, Hk, prefix in [(1, 4, 4, 0), (64, 32, 8, 32768), (0, 8, 1, 16), (4096, 64, 8, 16)]:
        assert lib.tw_prefix_workspace_size(B, Hq, Hk, prefix, ctypes.byref(n)) == _capi.TW_OK
        assert n.value >= 256 and n.value % 256 == 0
    for B, Hq, Hk, prefix, want in [(-1, 4, 4, 0, INV), (1, 3, 2, 0, INV), (1, 6, 2, 0, UNS),
                                    (1, 4, 2, 8, INV), (1, 4, 0, 0, INV)]:
        assert lib.tw_prefix_workspace_size(B, Hq, Hk, prefix, ctypes.byref(n)) == want
    assert lib.tw_prefix_workspace_size(1, 4, 2, 0, None) == INV


def test_page_table_model_keeps_every_page_once():
    """Random steps: pages are on the stack or in exactly one row, lengths and
    tables agree, nothing below the prefix moves."""
    rng = random.Random(5)
    for trial in range(40):
        B, W, keep = rng.randint(1, 9), rng.randint(2, 9), rng.randint(0, 1)
        pool = keep + rng.randint(1, B * (W - keep))
        table = [list(range(keep)) + [-1] * (W - keep) for _ in range(B)]
        free = [p for p in range(keep, pool)] + [0] * keep
        nf, lens = pool - keep, [0] * B
        for _ in range(12):
            new = [rng.choice([n, n + 1, n + rng.randint(0, 40), 0, n // 2, W * PAGE + 1])
                   for n in lens]
            before = list(lens)
            lens, nf, slots, offs = model_page_table(lens, new, table, free, nf, 500, PAGE * keep)
            held = [table[b][j] for b in range(B) for j in range(keep, max(keep, -(-lens[b] // PAGE)))]
            assert sorted(held + free[:nf]) == list(range(keep, pool))
            for b in range(B):
                assert table[b][:keep] == list(range(keep))
                assert lens[b] in (before[b], new[b])
            used = [s for s in slots if s >= 0]
            assert len(set(used)) == len(used)
