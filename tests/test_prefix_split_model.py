"""CPU model of how the shared-prefix attention shares its key tiles out
(csrc/prefix_decode.cu): the line of costs, the ranges of CTAs and streams, the
walk over them, and the join's search for a row's records, checked by brute
force: every tile is taken exactly once, every record has a place of its own
inside the workspace, and the join finds them all."""
import random
import re
import os

import numpy as np
import pytest

SRC = os.path.join(os.path.dirname(__file__), "..", "adaptive_top_sparse_quest_b200", "csrc")
CTAS = 148


def _constants():
    text = open(os.path.join(SRC, "prefix_decode.cu")).read()
    own = re.search(r"kOwnCost = (\d+), kOwnStart = (\d+), kUnitStart = (\d+)", text)
    tile = re.search(r"return a\.pair \? (\d+) : (\d+);", text)
    return [int(x) for x in own.groups()] + [int(x) for x in tile.groups()]


OWN, OWN_START, UNIT_START, PAIR_TILE, TILE = _constants()


def own_cost(nonempty, tiles):
    return nonempty * OWN_START + tiles * OWN


def shares(Hk, RT, KT, pair, kts):
    """Ranges of every CTA and where each stream's own tiles begin."""
    cost = PAIR_TILE if pair else TILE
    span = KT * cost + UNIT_START
    X1 = Hk * RT * span if KT else 0
    ne, cum = [0], [0]
    for kt in kts:
        ne.append(ne[-1] + (kt > 0))
        cum.append(cum[-1] + kt)
    X = X1 + own_cost(ne[-1], cum[-1]) * Hk

    def prefix_tile_at(x):
        if x <= 0:
            return 0
        u = x // span
        rest = x - u * span - UNIT_START
        return u * KT + (0 if rest <= 0 else -(-rest // cost))

    out = []
    for c in range(CTAS):
        x0, x1 = X * c // CTAS, X * (c + 1) // CTAS
        xm = (max(x0, X1) + max(x1, X1)) // 2 if pair else (x0 + x1) // 2
        r = dict(p0=prefix_tile_at(min(x0, X1)), p1=prefix_tile_at(min(x1, X1)))
        r["pm"] = r["p1"] if pair else prefix_tile_at(min(xm, X1))
        tiles, at = [cum[-1] * Hk] * 3, [None, None]
        for k, x in enumerate((x0, xm, x1)):
            pos = max(x, X1) - X1
            for b, kt in enumerate(kts):
                lo, unit = own_cost(ne[b], cum[b]) * Hk, own_cost(kt > 0, kt)
                if lo <= pos < lo + unit * Hk:
                    h, rest = divmod(pos - lo, unit)
                    rest -= OWN_START
                    t = 0 if rest <= 0 else -(-rest // OWN)
                    tiles[k] = cum[b] * Hk + h * kt + t
                    if t == kt:
                        h, t = h + 1, 0
                    if k < 2:
                        at[k] = (b + 1, 0, t) if h == Hk else (b, h, t)
        r.update(s0=tiles[0], sm=tiles[1], s1=tiles[2], at=at)
        out.append(r)
    return out, X1, X, span, ne, cum


def check(Hk, RT, KT, pair, kts):
    B = len(kts)
    rs, X1, X, span, ne, cum = shares(Hk, RT, KT, pair, kts)
    assert rs[0]["p0"] == 0 and rs[-1]["p1"] == Hk * RT * KT
    assert rs[0]["s0"] == 0 and rs[-1]["s1"] == cum[-1] * Hk
    own_seen, records = set(), set()
    for c, r in enumerate(rs):
        assert r["p0"] <= r["pm"] <= r["p1"] and r["s0"] <= r["sm"] <= r["s1"]
        if c:
            assert rs[c - 1]["p1"] == r["p0"] and rs[c - 1]["s1"] == r["s0"]
        for i in range(2):
            p = r["p0"] if pair or i == 0 else r["pm"]
            pe = r["p1"] if pair or i == 1 else r["pm"]
            while p < pe:
                u = p // KT
                p += min(pe - p, KT - (p - u * KT))
                slot = c + u if pair else 2 * c + i + u
                assert 0 <= slot < (CTAS + Hk * RT if pair else 2 * CTAS + Hk)
                assert (0, slot, pair and i) not in records
                records.add((0, slot, pair and i))
            s, se = (r["s0"], r["sm"]) if i == 0 else (r["sm"], r["s1"])
            if s >= se:
                continue
            b, h, t = r["at"][i]
            while s < se:
                while b < B - 1 and kts[b] == 0:
                    b += 1
                assert kts[b] > t and cum[b] * Hk + h * kts[b] + t == s
                n = min(se - s, kts[b] - t)
                slot = 2 * c + i + b * Hk + h
                assert 0 <= slot < 2 * CTAS + B * Hk and (1, slot) not in records
                records.add((1, slot))
                own_seen.update((b, h, t + x) for x in range(n))
                s, t, h = s + n, 0, h + 1
                if h == Hk:
                    b, h = b + 1, 0
    assert len(own_seen) == cum[-1] * Hk
    # the join looks at these CTAs for a unit's records
    per_x = np.float32(CTAS) / np.float32(max(X, 1))

    def candidates(x0, x1):
        return range(max(0, int(np.float32(x0) * per_x) - 1),
                     min(CTAS - 1, int(np.float32(x1) * per_x) + 1) + 1)

    for u in range(Hk * RT if KT else 0):
        got = sum(max(0, min(rs[c]["p1"], (u + 1) * KT) - max(rs[c]["p0"], u * KT))
                  for c in candidates(u * span, (u + 1) * span))
        assert got == KT
    for b, kt in enumerate(kts):
        for h in range(Hk if kt else 0):
            first = cum[b] * Hk + h * kt
            x0 = X1 + own_cost(ne[b], cum[b]) * Hk + h * own_cost(1, kt)
            got = sum(max(0, min(rs[c]["s1"], first + kt) - max(rs[c]["s0"], first))
                      for c in candidates(x0, x0 + own_cost(1, kt)))
            assert got == kt


@pytest.mark.parametrize("seed", range(8))
def test_every_tile_once_and_every_record_found(seed):
    rng = random.Random(seed)
    for _ in range(12):
        Hk, pair = rng.choice([1, 2, 8, 32]), rng.random() < 0.5
        RT = rng.choice([1, 1, 2, 4]) if pair else 1   # row tiles of 256; one below 128 rows
        KT = rng.choice([0, 0, 1, 2, 5, 32, 256, 1024])
        B = rng.choice([1, 2, 5, 30])
        top = rng.choice([1, 3, 10, 100])
        kts = [rng.choice([0, rng.randint(0, top), rng.randint(0, top)]) for _ in range(B)]
        if Hk * RT * KT + sum(kts):
            check(Hk, RT, KT, pair, kts)


def test_one_tile_and_one_long_sequence():
    check(1, 1, 1, False, [0])
    check(1, 1, 0, False, [1])
    check(2, 1, 0, False, [5000, 0, 1])
    check(8, 8, 1024, True, [1] * 64)
