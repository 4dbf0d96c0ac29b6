"""CPU model of the walk over a sequence's own key tiles in the shared-prefix
attention (csrc/prefix_decode.cu) while the lengths in memory change under the
kernel.  The results of such a call mean nothing, but every role of a block has
to stay inside the cache and the workspace and come to an end, whatever each
read of a length returns."""
import random

import pytest

from test_prefix_split_model import CTAS, shares

TILE, PAGE = 128, 16


def walk(B, Hk, P, read, c, i, s, se, b, h, t):
    """Segments (b, h, t0, n, keys, record) of stream i of block c."""
    while s < se:
        keys = 0
        while b < B:
            keys = read(b) - P
            if keys > 0:
                break
            b += 1
        kt = -(-keys // TILE)
        if b >= B or kt <= t:
            return
        n = min(se - s, kt - t)
        yield b, h, t, n, keys, 2 * c + i + b * Hk + h
        s, t, h = s + n, 0, h + 1
        if h == Hk:
            b, h = b + 1, 0


@pytest.mark.parametrize("seed", range(6))
def test_walk_stays_inside_whatever_the_lengths_become(seed):
    rng = random.Random(seed)
    for _ in range(40):
        Hk, B, P = rng.choice([1, 2, 8]), rng.choice([1, 2, 7, 40]), PAGE * rng.choice([0, 1, 9])
        N = P + rng.choice([1, 16, 200, 3000])
        top = rng.choice([P + 1, N, N])

        def read(b):
            assert 0 <= b < B
            return rng.choice([0, P, rng.randint(0, top), N])

        kts = [-(-max(0, read(b) - P) // TILE) for b in range(B)]
        rs = shares(Hk, 1, 0, False, kts)[0] if sum(kts) else []
        for c in rng.sample(range(CTAS), 20):
            if rs and rng.random() < 0.7:       # where the block's own sums put it
                r = rs[c]
                spans, at = [(r["s0"], r["sm"]), (r["sm"], r["s1"])], r["at"]
            else:                               # sums over lengths that changed between two reads
                spans = [tuple(rng.randint(0, 5 * B * Hk) for _ in range(2)) for _ in range(2)]
                at = [(rng.randint(0, B), rng.randrange(Hk), rng.randint(0, 9)) for _ in range(2)]
            for i in range(2):
                segs = 0
                for b, h, t0, n, keys, slot in walk(B, Hk, P, read, c, i, *spans[i],
                                                    *(at[i] or (0, 0, 0))):
                    segs += 1
                    assert 0 <= b < B and 0 <= h < Hk and n >= 1 and t0 >= 0
                    assert 0 < keys <= N - P and (t0 + n - 1) * TILE < keys
                    for x in range(t0, t0 + n):       # pages of a tile: some, inside the table
                        pages = min(TILE // PAGE, -(-(keys - x * TILE) // PAGE))
                        assert pages >= 1
                        assert P // PAGE + x * (TILE // PAGE) + pages <= -(-N // PAGE)
                    assert 0 <= slot < 2 * CTAS + B * Hk
                assert segs <= B * Hk
