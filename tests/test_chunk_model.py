"""A host model of the chunk attention's work partition and of its merge
ownership (csrc/chunk_partition.cuh), checked over many batches without a GPU:
every (item, tile) is covered exactly once, a CTA writes at most one record to
each of its two slots, every cut item has exactly one owner, and the records
the owner reads are exactly those its pieces wrote, in order. Also the tile,
page and mask arithmetic of a piece, and the oracle's chunk form."""
import random

import numpy as np
import pytest

import oracle

ROWS, KEYS, COST = 128, 64, 3


def tiles(s, rt, tpt, causal):
    q, n = s
    kend = max(0, n - q + min(q, (rt + 1) * tpt)) if causal else n
    return max(1, -(-kend // KEYS))


def items(seqs, Hkv, tpt, causal):
    """(b, g, rt, tiles) in line order."""
    out = []
    for b, s in enumerate(seqs):
        for g in range(Hkv):
            for rt in range(-(-s[0] // tpt)):
                out.append((b, g, rt, tiles(s, rt, tpt, causal)))
    return out


def pieces(line, c, P, per):
    total = sum(x[3] + COST for x in line)
    lo, hi = min(total, c * per), min(total, min(total, c * per) + per)
    pos = 0
    for it in line:
        length = it[3] + COST
        a, e = max(lo, pos), min(hi, pos + length)
        if a < e:
            t0, t1 = max(0, a - pos - COST), max(0, e - pos - COST)
            if t1 > t0:
                yield it, t0, t1, t0 == 0 and t1 == it[3], a == lo
        pos += length


def random_batch(rnd):
    G = rnd.choice((1, 2, 3, 4, 8, 16, 128))
    causal = rnd.random() < 0.8
    seqs = []
    for _ in range(rnd.randint(1, 9)):
        n = rnd.choice((0, 1, 63, 64, 65, rnd.randint(1, 3000)))
        q = rnd.choice((0, 1, min(n, 4), rnd.randint(0, max(1, n)), rnd.randint(0, 400)))
        seqs.append((q, n))
    return seqs, rnd.randint(1, 4), ROWS // G, causal, rnd.choice((1, 2, 7, 148))


@pytest.mark.parametrize("seed", range(60))
def test_every_tile_once_and_every_cut_item_merged_once(seed):
    rnd = random.Random(seed)
    seqs, Hkv, tpt, causal, P = random_batch(rnd)
    line = items(seqs, Hkv, tpt, causal)
    total = sum(x[3] + COST for x in line)
    per = max(COST + 1, -(-total // P))
    covered, written, whole = {}, {}, set()
    for c in range(P):
        slots = set()
        for it, t0, t1, complete, first in pieces(line, c, P, per):
            for t in range(t0, t1):
                assert covered.setdefault((it, t), c) == c and (it, t, c) not in whole
            if complete:
                assert it not in whole
                whole.add(it)
            else:
                slot = 2 * c + (0 if first else 1)
                assert slot not in slots
                slots.add(slot)
                written.setdefault(it, []).append((c, slot, t0, t1))
    assert len(covered) == sum(x[3] for x in line)
    assert whole | set(written) == set(line) and not whole & set(written)
    # the merge kernel's view
    merged = {}
    for c in range(P):
        lo, hi = min(total, c * per), min(total, min(total, c * per) + per)
        if lo >= hi:
            continue
        pos = 0
        for it in line:
            if lo < pos + it[3] + COST:
                break
            pos += it[3] + COST
        off = lo - pos
        if off <= COST or it[3] + COST - off > hi - lo:
            continue
        c0 = (pos + COST) // per
        c0_first = c0 * per >= pos
        assert it not in merged
        merged[it] = [2 * j + (0 if (j > c0 or c0_first) else 1) for j in range(c0, c + 1)]
    assert set(merged) == set(written)
    for it, recs in written.items():
        assert merged[it] == [slot for _, slot, _, _ in recs]
        assert [x[2] for x in recs[1:]] == [x[3] for x in recs[:-1]]
        assert recs[0][2] == 0 and recs[-1][3] == it[3]


@pytest.mark.parametrize("seed", range(30))
def test_masks_and_pages_of_every_row(seed):
    """Each row's mask keeps exactly its keys inside its item's tiles, every tile
    below the length lies in one page of the table, and the unmasked fast path is
    only taken where every live row sees the whole tile."""
    rnd = random.Random(100 + seed)
    seqs, Hkv, tpt, causal, _ = random_batch(rnd)
    ps = rnd.choice((64, 128, 256))
    for q, n in seqs:
        for rt in range(-(-q // tpt)):
            j0 = rt * tpt
            seen0 = n - q + j0 + 1 if causal else n
            nt = tiles((q, n), rt, tpt, causal)
            for x in range(min(tpt, q - j0)):
                klim = min(n, seen0 + x) if causal else n
                want = max(0, n - q + j0 + x + 1) if causal else n
                assert max(0, klim) == want <= nt * KEYS
                assert all(klim >= k0 + KEYS for k0 in range(0, nt * KEYS, KEYS)
                           if k0 + KEYS <= min(n, seen0))
            for k0 in range(0, nt * KEYS, KEYS):
                if k0 < n:
                    assert k0 // ps == min(n - 1, k0 + KEYS - 1) // ps < -(-n // ps)


def test_oracle_chunk_rows_are_decode_rows():
    """The oracle's chunk form against its decode, row by row, over a shuffled
    pool; rows without keys are zero."""
    rng = np.random.default_rng(0)
    Hq, Hkv, D, ps = 4, 2, 64, 64
    seqs = [(3, 70), (1, 1), (0, 5), (5, 3), (70, 130)]  # (5, 3): two rows see nothing
    pages = 12
    kp, vp = rng.standard_normal((2, pages, ps, Hkv, D))
    table = rng.permutation(pages)[: 5 * 3].reshape(-1)
    table = np.array([[0, 1, 2], [3, 0, 0], [4, 0, 0], [5, 0, 0], [9, 7, 11]])
    cu = np.concatenate([[0], np.cumsum([q for q, _ in seqs])])
    q, r = rng.standard_normal((2, cu[-1], Hq, D))
    lens = np.array([n for _, n in seqs])
    for causal in (True, False):
        got = oracle.parallax_prefill_paged(q, r, kp, vp, table, cu, lens, 0.1, causal)
        for b, (c, n) in enumerate(seqs):
            for j in range(c):
                row = cu[b] + j
                keys = max(0, n - c + j + 1) if causal else n
                want = oracle.parallax_decode_paged(q[row:row + 1], r[row:row + 1], kp, vp,
                                                    table[b:b + 1], np.array([keys]), 0.1)
                np.testing.assert_allclose(got[row:row + 1], want, rtol=1e-9, atol=1e-12)


def ceil_sum(a, T, m):
    """chunk_ceil_sum of csrc/chunk_partition.cuh."""
    period = (1 if T % KEYS == 0 else KEYS) if T >= KEYS else (KEYS // T if KEYS % T == 0 else KEYS)
    rise = period * T // KEYS
    u, v = divmod(m, period)
    total = 0
    for i in range(1, min(m, period) + 1):
        first = (a + i * T + KEYS - 1) // KEYS
        terms = u + (1 if i <= v else 0)
        total += terms * first + rise * (terms * (terms - 1) // 2)
    return total


@pytest.mark.parametrize("G", range(1, 129))
def test_the_closed_sum_is_the_sum_of_the_tiles(G):
    """Every row tile height, chunks of any offset and of up to 300 row tiles."""
    rnd, T = random.Random(G), ROWS // G
    for a in (0, 1, 63, 64, rnd.randint(0, 10 ** 6)):
        want = 0
        for m in range(300):
            assert ceil_sum(a, T, m) == want, (a, T, m)
            want += -(-(a + (m + 1) * T) // KEYS)


def search32(below, count):
    """The largest i with below(i) (below(0) holds), 32 candidates a step, as
    chunk_locate and NrBatch::search do it; counts the steps."""
    lo, hi, steps = 0, count, 0
    while hi - lo > 1:
        step = (hi - lo + 31) // 32
        votes = [lo + (x + 1) * step < hi and below(lo + (x + 1) * step) for x in range(32)]
        k = min((x for x in range(31) if not votes[x]), default=31)
        lo += k * step
        hi = min(hi, lo + step)
        steps += 1
    return lo, steps


def test_the_32_way_search_finds_every_place():
    for count in list(range(1, 200)) + [1023, 1024, 1025, 32769, 10 ** 6]:
        for at in {0, 1, 30, 31, 32, 33, count // 2, count - 2, count - 1} & set(range(count)):
            got, steps = search32(lambda i: i <= at, count)
            assert got == at and steps <= 5
    rnd = random.Random(0)  # no order among the votes: it still ends, in range
    for _ in range(200):
        got, steps = search32(lambda i: rnd.random() < 0.5, rnd.randint(1, 5000))
        assert 0 <= got < 5000 and steps <= 5


def test_the_divisor_is_exact():
    """NrDivisor: quotients of 31-bit numbers by a multiplication."""
    rnd = random.Random(1)
    for d in list(range(1, 300)) + [2 ** k + e for k in range(8, 31) for e in (-1, 0, 1)] + [2 ** 31 - 1]:
        s = 0
        while 2 ** s < d:
            s += 1
        m = (((2 ** s - d) << 32) // d + 1) & 0xffffffff
        for n in [0, 1, d - 1, d, d + 1, 2 ** 31 - 1] + [rnd.randrange(2 ** 31) for _ in range(50)] + \
                 [x * d + e for x in (rnd.randrange(2 ** 31 // d) for _ in range(10)) for e in (-1, 0)]:
            if 0 <= n < 2 ** 31:
                # (the sum mulhi + n stays below 2^32 for these n)
                assert ((m * n) >> 32) + n < 2 ** 32
                assert (((m * n) >> 32) + n) >> s == n // d, (n, d)
