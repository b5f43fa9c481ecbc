"""The chunk attention's partition and the norm kernels' division as the compiled code
computes them, on the host (parallax_testing.h), against the models of
test_chunk_model.py: the same pieces, records and merges for the same batches, lengths
up to the int range and lines past 2^32 included."""
import ctypes
import random

import numpy as np
import pytest

from parameterized_local_linear_b200 import binding, build
from test_chunk_model import COST, ROWS, items, pieces, random_batch

LMAX = 0x7fffffff // 64 * 64


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load_library()


def walk(lib, seqs, Hkv, tpt, causal, P, gaps=0, Lmax=LMAX, null_cu=False):
    """(pieces, merges) of the compiled walk; rows before the first sequence."""
    cu = np.concatenate([[gaps], gaps + np.cumsum([q for q, _ in seqs])]).astype(np.int32)
    lens = np.array([n for _, n in seqs], dtype=np.int32)
    total = int(cu[-1]) + gaps
    most = sum(-(-q // tpt) for q, _ in seqs) * Hkv + 2 * P
    out = np.zeros((most, 8), dtype=np.int32)
    merges = np.zeros((P, 5), dtype=np.int32)
    ptr = lambda a: a.ctypes.data_as(ctypes.c_void_p)
    n = lib.parallax_testing_chunk_walk(None if null_cu else ptr(cu), ptr(lens), len(seqs), total,
                                        Lmax, Hkv, tpt, int(causal), P, ptr(out), most, ptr(merges))
    assert n >= 0
    return out[:n].tolist(), merges.tolist()


def model(seqs, Hkv, tpt, causal, P, gaps=0):
    line = items(seqs, Hkv, tpt, causal)
    total = sum(x[3] + COST for x in line)
    per = max(COST + 1, -(-total // P))
    starts, pos = [], 0
    for it in line:
        starts.append(pos)
        pos += it[3] + COST
    s0 = np.concatenate([[gaps], gaps + np.cumsum([q for q, _ in seqs])])
    got, merges = [], []
    for c in range(P):
        note = [0] * 5
        lo, hi = min(total, c * per), min(total, (c + 1) * per)
        for k, (it, t0, t1, complete, first) in enumerate(pieces(line, c, P, per)):
            b, g, rt, nt = it
            got.append([c, b, g, rt, t0, t1, int(complete), int(first)])
        for it, start in zip(line, starts):
            end = start + it[3] + COST
            if start + COST < lo < end <= hi:  # ends here, after tiles in earlier ranges
                b, g, rt, _ = it
                c0 = (start + COST) // per
                note = [int(s0[b]) + rt * tpt, min(tpt, seqs[b][0] - rt * tpt), g, c0,
                        int(c0 * per >= start)]
        merges.append(note)
    return got, merges


@pytest.mark.parametrize("seed", range(200))
def test_walk_is_the_models(lib, seed):
    rnd = random.Random(1000 + seed)
    seqs, Hkv, tpt, causal, P = random_batch(rnd)
    gaps = rnd.choice((0, 0, 7))
    assert walk(lib, seqs, Hkv, tpt, causal, P, gaps) == model(seqs, Hkv, tpt, causal, P, gaps)


@pytest.mark.parametrize("G", [1, 3, 16, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_walk_of_far_lengths(lib, G, causal):
    """Lengths up to the int range, many heads and sequences: a line past 2^32."""
    rnd = random.Random(G)
    tpt = ROWS // G
    for seqs, Hkv in (([(1, LMAX)], 1), ([(700, LMAX), (0, 5), (3, LMAX - 1)], 8),
                      ([(tpt * 2, LMAX - rnd.randrange(10 ** 6)) for _ in range(40)], 8)):
        got = walk(lib, seqs, Hkv, tpt, causal, 148)
        assert got == model(seqs, Hkv, tpt, causal, 148)
    assert sum(x[3] + COST for x in items(seqs, Hkv, tpt, causal)) > 2 ** 32


def test_walk_clamps_its_lengths(lib):
    """Lengths outside the cache, and the form without cu_seqlens."""
    seqs = [(1, 130), (1, 0), (1, 64), (1, 5000)]
    want = model([(q, min(n, 256)) for q, n in seqs], 2, 64, False, 7)
    assert walk(lib, seqs, 2, 64, False, 7, Lmax=256) == want
    assert walk(lib, seqs, 2, 64, False, 7, Lmax=256, null_cu=True) == want
    assert walk(lib, [(1, -5), (1, 70)], 2, 64, True, 7) == model([(1, 0), (1, 70)], 2, 64, True, 7)


def test_division(lib):
    rnd = random.Random(2)
    f = lib.parallax_testing_divide
    for d in list(range(1, 300)) + [2 ** k + e for k in range(8, 31) for e in (-1, 0, 1)] + [2 ** 31 - 1]:
        ns = [0, 1, d - 1, d, d + 1, 2 ** 31 - 1] + [rnd.randrange(2 ** 31) for _ in range(30)]
        ns += [x * d + e for x in (rnd.randrange(2 ** 31 // d + 1) for _ in range(10)) for e in (-1, 0)]
        for n in ns:
            if 0 <= n < 2 ** 31:
                assert f(n, d) == n // d, (n, d)
