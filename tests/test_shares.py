"""Which tiles a CTA of the 4-bit decode attention takes (CPU; the arithmetic that the kernel is built from)."""
import ctypes
import os
import random
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "bit_plane_kv_gb300", "csrc")


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("shares") / "libshares.so")
    subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, os.path.join(HERE, "shares_harness.cpp"),
                    "-o", out], check=True)
    lib = ctypes.CDLL(out)
    lib.tile_owner.argtypes = [ctypes.c_longlong, ctypes.c_longlong, ctypes.c_int]
    return lib


def own_shares(lib, tiles, heads, ctas):
    buf = (ctypes.c_int * (5 * ctas))()
    n = lib.own_shares(len(tiles), heads, ctas, (ctypes.c_int * len(tiles))(*tiles), buf)
    assert n >= 0, "more CTAs than there are"
    return [tuple(buf[5 * i:5 * i + 5]) for i in range(n)]


def check_own(lib, tiles, heads, ctas):
    """Every tile once, in order; no share longer than 8/7 of the mean, rounded up."""
    shares = own_shares(lib, tiles, heads, ctas)
    want = [(s, h) for s, t in enumerate(tiles) for h in range(heads) if t]
    at = 0
    for s, h in want:
        done = 0
        while done < tiles[s]:
            cta, s1, h1, first, count = shares[at]
            assert (cta, s1, h1, first) == (at, s, h, done) and count > 0
            done += count
            at += 1
        assert done == tiles[s]
    assert at == len(shares) <= ctas
    total, units = sum(tiles) * heads, len(tiles) * heads
    longest = max(x[4] for x in shares)
    assert longest <= -(-total // (ctas - units))
    assert longest < 8 * total / (7 * ctas) + 1


@pytest.mark.parametrize("tiles,heads,ctas", [
    ([1024] * 56 + [233] * 20, 1, 608), ([8192] + [260] * 9, 7, 608), ([1] * 76, 1, 608), ([0, 5, 0], 8, 456),
    ([1 << 21] * 76, 1, 608), ([1, 1 << 21], 28, 456), ([71, 9, 40, 60, 33, 12, 70], 3, 456)])
def test_units_with_ctas_of_their_own(lib, tiles, heads, ctas):
    assert lib.own_rule(len(tiles) * heads, ctas)
    check_own(lib, tiles, heads, ctas)


def test_units_with_ctas_of_their_own_random(lib):
    rng = random.Random(3)
    for _ in range(4000):
        ctas, heads = 152 * rng.choice([3, 4]), rng.choice([1, 2, 3, 7, 8])
        seqs = rng.randint(1, ctas // 8 // heads)
        top = rng.choice([1, 2, 9, 100, 5000, 1 << 21])
        tiles = [rng.choice([0, 1, top, rng.randint(0, top), int(2 ** rng.uniform(0, top.bit_length() - 1))]) for _ in range(seqs)]
        if sum(tiles):
            check_own(lib, tiles, heads, ctas)


def test_equal_shares(lib):
    """They cover all tiles, differ by one at most, and a tile's owner is the CTA that has it."""
    rng = random.Random(4)
    for _ in range(3000):
        ctas = 152 * rng.choice([3, 4])
        W = int(2 ** rng.uniform(0, 37))
        NC = min(ctas, W)
        start = (ctypes.c_longlong * (NC + 1))()
        tiles = sorted({0, W - 1} | {rng.randrange(W) for _ in range(20)})
        tiles += [c * W // NC for c in range(0, NC, 7)] + [c * W // NC - 1 for c in range(1, NC, 7)]
        ok = lib.equal_shares(ctypes.c_longlong(W), NC, start, (ctypes.c_longlong * len(tiles))(*tiles), len(tiles))
        assert ok and start[0] == 0 and start[NC] == W
        sizes = {b - a for a, b in zip(start, start[1:])}
        assert min(sizes) >= 1 and max(sizes) - min(sizes) <= 1


def test_places_of_partial_results_and_tickets_have_one_owner(lib):
    """Equal shares: a CTA's two places for partial results, a unit's ticket (its first CTA's, where it goes on
    behind that) and the tickets of its groups of 16 shares (the first share's place) are nobody else's."""
    rng = random.Random(5)
    for _ in range(400):
        ctas, heads = 152 * rng.choice([3, 4]), rng.choice([1, 2, 4, 8])
        seqs = rng.randint(1, 300)
        tiles = [rng.choice([0, 1, 2, rng.randint(0, 40), rng.choice([3, 900])]) for _ in range(seqs)]
        W = sum(tiles) * heads
        if not W:
            continue
        NC, at = min(ctas, W), 0
        start = (ctypes.c_longlong * (NC + 1))()
        lib.equal_shares(ctypes.c_longlong(W), NC, start, None, 0)
        places, tickets, groups = set(), set(), set()
        for t in tiles:
            for _ in range(heads if t else 0):
                w0, w1, at = at, at + t, at + t
                first, last = lib.tile_owner(w0, W, NC), lib.tile_owner(w1 - 1, W, NC)
                assert start[first] <= w0 < start[first + 1] and start[last] < w1 <= start[last + 1]
                if first == last:
                    continue
                slots = [2 * c + (1 if c == first and start[first] < w0 else 0) for c in range(first, last + 1)]
                assert first not in tickets and not places & set(slots)
                tickets.add(first)
                places |= set(slots)
                if len(slots) > 32:
                    assert not groups & set(slots[::16])
                    groups |= set(slots[::16])
        assert at == W
