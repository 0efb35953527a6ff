"""The steps of the prompt attention's work items, and how a cluster's CTAs share them (CPU).

The row warps of a tile wait once for every step that the matrix warp issues: `nt` of them, the last one worked on
as half a step when the tile's flag says so.  A flagged tile without a step in a share would wait for scores that
nobody computes."""
import ctypes
import os
import random
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "bit_plane_kv_gb300", "csrc")
FIELDS = ("nt0", "nt1", "steps", "half", "from_", "k0", "lk", "off")


@pytest.fixture(scope="module")
def work(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("work") / "libwork.so")
    subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-I", CSRC,
                    os.path.join(HERE, "prefill_work_harness.cpp"), "-o", out], check=True)
    lib = ctypes.CDLL(out)

    def get(*args):
        buf = (ctypes.c_int * len(FIELDS))()
        lib.prefill_work(*args, buf)
        return dict(zip(FIELDS, buf))
    get.meetings = lib.prefill_meetings

    def edges(*args):
        buf = (ctypes.c_int * 64)()
        n = lib.prefill_edges(*args, buf)
        return {buf[4 * i]: tuple(buf[4 * i + 1:4 * i + 4]) for i in range(n)}
    get.edges = edges
    return get


def _items():
    """(lq, lk, tokens per tile, first token, flip)"""
    for lq, lk, gp in ((2048, 2080, 1), (3000, 3001, 1), (1500, 1540, 1), (5, 5000, 2), (60, 50, 4), (1, 1, 128)):
        for t0 in range(0, lq, 256 // gp):
            yield lq, lk, 128 // gp, t0, 0
    rng = random.Random(3)
    for _ in range(4000):
        gp = rng.choice([1, 1, 2, 4, 8, 32, 128])
        lq = max(1, int(2 ** rng.uniform(0, 13)))
        lk = max(0, lq + rng.choice([0, rng.randint(-lq, 300), int(2 ** rng.uniform(0, 16))]))
        t0 = rng.randrange((lq * gp + 255) // 256) * (256 // gp)
        yield lq, lk, 128 // gp, t0, rng.randint(0, 1) if lq - t0 <= 128 // gp else 0


def _keys(lq, lk, tw, t0, flip, w):
    """Keys that the last row of tile w sees, from the definition."""
    rows = range(t0 + (w ^ flip) * tw, min(t0 + (w ^ flip) * tw + tw, lq))
    return max(0, min(lk, rows[-1] + lk - lq + 1)) if rows else 0


def test_an_item_covers_the_keys_its_rows_see(work):
    for item in _items():
        g = work(*item, 0, 1)
        for w in (0, 1):
            keys = _keys(*item, w)
            assert g[f"nt{w}"] == -(-keys // 128), item
            assert (g["half"] >> w & 1) == (0 < keys and (keys - 1) % 128 < 64), item
        assert g["steps"] == max(g["nt0"], g["nt1"]) and g["from_"] == 0


@pytest.mark.parametrize("split", [2, 4, 8])
def test_shares_cover_every_step_once_and_half_a_step_only_where_it_is(work, split):
    for item in _items():
        whole = work(*item, 0, 1)
        steps = {0: [], 1: []}
        for rank in range(split):
            g = work(*item, rank, split)
            assert g["steps"] == max(g["nt0"], g["nt1"])
            assert g["k0"] == g["from_"] and g["from_"] + g["lk"] == item[1]
            assert g["from_"] + g["off"] == item[1] - item[0]
            for w in (0, 1):
                nt, half = g[f"nt{w}"], g["half"] >> w & 1
                assert 0 <= nt - half, f"{item} share {rank} of {split}: tile {w} has half a step and no step"
                first = g["from_"] // 128
                steps[w] += range(first, first + nt)
                last_here = nt > 0 and first + nt == whole[f"nt{w}"]
                assert half == (last_here and whole["half"] >> w & 1), (item, rank, w)
        for w in (0, 1):
            assert steps[w] == list(range(whole[f"nt{w}"])), item


@pytest.mark.parametrize("split", [1, 2, 8])
def test_value_rows_that_a_query_does_not_see_are_looked_over(work, split):
    """Every row that a tile's products read and that some query of the item does not see, those behind the
    sequence's end apart; in the steps between the first of them and the last they lie without a gap."""
    for n, item in enumerate(_items()):
        if split > 1 and n % 5:
            continue
        lq, lk, tw, t0, flip = item
        fewest = max(0, t0 + lk - lq + 1)                       # keys that the item's first query sees
        for rank in range(split):
            g, edges = work(*item, rank, split), work.edges(*item, rank, split)
            for j in range(g["steps"]):
                key0 = g["from_"] + 128 * j
                used = max(64 if g["half"] >> w & 1 and j + 1 == g[f"nt{w}"] else 128 for w in (0, 1) if j < g[f"nt{w}"])
                r0, r1, r2 = edges.get(j, (used, used, used))
                assert 0 <= r0 <= r1 <= r2 == used, (item, rank, j)
                assert r0 == min(max(0, fewest - key0), used)
                assert r1 == min(max(lk - key0, r0), used)
                assert j + 1 == g["steps"] or r1 == r2 == 128


def test_a_row_warp_passes_every_cluster_barrier_with_and_without_its_item(work):
    """The cluster's other warps wait there without a limit."""
    assert [work.meetings(2, met) for met in (0, 1, 2)] == [2, 2, 2]
    assert work.meetings(0, 0) == 0                              # no cluster
