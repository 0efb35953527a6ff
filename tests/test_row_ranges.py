"""The rotated queries' place against the rows that are read (CPU): the arithmetic by itself, and the calls' refusals."""
import ctypes
import os
import random
import subprocess

import pytest

from bit_plane_kv_gb300 import binding as B

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "bit_plane_kv_gb300", "csrc")


@pytest.fixture(scope="module")
def meet(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("ranges") / "libranges.so")
    subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, os.path.join(HERE, "row_ranges_harness.cpp"),
                    "-o", out], check=True)
    f = ctypes.CDLL(out).rows_meet
    return lambda a, b: bool(f((ctypes.c_longlong * 6)(*a), (ctypes.c_longlong * 6)(*b)))


def touched(base, tokens, heads, token, head, run):
    return {base + t * token + h * head + i for t in range(tokens) for h in range(heads) for i in range(run)}


def test_sets_against_their_bytes(meet):
    """False only where no byte is shared; exact where the steps of both axes are equal."""
    rng = random.Random(3)
    exact = agree = 0
    for _ in range(6000):
        run_a, run_b = rng.choice([1, 2, 4]), rng.choice([1, 2, 4, 8])
        head = rng.randint(1, 12)
        token = rng.choice([head * rng.randint(1, 5), rng.randint(1, 60)])
        if rng.random() < 0.3:
            token, head = head, token
        a = (100, rng.randint(1, 6), rng.randint(1, 4), token, head, run_a)
        same = rng.random() < 0.7
        b = (100 + rng.randint(-80, 80), rng.randint(1, 6), rng.randint(1, 4), token if same else rng.randint(1, 60),
             head if same else rng.randint(1, 12), run_b)
        shared = bool(touched(*a) & touched(*b))
        got = meet(a, b)
        assert got or not shared, (a, b)
        if all(a[i] == b[i] or 1 in (a[j], b[j]) for i, j in ((3, 1), (4, 2))):
            exact += 1
            assert got == shared, (a, b)
        agree += got == shared
    assert exact > 4000 and agree > 5000


@pytest.mark.parametrize("a,b,want", [
    # parts of one projection buffer [tokens][48 heads][128] in 16 bits
    ((0, 500, 32, 12288, 256, 256), (32 * 256, 500, 8, 12288, 256, 256), False),
    ((0, 500, 32, 12288, 256, 256), (31 * 256, 500, 8, 12288, 256, 256), True),
    ((0, 500, 32, 12288, 256, 256), (48 * 256, 500, 32, 12288, 256, 256), True),       # a token on
    ((0, 500, 24, 12288, 256, 256), (24 * 256, 500, 24, 12288, 256, 256), False),
    ((0, 500, 24, 12288, 512, 256), (256, 500, 24, 12288, 512, 256), False),           # every second head
    ((0, 500, 24, 12288, 512, 256), (256, 500, 24, 12288, 512, 512), True),            # in 32 bits
    ((0, 500, 1, 2048, 8, 256), (256, 500, 4, 2048, 256, 256), False),                 # one KV head
    ((0, 500, 32, 256, 500 * 256, 256), (32 * 500 * 256, 500, 8, 256, 500 * 256, 256), False),   # heads around tokens
    ((0, 500, 32, 256, 500 * 256, 256), (32 * 500 * 256 - 16, 500, 8, 256, 500 * 256, 256), True),
    ((0, 1 << 28, 65535, 1 << 39, 1 << 38, 256), (1 << 62, 1 << 28, 65535, 1 << 39, 1 << 38, 512), True),   # beyond 64 bits
])
def test_layouts_of_programs(meet, a, b, want):
    assert meet(a, b) is want and meet(b, a) is want


@pytest.fixture(scope="module")
def lib():
    from bit_plane_kv_gb300 import build as BUILD
    BUILD.build()
    return B.lib()


@pytest.mark.parametrize("call", ["fathom_nibble_append", "fathom_paged_append_rope"])
@pytest.mark.parametrize("q_out,q_dtype,word", [
    (256, B.BF16, "overlaps q"),                 # a head on
    (-512, B.BF16, "overlaps q"),
    (16, B.F32, "overlaps q"),
    (32 * 256, B.BF16, "overlaps k_new"),        # the queries' heads lie over K's
    (40 * 256 + 128, B.BF16, "overlaps v_new"),
    (48 * 256, B.BF16, "overlaps q"),            # a token on
    (48 * 256 * 19, B.F32, "overlaps q")])
def test_a_place_that_is_read_is_refused(lib, call, q_out, q_dtype, word):
    """Queries, keys and values are slices of one buffer [20 tokens][48 heads][128]; the place has their strides."""
    base, row = 1 << 20, 48 * 128
    at = lambda x: ctypes.c_void_p(base + x)
    heads = 32 if word == "overlaps q" else 4
    r = B.Rope(256, 100, 128, 0, None, base, base + q_out, heads, q_dtype, row, 128, row if q_dtype == B.BF16 else row // 2, 128)
    d = ctypes.c_void_p(256)
    tail = (at(32 * 256), at(40 * 256), 20, row, 128, d, d, ctypes.byref(r), None)
    if call == "fathom_nibble_append":
        p = B.NibblePages(2, 8, 128, 16, 8, 4, 8 * 2304, 2304)
        rc = lib.fathom_nibble_append(ctypes.byref(p), d, d, B.BF16, *tail)
    else:
        p = B.Pages(2, 8, 128, B.BF16, 16, 8, 4, 8 * 2048, 2048, 128)
        rc = lib.fathom_paged_append_rope(ctypes.byref(p), d, d, d, *tail)
    assert rc == 1 and lib.fathom_last_error().decode() == "rope: q_out " + word, lib.fathom_last_error()
