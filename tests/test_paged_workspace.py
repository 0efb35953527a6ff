"""One workspace of the paged decode attention serves calls of different sizes (CPU).

The workspace begins with tickets, words that are zero between calls; partial
results follow, whatever a call leaves there.  A buffer made for the largest of
several calls passes the size check of all of them, so no call's partial results
may lie where another call looks for tickets."""
import ctypes
import itertools
import random

import pytest

from bit_plane_kv_gb300 import binding as B


class Layout(ctypes.Structure):
    _fields_ = [("ctas", ctypes.c_int)] + [(f, ctypes.c_size_t) for f in ("ticket_off", "lse_off", "part_off", "ml_off",
                                                                         "logit_off", "total")]


@pytest.fixture(scope="module")
def layout_of():
    from bit_plane_kv_gb300 import build as BUILD
    BUILD.build()
    f = getattr(B.lib(), "_ZN6fathom22paged_workspace_layoutERK12fathom_pagesib")   # paged_workspace_layout
    f.restype, f.argtypes = Layout, [ctypes.POINTER(B.Pages), ctypes.c_int, ctypes.c_bool]

    def get(seqs, kv_heads, D, G, mass, max_pages=16):
        p = B.Pages(seqs=seqs, kv_heads=kv_heads, D=D, dtype=B.BF16, page_tokens=16, num_pages=64, max_pages=max_pages,
                    page_stride=16 * kv_heads * D, head_stride=D, token_stride=kv_heads * D)
        w = f(ctypes.byref(p), G, mass)
        assert w.total == B.lib().fathom_paged_workspace_size(ctypes.byref(p), G, int(mass)) > 0
        return w
    return get


def _calls():
    rng = random.Random(5)
    some = [(s, h, d, g, m) for s, h, d, g, m in itertools.product((1, 8, 1000), (1, 8), (64, 128), (1, 8), (False, True))]
    some += [(rng.randint(1, 8000), rng.choice([1, 2, 3, 8]), 8 * rng.randint(1, 16), rng.randint(1, 8),
              rng.random() < 0.5) for _ in range(100)]
    return some + [(65535, 1, 128, 4, True)]


def test_no_call_leaves_data_where_another_looks_for_tickets(layout_of):
    layouts = [(c, layout_of(*c)) for c in _calls()]
    for (ca, a), (cb, b) in itertools.product(layouts, layouts):
        assert a.ticket_off == b.ticket_off == 0
        data = min(b.lse_off, b.part_off, b.ml_off, b.logit_off)
        assert a.lse_off <= data, f"tickets of {ca} reach {a.lse_off}, data of {cb} start at {data}"


def test_every_cta_has_its_tickets(layout_of):
    """One of the unit that goes on behind it, two of groups of shares that it begins."""
    for c in _calls():
        w = layout_of(*c)
        assert w.lse_off - w.ticket_off >= 4 * 3 * w.ctas


def test_parts_do_not_overlap(layout_of):
    for seqs, heads, D, G, mass in _calls():
        w = layout_of(seqs, heads, D, G, mass)
        rows = seqs * heads * G
        assert w.part_off - w.lse_off >= (4 * rows if mass else 0)
        assert w.ml_off - w.part_off >= w.ctas * 2 * G * D * 4
        assert w.logit_off - w.ml_off >= w.ctas * 2 * G * 2 * 4
        assert w.total - w.logit_off >= (4 * rows * 256 if mass else 0)
        assert all(x % 256 == 0 for x in (w.lse_off, w.part_off, w.ml_off, w.logit_off, w.total))


def test_a_ticket_belongs_to_one_unit():
    """The kernel's shares, restated: CTA c of NC takes tiles c W / NC to (c + 1) W / NC of the W tiles of all units.
    Units that several CTAs share have first CTAs of their own, and the first shares of their groups of 16 lie at
    places of their own."""
    rng = random.Random(8)
    for _ in range(3000):
        ctas = rng.choice([1, 2, 3, 7, 304, 456])
        heads, seqs = rng.choice([1, 2, 8]), rng.randint(1, 12)
        top = rng.choice([2, 5, 30, 300, 3000])
        tiles = [t for _ in range(seqs) for t in [rng.randint(0, top)] * heads if t]
        W = sum(tiles)
        if W == 0:
            continue
        per_sm = 3 if ctas % 3 == 0 else 2
        NC = min(ctas, max(1, max(W // 4, min(W, ctas // per_sm))))
        firsts, groups, w0 = set(), set(), 0
        for n in tiles:
            first, last = ((w0 + 1) * NC - 1) // W, ((w0 + n) * NC - 1) // W
            assert first * W // NC <= w0 < (first + 1) * W // NC and last * W // NC < w0 + n <= (last + 1) * W // NC
            if first != last:
                assert first not in firsts
                firsts.add(first)
                before = first * W // NC < w0
                places = [2 * c + (before if c == first else 0) for c in range(first, last + 1, 16)] if last - first >= 32 else []
                assert not groups & set(places)
                groups |= set(places)
            w0 += n
        assert all(0 <= c < ctas for c in firsts) and all(0 <= x < 2 * ctas for x in groups)
