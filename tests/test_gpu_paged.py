"""The paged cache on the GPU (append, decode attention with attention mass,
eviction) against plain 64-bit forms; the tolerances are derived in paged_cases."""
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from bit_plane_kv_gb300 import binding as B

import paged_cases as P

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ decode
def attend(q, kp, vp, table, lens, mass=None, ws=None, **kw):
    pages = B.make_pages(kp, table)
    ws = B.alloc_paged_workspace(pages, G=q.shape[1], mass=mass is not None) if ws is None else ws
    return B.fathom_paged_attn(pages, q, kp, vp, table, i32(lens) if isinstance(lens, list) else lens, ws, mass=mass,
                               **kw)


def query(units, G, D, seed=1, scale=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return scale * torch.randn(units, G, D, generator=g, device="cuda")


def check_decode(out, q, kp, vp, table, lens, before=None, mass=None):
    o, w, tol, tol_w = P.decode(q, kp, vp, table, lens)
    assert torch.isfinite(out).all()
    far = (out.double() - o).abs()
    assert bool((far <= tol).all()), f"worst {(far / tol.clamp(min=1e-30)).max().item():.3f} of the tolerance"
    if mass is not None:
        want = before.double()
        want[:, : w.shape[1]] += w
        tol = torch.zeros_like(want)
        tol[:, : w.shape[1]] = tol_w
        tol += 2.0 ** -24 * want.abs() * (tol > 0)
        assert bool(((mass.double() - want).abs() <= tol).all())


LENS = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 500, 0, 1000]
DECODE = {
    "G 4, page 16": (LENS, 2, 4, 128, 16, BF, "token"),
    "G 1, fp16": (LENS, 3, 1, 128, 64, FP, "head"),
    "G 8": (LENS, 2, 8, 128, 32, BF, "token"),
    "G 8, fp16, 64 channels": (LENS, 2, 8, 64, 32, FP, "token"),
    "G 2, 96 channels": (LENS, 2, 2, 96, 128, BF, "head"),
    "G 3, 8 channels, page 1": ([1, 40, 7], 1, 3, 8, 1, FP, "token"),
    "G 5, 72 channels": ([300, 4], 2, 5, 72, 16, BF, "token"),
    "G 6, page 256": ([300, 4, 256, 257], 1, 6, 128, 256, FP, "head"),
    "G 7": ([100, 33], 1, 7, 64, 8, BF, "token"),
    "one unit of many shares": ([40000], 1, 8, 128, 64, BF, "token"),
    "one unit of many shares, 64 channels": ([51000], 1, 4, 64, 64, FP, "token"),
    "few units of many shares": ([30000, 5, 0, 21000], 1, 4, 128, 16, BF, "head"),
    "one token": ([1], 1, 1, 8, 16, BF, "token"),
    "all idle": ([0, 0, 0], 2, 4, 128, 16, BF, "token"),
    "long and short": ([9000, 3, 0, 700], 2, 4, 128, 64, BF, "token"),
    "many units": ([(37 * i) % 90 for i in range(300)], 4, 4, 64, 16, BF, "token"),
}


@pytest.mark.parametrize("with_mass", [False, True])
@pytest.mark.parametrize("name", list(DECODE))
def test_decode_matches_the_plain_form(name, with_mass):
    lens, H, G, D, page, dt, layout = DECODE[name]
    kp, vp, table, _ = P.pool(len(lens), H, D, page, -(-max(max(lens), 1) // page), dt, layout=layout)
    q = query(len(lens) * H, G, D)
    mass = torch.rand(len(lens) * H, table.shape[1] * page + 5, device="cuda") if with_mass else None
    before = mass.clone() if with_mass else None
    out = attend(q, kp, vp, table, lens, mass)
    check_decode(out, q, kp, vp, table, lens, before, mass)


def test_empty_sequences_give_zero():
    kp, vp, table, _ = P.pool(2, 2, 64, 16, 2, BF)
    out = attend(query(4, 4, 64), kp, vp, table, [0, -5])
    assert bool((out == 0).all())


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("scale", [0.0, 1e-6, 60.0])
def test_flat_tiny_and_sharp_queries(dt, scale):
    lens = [513, 70]
    kp, vp, table, _ = P.pool(2, 2, 128, 16, 40, dt)
    q = query(4, 4, 128, scale=scale)
    check_decode(attend(q, kp, vp, table, lens), q, kp, vp, table, lens)


def test_queries_beyond_the_cache_type_stay_finite():
    """fp32 queries larger than fp16 holds, against small fp16 keys."""
    kp, vp, table, _ = P.pool(1, 1, 64, 16, 10, FP)
    kp.mul_(2.0 ** -12)
    q = query(1, 4, 64) * 2.0 ** 18
    check_decode(attend(q, kp, vp, table, [150]), q, kp, vp, table, [150])


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_rows_behind_the_length_and_unnamed_pages_are_never_read(bad):
    lens, H, page = [70, 16, 1], 2, 16
    kp, vp, table, _ = P.pool(3, H, 128, page, 8, BF)
    q = query(6, 4, 128)
    want = attend(q, kp, vp, table, lens).clone()
    live = torch.zeros(kp.shape[0], page, dtype=torch.bool, device="cuda")
    for s, n in enumerate(lens):
        for i in range(n):
            live[int(table[s, i // page]), i % page] = True
    dead = ~live[:, None, :, None]
    kp.masked_fill_(dead, bad), vp.masked_fill_(dead, bad)
    assert torch.equal(attend(q, kp, vp, table, lens), want)


@pytest.mark.parametrize("lens", [[70, 300, 5], [20, 40000, 1]])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("what", ["q", "k", "v"])
def test_what_is_not_finite_stays_in_its_unit(what, bad, lens):
    """A NaN or an infinity that a unit does attend to: its own results only, and never finite ones where
    a NaN took part (also where a warp's 16 tokens are all NaN)."""
    H, G, D, page = 2, 4, 128, 64
    kp, vp, table, _ = P.pool(3, H, D, page, (max(lens) + page - 1) // page, BF)
    q = query(6, G, D)
    mass = torch.zeros(6, table.shape[1] * page, device="cuda")
    want = attend(q, kp, vp, table, lens, mass=mass)
    unit, seq, head = 3, 1, 1
    if what == "q":
        q[unit, 2, 9] = bad
    else:
        (kp if what == "k" else vp)[table[seq, 0], head, :16, 9] = bad
    mass2 = torch.zeros_like(mass)
    out = attend(q, kp, vp, table, lens, mass=mass2)
    others = [u for u in range(6) if u != unit]
    assert torch.equal(out[others], want[others]) and torch.equal(mass2[others], mass[others])
    if what == "v":
        rest = [c for c in range(D) if c != 9]
        assert torch.equal(out[unit][:, rest], want[unit][:, rest]) and torch.equal(mass2, mass)
        assert not torch.isfinite(out[unit, :, 9]).any()
    elif math.isnan(bad):
        heads = [2] if what == "q" else list(range(G))
        assert torch.isnan(out[unit, heads]).all() and torch.isnan(mass2[unit, : lens[seq]]).all()
        assert bool((mass2[unit, lens[seq]:] == 0).all())


def test_bad_page_table_entries_are_skipped():
    lens, page = [100, 64], 16
    kp, vp, table, _ = P.pool(2, 2, 128, page, 7, BF)
    table[0, 2], table[0, 5], table[1, 0] = -1, kp.shape[0], 1 << 30
    q = query(4, 4, 128)
    mass = torch.zeros(4, 7 * page, device="cuda")
    before = mass.clone()
    out = attend(q, kp, vp, table, lens, mass)
    check_decode(out, q, kp, vp, table, lens, before, mass)
    table[1] = -7                                          # a sequence with no page at all
    assert bool((attend(q, kp, vp, table, lens)[2:] == 0).all())


def test_lengths_are_clamped_to_the_table():
    kp, vp, table, _ = P.pool(1, 2, 64, 16, 3, BF)
    q = query(2, 4, 64)
    assert torch.equal(attend(q, kp, vp, table, [1 << 30]), attend(q, kp, vp, table, [48]))


def test_pages_shared_by_sequences():
    kp, vp, table, _ = P.pool(3, 2, 128, 16, 10, BF)
    table[1, :6], table[2, :3] = table[0, :6], table[0, :3]
    q, lens = query(6, 4, 128), [160, 130, 60]
    check_decode(attend(q, kp, vp, table, lens), q, kp, vp, table, lens)


def test_a_workspace_serves_call_after_call_and_graph_after_graph():
    kp, vp, table, _ = P.pool(5, 2, 128, 16, 60, BF)
    pages = B.make_pages(kp, table)
    ws = B.alloc_paged_workspace(pages, G=4, mass=True)
    lens = i32([900, 3, 0, 450, 77])
    mass = torch.zeros(10, pages.cap, device="cuda")
    q = query(10, 4, 128)
    want = attend(q, kp, vp, table, lens)
    for _ in range(3):
        assert torch.equal(attend(q, kp, vp, table, lens, ws=ws), want)
        attend(q, kp, vp, table, lens, mass, ws=ws)
    graphs, outs = [], []
    for _ in range(2):                                     # two graphs that share the workspace, one after the other
        g, o = torch.cuda.CUDAGraph(), torch.empty(10, 4, 128, device="cuda")
        with torch.cuda.graph(g):
            attend(q, kp, vp, table, lens, ws=ws, out=o)
        graphs.append(g)
        outs.append(o)
    lens.copy_(i32([60, 900, 1, 0, 333]))                  # another batch for the same graphs
    q.copy_(query(10, 4, 128, seed=5))
    want = attend(q, kp, vp, table, lens)
    for g in (graphs[0], graphs[1], graphs[0]):
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


def test_a_workspace_serves_calls_of_different_sizes_in_turn():
    """A serving loop's batch changes from step to step: one buffer, made for the largest call, gives what a fresh
    one gives (every output filled with NaN before)."""
    calls = [                                              # (lengths, KV heads, G, D, type, with mass)
        ([700 + i % 90 for i in range(256)], 4, 4, 128, BF, False),    # most units shared by two CTAs
        ([3000], 8, 4, 128, BF, False),
        ([60000], 1, 8, 64, FP, True),                                # joined in groups
        ([900 - i for i in range(300)], 2, 8, 64, FP, True),
        ([50000], 1, 4, 128, BF, True),
        ([1, 40, 9000], 2, 2, 72, BF, False),
    ]
    made = []
    for lens, H, G, D, dt, with_mass in calls:
        kp, vp, table, _ = P.pool(len(lens), H, D, 64, -(-max(lens) // 64), dt)
        q, pages = query(len(lens) * H, G, D), B.make_pages(kp, table)
        mass = torch.zeros(len(lens) * H, pages.cap, device="cuda") if with_mass else None
        want = attend(q, kp, vp, table, lens, mass)
        made.append((q, kp, vp, table, i32(lens), want, mass, B.paged_workspace_size(pages, G, with_mass)))
    ws = torch.zeros(max(m[-1] for m in made), dtype=torch.uint8, device="cuda")
    for i in (0, 1, 0, 2, 0, 3, 4, 3, 1, 5, 4, 2, 2, 0, 5, 3):
        q, kp, vp, table, lens, want, mass, _ = made[i]
        again = None if mass is None else torch.zeros_like(mass)
        out = attend(q, kp, vp, table, lens, again, ws=ws, out=torch.full_like(want, math.nan))
        assert torch.equal(out, want), f"call {i}"
        assert mass is None or torch.equal(again, mass), f"call {i}"


@pytest.mark.parametrize("lens,H,G,D,dt", [
    ([30000, 17, 0, 22001], 4, 4, 128, BF),                # long shares of few sequences
    ([50000, 17], 1, 8, 128, BF),                          # more shares than are joined at once
    ([2000 + 13 * i for i in range(150)], 2, 8, 64, FP),   # more than 128 sequences
])
def test_the_same_bits_every_time(lens, H, G, D, dt):
    kp, vp, table, _ = P.pool(len(lens), H, D, 64, -(-max(lens) // 64), dt)
    q = query(len(lens) * H, G, D)
    pages = B.make_pages(kp, table)
    ws = B.alloc_paged_workspace(pages, G=G, mass=True)
    mass = torch.zeros(len(lens) * H, pages.cap, device="cuda")
    before = mass.clone()
    out = attend(q, kp, vp, table, lens, mass, ws=ws)
    check_decode(out, q, kp, vp, table, lens, before, mass)
    for _ in range(5):
        again = torch.zeros_like(mass)
        assert torch.equal(attend(q, kp, vp, table, lens, again, ws=ws), out)
        assert torch.equal(again, mass)


def test_thousands_of_sequences():
    lens = [(7 * i) % 61 for i in range(1500)]
    kp, vp, table, _ = P.pool(1500, 1, 64, 16, 4, BF)
    q = query(1500, 2, 64)
    check_decode(attend(q, kp, vp, table, lens), q, kp, vp, table, lens)


def test_two_calls_at_once_with_their_own_workspaces():
    kp, vp, table, _ = P.pool(4, 2, 128, 32, 100, BF)
    lens = i32([3000, 100, 1, 2222])
    q = query(8, 4, 128)
    want = attend(q, kp, vp, table, lens)
    pages = B.make_pages(kp, table)
    ws = [B.alloc_paged_workspace(pages, G=4) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [attend(q, kp, vp, table, lens, ws=w, stream=s) for _ in range(4) for w, s in zip(ws, streams)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for x in got)


def test_pages_beyond_32_bit_offsets():
    """Four pages 2^30 elements apart: append, attention and eviction past 2^32 bytes."""
    H, D, page, step = 1, 64, 64, 1 << 30
    pools = [torch.empty(3 * step + H * page * D, dtype=BF, device="cuda").as_strided((4, H, page, D), (step, page * D, D, 1))
             for _ in range(2)]
    table = i32([[3, 1, 2, 0]])
    pages = B.make_pages(pools[0], table)
    new = torch.randn(200, 2, D, device="cuda").to(BF)
    B.fathom_paged_append(pages, *pools, table, new[:, :1], new[:, 1:], i32([0]), P.cumulated([200]))
    q = query(1, 4, D)
    check_decode(attend(q, *pools, table, [200]), q, *pools, table, [200])
    m = masses(1, 256)
    kept, _, _ = B.fathom_paged_evict(pages, *pools, table, i32([200]), m, 70, table, 4, 32)     # in place
    at = kept[0].long()
    assert torch.equal(torch.cat([pools[0][3, 0], pools[0][1, 0, :6]]), new[at, 0])
    assert torch.equal(torch.cat([pools[1][3, 0], pools[1][1, 0, :6]]), new[at, 1])


def test_cache_in_pinned_host_memory():
    kp, vp, table, _ = P.pool(2, 2, 128, 16, 20, BF, layout="head")
    q, lens = query(4, 4, 128), [300, 45]
    want = attend(q, kp, vp, table, lens)
    got = attend(q, kp.cpu().pin_memory(), vp.cpu().pin_memory(), table, lens)
    assert torch.equal(got, want)


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("page,H,D,dt,layout", [(16, 2, 128, BF, "token"), (64, 3, 72, FP, "head"), (1, 1, 8, BF, "token")])
def test_append_writes_the_named_places_only(page, H, D, dt, layout):
    seqs, per = 4, max(4, 96 // page)
    kp, vp, table, _ = P.pool(seqs, H, D, page, per, dt, layout=layout, extra=2)
    k0, v0 = kp.clone(), vp.clone()
    new, start = [5, 0, 40, 1], [0, 3, 17, per * page - 1]
    T = sum(new)
    kv = torch.randn(T + 3, 2 * H, D, device="cuda").to(dt)          # three tokens behind the last sequence
    B.fathom_paged_append(B.make_pages(kp, table), kp, vp, table, kv[:, :H], kv[:, H:], i32(start), P.cumulated(new))
    t = 0
    for s in range(seqs):
        for i in range(new[s]):
            p, slot = int(table[s, (start[s] + i) // page]), (start[s] + i) % page
            k0[p, :, slot], v0[p, :, slot] = kv[t, :H], kv[t, H:]
            t += 1
    assert torch.equal(kp, k0) and torch.equal(vp, v0)


def test_append_skips_what_has_no_place():
    kp, vp, table, _ = P.pool(4, 2, 64, 16, 2, BF, extra=1)
    k0, v0 = kp.clone(), vp.clone()
    table[1, 0], table[2, 1] = -1, kp.shape[0]
    new = torch.randn(4, 2, 64, device="cuda").to(BF)
    B.fathom_paged_append(B.make_pages(kp, table), kp, vp, table, new, new, i32([32, 3, 20, -1]))
    assert torch.equal(kp, k0) and torch.equal(vp, v0)               # past the end, no page, bad page, before 0
    B.fathom_paged_append(B.make_pages(kp, table), kp, vp, table, new, new, i32([31, 16, 0, 7]))
    for s, pos in enumerate([31, 16, 0, 7]):
        k0[int(table[s, pos // 16]), :, pos % 16] = new[s]
    assert torch.equal(kp, k0)


# ------------------------------------------------------------------ eviction
def evict_and_check(lens, H, D, page, keep, ns, nr, dt, mass, in_place, layout="token"):
    seqs, per = len(lens), mass.shape[1] // page
    dp = -(-keep // page)
    kp, vp, table, free = P.pool(seqs, H, D, page, per, dt, extra=seqs * dp, layout=layout)
    dst = free.reshape(seqs, dp).contiguous()
    if in_place:      # the table itself, or a copy of as much of it as the kept rows need
        dst = table if in_place is True else table[:, :dp].contiguous()
    k0, v0, m0 = kp.clone(), vp.clone(), mass.clone()
    out = None if in_place else torch.full((seqs * H, keep + 3), -2.0, device="cuda")
    pages = B.make_pages(kp, table)
    kept, new, mo = B.fathom_paged_evict(pages, kp, vp, table, i32(lens), mass, keep, dst, ns, nr, mass_out=out)
    wk, wv = k0.clone(), v0.clone()
    wm = m0.clone() if in_place else torch.full_like(mo, -2.0)
    tt, dd, mm = table.cpu().numpy(), dst.cpu().numpy(), m0.cpu().numpy()
    want = np.full((seqs * H, keep), -1, np.int32)
    for u in range(seqs * H):
        s, h = divmod(u, H)
        n = min(max(lens[s], 0), per * page)
        idx = np.array(P.kept_set(mm[u].tolist(), n, keep, ns, nr), np.int64)
        want[u, : len(idx)] = idx
        if len(idx) == 0:
            continue
        j = np.arange(len(idx))
        a, b = tt[s][idx // page], dd[s][j // page]
        a, b, i, j = (torch.from_numpy(np.asarray(x, np.int64)).cuda() for x in (a, b, idx % page, j % page))
        wk[b, h, j], wv[b, h, j] = k0[a, h, i], v0[a, h, i]
        wm[u, : len(idx)] = m0[u, torch.from_numpy(idx).cuda()]
    np.testing.assert_array_equal(kept.cpu().numpy(), want)
    assert new.tolist() == [min(min(max(n, 0), per * page), keep) for n in lens]
    assert torch.equal(kp.view(torch.int16), wk.view(torch.int16)) and torch.equal(vp, wv)
    assert torch.equal(torch.nan_to_num(mo, nan=9.0), torch.nan_to_num(wm, nan=9.0))


def masses(units, cap, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    m = torch.exp(2 * torch.randn(units, cap, generator=g, device="cuda"))
    m[torch.rand(m.shape, generator=g, device="cuda") < 0.2] = 0          # ties
    return m


@pytest.mark.parametrize("in_place", [False, True, "a copy of the table"])
@pytest.mark.parametrize("lens,H,D,page,keep,ns,nr,dt", [
    ([500, 64, 65, 0, 1, 40], 2, 128, 16, 64, 4, 32, BF),
    ([3000, 2999], 3, 128, 64, 1000, 4, 32, FP),
    ([700, 701, 130], 1, 72, 32, 129, 0, 0, BF),
    ([300, 299], 2, 64, 8, 36, 4, 32, FP),           # nothing but the forced tokens
    ([9, 10, 11], 1, 8, 1, 10, 3, 4, BF),
    ([1025, 2048, 2047], 2, 128, 16, 2047, 4, 32, BF),
    ([5000], 1, 128, 64, 1, 1, 0, BF),
    ([100], 1, 128, 16, 300, 4, 32, BF),             # more room than tokens
    ([9001, 4000], 1, 72, 16, 3500, 4, 32, FP),      # teams of CTAs over several chunks
    ([40000], 2, 64, 64, 20011, 4, 32, BF),          # clusters of CTAs choose
    ([200000], 1, 8, 64, 1000, 4, 32, BF),           # more tokens than a cluster holds
])
def test_eviction_keeps_and_moves_what_the_plain_form_does(lens, H, D, page, keep, ns, nr, dt, in_place):
    per = -(-max(max(lens), keep) // page)
    evict_and_check(lens, H, D, page, keep, ns, nr, dt, masses(len(lens) * H, per * page), in_place)


@pytest.mark.parametrize("in_place", [False, True, "a copy of the table"])
def test_many_units_and_the_head_major_layout(in_place):
    lens = [100 + 13 * i for i in range(40)]
    evict_and_check(lens, 8, 64, 16, 150, 4, 32, BF, masses(320, 640), in_place, layout="head")


@pytest.mark.parametrize("kind", ["equal", "zero", "nan", "inf", "negative", "two values"])
def test_ties_and_special_masses(kind):
    m = masses(2, 512, seed=4)
    g = torch.Generator(device="cuda").manual_seed(8)
    some = torch.rand(m.shape, generator=g, device="cuda") < 0.3
    if kind == "equal":
        m.fill_(0.25)
    elif kind == "zero":
        m.zero_()
        m[some] = -0.0                                # the same value as 0
    elif kind == "nan":
        m[some] = float("nan")
        m[some & (m.roll(1, 1) > 1)] = -float("nan")
    elif kind == "inf":
        m[some] = float("inf")
    elif kind == "negative":
        m[some] *= -1
    else:
        m = some.float()
    evict_and_check([500, 512], 1, 64, 16, 200, 4, 32, BF, m, False)


def test_a_bad_page_moves_nothing():
    kp, vp, table, free = P.pool(1, 1, 64, 16, 8, BF, extra=4)
    dst = free.reshape(1, 4).contiguous()
    table[0, 7], dst[0, 1] = -1, 1 << 20              # the recent tokens' page, and the rows 16 .. 31
    k0 = kp.clone()
    mass = masses(1, 128)
    kept, _, _ = B.fathom_paged_evict(B.make_pages(kp, table), kp, vp, table, i32([128]), mass, 64, dst, 4, 32)
    want = k0.clone()
    for j, i in enumerate(kept[0].tolist()):
        a, b = int(table[0, i // 16]), int(dst[0, j // 16])
        if 0 <= a < kp.shape[0] and 0 <= b < kp.shape[0]:
            want[b, 0, j % 16] = k0[a, 0, i % 16]
    assert torch.equal(kp, want)


def test_eviction_in_a_graph_and_on_a_stream():
    lens, keep = i32([400, 90]), 100
    kp, vp, table, free = P.pool(2, 2, 128, 16, 32, BF, extra=2 * 7)
    dst = free.reshape(2, 7).contiguous()
    pages, mass = B.make_pages(kp, table), masses(4, 512)
    out = [torch.empty(4, keep, dtype=torch.int32, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda"),
           torch.zeros(4, 112, device="cuda")]

    def call(stream=None):
        B.fathom_paged_evict(pages, kp, vp, table, lens, mass, keep, dst, kept_idx=out[0], lens_out=out[1],
                             mass_out=out[2], stream=stream)

    call()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    mass.copy_(masses(4, 512, seed=3))
    lens.copy_(i32([101, 512]))
    g.replay()
    got = [x.clone() for x in out] + [kp.clone()]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    call(stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, out + [kp]))
    for u in range(4):
        n = [101, 512][u // 2]
        assert out[0][u].tolist() == P.kept_set(mass[u].tolist(), n, keep, 4, 32)


def test_calls_by_clusters_captured_by_a_process_that_has_not_made_them():
    """Few rows against many keys, one unit of many shares, an eviction of long sequences in place: captured as a
    process's first calls, replayed twice, and the same as eager calls."""
    code = """
import sys
sys.path.insert(0, %r); sys.path.insert(0, %r)
import torch
from bit_plane_kv_gb300 import binding as B
import paged_cases as P
n = 30000
kp, vp, table, _ = P.pool(1, 1, 128, 64, 469, torch.bfloat16)
k0, v0 = kp.clone(), vp.clone()
pages = B.make_pages(kp, table)
ws = B.alloc_paged_workspace(pages, G=8, mass=True)
q, lens = torch.randn(1, 8, 128, device="cuda"), torch.full((1,), n, dtype=torch.int32, device="cuda")
mass, part = torch.zeros(1, 469 * 64, device="cuda"), torch.zeros(1, 5000, device="cuda")
p = torch.randn(9000, 3, 128, device="cuda").bfloat16()
cq, ck = P.cumulated([20]), P.cumulated([9000])

def calls():
    kp.copy_(k0), vp.copy_(v0), mass.zero_()
    a, _ = B.fathom_prefill_attn(p[:20, :1], p[:, 1:2], p[:, 2:], cq, ck)
    b = B.fathom_paged_attn(pages, q, kp, vp, table, lens, ws, mass=mass)
    c, d, e = B.fathom_paged_evict(pages, kp, vp, table, lens, mass, 5000, table, mass_out=part)
    return a, b, c, d, e, mass, kp, vp

g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
with torch.cuda.graph(g):
    got = calls()
g.replay()
g.replay()
torch.cuda.synchronize()
got = [x.clone() for x in got]
with torch.cuda.stream(side):
    want = calls()
torch.cuda.synchronize()
assert all(torch.equal(x, y) for x, y in zip(got, want))
assert want[2][0].tolist() == P.kept_set(mass[0].tolist(), n, 5000, 4, 32)
B.fathom_wait_status()
print("same")
""" % (os.path.dirname(os.path.dirname(os.path.abspath(__file__))), os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "same", r.stdout + r.stderr[-2000:]


def test_a_launch_that_fails_leaves_no_error_behind():
    """A launch that the runtime refuses (on the default stream, while a stream that waits for it is being captured):
    the call reports it, the next call of somebody else's does not."""
    code = """
import ctypes, sys
sys.path.insert(0, %r); sys.path.insert(0, %r)
import torch
from bit_plane_kv_gb300 import binding as B
import paged_cases as P
kp, vp, table, free = P.pool(2, 2, 128, 16, 8, torch.bfloat16, extra=8)
pages, L = B.make_pages(kp, table), B.lib()
ws = B.alloc_paged_workspace(pages, G=4, mass=True)
q, x = torch.randn(4, 4, 128, device="cuda"), torch.randn(40, 8, 128, device="cuda").bfloat16()
lens, cu = torch.full((2,), 100, dtype=torch.int32, device="cuda"), P.cumulated([7, 33])
mass, dst = torch.zeros(4, 128, device="cuda"), free.reshape(2, 4).contiguous()
out, kept = torch.zeros_like(x), torch.zeros(4, 60, dtype=torch.int32, device="cuda")
o, lens2, mass2 = torch.zeros_like(q), torch.zeros_like(lens), torch.zeros(4, 64, device="cuda")
a = [t.data_ptr() for t in (kp, vp, table)]
pr = B.Prompts(2, 8, 2, 128, B.BF16, 40, 40, 1024, 128, 1024, 128, 1024, 128, 1024, 128)
calls = {
    "prefill": lambda: L.fathom_prefill_attn(ctypes.byref(pr), x.data_ptr(), x.data_ptr(), x.data_ptr(), cu.data_ptr(),
                                             cu.data_ptr(), out.data_ptr(), None, None),
    "append": lambda: L.fathom_paged_append(ctypes.byref(pages), *a, x.data_ptr(), x.data_ptr(), 2, 1024, 128,
                                            lens.data_ptr(), None, None),
    "attn": lambda: L.fathom_paged_attn(ctypes.byref(pages), 4, q.data_ptr(), *a, lens.data_ptr(), o.data_ptr(), None, 0,
                                        ws.data_ptr(), ws.numel(), None),
    "mass": lambda: L.fathom_paged_attn(ctypes.byref(pages), 4, q.data_ptr(), *a, lens.data_ptr(), o.data_ptr(),
                                        mass.data_ptr(), 128, ws.data_ptr(), ws.numel(), None),
    "evict": lambda: L.fathom_paged_evict(ctypes.byref(pages), *a, lens.data_ptr(), mass.data_ptr(), 128, 60, 4, 32,
                                          dst.data_ptr(), 4, kept.data_ptr(), lens2.data_ptr(), mass2.data_ptr(), 64, None),
}
for call in calls.values():
    assert call() == 0
torch.cuda.synchronize()
rt = ctypes.CDLL("libcudart.so.%%s" %% torch.version.cuda.split(".")[0])
for name, call in calls.items():
    stream, graph = ctypes.c_void_p(), ctypes.c_void_p()
    assert rt.cudaStreamCreate(ctypes.byref(stream)) == 0
    assert rt.cudaStreamBeginCapture(stream, 0) == 0
    status, left = call(), rt.cudaGetLastError()
    rt.cudaStreamEndCapture(stream, ctypes.byref(graph))
    rt.cudaGetLastError()
    assert rt.cudaStreamDestroy(stream) == 0
    assert status == 2 and left == 0, (name, status, left)
    assert call() == 0
torch.cuda.synchronize()
print("clear")
""" % (os.path.dirname(os.path.dirname(os.path.abspath(__file__))), os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "clear", r.stdout + r.stderr[-2000:]


def test_first_calls_of_a_process_by_several_threads_at_once():
    """Every form of the kernels with large shared memory, called for the first time by eight threads together."""
    code = """
import sys, threading
sys.path.insert(0, %r); sys.path.insert(0, %r)
import torch
from bit_plane_kv_gb300 import binding as B
import paged_cases as P
N = 8
jobs = []
for dt in (torch.bfloat16, torch.float16):
    for D in (64, 96, 128):
        x = torch.randn(3000, 3, D, device="cuda").to(dt)
        for lq, lk in ((16, 3000), (300, 300)):                          # by clusters, and not
            cq, ck = P.cumulated([lq]), P.cumulated([lk])
            jobs.append(lambda s, x=x, lq=lq, lk=lk, cq=cq, ck=ck:
                        B.fathom_prefill_attn(x[:lq, :1], x[:lk, 1:2], x[:lk, 2:], cq, ck, stream=s)[0])
    for D in (64, 128):
        for G in (4, 8):
            kp, vp, table, _ = P.pool(1, 2, D, 16, 40, dt)
            pages, q = B.make_pages(kp, table), torch.randn(2, G, D, device="cuda")
            lens = torch.full((1,), 600, dtype=torch.int32, device="cuda")
            for mass in (False, True):
                jobs.append(lambda s, a=(pages, q, kp, vp, table, lens), G=G, mass=mass:
                            B.fathom_paged_attn(*a, B.alloc_paged_workspace(a[0], G=G, mass=mass),
                                                mass=torch.zeros(2, 640, device="cuda") if mass else None, stream=s))
torch.cuda.synchronize()
streams = [torch.cuda.Stream() for _ in range(N)]
got, wrong, gate = [[None] * len(jobs) for _ in range(N)], [], threading.Barrier(N)

def run(i):
    for j, job in enumerate(jobs):
        gate.wait()
        try:
            torch.cuda.set_device(0)
            got[i][j] = job(streams[i])
        except Exception as e:
            wrong.append((j, repr(e)))

threads = [threading.Thread(target=run, args=(i,)) for i in range(N)]
[t.start() for t in threads], [t.join() for t in threads]
torch.cuda.synchronize()
assert not wrong, (len(wrong), wrong[:3])
assert all(torch.equal(got[i][j], got[0][j]) for i in range(N) for j in range(len(jobs)))
print("same")
""" % (os.path.dirname(os.path.dirname(os.path.abspath(__file__))), os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "same", r.stdout + r.stderr[-2000:]


# ------------------------------------------------------------------ together
def test_prompt_append_decode_evict_decode():
    """A serving loop: packed prompts, their rows into the pages, decode steps that gather mass,
    an eviction, decode steps over what was kept; every step against the plain forms."""
    H, G, D, page, keep = 2, 4, 128, 16, 96
    lq = [150, 33, 260]
    g = torch.Generator(device="cuda").manual_seed(11)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    kp, vp, table, _ = P.pool(3, H, D, page, 20, BF, fill=float("nan"))
    pages = B.make_pages(kp, table)
    ws = B.alloc_paged_workspace(pages, G=G, mass=True)
    mass = torch.zeros(3 * H, pages.cap, device="cuda")
    q, k, v = (2 * rnd(sum(lq), H * G, D)).to(BF), rnd(sum(lq), H, D).to(BF), rnd(sum(lq), H, D).to(BF)
    cu = P.cumulated(lq)
    out, _ = B.fathom_prefill_attn(q, k, v, cu)
    o, _, tol, _ = P.prefill(q, k, v, lq, lq, D)
    assert bool(((out.double() - o).abs() <= tol).all())
    B.fathom_paged_append(pages, kp, vp, table, k, v, i32([0, 0, 0]), cu)
    lens = i32(lq)

    def step():
        B.fathom_paged_append(pages, kp, vp, table, rnd(3, H, D).to(BF), rnd(3, H, D).to(BF), lens)
        lens.add_(1)
        qd, before = 2 * rnd(3 * H, G, D), mass.clone()
        got = B.fathom_paged_attn(pages, qd, kp, vp, table, lens, ws, mass=mass)
        check_decode(got, qd, kp, vp, table, lens.tolist(), before, mass)

    for _ in range(3):
        step()
    want = [P.kept_set(mass[u].tolist(), lens.tolist()[u // H], keep, 4, 32) for u in range(3 * H)]
    kept, new, _ = B.fathom_paged_evict(pages, kp, vp, table, lens, mass, keep, table)     # in place
    assert new.tolist() == [96, 36, 96]
    assert [[i for i in row if i >= 0] for row in kept.tolist()] == want
    for s, n in enumerate(new.tolist()):      # the places behind the kept tokens start anew
        mass[s * H:(s + 1) * H, n:] = 0
    lens.copy_(new)
    for _ in range(2):
        step()


def test_contiguous_rows_are_pages_and_the_cut_back_rows_scan():
    """Rows [units][C][D] as pages: paged decode equals the dense decode, and after an eviction
    in place the rows go on through the bit-plane store, the plan, the scan and the sparse
    attention."""
    seqs, H, G, D, C, n, keep, k = 2, 2, 4, 128, 1024, 1000, 512, 256
    g = torch.Generator(device="cuda").manual_seed(2)
    kr, vr = (torch.randn(seqs * H, C, D, generator=g, device="cuda").to(BF) for _ in range(2))
    (kp, table), (vp, _) = B.rows_as_pages(kr, H), B.rows_as_pages(vr, H)
    pages = B.make_pages(kp, table)
    q, lens = query(seqs * H, G, D), i32([n, n])
    mass = torch.zeros(seqs * H, C, device="cuda")
    ws = B.alloc_paged_workspace(pages, G=G, mass=True)
    got = B.fathom_paged_attn(pages, q, kp, vp, table, lens, ws, mass=mass)
    full = B.make_shape(seqs * H, n, D, G, k, n_cap=C)
    want = B.fathom_dense_attn(full, kr, vr, q, B.alloc_workspace(full, B.WS_DENSE_ATTN))
    assert bool((B.fathom_rel_err(got, want) <= 2e-5).all())       # both fp32 throughout
    k0 = kr.clone()
    kept, _, _ = B.fathom_paged_evict(pages, kp, vp, table, lens, mass, keep, table)
    assert torch.equal(kr[:, :keep], torch.stack([k0[u, kept[u].long()] for u in range(seqs * H)]))
    cut = B.make_shape(seqs * H, keep, D, G, k, n_cap=C)
    planes, scales = B.fathom_quantize_pack(cut, kr)
    var = kr[:, :keep].float().var(1).contiguous()
    _, _, runs = B.fathom_plan(cut, q, var, i32([512] * seqs * H))          # every plane of every channel
    idx, _ = B.fathom_scan_topk(cut, planes, scales, runs, q, B.alloc_workspace(cut, B.WS_SCAN_TOPK))
    out = B.fathom_sparse_attn(cut, kr, vr, q, idx, B.alloc_workspace(cut, B.WS_SPARSE_ATTN))
    for u in range(seqs * H):
        x = q[u].double() @ kr[u, :keep].double().T / math.sqrt(D)
        for h in range(G):
            at = idx[u, h].long()
            w = torch.softmax(x[h, at], 0) @ vr[u, at].double()
            assert torch.linalg.norm(out[u, h].double() - w) <= 2e-3 * torch.linalg.norm(w)
