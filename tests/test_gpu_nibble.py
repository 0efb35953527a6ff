"""The 4-bit paged cache and the rotated append on the GPU, against plain 64-bit forms; the
tolerances are derived in nibble_cases."""
import math
import os
import subprocess
import sys

import pytest
import torch

from bit_plane_kv_gb300 import binding as B

import nibble_cases as N
import paged_cases as P

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def gen(seed=0):
    return torch.Generator(device="cuda").manual_seed(seed)


def rnd(*shape, seed=0):
    return torch.randn(*shape, generator=gen(seed), device="cuda")


def cache(seqs, H, D, page, per, seed=0, extra=0, scale_k=1.0, scale_v=1.0):
    """(kv_pages, page_table) of random rows."""
    count = seqs * per + extra
    k, v = rnd(count, H, page, D, seed=seed) * scale_k, rnd(count, H, page, D, seed=seed + 1) * scale_v
    order = torch.randperm(count, generator=gen(seed + 2), device="cuda").to(torch.int32)
    return N.pack(k, v), order[: seqs * per].reshape(seqs, per).contiguous()


def attend(q, kv, table, lens, ws=None, **kw):
    pages = B.make_nibble_pages(kv, table, q.shape[2])
    ws = B.alloc_nibble_workspace(pages, G=q.shape[1]) if ws is None else ws
    return B.fathom_nibble_attn(pages, q, kv, table, i32(lens) if isinstance(lens, list) else lens, ws, **kw)


def check_attend(out, lse, q, kv, table, lens):
    o, z, tol, tol_z = N.decode(q, *N.unpack(kv, q.shape[2]), table, lens)
    assert torch.isfinite(out).all()
    far = (out.double() - o).abs()
    assert bool((far <= tol).all()), f"worst {(far / tol.clamp(min=1e-300)).max().item():.3f} of the tolerance"
    empty = torch.isinf(z)
    assert bool((lse[empty] == -math.inf).all()) and bool(((lse.double() - z)[~empty].abs() <= tol_z[~empty]).all())


LENS = [1, 2, 15, 16, 17, 31, 63, 64, 65, 127, 128, 129, 500, 0, 1000]
ATTEND = {
    "G 4, page 16": (LENS, 2, 4, 128, 16),
    "G 1": (LENS, 3, 1, 128, 64),
    "G 8": (LENS, 2, 8, 128, 32),
    "G 8, 64 channels": (LENS, 2, 8, 64, 32),
    "G 2, 96 channels": (LENS, 2, 2, 96, 128),
    "G 3, 32 channels": ([1, 40, 7, 300], 1, 3, 32, 16),
    "G 5, 96 channels": ([300, 4], 2, 5, 96, 16),
    "G 6, page 256": ([300, 4, 256, 257], 1, 6, 128, 256),
    "G 7, 32 channels": ([100, 33], 1, 7, 32, 64),
    "one unit of many shares": ([40000], 1, 8, 128, 64),
    "one unit of many shares, 64 channels": ([51000], 1, 4, 64, 64),
    "few units of many shares": ([30000, 5, 0, 21000], 1, 4, 128, 16),
    "one token": ([1], 1, 1, 32, 16),
    "all idle": ([0, 0, 0], 2, 4, 128, 16),
    "long and short": ([9000, 3, 0, 700], 2, 4, 128, 64),
    "many units": ([(37 * i) % 90 for i in range(300)], 4, 4, 64, 16),
}


@pytest.mark.parametrize("name", list(ATTEND))
def test_attention_matches_the_plain_form(name):
    lens, H, G, D, page = ATTEND[name]
    kv, table = cache(len(lens), H, D, page, -(-max(max(lens), 1) // page))
    q = 2 * rnd(len(lens) * H, G, D, seed=5)
    out, lse = attend(q, kv, table, lens, want_lse=True)
    check_attend(out, lse, q, kv, table, lens)


def test_without_lse_the_result_is_the_same_and_empty_sequences_give_zero():
    kv, table = cache(3, 2, 64, 16, 4)
    q = rnd(6, 4, 64, seed=5)
    a = attend(q, kv, table, [50, 0, -5])
    b, z = attend(q, kv, table, [50, 0, -5], want_lse=True)
    assert torch.equal(a, b) and bool((a[2:] == 0).all()) and bool((z[2:] == -math.inf).all())


def test_lengths_beyond_the_table_are_cut():
    kv, table = cache(2, 1, 64, 16, 3)
    q = rnd(2, 4, 64, seed=5)
    assert torch.equal(attend(q, kv, table, [48, 48]), attend(q, kv, table, [49, 1 << 30]))


@pytest.mark.parametrize("scale", [0.0, 2.0 ** -70, 1e-6, 60.0])
def test_flat_tiny_and_sharp_queries(scale):
    kv, table = cache(2, 2, 128, 16, 40)
    q = rnd(4, 4, 128, seed=5) * scale
    out, lse = attend(q, kv, table, [513, 70], want_lse=True)
    check_attend(out, lse, q, kv, table, [513, 70])


def test_large_queries_meet_small_keys():
    kv, table = cache(2, 2, 128, 16, 40, scale_k=2.0 ** -13)
    q = rnd(4, 4, 128, seed=5) * 2.0 ** 13
    out, lse = attend(q, kv, table, [513, 70], want_lse=True)
    check_attend(out, lse, q, kv, table, [513, 70])


@pytest.mark.parametrize("power", [100, 115, 118, 123])
def test_huge_queries_choose_the_best_key(power):
    """Scores of 2^100 and more: one token has all the weight.  Channels of q are +-2^power, so scores are 2^power
    times sums of keys, whose differences are far above 2^-100."""
    kv, table = cache(1, 2, 64, 16, 40, scale_k=2.0 ** -3)
    q = rnd(2, 4, 64, seed=5).sign() * 2.0 ** power
    K, V = N.unpack(kv, 64)
    out, lse = attend(q, kv, table, [600], want_lse=True)
    for u in range(2):
        kk, vv = (x[table[0].long(), u].reshape(-1, 64)[:600] for x in (K, V))
        x = q[u].double() @ kk.T
        top = x.topk(2, 1)
        assert bool((top.values[:, 0] - top.values[:, 1] > 2.0 ** (power - 20)).all())
        # one weight of 1: its two pieces and the value, 2^-21
        assert bool(((out[u].double() - vv[top.indices[:, 0]]).abs() <= 2.0 ** -20 * vv[top.indices[:, 0]].abs()).all())
        if power < 115:
            assert bool(((lse[u].double() - top.values[:, 0] / 8).abs() <= 2.0 ** -20 * x.abs().amax(1) / 8).all())


def test_channels_of_very_different_sizes():
    q = 2 * rnd(4, 4, 128, seed=5)
    q[..., ::3] *= 2.0 ** -14
    q[..., 5] *= 64
    kv, table = cache(2, 2, 128, 16, 40)
    out, lse = attend(q, kv, table, [513, 70], want_lse=True)
    check_attend(out, lse, q, kv, table, [513, 70])


@pytest.mark.parametrize("kind", ["tiny", "subnormal", "largest", "growing", "falling", "zero", "mixed"])
def test_scales_of_values_over_the_whole_range(kind):
    n, page, D = 700, 16, 128
    per = -(-n // page)
    k, v = rnd(per, 1, page, D), rnd(per, 1, page, D, seed=1)
    at = torch.arange(per, device="cuda").double()[:, None, None, None] / per
    size = {"tiny": 2.0 ** -13, "subnormal": 2.0 ** -21, "largest": 20000.0, "growing": 2.0 ** (-14 + 28 * at),
            "falling": 2.0 ** (14 - 28 * at), "zero": 0.0,
            "mixed": 2.0 ** torch.randint(-14, 14, (per, 1, page, 1), generator=gen(3), device="cuda").double()}[kind]
    kv = N.pack(k, v.double() * size)
    table = torch.arange(per, dtype=torch.int32, device="cuda")[None].contiguous()
    q = rnd(1, 4, D, seed=5)
    out, lse = attend(q, kv, table, [n], want_lse=True)
    check_attend(out, lse, q, kv, table, [n])


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_places_behind_the_length_and_unnamed_pages_are_never_read(bad):
    lens, page, D = [70, 16, 1], 16, 128
    kv, table = cache(3, 2, D, page, 8, extra=4)
    q = rnd(6, 4, D, seed=5)
    want = attend(q, kv, table, lens).clone()
    x = kv.view(kv.shape[0], 2, 1, 18 * D)
    live = torch.zeros(kv.shape[0], 16, dtype=torch.bool, device="cuda")
    for s, n in enumerate(lens):
        for i in range(n):
            live[int(table[s, i // page]), i % page] = True
    dead = ~live
    bits = torch.tensor([bad], dtype=FP, device="cuda").view(torch.uint8)
    for base in (8 * D, 17 * D):                                            # scales [8][4][2] of tokens r, r + 8
        sc = x[..., base:base + D].reshape(kv.shape[0], 2, 8, 4, 2, 2)
        hit = dead.reshape(-1, 2, 8).transpose(1, 2)[:, None, :, None, :, None].expand_as(sc)
        x[..., base:base + D] = torch.where(hit, bits, sc).reshape(kv.shape[0], 2, 1, D)
    assert torch.equal(attend(q, kv, table, lens), want)


def test_bad_page_numbers_are_skipped():
    lens, page = [200, 90], 16
    kv, table = cache(2, 2, 64, page, 13)
    table[0, 3], table[0, 12], table[1, 0] = -1, kv.shape[0], 1 << 30
    q = rnd(4, 4, 64, seed=5)
    out, lse = attend(q, kv, table, lens, want_lse=True)
    check_attend(out, lse, q, kv, table, lens)
    table[1] = -7
    out, lse = attend(q, kv, table, lens, want_lse=True)
    check_attend(out, lse, q, kv, table, lens)
    assert bool((out[2:] == 0).all())


def test_nan_stays_with_what_depends_on_it():
    page, D, lens = 16, 128, [5000, 300]
    kv, table = cache(2, 2, D, page, 313)
    q = 2 * rnd(4, 4, D, seed=5)
    want = attend(q, kv, table, lens).clone()
    p = q.clone()
    p[0, 1, 7] = float("nan")                              # a query: its head
    got = attend(p, kv, table, lens)
    assert torch.isnan(got[0, 1]).all()
    got[0, 1] = want[0, 1]
    assert torch.equal(got, want)
    for part, what in ((0, "k"), (9 * D, "v")):            # token 3003 of unit 1, group 2
        x = kv.clone()
        at = part + 8 * D + 4 * ((3003 % 8) * 4 + 2) + 2 * (3003 % 16 // 8)
        x[int(table[0, 3003 // page]), 1, at:at + 2] = torch.tensor([float("nan")], dtype=FP, device="cuda").view(torch.uint8)
        got = attend(q, x, table, lens)
        if what == "k":
            assert torch.isnan(got[1]).all()
        else:
            assert torch.isnan(got[1, :, 64:96]).all() and torch.equal(got[1, :, :64], want[1, :, :64])
            assert torch.equal(got[1, :, 96:], want[1, :, 96:])
        got[1] = want[1]
        assert torch.equal(got, want)


def test_pages_may_be_strided_and_shared():
    lens, H, D, page = [100, 77], 3, 64, 32
    kv, table = cache(2, H, D, page, 4)
    table[1, 0] = table[0, 0]
    q = rnd(6, 4, D, seed=5)
    want = attend(q, kv, table, lens)
    heads_first = kv.transpose(0, 1).contiguous().transpose(0, 1)
    padded = torch.zeros(kv.shape[0], H + 2, kv.shape[2] + 48, dtype=torch.uint8, device="cuda")[:, 1:H + 1, 16:kv.shape[2] + 16]
    padded.copy_(kv)
    for x in (heads_first, padded):
        assert torch.equal(attend(q, x, table, lens), want)


def test_offsets_beyond_32_bits():
    """Pages 2^31 and 2^32 bytes behind the first one."""
    D, page = 128, 16
    kv, table = cache(1, 1, D, page, 5)
    q = rnd(1, 4, D, seed=5)
    want = attend(q, kv, table, [75])
    stride = (1 << 30) + 16
    big = torch.empty(4 * stride + kv.shape[2], dtype=torch.uint8, device="cuda").as_strided((5, 1, kv.shape[2]), (stride, 16, 1))
    big.copy_(kv)
    assert torch.equal(attend(q, big, table, [75]), want)
    k, v = B.fathom_nibble_read(B.make_nibble_pages(big, table, D), big, table, i32([0]), i32([0, 75]), 75, dtype=torch.float32)
    k2, v2 = B.fathom_nibble_read(B.make_nibble_pages(kv, table, D), kv, table, i32([0]), i32([0, 75]), 75, dtype=torch.float32)
    assert torch.equal(k, k2) and torch.equal(v, v2)
    B.fathom_nibble_append(B.make_nibble_pages(big, table, D), big, table, k[:75].to(FP), v[:75].to(FP), i32([0]), i32([0, 75]))
    B.fathom_nibble_append(B.make_nibble_pages(kv, table, D), kv, table, k[:75].to(FP), v[:75].to(FP), i32([0]), i32([0, 75]))
    assert torch.equal(big.contiguous(), kv)


def test_a_page_of_sixteen_million_tokens():
    """Places more than 2^31 bytes into a page: all tokens zero but the last 50."""
    D, page, last = 128, 1 << 24, 50
    kv, table = B.alloc_nibble_pages(1, 1, page, D), i32([[0]])
    pages = B.make_nibble_pages(kv, table, D)
    k, v = 3 * rnd(last, 1, D).to(BF), rnd(last, 1, D, seed=1).to(BF)
    start, cu = i32([page - last]), i32([0, last])
    B.fathom_nibble_append(pages, kv, table, k, v, start, cu)
    K, V = B.fathom_nibble_read(pages, kv, table, start, cu, last, dtype=torch.float32)
    assert torch.equal(K.double(), N.held(k.double())[0]) and torch.equal(V.double(), N.held(v.double())[0])
    q = 4 * rnd(1, 2, D, seed=5)
    out, lse = attend(q, kv, table, [page], want_lse=True)
    x = q[0].double() @ K[:, 0].double().T / math.sqrt(D)
    z = torch.logaddexp(torch.logsumexp(x, 1), torch.full((2,), math.log(page - last), device="cuda").double())
    w = torch.exp(x - z[:, None])
    # the scores of the zeros are exact; their sum of 2^24 / 608 / 64 additions per lane loses 432 * 2^-24 at most
    S = (q[0].double().abs() @ K[:, 0].double().abs().T / math.sqrt(D)).amax(1)
    tol = 2.0 ** -14 + 16 * 2.0 ** -24 * S + 2.0 ** -20 * S
    assert bool(((lse[0].double() - z).abs() <= tol).all())
    assert bool(((out[0].double() - w @ V[:, 0].double()).abs() <= 3 * tol[:, None] * (w @ V[:, 0].double().abs())).all())


def test_one_workspace_serves_calls_of_different_sizes():
    calls = []
    for lens, H, G, D in (([9000, 5], 2, 8, 128), ([40] * 300, 4, 1, 32), ([30000], 1, 4, 64), ([70, 0], 1, 5, 96)):
        kv, table = cache(len(lens), H, D, 16, -(-max(lens) // 16))
        calls.append((2 * rnd(len(lens) * H, G, D, seed=5), kv, table, lens))
    ws = B.alloc_nibble_workspace(B.make_nibble_pages(calls[0][1], calls[0][2], 128), G=8)
    want = [attend(*c) for c in calls]
    for i in (0, 1, 2, 3, 2, 0, 3, 1, 0):
        assert torch.equal(attend(*calls[i], ws=ws), want[i])


def test_the_same_bits_every_time_on_any_stream_and_in_a_graph():
    lens = [20000, 3, 800]
    kv, table = cache(3, 2, 128, 64, 313)
    q, n = 2 * rnd(6, 4, 128, seed=5), i32(lens)
    pages = B.make_nibble_pages(kv, table, 128)
    ws = [B.alloc_nibble_workspace(pages) for _ in range(2)]
    want, z = B.fathom_nibble_attn(pages, q, kv, table, n, ws[0], want_lse=True)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [B.fathom_nibble_attn(pages, q, kv, table, n, ws[i % 2], stream=streams[i % 2]) for i in range(20)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for x in got)
    out, lse, g = torch.empty_like(want), torch.empty_like(z), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.fathom_nibble_attn(pages, q, kv, table, n, ws[0], out=out, lse=lse)
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, z)
    n.copy_(i32([64, 0, 19999]))
    q.mul_(-1)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, attend(q, kv, table, [64, 0, 19999]))


# ------------------------------------------------------------------ appends
#: name: (D, rotated channels, pairs, type, page, KV heads, query heads, tokens of each sequence, cached before)
APPEND = {
    "halves": (128, 128, False, BF, 16, 8, 32, [1, 17, 40, 0, 3], [0, 5, 16, 2, 61]),
    "halves, fp16": (128, 128, False, FP, 64, 2, 2, [100, 1], [3, 64]),
    "pairs": (128, 128, True, BF, 16, 2, 6, [33, 20], [0, 7]),
    "part of the channels": (96, 48, False, BF, 16, 3, 3, [20, 2], [1, 0]),
    "part, pairs": (96, 52, True, FP, 32, 1, 4, [20, 2], [1, 40]),
    "halves that no vector fits": (64, 36, False, BF, 16, 2, 2, [20, 2], [1, 9]),
    "two channels": (64, 2, False, FP, 16, 1, 1, [9], [0]),
    "two channels, pairs": (32, 2, True, BF, 16, 5, 5, [9, 31], [0, 1]),
    "32 channels": (32, 32, False, BF, 128, 2, 2, [200, 1], [100, 0]),
    "many sequences": (64, 64, False, BF, 16, 1, 1, [(7 * i) % 5 for i in range(200)], [(3 * i) % 40 for i in range(200)]),
}


def new_rows(name, seed=0):
    D, R, pairs, dt, page, H, Hq, new, old = APPEND[name]
    qkv = rnd(sum(new), Hq + 2 * H, D, seed=seed).to(dt)
    pos = torch.cat([torch.arange(a, a + b) for a, b in zip(old, new)]).cuda()
    seq = torch.repeat_interleave(torch.arange(len(new)), torch.tensor(new)).cuda()
    table = N.rope_table(300, R)
    return qkv[:, :Hq], qkv[:, Hq:Hq + H], qkv[:, Hq + H:], pos, seq, table


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("name", list(APPEND))
def test_rotated_append_matches_the_plain_form(name, f32):
    D, R, pairs, dt, page, H, Hq, new, old = APPEND[name]
    q, k, v, pos, seq, rope = new_rows(name)
    per = -(-max(a + b for a, b in zip(old, new)) // page)
    kp, vp, table, _ = P.pool(len(new), H, D, page, per, dt, seed=3)
    k0, v0 = kp.clone(), vp.clone()
    _, _, qr = B.fathom_paged_append_rope(B.make_pages(kp, table), kp, vp, table, k, v, i32(old), rope, P.cumulated(new),
                                          interleaved=pairs, q=q, q_dtype=torch.float32 if f32 else None)
    at, slot = table[seq, pos // page].long(), pos % page
    assert N.near_rotated(kp[at, :, slot], k, rope, pos, pairs)
    assert torch.equal(kp[at, :, slot][..., R:], k[..., R:])
    v0[at, :, slot] = v
    assert torch.equal(vp, v0)
    k0[at, :, slot] = kp[at, :, slot]
    assert torch.equal(kp, k0)                                   # nothing else was written
    assert qr.dtype == (torch.float32 if f32 else dt) and N.near_rotated(qr, q, rope, pos, pairs)
    assert f32 or torch.equal(qr[..., R:], q[..., R:])


@pytest.mark.parametrize("rotate", [True, False])
@pytest.mark.parametrize("name", list(APPEND))
def test_4_bit_append_holds_the_exact_codes(name, rotate):
    D, R, pairs, dt, page, H, Hq, new, old = APPEND[name]
    q, k, v, pos, seq, rope = new_rows(name)
    per = -(-max(a + b for a, b in zip(old, new)) // page)
    kv, table = cache(len(new), H, D, page, per, seed=3)
    want_k, want_v = N.unpack(kv, D)
    pages, cu = B.make_nibble_pages(kv, table, D), P.cumulated(new)
    kw = dict(rope=rope, interleaved=pairs, q=q, q_dtype=torch.float32) if rotate else {}
    _, qr = B.fathom_nibble_append(pages, kv, table, k, v, i32(old), cu, **kw)
    at, slot = table[seq, pos // page].long(), pos % page
    y = N.rotated(k, rope, pos, pairs) if rotate else k.double()
    want_k[at, :, slot], want_v[at, :, slot] = N.held(y)[0], N.held(v.double())[0]
    got = N.unpack(kv, D)
    assert torch.equal(got[0], want_k) and torch.equal(got[1], want_v)
    if rotate:
        assert N.near_rotated(qr, q, rope, pos, pairs)
    else:
        assert qr is None
    for t in (torch.float32, BF, FP):                            # and read back
        a, b = B.fathom_nibble_read(pages, kv, table, i32(old), cu, sum(new), dtype=t)
        assert torch.equal(a, want_k[at, :, slot].float().to(t)) and torch.equal(b, want_v[at, :, slot].float().to(t))


@pytest.mark.parametrize("dt,table", [(BF, "angles"), (FP, "angles"), (BF, "quarters"), (FP, "any")])
def test_codes_of_many_rotated_keys_are_exact(dt, table):
    """Millions of them: a code taken from a key rounded to fp32 would differ here and there.  Quarter turns put
    keys on borders; a table may also hold numbers that are no cos and sin."""
    T, H, D = 6000, 4, 128
    k, v = rnd(T, H, D).to(dt), rnd(T, H, D, seed=1).to(dt)
    rope = N.rope_table(T, D)
    if table == "quarters":
        turns = torch.arange(T * 64, device="cuda").reshape(T, 64) % 4
        rope = torch.cat([torch.tensor([1.0, 0.0, -1.0, 0.0], device="cuda")[turns],
                          torch.tensor([0.0, 1.0, 0.0, -1.0], device="cuda")[turns]], 1)
    elif table == "any":
        rope = 3 * rnd(T, D, seed=2)
    kv, table = B.alloc_nibble_pages(-(-T // 64), H, 64, D), torch.arange(-(-T // 64), dtype=torch.int32, device="cuda")[None].contiguous()
    B.fathom_nibble_append(B.make_nibble_pages(kv, table, D), kv, table, k, v, i32([0]), i32([0, T]), rope=rope)
    K, V = N.unpack(kv, D)
    pos = torch.arange(T, device="cuda")
    want = N.held(N.rotated(k, rope, pos, False))[0]   # the products are exact in fp64, their sum to 2^-53
    assert torch.equal(K.transpose(1, 2).reshape(-1, H, D)[:T], want)
    assert torch.equal(V.transpose(1, 2).reshape(-1, H, D)[:T], N.held(v.double())[0])


@pytest.mark.parametrize("D", [32, 96, 128])
@pytest.mark.parametrize("dt", [BF, FP])
def test_codes_of_small_and_large_rows_are_exact(dt, D):
    """Rows from far below fp16's smallest number to beyond its largest, where the ways of coding change."""
    sizes = [2.0 ** e for e in (-27, -25, -24, -20, -15, -14, -13, -12, -11, 0, 13, 14, 15)] + ([2.0 ** 16, 2.0 ** 60] if dt == BF else [])
    T, H = 40 * len(sizes), 2
    size = torch.tensor(sizes, device="cuda").repeat_interleave(40)[:, None, None]
    k, v = ((rnd(T, H, D, seed=i) * size).clamp(-6e4, 6e4).to(dt) if dt == FP else (rnd(T, H, D, seed=i) * size).to(dt) for i in (0, 1))
    pages = -(-T // 16)
    kv, table = B.alloc_nibble_pages(pages, H, 16, D), torch.arange(pages, dtype=torch.int32, device="cuda")[None].contiguous()
    rope, pos = N.rope_table(T, D), torch.arange(T, device="cuda")
    B.fathom_nibble_append(B.make_nibble_pages(kv, table, D), kv, table, k, v, i32([0]), i32([0, T]), rope=rope)
    K, V = N.unpack(kv, D)
    assert torch.equal(K.transpose(1, 2).reshape(-1, H, D)[:T], N.held(N.rotated(k, rope, pos, False))[0])
    assert torch.equal(V.transpose(1, 2).reshape(-1, H, D)[:T], N.held(v.double())[0])


@pytest.mark.parametrize("dt", [BF, FP])
def test_values_on_borders_zeros_infinities_and_nan(dt):
    D = 64
    x = torch.zeros(9, 2, D, dtype=dt, device="cuda")
    x[0, 0, :32] = torch.arange(-16, 16, device="cuda").to(dt) / 2           # halves of a step, a = 8
    x[1, 0, :32] = torch.arange(-16, 16, device="cuda").to(dt) / 16
    x[2, 0, 3], x[2, 1, 40] = 1.0, -1.0                                      # a single value, the rest on a border
    x[3] = -0.0
    x[4, 0, 5], x[4, 1, 63] = float("nan"), -float("nan")
    x[5, 0, 5], x[5, 1, 63] = float("inf"), -float("inf")
    x[6] = torch.finfo(dt).tiny
    x[7] = 60000.0
    x[7, 1] *= -1
    if dt == BF:
        x[8, 0], x[8, 1] = 1e30, 1e-30
    kv, table = B.alloc_nibble_pages(2, 2, 16, D), i32([[1]])
    pages = B.make_nibble_pages(kv, table, D)
    B.fathom_nibble_append(pages, kv, table, x, x, i32([2]), i32([0, 9]))
    k, v = B.fathom_nibble_read(pages, kv, table, i32([2]), i32([0, 9]), 9, dtype=torch.float32)
    want = N.held(torch.nan_to_num(x.double(), nan=0.0, posinf=1e6, neginf=-1e6))[0]
    want[4, 0, :32] = want[4, 1, 32:] = float("nan")
    for got in (k, v):
        assert torch.equal(torch.nan_to_num(got, nan=7e7).double(), torch.nan_to_num(want, nan=7e7))


def test_rotated_rows_keep_infinities_and_nan():
    D = 64
    k = torch.ones(4, 1, D, dtype=BF, device="cuda")
    k[0, 0, 3], k[1, 0, 3], k[2, 0, 60] = float("inf"), float("nan"), -float("inf")
    rope = N.rope_table(10, D)
    rope[:, 32 + 3] = 0.5
    kp, vp, table, _ = P.pool(1, 1, D, 16, 1, BF)
    B.fathom_paged_append_rope(B.make_pages(kp, table), kp, vp, table, k, k, i32([2]), rope, i32([0, 4]))
    want = N.rotated(k, rope, torch.arange(2, 6, device="cuda"), False).float()
    got = kp[int(table[0, 0]), 0, 2:6].float()[:, None]
    for f in (torch.isnan, torch.isposinf, torch.isneginf):
        assert torch.equal(f(got), f(want))


def test_decode_steps_take_one_token_per_sequence_and_other_positions():
    S, H, D, page = 5, 2, 128, 16
    kv, table = cache(S, H, D, page, 4)
    rope = N.rope_table(1000, D)
    qkv = rnd(S, 8 + 2 * H, D, seed=9).to(BF)
    q, k, v = qkv[:, :8], qkv[:, 8:10], qkv[:, 10:]
    start, positions = i32([0, 15, 16, 63, 30]), i32([999, 0, 500, 7, 30])
    K, V = N.unpack(kv, D)
    kp, vp, t16, _ = P.pool(S, H, D, page, 4, BF)
    _, qr = B.fathom_nibble_append(B.make_nibble_pages(kv, table, D), kv, table, k, v, start, rope=rope, positions=positions,
                                   q=q, q_dtype=torch.float32)
    out = torch.zeros(S, 8, D, device="cuda")
    B.fathom_paged_append_rope(B.make_pages(kp, t16), kp, vp, t16, k, v, start, rope, positions=positions, q=q, q_out=out)
    assert torch.equal(out, qr)
    y, s = N.rotated(k, rope, positions.long(), False), torch.arange(S, device="cuda")
    at, slot = table[s, start.long() // page].long(), start.long() % page
    K[at, :, slot], V[at, :, slot] = N.held(y)[0], N.held(v.double())[0]
    got = N.unpack(kv, D)
    assert torch.equal(got[0], K) and torch.equal(got[1], V)
    assert N.near_rotated(kp[t16[s, start.long() // page].long(), :, slot], k, rope, positions.long(), False)


def test_tokens_without_a_place_are_skipped():
    H, D, page = 2, 64, 16
    kv, table = cache(3, H, D, page, 2)
    kp, vp, t16, _ = P.pool(3, H, D, page, 2, BF)
    bad = i32([[int(table[0, 0]), -1], [1 << 30, int(table[1, 1])], [int(table[2, 0]), int(table[2, 1])]])
    q, k, v = rnd(60, 4, D).to(BF), rnd(60, H, D, seed=1).to(BF), rnd(60, H, D, seed=2).to(BF)
    rope = N.rope_table(25, D)
    start, cu = i32([10, 10, -3]), i32([0, 20, 40, 55])            # 5 tokens behind the last sequence
    seq = torch.repeat_interleave(torch.arange(3), torch.tensor([20, 20, 15])).cuda()
    pos = (start[seq] + torch.arange(55, device="cuda") - cu[seq]).long()
    turned = (pos >= 0) & (pos < 25)
    K, V = N.unpack(kv, D)
    pages = B.make_nibble_pages(kv, bad, D)
    qo = torch.full((60, 4, D), 7.0, device="cuda")
    B.fathom_nibble_append(pages, kv, bad, k, v, start, cu, rope=rope, q=q, q_out=qo)
    page_of = bad[seq, (pos // page).clamp(0, 1)].long()
    ok = turned & (page_of >= 0) & (page_of < kv.shape[0])
    at, slot = page_of[ok], pos[ok] % page
    y = N.rotated(k[:55], rope, pos.clamp(0, 24), False)
    K[at, :, slot], V[at, :, slot] = N.held(y[ok])[0], N.held(v[:55][ok].double())[0]
    got = N.unpack(kv, D)
    assert torch.equal(got[0], K) and torch.equal(got[1], V)
    assert bool((qo[:55][~turned] == 7).all()) and bool((qo[55:] == 7).all()) and not bool((qo[:55][turned] == 7).all(-1).any())
    # without a rotation the positions count only where they name a place
    B.fathom_nibble_append(pages, kv, bad, k, v, start, cu)
    inside = (pos >= 0) & (pos < 32) & (page_of >= 0) & (page_of < kv.shape[0])
    K[page_of[inside], :, pos[inside] % page] = N.held(k[:55][inside].double())[0]
    assert torch.equal(N.unpack(kv, D)[0], K)
    # read back: the others' rows are left as they were
    a = torch.full((60, H, D), 9.0, device="cuda")
    b = a.clone()
    B.fathom_nibble_read(pages, kv, bad, start, cu, 60, k_out=a, v_out=b)
    assert torch.equal(a[:55][inside].double(), K[page_of[inside], :, pos[inside] % page])
    assert bool((a[:55][~inside] == 9).all()) and bool((a[55:] == 9).all()) and bool((b[55:] == 9).all())
    # 16-bit rows: the same tokens
    t16[0, 1], t16[1, 0] = -1, 1 << 30
    k0 = kp.clone()
    B.fathom_paged_append_rope(B.make_pages(kp, t16), kp, vp, t16, k, v, start, rope, cu)
    p16 = t16[seq, (pos // page).clamp(0, 1)].long()
    ok = turned & (p16 >= 0) & (p16 < kp.shape[0])
    assert N.near_rotated(kp[p16[ok], :, pos[ok] % page], k[:55][ok], rope, pos[ok], False)
    k0[p16[ok], :, pos[ok] % page] = kp[p16[ok], :, pos[ok] % page]
    assert torch.equal(kp, k0)


def test_reading_a_part_into_strided_rows():
    lens, H, D, page = [150, 90, 0], 3, 96, 32
    kv, table = cache(3, H, D, page, 5)
    K, V = N.unpack(kv, D)
    first, part = [40, 0, 0], [100, 90, 0]
    both = torch.zeros(190, 2 * H, D, dtype=BF, device="cuda")
    B.fathom_nibble_read(B.make_nibble_pages(kv, table, D), kv, table, i32(first), P.cumulated(part), 190, k_out=both[:, :H],
                         v_out=both[:, H:])
    at = 0
    for s in range(3):
        pos = torch.arange(first[s], first[s] + part[s], device="cuda")
        for x, y in ((K, both[:, :H]), (V, both[:, H:])):
            assert torch.equal(y[at:at + part[s]], x[table[s, pos // page].long(), :, pos % page].to(BF))
        at += part[s]


def test_appends_and_reads_captured_by_a_process_that_has_not_made_them():
    code = """
import sys
sys.path.insert(0, %r); sys.path.insert(0, %r)
import torch
from bit_plane_kv_gb300 import binding as B
import nibble_cases as N, paged_cases as P
H, D, S = 2, 128, 3
kv = B.alloc_nibble_pages(30, H, 16, D)
table = torch.arange(30, dtype=torch.int32, device="cuda").reshape(3, 10).contiguous()
kp, vp, t16, _ = P.pool(3, H, D, 16, 10, torch.bfloat16)
pages, p16 = B.make_nibble_pages(kv, table, D), B.make_pages(kp, t16)
ws = B.alloc_nibble_workspace(pages, G=4)
qkv = torch.randn(40, 12, D, device="cuda").bfloat16()
rope = N.rope_table(200, D)
start, cu, lens = torch.tensor([0, 7, 30], dtype=torch.int32, device="cuda"), P.cumulated([20, 5, 15]), torch.tensor([20, 12, 45], dtype=torch.int32, device="cuda")

def calls():
    _, q1 = B.fathom_nibble_append(pages, kv, table, qkv[:, 8:10], qkv[:, 10:], start, cu, rope=rope, q=qkv[:, :8], q_dtype=torch.float32)
    k, v = B.fathom_nibble_read(pages, kv, table, start, cu, 40)
    _, _, q2 = B.fathom_paged_append_rope(p16, kp, vp, t16, qkv[:, 8:10], qkv[:, 10:], start, rope, cu, q=qkv[:, :8], q_dtype=torch.float32)
    o, z = B.fathom_nibble_attn(pages, q1[:3].reshape(S * H, 4, D).contiguous(), kv, table, lens, ws, want_lse=True)
    return q1, k, v, q2, o, z, kv, kp, vp

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
print("same")
""" % (os.path.dirname(os.path.dirname(os.path.abspath(__file__))), os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "same", r.stdout + r.stderr[-2000:]


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("D,G,page", [(128, 4, 16), (64, 8, 32)])
def test_prompt_in_chunks_then_decode_steps(D, G, page):
    """A serving loop over a 4-bit cache: a prompt in two chunks (each appended, the cache's rows read back for
    the prompt attention of the second), then decode steps; against the plain forms on the values held."""
    H, S = 2, 2
    chunks = [[150, 33], [60, 41]]
    rope = N.rope_table(400, D)
    kv, table = cache(S, H, D, page, 256 // page, seed=7)
    pages = B.make_nibble_pages(kv, table, D)
    ws = B.alloc_nibble_workspace(pages, G=G)
    K, V = N.unpack(kv, D)
    have = [0, 0]
    for seed, new in enumerate(chunks):
        qkv = rnd(sum(new), H * G + 2 * H, D, seed=20 + seed).to(BF)
        q, k, v = qkv[:, :H * G], qkv[:, H * G:H * G + H], qkv[:, H * G + H:]
        start, cu = i32(have), P.cumulated(new)
        _, qr = B.fathom_nibble_append(pages, kv, table, k, v, start, cu, rope=rope, q=q)
        at = 0
        for s in range(S):
            pos = torch.arange(have[s], have[s] + new[s], device="cuda")
            p, slot = table[s, pos // page].long(), pos % page
            K[p, :, slot] = N.held(N.rotated(k[at:at + new[s]], rope, pos, False))[0]
            V[p, :, slot] = N.held(v[at:at + new[s]].double())[0]
            at += new[s]
        have = [a + b for a, b in zip(have, new)]
        cu_k = P.cumulated(have)
        kr, vr = B.fathom_nibble_read(pages, kv, table, i32([0, 0]), cu_k, sum(have))
        out, _ = B.fathom_prefill_attn(qr, kr, vr, cu, cu_k)
        o, _, tol, _ = P.prefill(qr, kr, vr, new, have, D)
        assert bool(((out.double() - o).abs() <= tol).all())
    lens = i32(have)
    for step in range(3):
        qkv = rnd(S, H * G + 2 * H, D, seed=40 + step).to(BF)
        k, v = qkv[:, H * G:H * G + H], qkv[:, H * G + H:]
        _, qr = B.fathom_nibble_append(pages, kv, table, k, v, lens, rope=rope, q=qkv[:, :H * G], q_dtype=torch.float32)
        pos, s = lens.long(), torch.arange(S, device="cuda")
        p, slot = table[s, pos // page].long(), pos % page
        K[p, :, slot] = N.held(N.rotated(k, rope, pos, False))[0]
        V[p, :, slot] = N.held(v.double())[0]
        lens.add_(1)
        q = qr.reshape(S * H, G, D)
        out, lse = B.fathom_nibble_attn(pages, q, kv, table, lens, ws, want_lse=True)
        o, z, tol, tol_z = N.decode(q, K, V, table, lens)
        assert bool(((out.double() - o).abs() <= tol).all()) and bool(((lse.double() - z).abs() <= tol_z).all())


def test_parts_of_a_sequence_join_by_their_log_sum_exps():
    """The first 160 tokens and the last 140 apart, weighed by exp(lse), as a caller does who keeps recent tokens
    elsewhere."""
    lens, H, D, page = [300], 2, 128, 16
    kv, table = cache(1, H, D, page, 19)
    q = rnd(2, 4, D, seed=5)
    whole, z = attend(q, kv, table, lens, want_lse=True)
    a, za = attend(q, kv, table[:, :10].contiguous(), [160], want_lse=True)
    b, zb = attend(q, kv, table[:, 10:].contiguous(), [140], want_lse=True)
    m = torch.logaddexp(za, zb)
    got = a * (za - m).exp()[..., None] + b * (zb - m).exp()[..., None]
    _, _, tol, tol_z = N.decode(q, *N.unpack(kv, D), table, lens)
    o = N.decode(q, *N.unpack(kv, D), table, lens)[0]
    assert bool(((m - z).abs() <= 2 * tol_z).all())
    # each part within its own tolerance, its factor within that of its log-sum-exp and two fp32 roundings
    A = N.decode(q, N.unpack(kv, D)[0], N.unpack(kv, D)[1].abs(), table, lens)[0]
    assert bool(((got.double() - o).abs() <= 2 * tol + (4 * tol_z + 2.0 ** -20)[..., None] * A).all())
    assert bool(((whole.double() - o).abs() <= tol).all())
