"""Causal attention of packed prompts on the GPU against the plain 64-bit form;
the tolerances are derived in paged_cases."""
import math
import os
import subprocess
import sys

import pytest
import torch

from bit_plane_kv_gb300 import binding as B

import paged_cases as P

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


def inputs(lq, lk, H, Hkv, D, dtype, seed=0, q_scale=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = (q_scale * torch.randn(sum(lq), H, D, generator=g, device="cuda")).to(dtype)
    k = torch.randn(sum(lk), Hkv, D, generator=g, device="cuda").to(dtype)
    v = torch.randn(sum(lk), Hkv, D, generator=g, device="cuda").to(dtype)
    return q, k, v


def check(out, lse, q, k, v, lq, lk):
    o, z, tol, tol_z = P.prefill(q, k, v, lq, lk, q.shape[2])
    assert torch.isfinite(out).all()
    far = (out.double() - o).abs()
    assert bool((far <= tol).all()), f"out: worst {(far / tol.clamp(min=1e-30)).max().item():.3f} of the tolerance"
    none = torch.isinf(z)
    assert torch.equal(torch.isinf(lse) & (lse < 0), none)
    far = (lse.double() - z)[~none].abs()
    assert bool((far <= tol_z[~none]).all())


SAME = [1, 2, 31, 63, 64, 65, 127, 128, 129, 257, 300]
CASES = {
    "whole prompts, G 4": (SAME, SAME, 8, 2, 128, BF),
    "whole prompts, one head, fp16": (SAME, SAME, 1, 1, 128, FP),
    "G 8, 64 channels": (SAME, SAME, 16, 2, 64, FP),
    "G 2, 96 channels": (SAME, SAME, 6, 3, 96, BF),
    "G 3": ([40, 200, 129], [40, 200, 129], 6, 2, 64, BF),
    "G 6, 72 channels": ([130, 7], [130, 7], 12, 2, 72, FP),
    "G 16, 8 channels": ([130, 7], [130, 7], 16, 1, 8, BF),
    "G 7": ([50], [50], 7, 1, 128, BF),
    "chunks": ([5, 128, 1, 300, 64], [300, 1000, 129, 301, 64], 8, 2, 128, BF),
    "chunks, fp16": ([1, 17, 250], [700, 513, 256], 4, 4, 128, FP),
    "empty rows and sequences": ([0, 10, 4, 0, 130, 3], [0, 0, 2, 50, 100, 3], 8, 2, 128, BF),
    "one token": ([1], [1], 1, 1, 8, FP),
    "long": ([1500], [1500], 4, 1, 128, BF),
    "128 heads on one": ([3, 130], [3, 140], 128, 1, 64, BF),
    "160 heads on one": ([9], [70], 160, 1, 72, FP),
    "many sequences": ([1 + i % 5 for i in range(100)], [1 + i % 5 + 3 * (i % 7) for i in range(100)], 4, 2, 64, BF),
    # few rows and many keys: clusters of CTAs share the keys (2, 4 and 8 of them; shares that a row does not reach)
    "few rows, 8 shares": ([3, 1, 40], [5000, 9, 41], 2, 1, 128, BF),
    "few rows, 8 shares, fp16": ([1, 16], [300, 6000], 8, 2, 128, FP),
    "few rows, 4 shares": ([7], [3000], 8, 4, 96, FP),
    "few rows, 4 shares, whole prompt": ([2100], [2100], 2, 2, 64, BF),
    "few rows, 2 shares": ([130, 3], [1500, 2], 4, 1, 64, FP),
    "few rows, odd channels": ([5], [4500], 3, 1, 72, BF),
    "few rows, some see nothing": ([60, 9], [50, 5000], 4, 1, 128, BF),
}


@pytest.mark.parametrize("name", list(CASES))
def test_prefill_matches_the_plain_form(name):
    lq, lk, H, Hkv, D, dt = CASES[name]
    q, k, v = inputs(lq, lk, H, Hkv, D, dt)
    out, lse = B.fathom_prefill_attn(q, k, v, P.cumulated(lq), P.cumulated(lk), want_lse=True)
    check(out, lse, q, k, v, lq, lk)


@pytest.mark.parametrize("lq,lk,H", [([2048], [2080], 1), ([3000], [3001], 3), ([1500, 1500], [1540, 1540], 1)])
def test_shares_that_a_tile_does_not_reach(lq, lk, H):
    """Few rows, one per token, after a prefix: some CTA's share of the keys has no step for the first tile, whose
    last step elsewhere is half a step.  No wait runs out."""
    q, k, v = inputs(lq, lk, H, H, 64, BF)
    out, lse = B.fathom_prefill_attn(q, k, v, P.cumulated(lq), P.cumulated(lk), want_lse=True)
    check(out, lse, q, k, v, lq, lk)
    B.fathom_wait_status()


def test_thousands_of_sequences():
    """Two-row sequences between longer ones: the search for a tile's sequence goes over many of them."""
    lq = [2 + 70 * (i % 97 == 0) for i in range(1500)]
    q, k, v = inputs(lq, lq, 2, 1, 64, BF)
    out, lse = B.fathom_prefill_attn(q, k, v, P.cumulated(lq), want_lse=True)
    check(out, lse, q, k, v, lq, lq)


def test_rows_beyond_32_bit_offsets():
    """Strides that put the later tokens past 2^32 bytes, of the inputs and of the result."""
    n, H, D, step = 300, 2, 64, 1 << 23
    g = torch.Generator(device="cuda").manual_seed(1)
    big = torch.empty(n * step, dtype=BF, device="cuda").as_strided((n, 4, 2, D), (step, 2 * D, D, 1))
    rows = torch.randn(n, 3, 2, D, generator=g, device="cuda").to(BF)
    big[:, :3].copy_(rows)
    q, k, v = big[:, 0], big[:, 1], big[:, 2]
    out, lse = B.fathom_prefill_attn(q, k, v, P.cumulated([100, 200]), out=big[:, 3], want_lse=True)
    check(out.contiguous(), lse, rows[:, 0].contiguous(), rows[:, 1].contiguous(), rows[:, 2].contiguous(), [100, 200],
          [100, 200])


def test_whole_prompts_need_one_list_of_lengths_and_no_lse():
    lq = [70, 200]
    q, k, v = inputs(lq, lq, 4, 2, 128, BF)
    out, lse = B.fathom_prefill_attn(q, k, v, P.cumulated(lq))
    both, _ = B.fathom_prefill_attn(q, k, v, P.cumulated(lq), P.cumulated(lq), want_lse=True)
    assert lse is None and torch.equal(out, both)


@pytest.mark.parametrize("scale", [0.0, 40.0])
def test_flat_and_sharp_rows(scale):
    lq = [260, 33]
    q, k, v = inputs(lq, lq, 4, 2, 128, BF, q_scale=scale)
    out, lse = B.fathom_prefill_attn(q, k, v, P.cumulated(lq), want_lse=True)
    check(out, lse, q, k, v, lq, lq)


def test_growing_scores_rescale_the_running_sums():
    """Keys whose scores climb by far more than any power the kernel may defer."""
    n = 900
    q, k, v = inputs([n], [n], 2, 1, 128, BF)
    k = (k.float() * torch.linspace(0.01, 30, n, device="cuda")[:, None, None]).to(BF)
    out, lse = B.fathom_prefill_attn(q, k, v, P.cumulated([n]), want_lse=True)
    check(out, lse, q, k, v, [n], [n])


@pytest.mark.parametrize("rising", [False, True])
def test_shares_of_unequal_weight_are_joined(rising):
    """The keys' scores climb or fall from one CTA's share of them to the next."""
    n = 5000
    q, k, v = inputs([4], [n], 2, 1, 128, BF)
    ramp = torch.linspace(0.01, 30, n, device="cuda")[:, None, None]
    k = (k.float() * (ramp if rising else ramp.flip(0))).to(BF)
    out, lse = B.fathom_prefill_attn(q, k, v, P.cumulated([4]), P.cumulated([n]), want_lse=True)
    check(out, lse, q, k, v, [4], [n])
    again, _ = B.fathom_prefill_attn(q, k, v, P.cumulated([4]), P.cumulated([n]))
    assert torch.equal(out, again)


def test_strided_slices_and_per_head_rows():
    lq = [77, 140]
    T, H, Hkv, D = sum(lq), 8, 2, 128
    g = torch.Generator(device="cuda").manual_seed(3)
    qkv = torch.randn(T, H + 2 * Hkv, D, generator=g, device="cuda").to(BF)
    q, k, v = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
    out_all = torch.full((T, H + 1, D), 7.0, dtype=BF, device="cuda")
    out, lse = B.fathom_prefill_attn(q, k, v, P.cumulated(lq), out=out_all[:, :H], want_lse=True)
    check(out, lse, q, k, v, lq, lq)
    assert bool((out_all[:, H] == 7).all())
    kr, vr = (x.permute(1, 0, 2).contiguous() for x in (k, v))      # [heads][tokens][D]
    again, _ = B.fathom_prefill_attn(q, kr.permute(1, 0, 2), vr.permute(1, 0, 2), P.cumulated(lq))
    assert torch.equal(again, out)
    qh = q.permute(1, 0, 2).contiguous().permute(1, 0, 2)
    oh = torch.empty(H, T, D, dtype=BF, device="cuda").permute(1, 0, 2)
    again, _ = B.fathom_prefill_attn(qh, k, v, P.cumulated(lq), out=oh)
    assert torch.equal(again, out)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_rows_of_others_never_reach_a_sequence(bad):
    """NaN and infinities in the padding behind the last sequence, and in a neighbour."""
    lq, lk = [100, 40, 60], [150, 40, 61]
    q, k, v = inputs([100, 40, 60, 50], [150, 40, 61, 90], 8, 2, 128, BF)
    cq, ck = P.cumulated(lq), P.cumulated(lk)
    want, _ = B.fathom_prefill_attn(q, k, v, cq, ck)
    want = want.clone()
    for x, n in ((q, 140), (k, 190), (v, 190)):
        x[n:] = bad                                # the third sequence and the padding behind it
    out = torch.full_like(q, 3.0)
    B.fathom_prefill_attn(q, k, v, cq, ck, out=out)
    assert torch.equal(out[:140], want[:140])
    assert bool((out[200:] == 3).all())            # rows behind the last sequence are left alone
    k[150:190], v[150:190] = bad, bad              # the second one too
    B.fathom_prefill_attn(q, k, v, cq, ck, out=out)
    assert torch.equal(out[:100], want[:100])


@pytest.mark.parametrize("lq,lk,H,Hkv,D,dt", [([300], [300], 4, 1, 128, BF), ([130], [200], 2, 2, 64, FP),
                                              ([5], [5000], 4, 2, 96, BF), ([40, 260], [40, 260], 3, 1, 72, FP)])
@pytest.mark.parametrize("what", ["k", "v"])
def test_rows_behind_a_query_never_reach_it(lq, lk, H, Hkv, D, dt, what):
    """NaN and infinities in keys and values of the sequence itself: only the queries that see them change,
    and of those, for a value, only its channel."""
    q, k, v = inputs(lq, lk, H, Hkv, D, dt)
    o, z, tol, tol_z = P.prefill(q, k, v, lq, lk, D)
    ends = torch.tensor([sum(lk[: i + 1]) for i in range(len(lk))])
    first_q = sum(lq[:-1])
    bad = [(int(ends[-1]) - 3, 0, float("nan")), (int(ends[-1]) - 70, D - 1, float("inf"))]     # of the last sequence
    for row, channel, x in bad:
        (k if what == "k" else v)[row, 0, channel] = x
    out, lse = B.fathom_prefill_attn(q, k, v, P.cumulated(lq), P.cumulated(lk), want_lse=True)
    # the first query that sees each of them
    sees = [max(first_q, first_q + lq[-1] - (int(ends[-1]) - row)) for row, _, _ in bad]
    clean = torch.ones_like(out, dtype=torch.bool)
    for t, (_, channel, _) in zip(sees, bad):
        hit = slice(0, H // Hkv)                                       # the query heads of KV head 0
        if what == "k":
            clean[t:, hit] = False
        else:
            assert not torch.isfinite(out[t:, hit, channel]).any()
            clean[t:, hit, channel] = False
    assert bool(((out.double() - o).abs() <= tol)[clean].all())
    rows = clean.any(2)
    assert bool(((lse.double() - z).abs() <= tol_z)[rows].all())


@pytest.mark.parametrize("dt", [BF, FP])
def test_infinite_values_seen_and_unseen(dt):
    """A channel that is infinite in every value row: infinite for every query, and never NaN from the rows
    behind; the other channels are the formula's."""
    lq, H, Hkv, D = [7, 200, 130], 4, 2, 128
    q, k, v = inputs(lq, lq, H, Hkv, D, dt, q_scale=0.5)    # weights far from underflow
    o, z, tol, tol_z = P.prefill(q, k, v, lq, lq, D)
    v[:, 1, 5], v[:, 1, 64] = float("inf"), float("-inf")
    out, lse = B.fathom_prefill_attn(q, k, v, P.cumulated(lq), want_lse=True)
    assert bool((out[:, 2:, 5] == float("inf")).all()) and bool((out[:, 2:, 64] == float("-inf")).all())
    clean = torch.ones_like(out, dtype=torch.bool)
    clean[:, 2:, 5] = clean[:, 2:, 64] = False
    assert bool(((out.double() - o).abs() <= tol)[clean].all())
    assert bool(((lse.double() - z).abs() <= tol_z).all())


@pytest.mark.parametrize("lq", [200, 16])
def test_an_odd_value_at_the_end_of_a_long_sequence(lq):
    """The next tokens of a sequence of 100 003, the last of whose values is NaN: the others do not see it."""
    lk, H, Hkv, D = 100003, 4, 1, 128
    q, k, v = inputs([lq], [lk], H, Hkv, D, BF)
    o, z, tol, tol_z = P.prefill(q, k, v, [lq], [lk], D)
    v[-1, 0, 17] = float("nan")
    out, lse = B.fathom_prefill_attn(q, k, v, P.cumulated([lq]), P.cumulated([lk]), want_lse=True)
    assert bool(torch.isnan(out[-1, :, 17]).all())
    assert bool(((out.double() - o).abs() <= tol)[:-1].all())
    assert bool(((lse.double() - z).abs() <= tol_z).all())
    B.fathom_wait_status()


ODD = {                   # (new tokens, tokens, heads, KV heads, channels, type)
    "tiles of 32 tokens": ([300, 77], [300, 500], 8, 2, 128, BF),
    "one row per token, fp16": ([513, 40], [700, 40], 2, 2, 64, FP),
    "tiles of one token": ([9], [70], 160, 1, 72, FP),
    "single tiles in turn": ([1 + i % 30 for i in range(200)], [1 + i % 30 + i % 7 for i in range(200)], 8, 8, 96, BF),
    "more items than are noted at once": ([1 + i % 16 for i in range(1500)], [1 + i % 16 + i % 3 for i in range(1500)], 4, 4,
                                          64, BF),
    "queries that see nothing": ([200, 60], [90, 300], 4, 2, 128, BF),
    "2 shares": ([300], [1500], 4, 1, 64, BF),
    "4 shares": ([129, 7], [3000, 9], 3, 3, 128, FP),
    "8 shares": ([16, 130], [300, 6000], 4, 1, 96, BF),
}


@pytest.mark.parametrize("name", list(ODD))
@pytest.mark.parametrize("count", [1, 7, 60])
def test_values_that_are_not_finite_reach_the_queries_that_see_them(name, count):
    """A query that sees such values has their sum in the channel; every other result is, bit for bit, the one for
    zeros in their place."""
    lq, lk, H, Hkv, D, dt = ODD[name]
    count = max(count, 3 * len(lq) * (count == 60))          # in most sequences, where there are many
    q, k, v = inputs(lq, lk, H, Hkv, D, dt, q_scale=0.25)    # weights far from underflow
    g = torch.Generator().manual_seed(count)
    seq = torch.randint(len(lk), (count,), generator=g).tolist()
    first_k, first_q = [sum(lk[:s]) for s in range(len(lk))], [sum(lq[:s]) for s in range(len(lq))]
    sums = torch.zeros(sum(lq), H, D, device="cuda")
    for i, s in enumerate(seq):
        # near the end, where some queries see the key and some do not
        key = lk[s] - 1 - int(torch.randint(min(lk[s], 2 * lq[s]), (1,), generator=g))
        h, c = int(torch.randint(Hkv, (1,), generator=g)), int(torch.randint(D, (1,), generator=g))
        bad = (math.nan, math.inf, -math.inf)[i % 3]
        v[first_k[s] + key, h, c] = bad
    for s in set(seq):
        for h in range(Hkv):
            odd = v[first_k[s]:first_k[s] + lk[s], h].float()
            odd = torch.where(torch.isfinite(odd), 0.0, odd).cumsum(0)       # of the keys up to each one
            sees = torch.arange(lq[s], device="cuda") + lk[s] - lq[s]
            part = torch.where((sees >= 0)[:, None], odd[sees.clamp(min=0)], 0.0)
            sums[first_q[s]:first_q[s] + lq[s], h * (H // Hkv):(h + 1) * (H // Hkv)] = part[:, None]
    zeros = torch.where(torch.isfinite(v), v, torch.zeros_like(v))
    cq, ck = P.cumulated(lq), P.cumulated(lk)
    want, lse = B.fathom_prefill_attn(q, k, zeros, cq, ck, want_lse=True)
    check(want, lse, q, k, zeros, lq, lk)
    out, lse2 = B.fathom_prefill_attn(q, k, v, cq, ck, want_lse=True)
    want = want.float() + sums
    assert not torch.isfinite(want).all()
    assert torch.equal(torch.nan_to_num(out.float(), nan=7e30), torch.nan_to_num(want, nan=7e30))
    assert torch.equal(lse, lse2)


@pytest.mark.parametrize("lq,lk,H", [(20000, 600000, 2), (10000, 300000, 8)])
def test_odd_values_of_a_long_sequence_with_more_work_than_the_device_holds(lq, lk, H):
    """Rows next to such values cost no more than others, however many keys they see: no wait of the work that
    follows runs out."""
    D = 64
    q, k, v = inputs([lq], [lk], H, H, D, BF, q_scale=0.25)
    cq, ck = P.cumulated([lq]), P.cumulated([lk])
    rows = [lk - 1, lk - 7000, lk - lq + 130]
    v[rows, 0] = 0.0
    want, lse = B.fathom_prefill_attn(q, k, v, cq, ck, want_lse=True)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    for row, bad in zip(rows, (math.nan, math.inf, -math.inf)):
        v[row, 0] = bad
    start.record()
    out, lse2 = B.fathom_prefill_attn(q, k, v, cq, ck, want_lse=True)
    end.record()
    B.fathom_wait_status()
    assert start.elapsed_time(end) < 1000
    seen = [row - (lk - lq) for row in rows]                 # the first query that sees each
    assert torch.equal(out[:, 1:], want[:, 1:]) and torch.equal(lse, lse2)
    assert torch.equal(out[:seen[2], 0], want[:seen[2], 0])
    assert bool((out[seen[2]:seen[1], 0] == -math.inf).all()) and bool(torch.isnan(out[seen[1]:, 0]).all())


@pytest.mark.parametrize("lq,lk", [(900, 900), (4, 5000)])
@pytest.mark.parametrize("rising", [False, True])
@pytest.mark.parametrize("power", [-120, -90, 100, 112])
def test_values_near_the_ends_of_bf16(lq, lk, rising, power):
    """Values of up to 4 x 2^112, of which fp32 holds the sum of 5000, and of no less than 2^-124, in whatever order
    the scores come."""
    q, k, v = inputs([lq], [lk], 2, 1, 128, BF)
    ramp = torch.linspace(0.01, 6, lk, device="cuda")[:, None, None]
    k = (k.float() * (ramp if rising else ramp.flip(0))).to(BF)
    v = (v.sign() * v.abs().clamp(1 / 16, 4) * 2.0 ** power).to(BF)
    out, lse = B.fathom_prefill_attn(q, k, v, P.cumulated([lq]), P.cumulated([lk]), want_lse=True)
    check(out, lse, q, k, v, [lq], [lk])


FEW_OR_MANY = {           # (new tokens, tokens, heads, KV heads, channels, type): the CTAs that share an item's keys
    "2 shares": (130, 1500, 4, 1, 64, FP),
    "4 shares": (7, 3000, 8, 4, 96, BF),
    "8 shares": (5, 5000, 4, 2, 128, BF),
    "8 shares, fp16": (3, 6000, 2, 1, 128, FP),
    "one CTA": (2600, 2600, 8, 8, 64, BF),
}


@pytest.mark.parametrize("name", list(FEW_OR_MANY))
@pytest.mark.parametrize("what", ["a query", "one key", "the first keys", "a share's keys", "the last keys"])
def test_a_nan_that_a_query_sees_reaches_its_results(name, what):
    """NaN in out and lse of every row that sees it, by however many CTAs its keys are shared; other rows as they were."""
    lq, lk, H, Hkv, D, dt = FEW_OR_MANY[name]
    q, k, v = inputs([lq], [lk], H, Hkv, D, dt)
    o, z, tol, tol_z = P.prefill(q, k, v, [lq], [lk], D)
    nan = torch.zeros(lq, H, dtype=torch.bool, device="cuda")
    G = H // Hkv
    if what == "a query":
        q[lq // 2, H - 1, 3] = math.nan
        nan[lq // 2, H - 1] = True
    else:
        steps = -(-lk // 128)
        first, last = {"one key": (lk - 2, lk - 1), "the first keys": (0, 700), "a share's keys": (steps // 8 * 128, 2 * steps // 8 * 128),
                       "the last keys": (7 * steps // 8 * 128, lk)}[what]
        k[first:last, Hkv - 1, D - 1] = math.nan
        sees = torch.arange(lq, device="cuda") + lk - lq >= first
        nan[:, (Hkv - 1) * G:] = sees[:, None]
    out, lse = B.fathom_prefill_attn(q, k, v, P.cumulated([lq]), P.cumulated([lk]), want_lse=True)
    assert bool(torch.isnan(out[nan]).all()) and bool(torch.isnan(lse[nan]).all())
    assert bool(((out.double() - o).abs() <= tol)[~nan].all())
    assert bool(((lse.double() - z).abs() <= tol_z)[~nan].all())


def test_lengths_are_clamped_to_the_arrays():
    q, k, v = inputs([50, 50], [50, 50], 4, 2, 128, BF)
    want, _ = B.fathom_prefill_attn(q, k, v, P.cumulated([50, 50]))
    cu = torch.tensor([0, 50, 1 << 30], dtype=torch.int32, device="cuda")
    got, _ = B.fathom_prefill_attn(q, k, v, cu)
    assert torch.equal(got, want)


def test_no_keys_at_all_and_no_queries():
    q, k, v = inputs([9], [0], 4, 2, 64, FP)
    out, lse = B.fathom_prefill_attn(q, k, v, P.cumulated([9]), P.cumulated([0]), want_lse=True)
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())
    q, k, v = inputs([0], [9], 4, 2, 64, FP)
    out, _ = B.fathom_prefill_attn(q, k, v, P.cumulated([0]), P.cumulated([9]))
    assert out.shape == (0, 4, 64)


def test_same_bits_on_streams_and_in_a_graph():
    lq, lk = [70, 260, 3], [70, 600, 9]
    q, k, v = inputs(lq, lk, 8, 2, 128, BF)
    cq, ck = P.cumulated(lq), P.cumulated(lk)
    want, _ = B.fathom_prefill_attn(q, k, v, cq, ck)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [B.fathom_prefill_attn(q, k, v, cq, ck, stream=s)[0] for s in streams for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for x in got)
    graph, out = torch.cuda.CUDAGraph(), torch.empty_like(q)
    with torch.cuda.graph(graph):
        B.fathom_prefill_attn(q, k, v, cq, ck, out=out)
    q2, _, _ = inputs(lq, lk, 8, 2, 128, BF, seed=9)
    want2, _ = B.fathom_prefill_attn(q2, k, v, cq, ck)
    q.copy_(q2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want2)


def test_no_bounded_wait_ran_out():
    q, k, v = inputs([300], [300], 4, 2, 128, BF)
    B.fathom_prefill_attn(q, k, v, P.cumulated([300]))
    B.fathom_wait_status()                             # covers every call of this process


def test_first_calls_of_a_process_inside_a_capture():
    """Every call, captured by a process that has not made it before, and replayed."""
    code = """
import sys
sys.path.insert(0, %r); sys.path.insert(0, %r)
import torch
from bit_plane_kv_gb300 import binding as B
import paged_cases as P
kp, vp, table, free = P.pool(2, 2, 128, 16, 8, torch.bfloat16, extra=8)
pages = B.make_pages(kp, table)
ws = B.alloc_paged_workspace(pages, G=4, mass=True)
q, new = torch.randn(4, 4, 128, device="cuda"), torch.randn(2, 2, 128, device="cuda").bfloat16()
lens, start = torch.full((2,), 100, dtype=torch.int32, device="cuda"), torch.full((2,), 99, dtype=torch.int32, device="cuda")
mass, dst = torch.zeros(4, 128, device="cuda"), free.reshape(2, 4).contiguous()
p = torch.randn(40, 8, 128, device="cuda").bfloat16()
cu = P.cumulated([7, 33])

def calls():
    a, _ = B.fathom_prefill_attn(p, p[:, :2], p[:, 2:4], cu)
    B.fathom_paged_append(pages, kp, vp, table, new, new, start)
    b = B.fathom_paged_attn(pages, q, kp, vp, table, lens, ws, mass=mass)
    c, _, d = B.fathom_paged_evict(pages, kp, vp, table, lens, mass, 60, dst, mass_out=torch.zeros(4, 64, device="cuda"))
    return a, b, c, d

g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    got = calls()
g.replay()
torch.cuda.synchronize()
got = [x.clone() for x in got]
mass.zero_()
want = calls()
torch.cuda.synchronize()
assert all(torch.equal(x, y) for x, y in zip(got, want))
print("same")
""" % (os.path.dirname(os.path.dirname(os.path.abspath(__file__))), os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "same", r.stdout + r.stderr[-2000:]
