"""Codes of rotated keys in a 4-bit cache against rational arithmetic, on the GPU: products below fp32's smallest
number or beyond its largest, and keys next to a border by less than 53 bits show."""
import random
from fractions import Fraction as F

import pytest
import torch

from bit_plane_kv_gb300 import binding as B

import nibble_cases as N

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


def to_half(v):
    """The fp16 number nearest to v >= 0, ties to even, at most 65504."""
    if v >= 65504:
        return F(65504)
    e = -14
    while v >= F(2) ** (e + 1):
        e += 1
    unit = F(2) ** (e - 10)
    n = v / unit
    low = n.numerator // n.denominator
    rest = n - low
    return (low + (rest > F(1, 2) or (rest == F(1, 2) and low % 2 == 1))) * unit


def held(y):
    """(values) that a group of 32 rationals becomes."""
    a = min(to_half(max(abs(v) for v in y)), F(65504))
    if a == 0:
        return [F(0)] * len(y)
    return [(min(max((v / (a / 8)).__floor__(), -8), 7) + F(1, 2)) * a / 8 for v in y]


def rotated(x, c, s, pairs):
    R = 2 * len(c)
    y = list(x)
    for i in range(R // 2):
        j, k = (2 * i, 2 * i + 1) if pairs else (i, i + R // 2)
        y[j], y[k] = x[j] * c[i] - x[k] * s[i], x[k] * c[i] + x[j] * s[i]
    return y


def append(x, rope, pairs):
    """What the cache holds of keys x [tokens][D] (one head) at positions 0 on."""
    T, D = x.shape
    per = -(-T // 16)
    kv, table = B.alloc_nibble_pages(per, 1, 16, D), torch.arange(per, dtype=torch.int32, device="cuda")[None].contiguous()
    zero, cu = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.tensor([0, T], dtype=torch.int32, device="cuda")
    B.fathom_nibble_append(B.make_nibble_pages(kv, table, D), kv, table, x[:, None], x[:, None], zero, cu, rope=rope, interleaved=pairs)
    return N.unpack(kv, D)[0].reshape(-1, D)[:T]


#: what keys and the table's numbers are taken from
KEYS = {BF: [0.0, 1.0, -1.0, 0.5, -0.75, 3.0, 2.0 ** -40, -2.0 ** -100, 2.0 ** -133, -2.0 ** -126, 3e38, -3e38, 2.0 ** 100],
        FP: [0.0, 1.0, -1.0, 0.5, -0.75, 3.0, 2.0 ** -24, -2.0 ** -24, 2.0 ** -14, 60000.0, -65504.0, 2.0 ** -10]}
TURNS = [0.0, 1.0, -1.0, 0.5, 1.5, -1.25, 2.0 ** -30, -2.0 ** -60, 2.0 ** -100, 2.0 ** -126, -2.0 ** -149, 1.0 + 2.0 ** -23, 0.1]


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("D,rot,pairs", [(64, 64, False), (128, 128, False), (64, 64, True), (96, 40, False), (32, 30, True)])
@pytest.mark.parametrize("large", [False, True])
def test_codes_of_products_beyond_fp32(dt, D, rot, pairs, large):
    """Keys that turn by any numbers, from below fp32's smallest products to beyond its largest sums."""
    rng = random.Random(D + rot + pairs)
    keys = [k for k in KEYS[dt] if large or abs(k) <= 3]
    T = 48
    x = torch.tensor([[rng.choice(keys) for _ in range(D)] for _ in range(T)]).to(dt)
    rope = torch.tensor([[rng.choice(TURNS) for _ in range(rot)] for _ in range(T)], dtype=torch.float32)
    got = append(x.cuda(), rope.cuda(), pairs).cpu()
    for t in range(T):
        row, table = [F(v) for v in x[t].double().tolist()], [F(v) for v in rope[t].double().tolist()]
        y = rotated(row, table[: rot // 2], table[rot // 2:], pairs)
        want = [v for g in range(0, D, 32) for v in held(y[g:g + 32])]
        wrong = [i for i, (v, w) in enumerate(zip(got[t].tolist(), want)) if F(v) != w]
        assert not wrong, (t, wrong, [float(y[i]) for i in wrong], [float(want[i]) for i in wrong], [got[t, i].item() for i in wrong])


@pytest.mark.parametrize("pairs", [False, True])
def test_keys_a_hair_from_a_border(pairs):
    """x c lies on a border, x' s moves it by 2^-70 to 2^-250 to either side."""
    D, T = 64, 40
    x, rope = torch.zeros(T, D), torch.zeros(T, D)
    first, second = (slice(0, D, 2), slice(1, D, 2)) if pairs else (slice(0, 32), slice(32, 64))
    rng = random.Random(7)
    for t in range(T):
        x[t, first] = torch.tensor([rng.randint(-8, 8) / 8 for _ in range(32)])
        if t % 2:
            x[t, first] = torch.where(x[t, first] == 0, torch.tensor(2.0 ** -100), x[t, first])
        x[t, second] = torch.tensor([rng.choice([-1, 1]) * 2.0 ** -rng.randint(35, 126) for _ in range(32)])
        x[t, 0] = 1.0
        rope[t, :32] = 1.0
        rope[t, 32:] = torch.tensor([2.0 ** -rng.randint(35, 126) for _ in range(32)])
        rope[t, 32] = 0.0                                     # the largest is 1
    x = x.to(BF)
    got = append(x.cuda(), rope.cuda(), pairs).cpu()
    for t in range(T):
        row, table = [F(v) for v in x[t].double().tolist()], [F(v) for v in rope[t].double().tolist()]
        y = rotated(row, table[:32], table[32:], pairs)
        want = [v for g in (0, 32) for v in held(y[g:g + 32])]
        wrong = [i for i, (v, w) in enumerate(zip(got[t].tolist(), want)) if F(v) != w]
        assert not wrong, (t, wrong)
