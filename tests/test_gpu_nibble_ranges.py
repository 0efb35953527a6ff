"""Decode attention over the 4-bit cache where channel groups, tokens and queries differ in size by
many powers of two, on the GPU against 64 bits.

Bounds as derived in nibble_cases, with two terms of their own:
* Rows of V.  A weight times a scale is held in two fp16 pieces.  Where all scales that a warp has seen in the
  unit lie within a factor of 2^9 of each other, they are scaled to 2^-7 .. 4: the second piece of a weight is off by
  2^-25 times the scale, the product's pieces by 2^-24 together, so 2^-22.5 per token at most, beside the
  largest weight's 2^13 times a scale of 2^-7 and more times a value of a 16th of it and more, 2^2: 2^-24.5 of the
  sum A of w |v| in the same channel per token of the warp, of which there are n / 4 + 32 at most.
  Elsewhere products are scaled block by block by their largest, 2^-38 of it per token, 2^-30 A in all.
  So (n / 4 + 32) 2^-24 A, and nothing that depends on the largest scale.
* Queries.  A channel is held to 2^-22 of its group's largest, and of the row's largest to 2^-45:
  Q = sum over groups of max |q| sum |k|, and 2^-44 of max |q| sum |k| over the row."""
import math

import pytest
import torch

from bit_plane_kv_gb300 import binding as B

import nibble_cases as N

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def gen(seed=0):
    return torch.Generator(device="cuda").manual_seed(seed)


def rnd(*shape, seed=0):
    return torch.randn(*shape, generator=gen(seed), device="cuda").double()


def attend(q, k, v, lens):
    """(out, lse, what the cache holds of K, of V) with pages of 16 tokens; k, v [sequences][heads][tokens][D]."""
    S, H, n, D = k.shape
    per = n // 16
    rows = [x.reshape(S, H, per, 16, D).transpose(1, 2).reshape(S * per, H, 16, D) for x in (k, v)]
    kv, table = N.pack(*rows), torch.arange(S * per, dtype=torch.int32, device="cuda").reshape(S, per)
    pages = B.make_nibble_pages(kv, table, D)
    out, lse = B.fathom_nibble_attn(pages, q, kv, table, i32(lens), B.alloc_nibble_workspace(pages, G=q.shape[1]), want_lse=True)
    held = [x.reshape(S, per, H, 16, D).transpose(1, 2).reshape(S, H, n, D) for x in N.unpack(kv, D)]
    return out, lse, *held


def check(out, lse, q, K, V, lens):
    U, G, D = q.shape
    H = K.shape[1]
    for u in range(U):
        s, h = divmod(u, H)
        n = lens[s]
        kk, vv, qq = K[s, h, :n], V[s, h, :n], q[u].double()
        x = qq @ kk.T / math.sqrt(D)
        S = (qq.abs() @ kk.abs().T / math.sqrt(D)).amax(1)
        most, size = qq.abs().reshape(G, -1, 32).amax(2), kk.abs().reshape(n, -1, 32).sum(2)
        Q = (most @ size.T).amax(1) / math.sqrt(D) + 2.0 ** -24 * most.amax(1) * size.sum(1).amax() / math.sqrt(D)
        z = torch.logsumexp(x, 1)
        A = torch.exp(x - z[:, None]) @ vv.abs()
        ds = 16 * 2.0 ** -24 * S + 2.0 ** -20 * Q
        r = 2 * (ds + 2.0 ** -23 * (2.2 * S + 10)) + 3 * 2.0 ** -22
        k = (n / 64 + 128) * 2.0 ** -23
        far = (out[u].double() - torch.exp(x - z[:, None]) @ vv).abs()
        tol = (2 * r + 2.0 ** -21 + 2 * k + (n / 4 + 32) * 2.0 ** -24)[:, None] * A
        assert bool((r < 0.1).all())                              # the first order is enough
        assert torch.isfinite(out[u]).all()
        assert bool((far <= tol).all()), f"unit {u}: worst {(far / tol.clamp(min=1e-300)).max().item():.3g} of the tolerance"
        assert bool(((lse[u].double() - z).abs() <= r + k + ds + 2.0 ** -22 * z.abs()).all())


# ------------------------------------------------------------------ values
@pytest.mark.parametrize("D,G", [(128, 4), (128, 8), (64, 3), (64, 7), (96, 5), (96, 1), (32, 4), (32, 8)])
@pytest.mark.parametrize("kind", ["groups", "groups, the other way", "first tokens", "last tokens", "tokens and groups"])
def test_values_of_very_different_sizes(kind, D, G):
    """A group or a token of large values takes nothing from the others."""
    S, H, n = 2, 2, 1504
    k, v = 0.3 * rnd(S, H, n, D), rnd(S, H, n, D, seed=1)
    g = torch.arange(D, device="cuda") // 32
    if kind.startswith("groups"):
        v *= 2.0 ** (8 - 7 * (g if kind == "groups" else D // 32 - 1 - g))
    elif kind == "tokens and groups":
        v *= 2.0 ** torch.randint(-13, 14, (S, H, n, D // 32, 1), generator=gen(3), device="cuda").double().expand(-1, -1, -1, -1, 32).reshape(S, H, n, D)
    else:
        v[:, :, :70 if kind == "first tokens" else None] *= 2.0 ** 12
        if kind == "last tokens":
            v[:, :, :-70] *= 2.0 ** -25
        else:
            v[:, :, 70:] *= 2.0 ** -10
    q = rnd(S * H, G, D, seed=5).float()
    lens = [n - 5, 333]
    out, lse, K, V = attend(q, k, v, lens)
    check(out, lse, q, K, V, lens)


@pytest.mark.parametrize("D,G", [(128, 4), (128, 8), (64, 4), (96, 6), (32, 2)])
@pytest.mark.parametrize("where", ["first", "middle", "last", "every fifth"])
def test_large_values_of_negligible_weight(where, D, G):
    """Tokens of values 2^22 times the others' whose softmax weights are below 2^-50."""
    S, H, n = 2, 1, 1104
    sign = rnd(S, H, 1, D, seed=2).sign()
    k, v = sign + 0.2 * rnd(S, H, n, D), 2.0 ** -11 * rnd(S, H, n, D, seed=1)
    big = {"first": slice(0, 40), "middle": slice(500, 520), "last": slice(1060, 1104), "every fifth": slice(2, None, 5)}[where]
    k[:, :, big] *= -1
    v[:, :, big] *= 2.0 ** 22
    q = (sign.reshape(S, 1, D) * (25 / math.sqrt(D)) + 0.1 * rnd(S, G, D, seed=5)).float()
    lens = [n, 1090]
    out, lse, K, V = attend(q, k, v, lens)
    check(out, lse, q, K, V, lens)


def test_large_and_small_values_over_many_shares():
    """The same where CTAs share a unit."""
    D, n = 128, 24000
    size = 2.0 ** torch.randint(-12, 12, (1, 1, n // 16, 1), generator=gen(3), device="cuda").double().repeat_interleave(16, 2)
    k, v = rnd(1, 1, n, D), rnd(1, 1, n, D, seed=1) * size * 2.0 ** (3 * (torch.arange(D, device="cuda") // 32) - 6)
    q = rnd(1, 4, D, seed=5).float()
    out, lse, K, V = attend(q, k, v, [n])
    check(out, lse, q, K, V, [n])


# ------------------------------------------------------------------ queries
@pytest.mark.parametrize("D,G", [(128, 4), (128, 7), (64, 8), (64, 1), (96, 3)])
@pytest.mark.parametrize("bits", [-27, -24, -20, -12, -5, 5, 12, 20, 24, 27])
def test_large_channels_of_a_query_over_small_ones_of_the_keys(bits, D, G):
    """Groups whose queries differ by up to 2^27 and whose keys by the inverse of it, so that all count alike."""
    S, H, n = 2, 2, 1104
    g = torch.arange(D, device="cuda").double().div(32, rounding_mode="floor") / (D // 32 - 1)
    k, v = rnd(S, H, n, D) * 2.0 ** (bits * (g - 0.5)), rnd(S, H, n, D, seed=1)
    q = (rnd(S * H, G, D, seed=5) * 2.0 ** (-bits * (g - 0.5))).float()
    lens = [n, 75]
    out, lse, K, V = attend(q, k, v, lens)
    check(out, lse, q, K, V, lens)


@pytest.mark.parametrize("factor", [64.0, 1000.0, 1e6])
def test_one_large_channel_of_a_query(factor):
    S, H, n, D = 1, 2, 1104, 128
    k, v = rnd(S, H, n, D), rnd(S, H, n, D, seed=1)
    k[..., :32] /= factor
    q = rnd(S * H, 4, D, seed=5)
    q[..., 5] *= factor
    q = q.float()
    out, lse, K, V = attend(q, k, v, [n])
    check(out, lse, q, K, V, [n])


LARGEST = torch.finfo(torch.float32).max


@pytest.mark.parametrize("D,G,n", [(64, 4, 608), (128, 8, 608), (32, 1, 20000)])
@pytest.mark.parametrize("size", [2.0 ** p for p in (100, 105, 112, 114, 115, 116, 117, 118, 122, 126, 127)] + [LARGEST])
def test_scores_up_to_the_largest_numbers(size, D, G, n):
    """Queries of up to fp32's largest number: one token has all the weight, and the log-sum-exp is its score.
    Channels of q are +-size, so the scores, size times sums of keys, are far apart."""
    k, v = 2.0 ** -13 * rnd(1, 2, n, D), rnd(1, 2, n, D, seed=1)
    q = (rnd(2, G, D, seed=5).sign() * size).float()
    out, lse, K, V = attend(q, k, v, [n])
    for u in range(2):
        kk, vv = K[0, u], V[0, u]
        x = q[u].double() @ kk.T
        top = x.topk(2, 1)
        assert bool((top.values[:, 0] - top.values[:, 1] > size * 2.0 ** -24).all())
        # one weight of 1: its two pieces and the value, 2^-21
        assert bool(((out[u].double() - vv[top.indices[:, 0]]).abs() <= 2.0 ** -20 * vv[top.indices[:, 0]].abs()).all())
        # the score's roundings, ds above with Q <= S, and fewer than 16 of the factor's
        want, S = top.values[:, 0] / math.sqrt(D), (q[u].double().abs() @ kk.abs().T).amax(1) / math.sqrt(D)
        assert bool((want < LARGEST).all())
        assert bool(((lse[u].double() - want).abs() <= 2.0 ** -18 * S).all()), f"{lse[u]} for {want}"


@pytest.mark.parametrize("n", [16, 30000])
@pytest.mark.parametrize("score", [1e37, 1e38, 2.3e38, 2.5e38, 3.3e38])
def test_a_log_sum_exp_next_to_the_largest_number(score, n):
    """In powers of two the last two lie beyond it."""
    D, G = 64, 4
    sign = rnd(1, 1, 1, D, seed=2).sign()
    k, v = torch.zeros(1, 1, n, D, device="cuda").double(), rnd(1, 1, n, D, seed=1)
    k[:, :, n // 3] = sign
    q = (sign.reshape(1, 1, D) * (score / math.sqrt(D) / (15 / 16))).float().repeat(1, G, 1)
    q[:, 1] *= -1                                               # the others' score, 0, is the largest
    out, lse, K, V = attend(q, k, v, [n])
    x = q[0].double() @ K[0, 0].T / math.sqrt(D)
    want = torch.logsumexp(x, 1)
    assert bool((want < LARGEST).all()) and torch.isfinite(lse).all()
    assert bool(((lse[0].double() - want).abs() <= 2.0 ** -18 * x.abs().amax(1)).all())
    assert bool(((out[0, 0].double() - V[0, 0, n // 3]).abs() <= 2.0 ** -20 * V[0, 0, n // 3].abs()).all())
    assert bool(((lse[0, 1] - math.log(n - 1)).abs() <= 2.0 ** -12)) and torch.isfinite(out).all()


def test_a_log_sum_exp_beyond_the_largest_number_is_infinite():
    D = 64
    k, v = torch.ones(1, 1, 32, D, device="cuda").double(), rnd(1, 1, 32, D, seed=1)
    q = torch.full((1, 2, D), LARGEST, device="cuda")
    q[0, 1] = -q[0, 1]
    out, lse, K, V = attend(q, k, v, [32])
    assert lse[0, 0] == math.inf and lse[0, 1] == -math.inf and torch.isfinite(out).all()


# ------------------------------------------------------------------ what may lie beside values of different sizes
def wide_cache(S, H, n, D):
    """Pages whose V scales are 2^-21 to 2^15."""
    k, v = rnd(S * n // 16, H, 16, D), rnd(S * n // 16, H, 16, D, seed=1)
    v *= 2.0 ** torch.randint(-11, 12, (S * n // 16, H, 16, 1), generator=gen(3), device="cuda").double()
    v *= 2.0 ** (2 - 3 * (torch.arange(D, device="cuda") // 32))
    return N.pack(k, v), torch.arange(S * n // 16, dtype=torch.int32, device="cuda").reshape(S, n // 16)


@pytest.mark.parametrize("D,G", [(128, 4), (64, 8), (96, 3)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_places_behind_the_length_and_missing_pages_beside_values_of_different_sizes(bad, D, G):
    S, H, n = 3, 2, 1024
    kv, table = wide_cache(S, H, n, D)
    lens, q = [1003, 70, 1], rnd(S * H, G, D, seed=5).float()
    table[0, 5], table[0, 33], table[1, 0] = -1, 1 << 30, kv.shape[0]
    pages = B.make_nibble_pages(kv, table, D)
    ws = B.alloc_nibble_workspace(pages, G=G)
    want, z = B.fathom_nibble_attn(pages, q, kv, table, i32(lens), ws, want_lse=True)
    K, V = N.unpack(kv, D)
    keep = torch.ones(S, n, dtype=torch.bool, device="cuda")
    for s, p in ((0, 5), (0, 33), (1, 0)):
        keep[s, 16 * p:16 * p + 16] = False
    for s in range(S):
        for h in range(H):
            rows = [x[s * n // 16:(s + 1) * n // 16, h].reshape(n, D)[:lens[s]][keep[s, :lens[s]]] for x in (K, V)]
            u = s * H + h
            check(want[u:u + 1], z[u:u + 1], q[u:u + 1], rows[0][None, None], rows[1][None, None], [rows[0].shape[0]])
    x = kv.view(S, n // 16, H, 18 * D)                                      # a page is a block
    bits = torch.tensor([bad], dtype=torch.float16, device="cuda").view(torch.uint8)
    for s in range(S):
        for p in range(n // 16):
            for t in range(16):
                if 16 * p + t >= lens[s] or not keep[s, 16 * p]:
                    for base in (8 * D, 17 * D):
                        for g in range(D // 32):
                            at = base + 4 * ((t & 7) * (D // 32) + g) + 2 * (t >> 3)
                            x[s, p, :, at:at + 2] = bits
    n_of = i32(lens)
    graph, out, lse = torch.cuda.CUDAGraph(), torch.empty_like(want), torch.empty_like(z)
    with torch.cuda.graph(graph):
        B.fathom_nibble_attn(pages, q, kv, table, n_of, ws, out=out, lse=lse)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, z)


def test_a_nan_beside_values_of_different_sizes_stays_in_its_group():
    D, n = 128, 1024
    kv, table = wide_cache(2, 2, n, D)
    pages, q = B.make_nibble_pages(kv, table, D), rnd(4, 4, D, seed=5).float()
    ws = B.alloc_nibble_workspace(pages)
    want = B.fathom_nibble_attn(pages, q, kv, table, i32([n, n]), ws)
    at = 17 * D + 4 * ((600 % 8) * 4 + 2) + 2 * (600 % 16 // 8)             # token 600 of unit 1, group 2 of V
    kv[600 // 16, 1, at:at + 2] = torch.tensor([float("nan")], dtype=torch.float16, device="cuda").view(torch.uint8)
    got = B.fathom_nibble_attn(pages, q, kv, table, i32([n, n]), ws)
    assert torch.isnan(got[1, :, 64:96]).all()
    got[1, :, 64:96] = want[1, :, 64:96]
    assert torch.equal(got, want)
