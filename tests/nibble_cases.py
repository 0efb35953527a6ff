"""Plain 64-bit forms of the rotated append and of the 4-bit cache, and how far a kernel
may be from them.

Rotation, y = x c + p s: the product p s is rounded to fp32 and the fused sum once more, so a
result in fp32 is within 2^-24 (|p s| + |y|) <= 2^-23 Y, Y = |x c| + |p s|; in 16 bits one more
rounding, u (|y| + 2^-23 Y), u = eps / 2 of the type, or half a subnormal step.

Codes, scales and what is read back in fp32 are exact: the same numbers.  Read back in 16
bits: the exact value's rounding, the same bits.

Decode attention.  S = max_j sum_c |q_c k_jc| / sqrt(D), Q = max_c |q_c| max_j sum_c |k_jc|
/ sqrt(D), A = sum_j w_j |v_j| per channel with the exact weights w_j, a the largest scale
of V.
* q is whole numbers of units of 2^-10 / 1.0625 of its largest channel or less, in two
  pieces, the second off by 2^-13 of a unit, and a neighbour's by a 16th of that: 2^-22 Q.
  A group's sum is exact up to 2^24 units / 16, beyond which nothing typical gets, and else off
  by 2^-24 S; joining its pieces, four scales, their sums and the factor in front are at most
  12 fp32 roundings.  - 7.5 sum(q) of a group is rounded once, 2^-24 7.5 32 max|q| a / 8, and
  the group's |k| are a / 16 at least and once 15 a / 16, 2.8 a together: 2^-21.5 Q.  So
  ds = 16 * 2^-24 S + 2^-20 Q.
* The exponential's argument is an fp32 difference of scores, of up to 1.45 * 2 S in its
  units, and a fused operation that adds 13: 2^-23 (3 S + 14) / 1.4.  The exponential itself
  and two rescalings: 3 * 2^-22.  So a weight's relative error is at most
  r = 2 (ds + 2^-23 (2.2 S + 10)) + 3 * 2^-22 (the first factor for e^x - 1).
* A weight times a scale in two fp16 pieces: 2^-21 of it, and 2^-24 where pieces are
  subnormal, the largest product being at least 2^13 a / 4 there: 2^-35 a per token in units
  of the largest weight, so n 2^-35 a 7.5 / 8 / l in the result, l = sum_j exp(s_j - max) >= 1.
* Sums: at most 16 tensor core steps of a cut-off fp32 (2^-23) each, then chains of
  n / 1024 fp32 additions per warp, 4 warps, and at most 64 shares; the weights' own sum is
  a chain of n / 64 additions: K = (n / 64 + 128) 2^-23, in numerator and denominator.
So the result is within (2 r + 2^-21 + 2 K) A + n 2^-35 a / l, the log-sum-exp within
r + K + ds + 2^-22 |lse|.
"""
import math

import numpy as np
import torch


def rotated(x, table, pos, pairs):
    """x [tokens][heads][D] in fp64, its first table.shape[1] channels rotated by the table's rows at pos."""
    R = table.shape[1]
    y = x.double().clone()
    c, s = table[pos].double()[:, None].chunk(2, -1)
    i = torch.arange(R // 2, device=x.device)
    a, b = (2 * i, 2 * i + 1) if pairs else (i, i + R // 2)
    xa, xb = x[..., a].double(), x[..., b].double()
    y[..., a], y[..., b] = xa * c - xb * s, xb * c + xa * s
    return y


def turn_size(x, table, pos, pairs):
    """Y of each channel (0 where nothing turns)."""
    R = table.shape[1]
    y = torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    c, s = table[pos].double().abs()[:, None].chunk(2, -1)
    i = torch.arange(R // 2, device=x.device)
    a, b = (2 * i, 2 * i + 1) if pairs else (i, i + R // 2)
    xa, xb = x[..., a].double().abs(), x[..., b].double().abs()
    y[..., a], y[..., b] = xa * c + xb * s, xb * c + xa * s
    return y


def near_rotated(got, x, table, pos, pairs):
    """Whether `got` is x rotated, within the bound above."""
    want, size = rotated(x, table, pos, pairs), turn_size(x, table, pos, pairs)
    tol = 2.0 ** -23 * size
    if got.dtype != torch.float32:
        u = torch.finfo(got.dtype).eps / 2
        tol = tol + u * (want.abs() + tol) + (2.0 ** -25 if got.dtype == torch.float16 else 2.0 ** -134)
    return bool(((got.double() - want).abs() <= tol).all())


def to_half(x):
    """fp64 rounded once to fp16 (torch rounds to fp32 in between: 3 scales of 48000 come out one step off)."""
    return torch.from_numpy(x.cpu().numpy().astype(np.float16)).to(x.device)


def held(x):
    """(values, scales) that a 4-bit cache holds of rows x [..][D] fp64: values fp64."""
    g = x.reshape(*x.shape[:-1], -1, 32)
    a = to_half(g.abs().amax(-1).clamp(max=65504.0))
    s = a.double()[..., None] / 8
    c = torch.where(s > 0, torch.floor(g / s), torch.zeros_like(g)).clamp(-8, 7)
    return ((c + 0.5) * s).reshape(x.shape), a


def rope_table(positions, R, base=10000.0, device="cuda"):
    f = base ** (-torch.arange(0, R, 2, dtype=torch.float64, device=device) / R)
    angle = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * f
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def pack(k, v):
    """Rows k, v [pages][heads][tokens][D] as pages of a 4-bit cache (codes by the rule, from fp64)."""
    n, H, P, D = k.shape
    G, parts = D // 32, []
    for x in (k, v):
        values, a = held(x.double())
        s = a.double()[..., None] / 8
        c = torch.where(s > 0, torch.round(values.reshape(n, H, P, G, 32) / s.clamp(min=1e-30) + 7.5), torch.full_like(s, 8))
        c = c.expand(n, H, P, G, 32).to(torch.uint8)
        codes = c[..., 0::2] | (c[..., 1::2] << 4)
        codes = codes.reshape(n, H, P // 16, 16, G, 16).transpose(3, 4).reshape(n, H, P // 16, 8 * D)
        a = a.reshape(n, H, P // 16, 2, 8, G).permute(0, 1, 2, 4, 5, 3).contiguous()
        parts += [codes, a.view(torch.uint8).reshape(n, H, P // 16, D)]
    return torch.cat(parts, -1).reshape(n, H, -1).contiguous()


def unpack(kv, D):
    """(K, V) [pages][heads][tokens][D] fp64 of 4-bit pages."""
    n, H, size = kv.shape
    b = kv.reshape(n, H, size // (18 * D), 18 * D)
    out = []
    for base in (0, 9 * D):
        codes = b[..., base:base + 8 * D].reshape(n, H, -1, D // 32, 16, 16).transpose(3, 4)
        c = torch.stack([codes & 15, codes >> 4], -1).reshape(n, H, -1, 16, D // 32, 32)
        a = b[..., base + 8 * D:base + 9 * D].contiguous().view(torch.float16).reshape(n, H, -1, 8, D // 32, 2)
        a = a.permute(0, 1, 2, 5, 3, 4).reshape(n, H, -1, 16, D // 32, 1).double()
        out.append(((c.double() - 7.5) * a / 8).reshape(n, H, -1, D))
    return out


def decode(q, K, V, table, lens):
    """(out, lse, tolerance of out, tolerance of lse) in fp64; K, V [pages][heads][page][D] fp64."""
    U, G, D = q.shape
    H, P = K.shape[1], K.shape[2]
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.full((U, G), -math.inf, dtype=torch.float64, device=q.device)
    tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    for u in range(U):
        s, h = divmod(u, H)
        n = min(max(int(lens[s]), 0), table.shape[1] * P)
        ids = table[s, : -(-n // P)].long() if n else table[s, :0].long()
        keep = torch.zeros(ids.numel() * P, dtype=torch.bool, device=q.device)
        keep[:n] = True
        good = (ids >= 0) & (ids < K.shape[0])
        keep &= good.repeat_interleave(P)
        ids = ids.clamp(0, K.shape[0] - 1)
        kk, vv = (x[ids, h].reshape(-1, D)[keep] for x in (K, V))
        if not kk.shape[0]:
            continue
        qq = q[u].double()
        x = qq @ kk.T / math.sqrt(D)
        S = (qq.abs() @ kk.abs().T / math.sqrt(D)).amax(1)
        Q = qq.abs().amax(1) * kk.abs().sum(1).amax() / math.sqrt(D)
        z = torch.logsumexp(x, 1)
        w = torch.exp(x - z[:, None])
        ds = 16 * 2.0 ** -24 * S + 2.0 ** -20 * Q
        r = 2 * (ds + 2.0 ** -23 * (2.2 * S + 10)) + 3 * 2.0 ** -22
        k = (n / 64 + 128) * 2.0 ** -23
        A = w @ vv.abs()
        big = vv.abs().amax() * 8 / 7                       # the largest scale is at most this
        l = torch.exp(z - x.amax(1))
        out[u], lse[u] = w @ vv, z
        tol[u] = (2 * r + 2.0 ** -21 + 2 * k)[:, None] * A + (n * 2.0 ** -35 * big / l)[:, None]
        tol_lse[u] = r + k + ds + 2.0 ** -22 * z.abs()
    return out, lse, tol, tol_lse
