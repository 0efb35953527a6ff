"""Plain 64-bit forms of the prompt and paged-cache operators, and how far a
kernel may be from them.

Notation: u = eps / 2 of the rows' type (a rounding is off by at most half a
step), w_j the exact softmax weights of a row, A = sum_j w_j |v_j| per channel,
S = max_j sum_c |q_c k_jc| / sqrt(D).

* A score is a fp32 sum of at most D exact products (of pieces of q, for the
  decode attention, that leave at most 2^-22 of |q_c|): it is off by at most
  ds = (D + 8) 2^-23 S, each addition counted as a full fp32 step because the
  tensor cores may cut instead of rounding.
* A weight exp(s - m) then has the relative error e^(ds) - 1 <= 2 ds (ds < 1/2),
  plus 2^-20 for the fp32 argument, the exponential and its rescalings.
* Sums over n tokens are chains of at most n / 16 + 64 fp32 additions
  (16 products per tensor core step; the split parts are joined in at most 64
  more): relative error (n / 16 + 64) 2^-23 of the summed magnitudes.  It
  enters numerator and denominator.
So with r = 2 ds + 2^-20 + (n / 16 + 64) 2^-23, a fp32 output is within 2 r A
of the exact one, a log-sum-exp within r + ds + 2^-22 |lse|, a token's mass
within 2 r of its own weight sum (plus one fp32 rounding of the running mass).

The prompt attention also rounds each weight to the rows' type before the
second product (u A) and the output at the end (u |o|).  In fp16 a weight below
2^-14 of the row's largest is a subnormal, off by at most 2^-25 in absolute
terms, against a denominator l = sum_j exp(s_j - m) >= 1: 2^-25 sum_j |v_j| / l.
"""
import math

import torch


def prefill(q, k, v, lq, lk, D):
    """(out, lse, tolerance of out, tolerance of lse) in fp64, one (sequence, head) at a time."""
    H, Hkv = q.shape[1], k.shape[1]
    u = torch.finfo(q.dtype).eps / 2
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=q.device)
    tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    q0 = k0 = 0
    for a, b in zip(lq, lk):
        if a and b:
            seen = torch.ones(a, b, dtype=torch.bool, device=q.device).tril(b - a)
            some = seen.any(1)
            for h in range(H):
                qq, kk, vv = (x.double() for x in (q[q0:q0 + a, h], k[k0:k0 + b, h // (H // Hkv)],
                                                   v[k0:k0 + b, h // (H // Hkv)]))
                s = (qq @ kk.T / math.sqrt(D)).masked_fill(~seen, -math.inf)[some]
                S = ((qq.abs() @ kk.abs().T) / math.sqrt(D)).masked_fill(~seen, 0)[some].amax(1)
                z = torch.logsumexp(s, 1)
                w = torch.exp(s - z[:, None])
                at = torch.nonzero(some)[:, 0] + q0
                out[at, h], lse[at, h] = w @ vv, z
                ds = (D + 8) * 2.0 ** -23 * S
                r = 2 * ds + 2.0 ** -20 + (b / 16 + 64) * 2.0 ** -23
                A = w @ vv.abs()
                tol[at, h] = 2 * r[:, None] * A + u * A + u * (w @ vv).abs() * (1 + u)
                if q.dtype == torch.float16:
                    l = torch.exp(z - s.amax(1))
                    few = seen[some].double() @ vv.abs()
                    tol[at, h] += 2.0 ** -25 * few / l[:, None] + 2.0 ** -25
                tol_lse[at, h] = r + ds + 2.0 ** -22 * z.abs()
        q0, k0 = q0 + a, k0 + b
    return out, lse, tol, tol_lse


def rows_of(pages, table, n, h):
    """The first n rows of head h that one row of a page table names (bad entries: None)."""
    P = pages.shape[2]
    t = table.tolist()
    keep = [i for i in range(n) if 0 <= t[i // P] < pages.shape[0]]
    idx = torch.tensor([t[i // P] for i in keep], dtype=torch.long, device=pages.device)
    slot = torch.tensor([i % P for i in keep], dtype=torch.long, device=pages.device)
    return pages[idx, h, slot], keep


def decode(q, k_pages, v_pages, table, lens):
    """(out, weights per token [units][cap], tolerance of out, tolerance of the weights) in fp64."""
    seqs, H, P, D = table.shape[0], k_pages.shape[1], k_pages.shape[2], k_pages.shape[3]
    cap = table.shape[1] * P
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    mass = torch.zeros(q.shape[0], cap, dtype=torch.float64, device=q.device)
    tol, tol_mass = torch.zeros_like(out), torch.zeros_like(mass)
    for u in range(seqs * H):
        s, h = divmod(u, H)
        n = min(max(int(lens[s]), 0), cap)
        kk, at = rows_of(k_pages, table[s], n, h)
        vv, _ = rows_of(v_pages, table[s], n, h)
        if not at:
            continue
        kk, vv, qq = kk.double(), vv.double(), q[u].double()
        x = qq @ kk.T / math.sqrt(D)
        w = torch.softmax(x, 1)
        S = (qq.abs() @ kk.abs().T / math.sqrt(D)).amax(1)
        ds = (D + 8) * 2.0 ** -23 * S
        r = (2 * ds + 2.0 ** -20 + (n / 16 + 64) * 2.0 ** -23)[:, None]
        out[u] = w @ vv
        tol[u] = 2 * r * (w @ vv.abs())
        at = torch.tensor(at, device=q.device)
        mass[u, at] = w.sum(0)
        tol_mass[u, at] = (2 * r * w).sum(0)
    return out, mass, tol, tol_mass


def kept_set(mass, n, keep, n_sink, n_recent):
    """The kept tokens of one unit, ascending."""
    if n <= keep:
        return list(range(n))
    m = [math.inf if math.isnan(x) else x for x in mass[:n]]
    nan = [math.isnan(x) for x in mass[:n]]
    middle = sorted(range(n_sink, n - n_recent), key=lambda t: (not nan[t], -m[t], t))
    return sorted(list(range(n_sink)) + middle[: keep - n_sink - n_recent] + list(range(n - n_recent, n)))


def cumulated(lens, device="cuda"):
    out = [0]
    for x in lens:
        out.append(out[-1] + x)
    return torch.tensor(out, dtype=torch.int32, device=device)


def pool(seqs, heads, D, page, pages_per_seq, dtype, seed=0, extra=0, layout="token", fill=None):
    """K and V pages and a scrambled page table; layout "token": [page][token][head][D] in
    memory, "head": [page][head][token][D]."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    count = seqs * pages_per_seq + extra
    shape = (count, page, heads, D) if layout == "token" else (count, heads, page, D)
    both = []
    for _ in range(2):
        x = torch.randn(shape, generator=g, device="cuda").to(dtype) if fill is None else \
            torch.full(shape, fill, dtype=dtype, device="cuda")
        both.append(x.permute(0, 2, 1, 3) if layout == "token" else x)
    order = torch.randperm(count, generator=g, device="cuda").to(torch.int32)
    table = order[: seqs * pages_per_seq].reshape(seqs, pages_per_seq).contiguous()
    return both[0], both[1], table, order[seqs * pages_per_seq:]
