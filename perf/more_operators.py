"""Cases of the rotated append and of the 4-bit paged cache: new rows appended to a paged cache of 16-bit rows with
the position rotation applied on the way (to the step's queries too), the same into a cache held in 4 bits, decode
attention of one new token per sequence over that cache, and its rows read back for the next chunk of a prompt.

A 4-bit cache is a uint8 tensor [pages][kv_heads][page_tokens / 16 * 18 * D].  Blocks of 16 tokens lie one after the
other, 18 * D bytes each: the codes of K [D / 32][16 tokens][16 bytes] (channel 2 b of a group of 32 in the low four
bits of byte b, channel 2 b + 1 in the high four), the scales a of K, fp16, [8][D / 32][2] (tokens r and r + 8 of the
block side by side), then codes and scales of V.  A code c stands for (c - 7.5) a / 8.

With ``own`` false, ``run`` computes the operators with elementary torch operations (rotated keys in 64 bits before
they are coded, where a value may lie next to a border, everything else in 32 bits, rounded once at the end); with
``own`` true it makes the library's calls.  ``exact`` computes them in 64 bits from the definition.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the rows and queries of one decode step of 61 sessions, 8 KV heads x 4 query heads
        dict(name="rope step", op="rope", dtype="bf16", seqs=61, kv_heads=8, G=4, D=128, rot=128, pairs=False, n=4096,
             page=16, new=1),
        # a chunk of five prompts: half of the channels rotated, neighbours as pairs, few heads
        dict(name="rope chunk", op="rope", dtype="fp16", seqs=5, kv_heads=2, G=3, D=96, rot=48, pairs=True, n=1500,
             page=32, new=301),
        # the rows and queries of 16 packed prompts of ragged lengths, sliced from a fused projection
        dict(name="rope prompts", op="rope", dtype="bf16", seqs=16, kv_heads=8, G=4, D=128, rot=128, pairs=False, n=4096,
             page=64, new=2048),
        # one decode step of 61 sessions into a 4-bit cache, and what it holds then
        dict(name="append4 step", op="append4", dtype="bf16", seqs=61, kv_heads=8, G=4, D=128, rot=128, pairs=False,
             n=4096, page=16, new=1),
        # 16 packed prompts into a 4-bit cache, and what it holds then
        dict(name="append4 prompts", op="append4", dtype="bf16", seqs=16, kv_heads=8, G=4, D=128, rot=128, pairs=False,
             n=4096, page=64, new=2048),
        # one session's tokens read back for the next chunk of its prompt
        dict(name="read4 12k", op="read4", dtype="bf16", seqs=1, kv_heads=8, D=128, n=12000, page=64, ragged=False),
        # a batch of short sessions read back, 64 channels, fp16
        dict(name="read4 23x700", op="read4", dtype="fp16", seqs=23, kv_heads=4, D=64, n=700, page=16, ragged=True),
        # one user's short session: latency counts
        dict(name="attn4 one 4k", op="attn4", seqs=1, kv_heads=8, G=4, D=128, n=4096, page=16, ragged=False),
        # one long session
        dict(name="attn4 one 128k", op="attn4", seqs=1, kv_heads=8, G=4, D=128, n=131072, page=64, ragged=False),
        # 32 sessions of ragged lengths up to 32k tokens
        dict(name="attn4 32x32k", op="attn4", seqs=32, kv_heads=8, G=4, D=128, n=32768, page=64, ragged=True),
        # many short sessions, 8 query heads per KV head, 64 channels
        dict(name="attn4 61x3k", op="attn4", seqs=61, kv_heads=4, G=8, D=64, n=3001, page=32, ragged=True),
        # an odd layout: 3 KV heads x 5 query heads, 96 channels
        dict(name="attn4 7x9k", op="attn4", seqs=7, kv_heads=3, G=5, D=96, n=9001, page=128, ragged=True),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append4", "attn4", "attn4", "read4"])
    case = dict(op=op, kv_heads=rng.choice([1, 2, 3, 4, 8]), D=rng.choice([32, 64, 96, 128, 128, 128]),
                page=rng.choice([16, 32, 64, 128]))
    if op == "attn4":
        n = _log(rng, 1, 60000)
        case.update(seqs=max(1, min(_log(rng, 1, 64), 600000 // n)), G=rng.randint(1, 8), n=n, ragged=rng.random() < 0.8)
    elif op == "read4":
        n = _log(rng, 1, 12000)
        case.update(dtype=rng.choice(["bf16", "fp16"]), seqs=max(1, min(_log(rng, 1, 32), 24000 // n)), n=n,
                    ragged=rng.random() < 0.8)
    else:
        n = _log(rng, 64, 4096)
        D = case["D"] = rng.choice([32, 64, 96, 128, 128, 128] if op == "append4" else [128, 128, 8 * rng.randint(1, 16)])
        case.update(dtype=rng.choice(["bf16", "fp16"]), seqs=_log(rng, 1, 64), G=rng.choice([1, 2, 3, 4, 8]), n=n,
                    rot=rng.choice([D, D, 2 * rng.randint(1, D // 2)]), pairs=rng.random() < 0.3,
                    new=rng.choice([1, _log(rng, 1, min(n, 400))]))
    return case


def _lengths(count, n, ragged, salt=0):
    """The lengths of a batch, the longest n: a matter of the case, not of the seed."""
    if not ragged:
        return [n] * count
    r = random.Random(count * 1000003 + n * 7 + salt)
    return [n] + [r.randint(max(1, n // 8), n) for _ in range(count - 1)]


def _append_lengths(case):
    """(tokens cached before, new tokens) of each sequence; together at most n."""
    new = _lengths(case["seqs"], case["new"], True, 1)
    old = _lengths(case["seqs"], case["n"] - case["new"] + 1, True, 2)
    return [x - 1 for x in old], new


def work(case):
    D, H = case["D"], case["kv_heads"]
    if case["op"] == "attn4":
        tokens = sum(_lengths(case["seqs"], case["n"], case["ragged"]))
        return {"bytes": 9 * D // 8 * H * tokens + 8 * D * case["seqs"] * H * case["G"],
                "flops": 4 * D * H * case["G"] * tokens}
    if case["op"] == "read4":
        tokens = sum(_lengths(case["seqs"], case["n"], case["ragged"]))
        return {"bytes": (9 * D // 8 + 4 * D) * H * tokens, "flops": 2 * D * H * tokens}
    old, new = _append_lengths(case)
    tokens = sum(new)
    seen = set()
    for a, b in zip(old, new):
        seen.update(range(a, a + b))
    q_bytes = case["G"] * D * (2 + (4 if case["new"] == 1 else 2))     # read, and written rotated
    if case["op"] == "rope":
        kv_bytes = 8 * D
    else:   # written in 4 bits, and read from there and written as rows
        kv_bytes = 4 * D + 9 * D // 8 + 4 * D
    return {"bytes": tokens * H * (kv_bytes + q_bytes) + len(seen) * case["rot"] * 4,
            "flops": 3 * case["rot"] * H * (1 + case["G"]) * tokens}


# ------------------------------------------------------------------ inputs
def _cumulated(lens):
    out = [0]
    for x in lens:
        out.append(out[-1] + x)
    return torch.tensor(out, dtype=torch.int32, device="cuda")


def _page_table(g, seqs, per):
    """A page table [seqs][per], the pages in no order."""
    return torch.randperm(seqs * per, generator=g, device="cuda").to(torch.int32).reshape(seqs, per)


def _pack(k, v):
    """Rows k, v [pages][heads][tokens][D] fp32 as 4-bit pages."""
    n, H, P, D = k.shape
    g, parts = D // 32, []
    for x in (k, v):
        x = x.reshape(n, H, P // 16, 16, g, 32)
        a = x.abs().amax(-1).clamp(max=65504).half()
        c = (torch.floor(x / (a.float() / 8).clamp(min=1e-30)[..., None]).clamp(-8, 7) + 8).to(torch.uint8)
        codes = (c[..., 0::2] | (c[..., 1::2] << 4)).transpose(3, 4)                   # [..][g][16][16]
        scales = a.reshape(n, H, P // 16, 2, 8, g).permute(0, 1, 2, 4, 5, 3)          # [..][8][g][2]
        parts += [codes.reshape(n, H, P // 16, D * 8), scales.contiguous().view(torch.uint8).reshape(n, H, P // 16, D)]
    return torch.cat(parts, -1).reshape(n, H, -1)


def _pages4(case, g, pages):
    """4-bit pages of keys, whose channels differ in size, and values."""
    H, D, P = case["kv_heads"], case["D"], case["page"]
    out = torch.empty(pages, H, P // 16 * 18 * D, dtype=torch.uint8, device="cuda")
    size = torch.exp(0.5 * torch.randn(H, 1, D, generator=g, device="cuda"))
    step = max(1, (1 << 25) // (H * P * D))
    for i in range(0, pages, step):
        m = min(step, pages - i)
        k, v = (torch.randn(m, H, P, D, generator=g, device="cuda") for _ in range(2))
        out[i:i + m] = _pack(k * size, v)
    return out


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    H, D, S, P = case["kv_heads"], case["D"], case["seqs"], case["page"]
    per = -(-case["n"] // P)
    st = {"case": case, "table": _page_table(g, S, per)}
    if case["op"] in ("attn4", "read4"):
        lens = _lengths(S, case["n"], case["ragged"])
        st.update(kv=_pages4(case, g, S * per), lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
        if case["op"] == "attn4":
            st["q"] = 2 * torch.randn(S * H, case["G"], D, generator=g, device="cuda")
            if own:   # what a program keeps from call to call
                from bit_plane_kv_gb300 import binding as B
                st["pages"] = B.make_nibble_pages(st["kv"], st["table"], D)
                st["ws"] = B.alloc_nibble_workspace(st["pages"], G=case["G"])
        else:
            st.update(first=torch.zeros_like(st["lens"]), cu=_cumulated(lens), total=sum(lens),
                      seq=torch.repeat_interleave(torch.arange(S), torch.tensor(lens)).cuda())
        return st
    dt, R, Hq = DTYPES[case["dtype"]], case["rot"], H * case["G"]
    old, new = _append_lengths(case)
    qkv = torch.randn(sum(new), Hq + 2 * H, D, generator=g, device="cuda").to(dt)   # a fused projection's output
    # cos and sin of position * 10000^(-2 i / R), the angles in 64 bits
    freq = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64, device="cuda") / R)
    angle = torch.arange(case["n"], dtype=torch.float64, device="cuda")[:, None] * freq
    st.update(q=qkv[:, :Hq], k_new=qkv[:, Hq:Hq + H], v_new=qkv[:, Hq + H:], start=torch.tensor(old, dtype=torch.int32).cuda(),
              cu=_cumulated(new), total=sum(new), seq=torch.repeat_interleave(torch.arange(S), torch.tensor(new)).cuda(),
              rope=torch.cat([angle.cos(), angle.sin()], 1).float(), q_type=torch.float32 if case["new"] == 1 else dt)
    if case["op"] == "rope":
        st["k_pages"], st["v_pages"] = (torch.zeros(S * per, P, H, D, dtype=dt, device="cuda").permute(0, 2, 1, 3)
                                        for _ in range(2))
    else:
        st["kv"] = torch.zeros(S * per, H, P // 16 * 18 * D, dtype=torch.uint8, device="cuda")
    return st


# ------------------------------------------------------------------ one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return _own(state, op)
    return {"rope": _rope, "append4": _append4, "read4": _read4, "attn4": _attn4}[op](state)


def _own(st, op):
    from bit_plane_kv_gb300 import binding as B
    c = st["case"]
    if op == "attn4":
        return {"out": B.fathom_nibble_attn(st["pages"], st["q"], st["kv"], st["table"], st["lens"], st["ws"])}
    cu = None if c.get("new") == 1 else st["cu"]     # a decode step: one token per sequence
    if op == "rope":
        pages = B.make_pages(st["k_pages"], st["table"])
        _, _, q = B.fathom_paged_append_rope(pages, st["k_pages"], st["v_pages"], st["table"], st["k_new"], st["v_new"],
                                             st["start"], st["rope"], cu, interleaved=c["pairs"], q=st["q"],
                                             q_dtype=st["q_type"])
        return {"k": st["k_pages"], "v": st["v_pages"], "q": q}
    pages = B.make_nibble_pages(st["kv"], st["table"], c["D"])
    q, first = {}, st.get("first")
    if op == "append4":
        first = st["start"]
        q["q"] = B.fathom_nibble_append(pages, st["kv"], st["table"], st["k_new"], st["v_new"], first, cu,
                                        rope=st["rope"], interleaved=c["pairs"], q=st["q"], q_dtype=st["q_type"])[1]
    k, v = B.fathom_nibble_read(pages, st["kv"], st["table"], first, st["cu"], st["total"], dtype=DTYPES[c["dtype"]])
    return {"k": k, "v": v, **q}


def _places(st):
    """(position, page, place in the page) of each packed token."""
    seq, start, P = st["seq"], st.get("first", st.get("start")), st["case"]["page"]
    pos = (start[seq] + torch.arange(seq.shape[0], device=seq.device) - st["cu"][seq]).long()
    return pos, st["table"][seq, pos // P].long(), pos % P


def _rotated(st, x, pos):
    """x [tokens][heads][D] rotated, in x's type (32 or 64 bits)."""
    R, half = st["case"]["rot"], st["case"]["rot"] // 2
    row = st["rope"][pos].to(x.dtype)[:, None]
    cos, sin = row[..., :half], row[..., half:]
    a, b = (slice(0, R, 2), slice(1, R, 2)) if st["case"]["pairs"] else (slice(0, half), slice(half, R))
    y = x.clone()
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., b] * cos + x[..., a] * sin
    return y


def _rope(st):
    pos, page, slot = _places(st)
    st["k_pages"][page, :, slot] = _rotated(st, st["k_new"].float(), pos).to(st["k_new"].dtype)
    st["v_pages"][page, :, slot] = st["v_new"]
    return {"k": st["k_pages"], "v": st["v_pages"], "q": _rotated(st, st["q"].float(), pos).to(st["q_type"])}


def _append4(st):
    c = st["case"]
    H, D, T = c["kv_heads"], c["D"], st["total"]
    pos, page, slot = _places(st)
    blocks = st["kv"].view(st["kv"].shape[0], H, -1, 18 * D)
    at = (page[:, None], torch.arange(H, device=page.device), (slot // 16)[:, None])
    t, out = slot % 16, {}
    group, byte = torch.arange(D // 32, device=page.device), torch.arange(16, device=page.device)
    code_at = group[:, None] * 256 + t[:, None, None] * 16 + byte                      # [T][groups][16]
    scale_at = ((t % 8)[:, None] * (D // 32) + group) * 4 + (t // 8)[:, None] * 2      # [T][groups]
    for name, x, base in (("k", _rotated(st, st["k_new"].double(), pos), 0), ("v", st["v_new"].double(), 9 * D)):
        x = x.reshape(T, H, D // 32, 32)
        a = x.abs().amax(-1).clamp(max=65504).half()
        s = a.double() / 8
        code = torch.where(s[..., None] > 0, torch.floor(x / s.clamp(min=1e-30)[..., None]), torch.zeros_like(x))
        code = code.clamp(-8, 7) + 8
        u = code.to(torch.uint8)
        blocks[(*(i[..., None, None] for i in at), base + code_at[:, None])] = u[..., 0::2] | (u[..., 1::2] << 4)
        both = a.contiguous().view(torch.uint8).reshape(T, H, D // 32, 2)
        for e in (0, 1):
            blocks[(*(i[..., None] for i in at), base + 8 * D + scale_at[:, None] + e)] = both[..., e]
        out[name] = ((code.float() - 7.5) * (a.float() / 8)[..., None]).reshape(T, H, D).to(st["k_new"].dtype)
    out["q"] = _rotated(st, st["q"].float(), pos).to(st["q_type"])
    return out


def _values(blocks, D):
    """K and V [..][16][D] fp32 of blocks [..][18 D]."""
    out, lead = [], blocks.shape[:-1]
    for base in (0, 9 * D):
        b = blocks[..., base:base + 8 * D].reshape(*lead, D // 32, 16, 16)
        a = blocks[..., base + 8 * D:base + 9 * D].contiguous().view(torch.float16).reshape(*lead, 8, D // 32, 2)
        a = a.float().movedim(-1, -3).reshape(*lead, 16, D // 32)                      # [..][token][group]
        c = torch.stack([b & 15, b >> 4], -1).reshape(*lead, D // 32, 16, 32).transpose(-3, -2)
        out.append(((c.float() - 7.5) * (a / 8)[..., None]).reshape(*lead, 16, D))
    return out


def _read4(st):
    c = st["case"]
    H, D, P, S = c["kv_heads"], c["D"], c["page"], c["seqs"]
    blocks = st["kv"][st["table"].long()].reshape(S, -1, H, P // 16, 18 * D).transpose(2, 3)    # [S][pages][blocks][H]
    pos, _, _ = _places(st)
    return {x: y.transpose(3, 4).reshape(S, -1, H, D)[st["seq"], pos].to(DTYPES[c["dtype"]])
            for x, y in zip("kv", _values(blocks, D))}


def _attn4(st):
    c = st["case"]
    H, D, P, S = c["kv_heads"], c["D"], c["page"], c["seqs"]
    blocks = st["kv"][st["table"].long()].transpose(1, 2).reshape(S * H, -1, 18 * D)
    k, v = (x.reshape(S * H, -1, D) for x in _values(blocks, D))
    s = torch.matmul(st["q"], k.transpose(1, 2)).mul_(1.0 / math.sqrt(D))
    lens = st["lens"].repeat_interleave(H)
    s.masked_fill_(torch.arange(s.shape[-1], device=s.device) >= lens[:, None, None], float("-inf"))
    p = s.sub_(s.amax(-1, keepdim=True)).exp_()
    return {"out": torch.matmul(p, v) / p.sum(-1, keepdim=True)}


# ------------------------------------------------------------------ the definition, in 64 bits
def _turned(x, rope, first, pairs):
    """x [tokens][heads][D] at the positions from `first` on, as complex numbers times cos + i sin."""
    R = rope.shape[1]
    z = torch.complex(*rope[first:first + x.shape[0]].double().chunk(2, 1))[:, None]
    x = x.double()
    if pairs:
        y = torch.view_as_real(torch.view_as_complex(x[..., :R].reshape(*x.shape[:2], -1, 2).contiguous()) * z).flatten(2)
    else:
        y = torch.complex(*x[..., :R].contiguous().chunk(2, 2)) * z
        y = torch.cat([y.real, y.imag], 2)
    return torch.cat([y, x[..., R:]], 2)


def _held(x):
    """What a 4-bit cache holds of x [..][D]."""
    y = torch.empty_like(x)
    for i in range(0, x.shape[-1], 32):
        part = x[..., i:i + 32]
        s = part.abs().amax(-1, keepdim=True).clamp(max=65504).to(torch.float16).double() / 8
        m = torch.floor(part / torch.where(s > 0, s, torch.ones_like(s)))
        y[..., i:i + 32] = (torch.clamp(m, -8, 7) + 0.5) * s
    return y


def exact(case, seed):
    st = prepare(case, seed)
    H, D, S, P = case["kv_heads"], case["D"], case["seqs"], case["page"]
    if case["op"] in ("rope", "append4"):
        old, new = _append_lengths(case)
        k, v, q, at = [], [], [], 0
        for a, b in zip(old, new):
            for rows, x in ((k, st["k_new"]), (q, st["q"])):
                rows.append(_turned(x[at:at + b], st["rope"], a, case["pairs"]))
            v.append(st["v_new"][at:at + b].double())
            at += b
        q = torch.cat(q)
        if case["op"] == "append4":
            return {"k": _held(torch.cat(k)), "v": _held(torch.cat(v)), "q": q}
        pages = {}
        for name, rows in (("k", k), ("v", v)):
            pages[name] = st[name + "_pages"].double()
            for s in range(S):
                done = 0
                while done < new[s]:   # page by page
                    p, slot = divmod(old[s] + done, P)
                    m = min(P - slot, new[s] - done)
                    pages[name][int(st["table"][s, p]), :, slot:slot + m] = rows[s][done:done + m].transpose(0, 1)
                    done += m
        return {**pages, "q": q}

    def held_rows(s, h, n):
        """K and V of the first n tokens, from the bytes, token by token of a block."""
        b = st["kv"][st["table"][s, : -(-n // P)].long(), h].reshape(-1, 18 * D)
        both = []
        for base in (0, 9 * D):
            rows = torch.empty(b.shape[0], 16, D, dtype=torch.float64, device="cuda")
            scale = b[:, base + 8 * D:base + 9 * D].contiguous().view(torch.float16).double()
            for t in range(16):
                for g in range(D // 32):
                    code = b[:, base + g * 256 + t * 16:base + g * 256 + t * 16 + 16].double()
                    high = torch.floor(code / 16)
                    a = scale[:, (t % 8 * (D // 32) + g) * 2 + t // 8, None] / 8
                    rows[:, t, 32 * g:32 * g + 32:2] = (code - 16 * high - 7.5) * a
                    rows[:, t, 32 * g + 1:32 * g + 32:2] = (high - 7.5) * a
            both.append(rows.reshape(-1, D)[:n])
        return both

    lens = _lengths(S, case["n"], case["ragged"])
    if case["op"] == "read4":
        rows = [[held_rows(s, h, lens[s]) for h in range(H)] for s in range(S)]
        return {x: torch.cat([torch.stack([r[i] for r in one], 1) for one in rows]) for i, x in enumerate("kv")}
    out = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
    for u in range(S * H):
        k, v = held_rows(u // H, u % H, lens[u // H])
        out[u] = torch.softmax(st["q"][u].double() @ k.T / math.sqrt(D), 1) @ v
    return {"out": out}
