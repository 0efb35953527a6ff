"""Cases of the prompt and paged-cache operators: prefill attention over packed prompts, the append of
new rows to a paged cache, decode attention of one new token over it (with the attention weight that each
cached token has drawn, its "mass"), and the eviction of the tokens with the least mass.

With ``own`` false, ``run`` computes the operators with elementary torch operations in 32 bits, rounded
once at the end; with ``own`` true it makes the library's calls.  ``exact`` computes them in 64 bits,
one unit at a time.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
N_SINK, N_RECENT = 4, 32


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a handful of one-line prompts, as a chat server takes them in: latency counts
        dict(name="prefill short", op="prefill", dtype="fp16", seqs=5, kv_heads=8, G=1, D=64, n=61, chunk=0,
             ragged=True),
        # a batch of prompts of ragged lengths packed into one call (8 KV heads x 4 query heads, 128 channels)
        dict(name="prefill packed", op="prefill", dtype="bf16", seqs=12, kv_heads=8, G=4, D=128, n=2048, chunk=0,
             ragged=True),
        # the last chunk of a long prompt, against all the keys before it; G = 2, channels not a power of two
        dict(name="prefill chunk", op="prefill", dtype="fp16", seqs=2, kv_heads=8, G=2, D=96, n=12000, chunk=1000,
             ragged=True),
        # one long prompt
        dict(name="prefill 16k", op="prefill", dtype="bf16", seqs=1, kv_heads=8, G=4, D=128, n=16384, chunk=0,
             ragged=False),
        # one user's short session
        dict(name="decode one 4k", op="decode", dtype="bf16", seqs=1, kv_heads=8, G=4, D=128, n=4096, page=16,
             mass=False, ragged=False),
        # 32 sessions of ragged lengths up to 32k tokens
        dict(name="decode 32x32k", op="decode", dtype="bf16", seqs=32, kv_heads=8, G=4, D=128, n=32768, page=64,
             mass=False, ragged=True),
        # many short sessions, 8 query heads per KV head, 64 channels, fp16
        dict(name="decode 61x3k", op="decode", dtype="fp16", seqs=61, kv_heads=4, G=8, D=64, n=3001, page=32,
             mass=False, ragged=True),
        # 8 sessions whose cache keeps each token's attention mass for a later eviction
        dict(name="decode mass 8x16k", op="decode", dtype="bf16", seqs=8, kv_heads=8, G=4, D=128, n=16384, page=64,
             mass=True, ragged=True),
        # the rows of one decode step of 61 sessions
        dict(name="append step", op="append", dtype="bf16", seqs=61, kv_heads=8, D=128, n=4096, page=16, new=1),
        # the rows of 16 packed prompts of ragged lengths, sliced from a fused projection
        dict(name="append prompts", op="append", dtype="bf16", seqs=16, kv_heads=8, D=128, n=4096, page=64,
             new=2048),
        # one session cut back to a quarter of its length
        dict(name="evict one 8k", op="evict", dtype="bf16", seqs=1, kv_heads=8, D=128, n=8192, page=16, keep=2048,
             ragged=False),
        # 32 sessions of ragged lengths cut back to 4096 tokens each
        dict(name="evict 32x16k", op="evict", dtype="bf16", seqs=32, kv_heads=8, D=128, n=16384, page=64, keep=4096,
             ragged=True),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "decode", "decode", "append", "evict"])
    case = dict(op=op, dtype=rng.choice(["bf16", "fp16"]), kv_heads=rng.choice([1, 2, 3, 4, 8]),
                D=rng.choice([64, 128, 128, 128, 8 * rng.randint(2, 16)]))
    if op == "prefill":
        n = _log(rng, 1, 9000)
        case.update(seqs=max(1, min(_log(rng, 1, 24), 24000 // n)), G=rng.choice([1, 2, 3, 4, 8]), n=n,
                    chunk=rng.choice([0, 0, _log(rng, 1, n)]), ragged=rng.random() < 0.8)
    elif op == "decode":
        n = _log(rng, 1, 40000)
        case.update(seqs=max(1, min(_log(rng, 1, 64), 400000 // n)), G=rng.choice([1, 2, 3, 4, 6, 8]), n=n,
                    page=rng.choice([16, 32, 64, 128]), mass=rng.random() < 0.4, ragged=rng.random() < 0.8)
    elif op == "append":
        n = _log(rng, 64, 8000)
        case.update(seqs=_log(rng, 1, 64), n=n, page=rng.choice([16, 32, 64, 128]),
                    new=rng.choice([1, _log(rng, 1, max(1, min(n, 1500)))]))
    else:
        n = _log(rng, 100, 20000)
        case.update(seqs=max(1, min(_log(rng, 1, 32), 400000 // n)), n=n, page=rng.choice([16, 32, 64, 128]),
                    keep=_log(rng, N_SINK + N_RECENT, max(N_SINK + N_RECENT, n // 2)), ragged=rng.random() < 0.8)
    return case


def _lengths(count, n, ragged, salt=0):
    """The lengths of a batch, the longest n: a matter of the case, not of the seed."""
    if not ragged:
        return [n] * count
    r = random.Random(count * 1000003 + n * 7 + salt)
    return [n] + [r.randint(max(1, n // 8), n) for _ in range(count - 1)]


def _prompt_lengths(case):
    """(new tokens, tokens in all) of each sequence."""
    k = _lengths(case["seqs"], case["n"], case["ragged"])
    q = [min(x, case["chunk"]) if case["chunk"] else x for x in k]
    return q, k


def _append_lengths(case):
    """(tokens cached before, new tokens) of each sequence; together at most n."""
    new = _lengths(case["seqs"], case["new"], True, 1)
    old = _lengths(case["seqs"], case["n"] - case["new"] + 1, True, 2)
    return [x - 1 for x in old], new


def work(case):
    D, H = case["D"], case["kv_heads"]
    if case["op"] == "prefill":
        q, k = _prompt_lengths(case)
        pairs = sum(a * b - a * (a - 1) // 2 for a, b in zip(q, k))   # query i sees keys 0 .. i + (b - a)
        return {"bytes": 2 * D * H * (2 * case["G"] * sum(q) + 2 * sum(k)), "flops": 4 * D * H * case["G"] * pairs}
    if case["op"] == "decode":
        tokens = sum(_lengths(case["seqs"], case["n"], case["ragged"]))
        rows = case["seqs"] * H * case["G"]
        return {"bytes": 4 * D * H * tokens + 8 * D * rows + (8 * H * tokens if case["mass"] else 0),
                "flops": 4 * D * H * case["G"] * tokens}
    if case["op"] == "append":
        return {"bytes": 8 * D * H * sum(_append_lengths(case)[1]), "flops": 0}
    lens = _lengths(case["seqs"], case["n"], case["ragged"])
    kept = sum(min(x, case["keep"]) for x in lens)
    return {"bytes": H * (4 * sum(lens) + kept * (8 * D + 8)), "flops": 0}


# ------------------------------------------------------------------ inputs
def _cumulated(lens, device):
    out = [0]
    for x in lens:
        out.append(out[-1] + x)
    return torch.tensor(out, dtype=torch.int32, device=device)


def _pool(case, g, tokens, extra_pages, fill):
    """K and V pages [pages][kv_heads][page][D] (held as [pages][page][kv_heads][D], as a projection
    writes them) and a page table [seqs][pages per sequence], the pages in no order."""
    page, seqs = case["page"], case["seqs"]
    per = -(-tokens // page)
    count = seqs * per + extra_pages
    shape = (count, page, case["kv_heads"], case["D"])
    dt = DTYPES[case["dtype"]]
    pools = []
    for _ in range(2):
        p = torch.zeros(shape, dtype=dt, device="cuda")
        if fill:
            p.normal_(generator=g)
        pools.append(p.permute(0, 2, 1, 3))
    order = torch.randperm(count, generator=g, device="cuda").to(torch.int32)
    return pools[0], pools[1], order[: seqs * per].reshape(seqs, per).contiguous(), order[seqs * per:]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    H, D, dt = case["kv_heads"], case["D"], DTYPES[case["dtype"]]
    st = {"case": case}
    if case["op"] == "prefill":
        lq, lk = _prompt_lengths(case)
        # keys and values as slices of one fused projection's output, tokens outermost
        kv = torch.randn(sum(lk), 2 * H, D, generator=g, device="cuda").to(dt)
        st.update(q=(2 * torch.randn(sum(lq), H * case["G"], D, generator=g, device="cuda")).to(dt), k=kv[:, :H],
                  v=kv[:, H:], cu_q=_cumulated(lq, "cuda"), cu_k=_cumulated(lk, "cuda"))
        # where the packed tokens lie in a padded batch, for the plain form
        st.update(pad_q=_padded(lq), pad_k=_padded(lk), lq=torch.tensor(lq, device="cuda"),
                  lk=torch.tensor(lk, device="cuda"))
    elif case["op"] == "decode":
        lens = _lengths(case["seqs"], case["n"], case["ragged"])
        kp, vp, table, _ = _pool(case, g, case["n"], 0, True)
        st.update(k_pages=kp, v_pages=vp, table=table, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                  q=2 * torch.randn(case["seqs"] * H, case["G"], D, generator=g, device="cuda"))
        if case["mass"]:
            cap = table.shape[1] * case["page"]
            st["mass"] = torch.rand(case["seqs"] * H, cap, generator=g, device="cuda")
    elif case["op"] == "append":
        old, new = _append_lengths(case)
        kp, vp, table, _ = _pool(case, g, case["n"], 0, False)
        kv = torch.randn(sum(new), 2 * H, D, generator=g, device="cuda").to(dt)
        seq = torch.repeat_interleave(torch.arange(case["seqs"]), torch.tensor(new)).cuda()
        st.update(k_pages=kp, v_pages=vp, table=table, k_new=kv[:, :H], v_new=kv[:, H:], seq=seq,
                  start=torch.tensor(old, dtype=torch.int32, device="cuda"), cu_new=_cumulated(new, "cuda"))
    else:
        lens = _lengths(case["seqs"], case["n"], case["ragged"])
        keep_pages = -(-case["keep"] // case["page"])
        kp, vp, table, free = _pool(case, g, case["n"], case["seqs"] * keep_pages, True)
        cap = table.shape[1] * case["page"]
        # attention mass is heavy-tailed, and nothing for some tokens
        mass = torch.exp(2 * torch.randn(case["seqs"] * H, cap, generator=g, device="cuda"))
        mass[torch.rand(mass.shape, generator=g, device="cuda") < 0.1] = 0
        st.update(k_pages=kp, v_pages=vp, table=table, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                  mass=mass, dst=free.reshape(case["seqs"], keep_pages).contiguous(),
                  mass_out=torch.zeros(case["seqs"] * H, keep_pages * case["page"], device="cuda"))
    if own and case["op"] != "prefill":   # what a program keeps from call to call: the plan and its workspace
        from bit_plane_kv_gb300 import binding as B
        st["pages"] = B.make_pages(st["k_pages"], st["table"])
        if case["op"] == "decode":
            st["ws"] = B.alloc_paged_workspace(st["pages"], G=case["G"], mass=case["mass"])
    return st


def _padded(lens):
    """(index of each place of the padded batch [seqs][longest] in the packed tokens, index of each packed
    token in the padded batch)."""
    n, L = torch.tensor(lens), max(lens)
    first = torch.cumsum(n, 0) - n
    at = first[:, None] + torch.arange(L)
    inside = torch.arange(L) < n[:, None]
    return torch.where(inside, at, 0).cuda(), torch.nonzero(inside.reshape(-1)).reshape(-1).cuda()


# ------------------------------------------------------------------ one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return _own(state, op)
    return {"prefill": _prefill, "decode": _decode, "append": _append, "evict": _evict}[op](state)


def _own(st, op):
    from bit_plane_kv_gb300 import binding as B
    if op == "prefill":
        out, lse = B.fathom_prefill_attn(st["q"], st["k"], st["v"], st["cu_q"], st["cu_k"], want_lse=True)
        return {"out": out, "lse": lse}
    if op == "decode":
        out = B.fathom_paged_attn(st["pages"], st["q"], st["k_pages"], st["v_pages"], st["table"], st["lens"],
                                  st["ws"], mass=st.get("mass"))
        return {"out": out, "mass": st["mass"]} if "mass" in st else {"out": out}
    if op == "append":
        B.fathom_paged_append(st["pages"], st["k_pages"], st["v_pages"], st["table"], st["k_new"], st["v_new"],
                              st["start"], st["cu_new"])
        return {"k": st["k_pages"], "v": st["v_pages"]}
    kept, lens, mass = B.fathom_paged_evict(st["pages"], st["k_pages"], st["v_pages"], st["table"], st["lens"],
                                            st["mass"], st["case"]["keep"], st["dst"], n_sink=N_SINK,
                                            n_recent=N_RECENT, mass_out=st["mass_out"])
    return {"kept": kept, "lens": lens, "mass": mass, "k": _rows(st["k_pages"], st["dst"]),
            "v": _rows(st["v_pages"], st["dst"])}


def _rows(pages, table):
    """The rows that a page table names, [seqs][kv_heads][tokens][D]."""
    p = pages[table.long()]                                      # [seqs][pages][heads][page][D]
    return p.transpose(1, 2).reshape(p.shape[0], p.shape[2], -1, p.shape[4])


def _softmax_parts(s):
    """exp(s - m) in place, its row sums and m (0 where a row has no finite score)."""
    m = s.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p = s.sub_(m).exp_()
    return p, p.sum(-1, keepdim=True), m


def _prefill(st):
    c = st["case"]
    H, G, D, S = c["kv_heads"], c["G"], c["D"], c["seqs"]
    (at_q, from_q), (at_k, _) = st["pad_q"], st["pad_k"]
    Lq, Lk = at_q.shape[1], at_k.shape[1]
    q = st["q"].float()[at_q].reshape(S, Lq, H, G, D).permute(0, 2, 3, 1, 4).reshape(S, H, G * Lq, D)
    k = st["k"].float()[at_k].permute(0, 2, 3, 1)                # [S][H][D][Lk]
    v = st["v"].float()[at_k].permute(0, 2, 1, 3)                # [S][H][Lk][D]
    s = torch.matmul(q, k).mul_(1.0 / math.sqrt(D)).reshape(S, H, G, Lq, Lk)
    i = torch.arange(Lq, device=s.device)[None, :, None] + (st["lk"] - st["lq"])[:, None, None]
    j = torch.arange(Lk, device=s.device)[None, None, :]
    s.masked_fill_((j > i)[:, None, None], float("-inf"))        # causal; the padded keys lie behind every query
    p, l, m = _softmax_parts(s)
    o = torch.matmul(p.reshape(S, H, G * Lq, Lk), v).reshape(S, H, G, Lq, D) / l
    out = o.permute(0, 3, 1, 2, 4).reshape(S * Lq, H * G, D)[from_q]
    lse = (m + l.log())[..., 0].permute(0, 3, 1, 2).reshape(S * Lq, H * G)[from_q]
    return {"out": out.to(st["q"].dtype), "lse": lse}


def _decode(st):
    c = st["case"]
    S, H, D = c["seqs"], c["kv_heads"], c["D"]
    k, v = (_rows(st[x], st["table"]).float().reshape(S * H, -1, D) for x in ("k_pages", "v_pages"))
    s = torch.matmul(st["q"], k.transpose(1, 2)).mul_(1.0 / math.sqrt(D))
    lens = st["lens"].repeat_interleave(H)
    dead = torch.arange(s.shape[-1], device=s.device) >= lens[:, None, None]
    p, l, _ = _softmax_parts(s.masked_fill_(dead, float("-inf")))
    out = torch.matmul(p, v) / l
    if "mass" not in st:
        return {"out": out}
    st["mass"] += p.div_(l).sum(1)
    return {"out": out, "mass": st["mass"]}


def _append(st):
    page, seq = st["case"]["page"], st["seq"]
    token = torch.arange(seq.shape[0], device=seq.device)
    pos = (st["start"][seq] + token - st["cu_new"][seq]).long()
    at = st["table"][seq, pos // page].long()
    st["k_pages"][at, :, pos % page] = st["k_new"]
    st["v_pages"][at, :, pos % page] = st["v_new"]
    return {"k": st["k_pages"], "v": st["v_pages"]}


def _evict(st):
    c = st["case"]
    S, H, page, keep = c["seqs"], c["kv_heads"], c["page"], c["keep"]
    mass, lens = st["mass"], st["lens"].repeat_interleave(H)[:, None]
    t = torch.arange(mass.shape[1], device=mass.device)
    forced = (t < N_SINK) | (t >= lens - N_RECENT)
    key = mass.masked_fill(forced, float("inf")).masked_fill(t >= lens, float("-inf"))
    first = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :keep]   # ties: the lower index
    if first.shape[1] < keep:
        first = torch.cat([first, first.new_full((S * H, keep - first.shape[1]), mass.shape[1])], 1)
    kept = torch.where(first < lens, first, mass.shape[1]).sort(1).values
    ok = kept < mass.shape[1]
    src = kept.clamp(max=mass.shape[1] - 1)
    j = torch.arange(keep, device=mass.device)
    s = torch.arange(S, device=mass.device)[:, None, None]
    h = torch.arange(H, device=mass.device)[None, :, None]
    src3, ok3 = src.reshape(S, H, keep), ok.reshape(S, H, keep)
    from_page, to_page = st["table"][s, src3 // page].long(), st["dst"][s, j // page].long()
    for name in ("k_pages", "v_pages"):
        p = st[name]
        p[to_page, h, j % page] = torch.where(ok3[..., None], p[from_page, h, src3 % page], p[to_page, h, j % page])
    out = st["mass_out"]
    out[:, :keep] = torch.where(ok, mass.gather(1, src), out[:, :keep])
    return {"kept": torch.where(ok, kept, -1).to(torch.int32), "lens": st["lens"].clamp(max=keep), "mass": out,
            "k": _rows(st["k_pages"], st["dst"]), "v": _rows(st["v_pages"], st["dst"])}


# ------------------------------------------------------------------ the definition, in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    H, D, S = case["kv_heads"], case["D"], case["seqs"]
    if case["op"] == "prefill":
        lq, lk = _prompt_lengths(case)
        G = case["G"]
        out = torch.zeros(sum(lq), H * G, D, dtype=torch.float64, device="cuda")
        lse = torch.zeros(sum(lq), H * G, dtype=torch.float64, device="cuda")
        q0 = k0 = 0
        for a, b in zip(lq, lk):
            seen = torch.ones(a, b, dtype=torch.bool, device="cuda").tril(b - a)
            for h in range(H * G):
                k, v = (st[x][k0:k0 + b, h // G].double() for x in "kv")
                x = (st["q"][q0:q0 + a, h].double() @ k.T) / math.sqrt(D)
                x[~seen] = -math.inf
                lse[q0:q0 + a, h] = torch.logsumexp(x, 1)
                out[q0:q0 + a, h] = torch.exp(x - lse[q0:q0 + a, h, None]) @ v
            q0, k0 = q0 + a, k0 + b
        return {"out": out, "lse": lse}
    page = case["page"]
    if case["op"] == "decode":
        lens = _lengths(S, case["n"], case["ragged"])
        out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
        mass = st["mass"].double() if case["mass"] else None
        for u in range(S * H):
            s, h = divmod(u, H)
            ids = st["table"][s, : -(-lens[s] // page)].long()
            k, v = (st[x][ids, h].reshape(-1, D)[: lens[s]].double() for x in ("k_pages", "v_pages"))
            x = torch.softmax(st["q"][u].double() @ k.T / math.sqrt(D), 1)
            out[u] = x @ v
            if mass is not None:
                mass[u, : lens[s]] += x.sum(0)
        return {"out": out, "mass": mass} if case["mass"] else {"out": out}
    if case["op"] == "append":
        old, new = _append_lengths(case)
        pages = {"k": st["k_pages"].double(), "v": st["v_pages"].double()}
        for x in "kv":
            at = 0
            for s in range(S):
                rows = st[x + "_new"][at:at + new[s]].double()
                at += new[s]
                done = 0
                while done < new[s]:   # page by page
                    p, slot = divmod(old[s] + done, page)
                    m = min(page - slot, new[s] - done)
                    pages[x][int(st["table"][s, p]), :, slot:slot + m] = rows[done:done + m].transpose(0, 1)
                    done += m
        return pages
    lens, keep = _lengths(S, case["n"], case["ragged"]), case["keep"]
    mass_out = st["mass_out"].double()
    rows = {x: _rows(st[x + "_pages"], st["dst"]).double() for x in "kv"}
    mass = st["mass"].cpu().numpy()
    for u in range(S * H):
        s, h = divmod(u, H)
        n, m = lens[s], mass[u]
        middle = sorted(range(min(N_SINK, n), max(min(N_SINK, n), n - N_RECENT)), key=lambda t: (-m[t], t))
        forced = n - len(middle)
        kept = list(range(n)) if n <= keep else sorted(
            list(range(N_SINK)) + middle[: keep - forced] + list(range(n - N_RECENT, n)))
        at = torch.tensor(kept, device="cuda")
        mass_out[u, : len(kept)] = st["mass"][u, at].double()
        ids = st["table"][s].long()
        for x in "kv":
            rows[x][s, h, : len(kept)] = st[x + "_pages"][ids[at // page], h, at % page].double()
    return {"kept": None, "lens": None, "mass": mass_out, "k": rows["k"], "v": rows["v"]}
