"""Decode attention over the 4-bit cache where the batch's units have no CTAs of their own: the CTAs take equal shares
of all tiles, units cross them, a CTA joins two units, a unit has more than 32 shares; against the plain form
(tolerances in nibble_cases)."""
import pytest
import torch

from bit_plane_kv_gb300 import binding as B

import nibble_cases as N

pytestmark = pytest.mark.gpu


def ragged(count, n, salt=0):
    return [(7919 * (i + salt) * (i + salt) + 104729 * i) % (n + 1) for i in range(count)]


#: name: (lengths, KV heads, query heads of each, D, tokens of a page)
SPLIT = {
    "256 units of up to 1500 tokens": (ragged(32, 1500), 8, 4, 128, 64),
    "244 units, 8 heads, 64 channels": (ragged(61, 3001), 4, 8, 64, 32),
    "80 units, one of 100000 tokens in the middle": ([500] * 40 + [100000] + [500] * 39, 1, 4, 128, 64),
    "the same, 8 heads": ([500] * 40 + [70000] + [500] * 39, 1, 8, 128, 64),
    "100 units, the first of 60000 tokens": ([60000] + ragged(99, 700), 1, 2, 64, 16),
    "100 units, the last of 60001 tokens, 96 channels": (ragged(99, 700, 3) + [60001], 1, 5, 96, 128),
    "two of 40000 tokens side by side, 3 heads": (ragged(30, 900) + [40000, 39999] + ragged(30, 900, 9), 3, 1, 32, 32),
    "300 sequences of up to 2500 tokens": (ragged(300, 2500), 1, 4, 64, 16),
    "300 sequences, empty ones and one of 50000 tokens": ([n if i % 3 else 0 for i, n in enumerate(ragged(150, 600))] + [50000]
                                                          + [n if i % 7 else 0 for i, n in enumerate(ragged(149, 600, 5))], 2, 3, 32, 16),
    "129 sequences": (ragged(129, 1200), 2, 6, 128, 16),
    "128 sequences": (ragged(128, 1200), 2, 4, 96, 16),
    "1000 sequences of 100 tokens, one of 20000": ([100] * 700 + [20000] + [100] * 299, 1, 4, 128, 16),
    "77 units of equal tokens": ([1024] * 77, 1, 4, 128, 16),
}


def batch(name):
    lens, H, G, D, page = SPLIT[name]
    own = -(-torch.tensor(lens) // page)                    # pages of each sequence, numbered in no order
    g = torch.Generator(device="cuda").manual_seed(1)
    count = int(own.sum()) + 1
    k, v = (torch.randn(count, H, page, D, generator=g, device="cuda") for _ in range(2))
    order = torch.randperm(count, generator=g, device="cuda").to(torch.int32).tolist()
    table, at = torch.full((len(lens), int(own.max())), -1, dtype=torch.int32), 0
    for s, n in enumerate(own.tolist()):
        table[s, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
    q = 2 * torch.randn(len(lens) * H, G, D, generator=g, device="cuda")
    return q, N.pack(k, v), table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("name", list(SPLIT))
def test_equal_shares_match_the_plain_form(name):
    lens, H, G, D, page = SPLIT[name]
    ctas = (4 if G <= 4 else 3) * torch.cuda.get_device_properties(0).multi_processor_count
    assert len(lens) * H * 8 > ctas                         # else each unit has CTAs of its own
    q, kv, table, n = batch(name)
    pages = B.make_nibble_pages(kv, table, D)
    ws = B.alloc_nibble_workspace(pages, G=G)
    out, lse = B.fathom_nibble_attn(pages, q, kv, table, n, ws, want_lse=True)
    again = B.fathom_nibble_attn(pages, q, kv, table, n, ws)
    o, z, tol, tol_z = N.decode(q, *N.unpack(kv, D), table, lens)
    far = (out.double() - o).abs()
    assert torch.isfinite(out).all()
    assert bool((far <= tol).all()), f"worst {(far / tol.clamp(min=1e-300)).max().item():.3f} of the tolerance"
    empty = torch.isinf(z)
    assert bool((lse[empty] == -torch.inf).all()) and bool(((lse.double() - z)[~empty].abs() <= tol_z[~empty]).all())
    assert torch.equal(out, again)


def test_batches_of_both_kinds_share_a_workspace():
    calls = [batch(x) for x in ("80 units, one of 100000 tokens in the middle", "129 sequences", "256 units of up to 1500 tokens")]
    g = torch.Generator(device="cuda").manual_seed(3)
    k, v = (torch.randn(300, 1, 64, 128, generator=g, device="cuda") for _ in range(2))
    calls.append((torch.randn(2, 4, 128, generator=g, device="cuda"), N.pack(k, v),
                  torch.arange(300, dtype=torch.int32, device="cuda").reshape(2, 150), torch.tensor([9600, 7], dtype=torch.int32, device="cuda")))
    pages = [B.make_nibble_pages(kv, table, q.shape[2]) for q, kv, table, _ in calls]
    want = [B.fathom_nibble_attn(p, *c, B.alloc_nibble_workspace(p, G=c[0].shape[1])) for p, c in zip(pages, calls)]
    ws = B.alloc_nibble_workspace(pages[1], G=8)
    for i in (0, 1, 2, 3, 0, 3, 2, 1, 0):
        assert torch.equal(B.fathom_nibble_attn(pages[i], *calls[i], ws), want[i])
