"""Where rotated queries may go, and how many heads there may be, on the GPU."""
import pytest
import torch

from bit_plane_kv_gb300 import binding as B

import nibble_cases as N
import paged_cases as P

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("f32", [False, True])
def test_rotated_queries_between_the_rows_of_one_buffer(f32):
    """[tokens][heads][D] of one projection with room for the rotated queries behind its heads; a head on is refused."""
    H, Hq, D, new, old = 2, 6, 64, [40, 3, 1], [5, 0, 20]
    T, room = sum(new), Hq * (2 if f32 else 1)
    buf = torch.randn(T, Hq + 2 * H + room, D, device="cuda").to(BF)
    q, k, v = buf[:, :Hq], buf[:, Hq:Hq + H], buf[:, Hq + H:Hq + 2 * H]
    rest = buf.view(-1).view(torch.float32).view(T, -1) if f32 else buf.view(T, -1)
    q_out = rest[:, (Hq + 2 * H) * D // (2 if f32 else 1):].unflatten(1, (Hq, D))
    rope, cu = N.rope_table(100, D), P.cumulated(new)
    table = torch.arange(9, dtype=torch.int32, device="cuda").reshape(3, 3)
    kv, kv2 = (B.alloc_nibble_pages(9, H, 16, D) for _ in range(2))
    pages = B.make_nibble_pages(kv, table, D)
    dt = torch.float32 if f32 else BF
    _, want = B.fathom_nibble_append(pages, kv2, table, k, v, i32(old), cu, rope=rope, q=q, q_dtype=dt)
    before = buf[:, :Hq + 2 * H].clone()
    B.fathom_nibble_append(pages, kv, table, k, v, i32(old), cu, rope=rope, q=q, q_out=q_out)
    assert torch.equal(q_out, want) and torch.equal(kv, kv2) and torch.equal(buf[:, :Hq + 2 * H], before)
    for wrong in ((q_out[:, :Hq - 1], q_out[:, 1:]), (q[:, :Hq - 1], q[:, 1:])):
        if wrong[0].dtype is BF:
            with pytest.raises(B.FathomError, match="overlaps"):
                B.fathom_nibble_append(pages, kv, table, k, v, i32(old), cu, rope=rope, q=wrong[0], q_out=wrong[1])
    assert torch.equal(kv, kv2) and torch.equal(buf[:, :Hq + 2 * H], before)


def test_as_many_heads_as_the_layout_allows():
    """65535 query heads and 65535 KV heads of 32 channels: as many rows of a token as there can be."""
    H = Hq = 65535
    D, page = 32, 16
    k, v, q = (torch.randn(1, n, D, device="cuda").to(BF) for n in (H, H, Hq))
    table, rope = i32([[0]]), N.rope_table(20, D)
    kp, vp = torch.zeros(1, H, page, D, dtype=BF, device="cuda"), torch.zeros(1, H, page, D, dtype=BF, device="cuda")
    pos = i32([3]).long()
    _, _, r = B.fathom_paged_append_rope(B.make_pages(kp, table), kp, vp, table, k, v, i32([3]), rope, q=q)
    assert torch.equal(vp[0, :, 3], v[0]) and N.near_rotated(kp[0, :, 3][None], k, rope, pos, False) and N.near_rotated(r, q, rope, pos, False)
    kv = B.alloc_nibble_pages(1, H, page, D)
    pages = B.make_nibble_pages(kv, table, D)
    _, r4 = B.fathom_nibble_append(pages, kv, table, k, v, i32([3]), rope=rope, q=q)
    assert torch.equal(r4, r)
    k4, v4 = B.fathom_nibble_read(pages, kv, table, i32([3]), i32([0, 1]), 1, dtype=torch.float32)
    assert torch.equal(k4[0].double(), N.held(N.rotated(k, rope, pos, False))[0][0]) and torch.equal(v4[0].double(), N.held(v.double())[0][0])
