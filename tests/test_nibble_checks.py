"""Refusals of the rotated append and of the 4-bit cache's calls, on CPU: the C ABI's own
checks (nothing is enqueued), the binding's checks before the library call, the injected
launch fault; and the workspace's layout."""
import ctypes
import os
import random
import subprocess
import sys

import numpy as np
import pytest
import torch

from bit_plane_kv_gb300 import binding as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
d = ctypes.c_void_p(256)          # never dereferenced: the argument checks come first
e = ctypes.c_void_p(512)
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    from bit_plane_kv_gb300 import build as BUILD
    BUILD.build()
    return B.lib()


def pages(**kw):
    f = dict(seqs=2, kv_heads=2, D=128, page_tokens=16, num_pages=8, max_pages=4, page_stride=4608, head_stride=2304)
    f.update(kw)
    return B.NibblePages(**f)


def pages16(**kw):
    f = dict(seqs=2, kv_heads=2, D=128, dtype=B.BF16, page_tokens=16, num_pages=8, max_pages=4, page_stride=4096,
             head_stride=128, token_stride=256)
    f.update(kw)
    return B.Pages(**f)


def rope(**kw):
    f = dict(table=256, rows=100, rot=128, interleaved=0, positions=None, q=256, q_out=512, q_heads=8, q_dtype=B.BF16,
             q_token=1024, q_head=128, out_token=1024, out_head=128)
    f.update(kw)
    return B.Rope(**f)


def refused(lib, rc, code, word):
    assert rc == code
    assert word in lib.fathom_last_error().decode(), lib.fathom_last_error()


def append(lib, p=None, dt=B.BF16, total=2, tok=256, head=128, args=(d, d, d, d), start=d, cu=None, r=None):
    kv, table, k, v = args
    return lib.fathom_nibble_append(ctypes.byref(p or pages()), kv, table, dt, k, v, total, tok, head, start, cu,
                                    ctypes.byref(r) if r else None, None)


def append16(lib, p=None, total=2, tok=256, head=128, args=(d, d, d, d, d), start=d, cu=None, r=None):
    return lib.fathom_paged_append_rope(ctypes.byref(p or pages16()), *args, total, tok, head, start, cu,
                                        ctypes.byref(r) if r else None, None)


def read(lib, p=None, args=(d, d, d, d), total=5, out=(d, d), dt=B.F32, tok=256, head=128):
    return lib.fathom_nibble_read(ctypes.byref(p or pages()), *args, total, *out, dt, tok, head, None)


def attn(lib, p=None, G=4, args=(d, d, d, d, d), lse=None, ws=ctypes.c_void_p(1 << 20), n=BIG):
    return lib.fathom_nibble_attn(ctypes.byref(p or pages()), G, *args, lse, ws, n, None)


@pytest.mark.parametrize("kw,word", [
    (dict(seqs=0), "seqs"), (dict(seqs=40000), "65535"), (dict(kv_heads=0), "kv_heads"), (dict(D=0), "D must"),
    (dict(D=48), "D must"), (dict(D=160), "D must"), (dict(page_tokens=8), "power of two"), (dict(page_tokens=48), "power of two"),
    (dict(num_pages=0), "num_pages"), (dict(max_pages=0), "max_pages"), (dict(max_pages=1 << 25), "2^28"),
    (dict(page_stride=-16), "strides"), (dict(head_stride=2312), "strides"), (dict(page_stride=0), "strides")])
def test_layouts_are_refused(lib, kw, word):
    p = pages(**kw)
    assert lib.fathom_nibble_workspace_size(ctypes.byref(p), 4) == 0
    assert word in lib.fathom_last_error().decode()
    for call in (append, read, attn):
        refused(lib, call(lib, p), 1, word)


def test_attention_refuses(lib):
    for G in (0, 9):
        refused(lib, attn(lib, G=G), 1, "G must")
    for i, name in enumerate(["q", "kv_pages", "page_table", "lens", "out"]):
        refused(lib, attn(lib, args=[None if j == i else d for j in range(5)]), 1, f"{name} is NULL")
    for i in (0, 1, 4):
        refused(lib, attn(lib, args=[ctypes.c_void_p(264) if j == i else d for j in range(5)]), 1, "aligned")
    refused(lib, attn(lib, ws=None), 1, "workspace is NULL")
    need = lib.fathom_nibble_workspace_size(ctypes.byref(pages()), 4)
    assert need > 0 and need % 256 == 0
    refused(lib, attn(lib, n=need - 1), 3, "too small")
    refused(lib, attn(lib, ws=ctypes.c_void_p((1 << 20) + 16)), 1, "256-byte")
    assert lib.fathom_nibble_attn(None, 4, d, d, d, d, d, None, d, BIG, None) == 1


def test_appends_refuse(lib):
    for call, names in ((append, ["kv_pages", "page_table", "k_new", "v_new"]),
                        (append16, ["k_pages", "v_pages", "page_table", "k_new", "v_new"])):
        good = dict(r=rope())
        refused(lib, call(lib, total=3, **good), 1, "total_new")
        refused(lib, call(lib, total=-1, cu=d, **good), 1, "total_new")
        refused(lib, call(lib, total=(1 << 28) + 1, cu=d, **good), 1, "total_new")
        refused(lib, call(lib, tok=4, **good), 1, "strides")
        refused(lib, call(lib, head=-8, **good), 1, "strides")
        for i, name in enumerate(names):
            refused(lib, call(lib, args=[None if j == i else d for j in range(len(names))], **good), 1, f"{name} is NULL")
        refused(lib, call(lib, args=[ctypes.c_void_p(258) if n == "k_new" else d for n in names], **good), 1, "aligned")
        refused(lib, call(lib, start=None, **good), 1, "start is NULL")
        assert call(lib, total=0, args=[None] * len(names), start=None, **good) == 0
    for dt in (B.F32, 3):
        refused(lib, append(lib, dt=dt), 1, "dtype")
    refused(lib, append(lib, args=(ctypes.c_void_p(264), d, d, d)), 1, "aligned")
    refused(lib, append16(lib), 1, "rope is NULL")
    refused(lib, append16(lib, pages16(D=12), r=rope()), 1, "D must")


@pytest.mark.parametrize("kw,word", [
    (dict(table=None), "table is NULL"), (dict(table=264), "aligned"), (dict(rows=0), "rows"), (dict(rot=0), "rot"), (dict(rot=7), "rot"),
    (dict(rot=130), "rot"), (dict(interleaved=2), "interleaved"), (dict(q_out=None), "q_out is NULL"), (dict(q_out=256), "may not be q"),
    (dict(q_heads=0), "q_heads"), (dict(q_heads=65536), "q_heads"), (dict(q_dtype=B.F16), "q_dtype"), (dict(q_dtype=5), "q_dtype"),
    (dict(q_token=4), "strides"), (dict(q_head=0), "strides"), (dict(out_token=-8), "strides"), (dict(out_head=12), "strides"),
    (dict(q=264), "aligned"), (dict(q_out=520), "aligned")])
def test_rotations_are_refused(lib, kw, word):
    refused(lib, append(lib, r=rope(**kw)), 1, word)
    refused(lib, append16(lib, r=rope(**kw)), 1, word)


def test_read_refuses(lib):
    refused(lib, read(lib, total=-1), 1, "total")
    refused(lib, read(lib, dt=3), 1, "out_dtype")
    refused(lib, read(lib, tok=4), 1, "strides")
    refused(lib, read(lib, head=100), 1, "strides")
    for i, name in enumerate(["kv_pages", "page_table", "start", "cu"]):
        refused(lib, read(lib, args=[None if j == i else d for j in range(4)]), 1, f"{name} is NULL")
    refused(lib, read(lib, out=(None, d)), 1, "k_out is NULL")
    refused(lib, read(lib, out=(d, None)), 1, "v_out is NULL")
    refused(lib, read(lib, out=(d, ctypes.c_void_p(264))), 1, "aligned")
    assert read(lib, total=0, args=(None,) * 4, out=(None, None)) == 0


def test_injected_launch_fault_reaches_every_call():
    code = """
import ctypes, sys
sys.path.insert(0, %r); sys.path.insert(0, %r)
import test_nibble_checks as T
L = T.B.lib()
for rc in (T.append(L, r=T.rope()), T.append(L), T.append16(L, r=T.rope()), T.read(L), T.attn(L)):
    assert rc == 2 and "injected" in L.fathom_last_error().decode(), (rc, L.fathom_last_error())
""" % (ROOT, os.path.join(ROOT, "tests"))
    r = subprocess.run([sys.executable, "-c", code], env=dict(os.environ, FATHOM_FAULT="launch"), capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


# ------------------------------------------------------------------ the binding
class Reached(Exception):
    pass


@pytest.fixture
def no_library(monkeypatch):
    def fake_call(name, *args):
        raise Reached(name)
    monkeypatch.setattr(B, "_call", fake_call)
    monkeypatch.setattr(B, "_stream", lambda stream=None: None)
    monkeypatch.setattr(B, "_reachable", lambda t: True)
    monkeypatch.setattr(B, "_on_device", lambda t: True)


I32, BF, F32 = torch.int32, torch.bfloat16, torch.float32


def z(*shape, dtype=F32):
    return torch.zeros(*shape, dtype=dtype)


def _cache():
    kv, table = B.alloc_nibble_pages(9, 2, 32, 64, device="cpu"), z(3, 4, dtype=I32)
    return dict(pages=B.make_nibble_pages(kv, table, 64), kv_pages=kv, page_table=table)


def _rows():
    return dict(k_new=z(5, 2, 64, dtype=BF), v_new=z(5, 2, 64, dtype=BF), start=z(3, dtype=I32), cu_new=z(4, dtype=I32),
                rope=z(50, 64), positions=z(5, dtype=I32), q=z(5, 8, 64, dtype=BF), q_out=z(5, 8, 64))


def _append_args():
    return dict(_cache(), **_rows())


def _append16_args():
    kp, table = z(9, 2, 16, 64, dtype=BF), z(3, 4, dtype=I32)
    return dict(pages=B.make_pages(kp, table), k_pages=kp, v_pages=kp.clone(), page_table=table, **_rows())


def _read_args():
    return dict(_cache(), start=z(3, dtype=I32), cu=z(4, dtype=I32), total=7, k_out=z(7, 2, 64), v_out=z(7, 2, 64))


def _attn_args():
    return dict(_cache(), q=z(6, 4, 64), lens=z(3, dtype=I32), workspace=z(64, dtype=torch.uint8), out=z(6, 4, 64), lse=z(6, 4))


CALLS = {"fathom_nibble_append": _append_args, "fathom_paged_append_rope": _append16_args, "fathom_nibble_read": _read_args,
         "fathom_nibble_attn": _attn_args}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_valid_arguments_reach_the_library_call(no_library, name):
    with pytest.raises(Reached):
        getattr(B, name)(**CALLS[name]())


def _tensors(name):
    return [a for a, v in CALLS[name]().items() if isinstance(v, torch.Tensor) and a != "workspace"]


@pytest.mark.parametrize("name,arg", [(n, a) for n in sorted(CALLS) for a in _tensors(n)])
def test_tensors_of_other_sizes_types_or_layouts_are_refused(no_library, name, arg):
    good = CALLS[name]()[arg]
    wrong = [good.double()]
    if arg != "rope":                                  # any number of positions and of rotated channels is a table
        wrong.append(good.reshape(-1)[:-1].clone())
    else:
        wrong += [good.reshape(-1), good[:0]]
    if good.dim() > 1:
        wrong.append(good.transpose(-1, -2).contiguous().transpose(-1, -2))   # the same sizes, the last axis strided
        if arg not in ("rope", "q") or name == "fathom_nibble_attn":
            wrong.append(good[:, :-1].clone())
    for t in wrong:
        kw = CALLS[name]()
        kw[arg] = t
        with pytest.raises((ValueError, TypeError)):
            getattr(B, name)(**kw)


def test_the_binding_refuses_what_does_not_fit_together(no_library):
    for name in ("fathom_nibble_append", "fathom_paged_append_rope"):
        call = getattr(B, name)
        for change in (dict(cu_new=None), dict(v_new=z(5, 3, 64, dtype=BF)[:, :2]), dict(rope=None), dict(q=None),
                       dict(q_out=None, q=None, q_dtype=F32), dict(k_new=None), dict(start=None),
                       dict(v_new=z(5, 2, 64, dtype=torch.float16))):
            with pytest.raises((ValueError, TypeError)):
                call(**dict(CALLS[name](), **change))
        with pytest.raises(TypeError, match="q_dtype"):
            call(**dict(CALLS[name](), q_out=None, q_dtype=torch.float16))
    for change in (dict(k_out=None), dict(v_out=z(7, 3, 64)[:, :2]), dict(k_out=None, v_out=None, total=-1),
                   dict(k_out=None, v_out=None, dtype=torch.float64), dict(start=None), dict(cu=None)):
        with pytest.raises((ValueError, TypeError)):
            B.fathom_nibble_read(**dict(_read_args(), **change))
    with pytest.raises(ValueError):
        B.make_nibble_pages(z(9, 2, 100, dtype=torch.uint8), z(3, 4, dtype=I32), 64)
    with pytest.raises(TypeError):
        B.make_nibble_pages(z(9, 2, 18 * 64), z(3, 4, dtype=I32), 64)


def test_host_tensors_are_refused_without_a_device():
    for name, make in CALLS.items():
        with pytest.raises(ValueError, match="CUDA"):
            getattr(B, name)(**make())


def test_counts_beyond_32_bits_are_refused(no_library):
    big = (1 << 32) + 5
    for name in ("fathom_nibble_append", "fathom_paged_append_rope"):
        kw = CALLS[name]()
        kw.update(k_new=z(1, 2, 64, dtype=BF).expand(big, 2, 64), v_new=z(1, 2, 64, dtype=BF).expand(big, 2, 64))
        with pytest.raises(ValueError, match="32 bits"):
            getattr(B, name)(**kw)
    with pytest.raises(ValueError, match="32 bits"):
        B.make_nibble_pages(z(1, 2, 18 * 64, dtype=torch.uint8).expand(big, 2, 18 * 64), z(3, 4, dtype=I32), 64)
    with pytest.raises(ValueError, match="32 bits"):
        B.fathom_nibble_read(**dict(_read_args(), total=big, k_out=None, v_out=None))


# ------------------------------------------------------------------ the workspace
class Layout(ctypes.Structure):
    _fields_ = [("sms", ctypes.c_int)] + [(f, ctypes.c_size_t) for f in ("part_off", "ml_off", "total")]


def test_no_call_leaves_data_where_another_looks_for_tickets(lib):
    """Tickets come first and in the same number whatever the call, three for each of four CTAs per SM; partial
    results, two per CTA, follow."""
    f = getattr(lib, "_ZN6fathom23nibble_workspace_layoutERK19fathom_nibble_pagesi")   # nibble_workspace_layout
    f.restype, f.argtypes = Layout, [ctypes.POINTER(B.NibblePages), ctypes.c_int]
    starts = set()
    for seqs, heads in ((1, 1), (1000, 8), (65535, 1)):
        for D in (32, 64, 96, 128):
            for G in range(1, 9):
                p = pages(seqs=seqs, kv_heads=heads, D=D, page_stride=heads * 18 * D, head_stride=18 * D)
                w = f(ctypes.byref(p), G)
                assert w.total == lib.fathom_nibble_workspace_size(ctypes.byref(p), G)
                assert w.part_off >= 4 * 3 * 4 * w.sms
                assert w.ml_off - w.part_off >= 4 * w.sms * 2 * G * D * 4 and w.total - w.ml_off >= 4 * w.sms * 2 * G * 2 * 4
                assert all(x % 256 == 0 for x in (w.part_off, w.ml_off, w.total))
                starts.add(w.part_off)
    assert len(starts) == 1


def test_shares_of_few_units_cover_every_tile_once():
    """The kernel's own CTAs of a unit, restated: of `grid` CTAs each unit of t > 0 tiles gets
    min(t, max(1, t * part)), part = (grid - units) / all tiles in fp32; CTA j of its c takes tiles
    j t / c to (j + 1) t / c.  No more CTAs than there are, and the longest share is an eighth and a tile more than
    the mean at most."""
    f = np.float32
    rng = random.Random(3)
    for _ in range(4000):
        grid = 152 * rng.choice([3, 4])
        heads = rng.choice([1, 2, 3, 8])
        seqs = rng.randint(1, grid // 8 // heads)
        top = rng.choice([1, 2, 9, 100, 5000, 1 << 21])
        tiles = [rng.randint(0, top) for _ in range(seqs)]
        total = sum(tiles)
        if not total:
            continue
        part = f(grid - seqs * heads) / (f(total) * f(heads))
        count = [min(t, max(1, int(f(t) * part))) if t else 0 for t in tiles]
        assert sum(count) * heads <= grid
        mean = total * heads / (grid - seqs * heads)
        for t, c in zip(tiles, count):
            ends = [j * t // c for j in range(c + 1)] if c else [0]
            assert ends[-1] == t and all(a < b for a, b in zip(ends, ends[1:]))
            assert all((j + 1) * t < 1 << 32 for j in range(c))
            longest = max((b - a for a, b in zip(ends, ends[1:])), default=0)
            assert longest <= 1 + mean * (2 if c < 8 else 1.125)
