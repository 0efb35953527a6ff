"""Refusals of the prompt and paged-cache calls, on CPU: the C ABI's own checks
(nothing is enqueued), the binding's checks before the library call, and the
injected launch fault."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

from bit_plane_kv_gb300 import binding as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
d = ctypes.c_void_p(256)          # never dereferenced: the argument checks come first
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    from bit_plane_kv_gb300 import build as BUILD
    BUILD.build()
    return B.lib()


def prompts(**kw):
    f = dict(seqs=2, heads=8, kv_heads=2, D=128, dtype=B.BF16, total_q=10, total_k=10, q_token=1024, q_head=128,
             k_token=256, k_head=128, v_token=256, v_head=128, out_token=1024, out_head=128)
    f.update(kw)
    return B.Prompts(**f)


def pages(**kw):
    f = dict(seqs=2, kv_heads=2, D=128, dtype=B.BF16, page_tokens=16, num_pages=8, max_pages=4, page_stride=4096,
             head_stride=128, token_stride=256)
    f.update(kw)
    return B.Pages(**f)


def refused(lib, rc, code, word):
    assert rc == code
    assert word in lib.fathom_last_error().decode()


@pytest.mark.parametrize("kw,word", [
    (dict(seqs=0), "seqs"), (dict(seqs=65536), "seqs"), (dict(heads=9), "multiple of kv_heads"),
    (dict(kv_heads=0), "kv_heads"), (dict(heads=0), "heads"), (dict(D=4), "multiple of 8"), (dict(D=100), "multiple of 8"),
    (dict(D=136), "multiple of 8"), (dict(dtype=B.F32), "dtype"), (dict(dtype=3), "dtype"), (dict(total_q=-1), "total_q"),
    (dict(total_k=(1 << 28) + 1), "total_k"), (dict(q_token=1020), "strides"), (dict(k_head=0), "strides"),
    (dict(v_token=-256), "strides"), (dict(out_head=4), "strides"),
])
def test_prefill_refuses_shapes(lib, kw, word):
    refused(lib, lib.fathom_prefill_attn(ctypes.byref(prompts(**kw)), d, d, d, d, d, d, None, None), 1, word)


def test_prefill_refuses_pointers(lib):
    args = [d, d, d, d, d, d]
    for i, name in enumerate(["q", "k", "v", "cu_q", "cu_k", "out"]):
        a = list(args)
        a[i] = None
        refused(lib, lib.fathom_prefill_attn(ctypes.byref(prompts()), *a, None, None), 1, f"{name} is NULL")
    for i in (0, 1, 2, 5):
        a = list(args)
        a[i] = ctypes.c_void_p(264)
        refused(lib, lib.fathom_prefill_attn(ctypes.byref(prompts()), *a, None, None), 1, "aligned")
    refused(lib, lib.fathom_prefill_attn(None, *args, None, None), 1, "prompts is NULL")
    assert lib.fathom_prefill_attn(ctypes.byref(prompts(total_q=0)), *[None] * 6, None, None) == 0   # nothing to do


BAD_PAGES = [(dict(seqs=0), "seqs"), (dict(seqs=40000), "65535"), (dict(kv_heads=0), "kv_heads"), (dict(D=12), "D must"),
             (dict(dtype=0), "dtype"), (dict(page_tokens=0), "power of two"), (dict(page_tokens=48), "power of two"),
             (dict(num_pages=0), "num_pages"), (dict(max_pages=0), "max_pages"), (dict(max_pages=1 << 25), "2^28"),
             (dict(page_stride=-8), "strides"), (dict(head_stride=100), "strides"), (dict(token_stride=0), "strides")]


@pytest.mark.parametrize("kw,word", BAD_PAGES)
def test_paged_calls_refuse_layouts(lib, kw, word):
    p = ctypes.byref(pages(**kw))
    assert lib.fathom_paged_workspace_size(p, 4, 0) == 0
    assert word in lib.fathom_last_error().decode()
    refused(lib, lib.fathom_paged_attn(p, 4, d, d, d, d, d, d, None, 0, d, BIG, None), 1, word)
    refused(lib, lib.fathom_paged_append(p, d, d, d, d, d, 2, 256, 128, d, None, None), 1, word)
    refused(lib, lib.fathom_paged_evict(p, d, d, d, d, d, 64, 40, 4, 32, d, 4, d, ctypes.c_void_p(512), d, 64, None), 1, word)


def test_paged_attn_refuses(lib):
    p = ctypes.byref(pages())
    ws = ctypes.c_void_p(1 << 20)

    def call(G=4, args=(d, d, d, d, d, d), mass=None, stride=64, w=ws, n=BIG):
        return lib.fathom_paged_attn(p, G, *args, mass, stride, w, n, None)

    for G in (0, 9):
        refused(lib, call(G=G), 1, "G must")
    for i, name in enumerate(["q", "k_pages", "v_pages", "page_table", "lens", "out"]):
        refused(lib, call(args=[None if j == i else d for j in range(6)]), 1, f"{name} is NULL")
    refused(lib, call(args=(d, ctypes.c_void_p(264), d, d, d, d)), 1, "aligned")
    refused(lib, call(mass=d, stride=63), 1, "mass_stride")
    refused(lib, call(w=None), 1, "workspace is NULL")
    need = lib.fathom_paged_workspace_size(p, 4, 0)
    assert need > 0 and need % 256 == 0
    refused(lib, call(n=need - 1), 3, "too small")
    refused(lib, call(mass=d, n=need), 3, "too small")
    assert lib.fathom_paged_workspace_size(p, 4, 1) > need
    refused(lib, call(w=ctypes.c_void_p((1 << 20) + 16)), 1, "256-byte")


def test_paged_append_refuses(lib):
    p = ctypes.byref(pages())

    def call(total=2, tok=256, head=128, args=(d, d, d, d, d), start=d, cu=None):
        return lib.fathom_paged_append(p, *args, total, tok, head, start, cu, None)

    refused(lib, call(total=3), 1, "total_new")
    refused(lib, call(total=-1, cu=d), 1, "total_new")
    refused(lib, call(tok=4), 1, "strides")
    refused(lib, call(head=-8), 1, "strides")
    for i, name in enumerate(["k_pages", "v_pages", "page_table", "k_new", "v_new"]):
        refused(lib, call(args=[None if j == i else d for j in range(5)]), 1, f"{name} is NULL")
    refused(lib, call(args=(d, d, d, ctypes.c_void_p(258), d)), 1, "aligned")
    refused(lib, call(start=None), 1, "start is NULL")
    assert call(total=0) == 0


def test_paged_evict_refuses(lib):
    p = ctypes.byref(pages())
    e = ctypes.c_void_p(512)

    def call(keep=40, ns=4, nr=32, dst=3, ms=64, os_=40, ptr=None, out=d, mass_out=e, lens_out=e):
        a = dict(zip(["k_pages", "v_pages", "page_table", "lens", "mass", "dst_table", "kept_idx"], [d] * 7))
        if ptr:
            a[ptr] = None
        return lib.fathom_paged_evict(p, a["k_pages"], a["v_pages"], a["page_table"], a["lens"], a["mass"], ms, keep, ns,
                                      nr, a["dst_table"], dst, a["kept_idx"], lens_out, mass_out, os_, None)

    for kw, word in [(dict(keep=0), "keep must"), (dict(ns=-1), "n_sink"), (dict(nr=37), "n_sink"), (dict(dst=2), "dst_pages"),
                     (dict(dst=0), "dst_pages"), (dict(ms=63), "mass_stride"), (dict(os_=39), "mass_out_stride"),
                     (dict(lens_out=d), "lens_out"), (dict(mass_out=d, os_=63), "same stride"),
                     (dict(lens_out=None), "lens_out is NULL"), (dict(mass_out=None), "mass_out is NULL")]:
        refused(lib, call(**kw), 1, word)
    for name in ["k_pages", "v_pages", "page_table", "lens", "mass", "dst_table", "kept_idx"]:
        refused(lib, call(ptr=name), 1, f"{name} is NULL")


def test_injected_launch_fault_reaches_every_call():
    code = """
import ctypes, sys
sys.path.insert(0, %r); sys.path.insert(0, %r)
import test_paged_checks as T
L, d, e = T.B.lib(), T.d, ctypes.c_void_p(512)
p = ctypes.byref(T.pages())
for rc in (L.fathom_prefill_attn(ctypes.byref(T.prompts()), d, d, d, d, d, d, None, None),
           L.fathom_paged_attn(p, 4, d, d, d, d, d, d, None, 0, d, 1 << 40, None),
           L.fathom_paged_append(p, d, d, d, d, d, 2, 256, 128, d, None, None),
           L.fathom_paged_evict(p, d, d, d, d, d, 64, 40, 4, 32, d, 4, d, e, d, 64, None)):
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


I32 = torch.int32
BF = torch.bfloat16


def z(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype)


def _prefill_args():
    return dict(q=z(10, 8, 64, dtype=BF), k=z(12, 2, 64, dtype=BF), v=z(12, 2, 64, dtype=BF), cu_q=z(3, dtype=I32),
                cu_k=z(3, dtype=I32), out=z(10, 8, 64, dtype=BF), lse=z(10, 8))


def _cache_args():
    kp, table = z(9, 2, 16, 64, dtype=BF), z(3, 4, dtype=I32)
    return dict(pages=B.make_pages(kp, table), k_pages=kp, v_pages=kp.clone(), page_table=table)


def _attn_args():
    return dict(_cache_args(), q=z(6, 4, 64), lens=z(3, dtype=I32), workspace=z(64, dtype=torch.uint8), out=z(6, 4, 64),
                mass=z(6, 64))


def _append_args():
    return dict(_cache_args(), k_new=z(5, 2, 64, dtype=BF), v_new=z(5, 2, 64, dtype=BF), start=z(3, dtype=I32),
                cu_new=z(4, dtype=I32))


def _evict_args():
    return dict(_cache_args(), lens=z(3, dtype=I32), mass=z(6, 64), keep=40, dst_table=z(3, 3, dtype=I32),
                kept_idx=z(6, 40, dtype=I32), lens_out=z(3, dtype=I32), mass_out=z(6, 48))


CALLS = {"fathom_prefill_attn": _prefill_args, "fathom_paged_attn": _attn_args, "fathom_paged_append": _append_args,
         "fathom_paged_evict": _evict_args}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_valid_arguments_reach_the_library_call(no_library, name):
    with pytest.raises(Reached):
        getattr(B, name)(**CALLS[name]())


def _tensors(name):
    return [a for a, v in CALLS[name]().items() if isinstance(v, torch.Tensor) and a != "workspace"]


@pytest.mark.parametrize("name,arg", [(n, a) for n in sorted(CALLS) for a in _tensors(n)])
def test_tensors_of_other_sizes_types_or_layouts_are_refused(no_library, name, arg):
    good = CALLS[name]()[arg]
    wrong = [good.reshape(-1)[:-1].clone(), good.double()]
    if good.dim() > 1:
        wrong.append(good.transpose(-1, -2).contiguous().transpose(-1, -2))   # the same sizes, the last axis strided
        wrong.append(good[:, :-1].clone() if arg not in ("mass", "mass_out", "dst_table") else good[:-1].clone())
    for t in wrong:
        kw = CALLS[name]()
        kw[arg] = t
        with pytest.raises((ValueError, TypeError)):
            getattr(B, name)(**kw)


@pytest.mark.parametrize("name,arg", [("fathom_prefill_attn", "k"), ("fathom_prefill_attn", "q"),
                                      ("fathom_prefill_attn", "cu_q"), ("fathom_paged_attn", "q"),
                                      ("fathom_paged_attn", "lens"), ("fathom_paged_append", "start"),
                                      ("fathom_paged_append", "k_new"), ("fathom_paged_evict", "mass"),
                                      ("fathom_paged_evict", "dst_table")])
def test_missing_tensors_are_refused(no_library, name, arg):
    kw = CALLS[name]()
    kw[arg] = None
    with pytest.raises((ValueError, AttributeError)):
        getattr(B, name)(**kw)


def test_the_binding_refuses_what_does_not_fit_together(no_library):
    kw = _append_args()
    kw["cu_new"] = None                                    # five tokens for three sequences
    with pytest.raises(ValueError, match="k_new"):
        B.fathom_paged_append(**kw)
    kw = _append_args()
    kw["v_new"] = z(5, 3, 64, dtype=BF)[:, :2]             # other strides than k_new
    with pytest.raises(ValueError, match="v_new"):
        B.fathom_paged_append(**kw)
    kw = _attn_args()
    kw["v_pages"] = z(9, 16, 2, 64, dtype=BF).permute(0, 2, 1, 3)
    with pytest.raises(ValueError, match="v_pages"):
        B.fathom_paged_attn(**kw)
    kw = _attn_args()
    kw["k_pages"] = kw["k_pages"].half()
    with pytest.raises(TypeError, match="k_pages"):
        B.fathom_paged_attn(**kw)
    with pytest.raises(ValueError):
        B.fathom_prefill_attn(z(4, 2, 64, dtype=BF), z(4, 2, 64, dtype=BF), z(4, 2, 64, dtype=BF), z(1, dtype=I32))


def test_host_tensors_are_refused_without_a_device():
    kw = _prefill_args()
    with pytest.raises(ValueError, match="CUDA"):
        B.fathom_prefill_attn(**kw)


def test_rows_as_pages_names_every_row_once():
    seqs, H, C, D, P = 3, 2, 64, 8, 16
    rows = torch.arange(seqs * H * C * D, dtype=torch.float32).reshape(seqs * H, C, D)
    view, table = B.rows_as_pages(rows, H, P)
    assert view.data_ptr() == rows.data_ptr() and tuple(table.shape) == (seqs, C // P)
    for u in range(seqs * H):
        s, h = divmod(u, H)
        assert torch.equal(torch.cat([view[int(t), h] for t in table[s]]), rows[u])
    with pytest.raises(ValueError):
        B.rows_as_pages(rows, H, 48)
    with pytest.raises(ValueError):
        B.rows_as_pages(rows, 4, P)


def test_counts_beyond_32_bits_are_refused(no_library):
    """The library's counts are 32-bit; a larger one must not wrap around into one that it accepts."""
    big = (1 << 32) + 5
    kw = _prefill_args()
    kw.update(q=z(1, 8, 64, dtype=BF).expand(big, 8, 64), out=z(1, 8, 64, dtype=BF).expand(big, 8, 64), lse=None)
    with pytest.raises(ValueError, match="32 bits"):
        B.fathom_prefill_attn(**kw)
    kw = _prefill_args()
    kw.update(k=z(1, 2, 64, dtype=BF).expand(big, 2, 64), v=z(1, 2, 64, dtype=BF).expand(big, 2, 64))
    with pytest.raises(ValueError, match="32 bits"):
        B.fathom_prefill_attn(**kw)
    with pytest.raises(ValueError, match="32 bits"):
        B.make_pages(z(1, 2, 16, 64, dtype=BF).expand(big, 2, 16, 64), z(3, 4, dtype=I32))
    kw = _append_args()
    kw.update(k_new=z(1, 2, 64, dtype=BF).expand(big, 2, 64), v_new=z(1, 2, 64, dtype=BF).expand(big, 2, 64))
    with pytest.raises(ValueError, match="32 bits"):
        B.fathom_paged_append(**kw)
    for name in ("keep", "n_sink", "n_recent"):
        kw = _evict_args()
        kw.update({name: (1 << 32) + kw.get(name, 4)}, mass_out=z(6, 48), kept_idx=None)
        with pytest.raises(ValueError, match="32 bits"):
            B.fathom_paged_evict(**kw)
