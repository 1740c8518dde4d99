"""The rotary and paged entry points without a GPU: what they refuse, before any launch, and the
one-token-at-a-time plan that the GPU tests compare with."""
import ctypes

import numpy as np
import pytest

import exact_io_aware_98_b200 as fa
from exact_io_aware_98_b200 import build as fabuild
from paged_util import plan_ref

OK, INVALID, UNSUPPORTED, ALIGN, CUDA, TIMEOUT, WORKSPACE = 0, -1, -2, -3, -4, -5, -6
A = 0x100000  # an aligned fake device address; never dereferenced by these calls
L3, L8 = ctypes.c_int64 * 3, ctypes.c_int64 * 8


@pytest.fixture(scope="module")
def lib():
    fabuild.build()
    return fa.load()


def _rope(lib, x=A, y=A + 4096, pos=None, f=A, B=1, H=2, N=4, d=64, rot=64, xs=(512, 256, 64),
          ys=(512, 256, 64), ps=0, mag=1.0, opt=0, dtype=0):
    return lib.fa_rope(x, y, pos, f, B, H, N, d, rot, L3(*xs), L3(*ys), ps, mag, opt, dtype, None)


def test_rope_codes(lib):
    for kw in (dict(dtype=9), dict(opt=4), dict(H=0), dict(N=-1), dict(B=-1), dict(d=0), dict(rot=63),
               dict(rot=66), dict(rot=0), dict(mag=float("nan")), dict(x=None), dict(y=None), dict(f=None),
               dict(ys=(512, 0, 64)), dict(ys=(512, 256, 0)), dict(y=A, ys=(512, 64, 128))):
        assert _rope(lib, **kw) == INVALID, kw
    assert _rope(lib, d=2048, rot=64) == UNSUPPORTED
    assert _rope(lib, N=1 << 25) == UNSUPPORTED
    assert _rope(lib, x=A + 1) == ALIGN and _rope(lib, f=A + 4) == ALIGN and _rope(lib, pos=A + 2) == ALIGN
    assert _rope(lib, N=0) == OK and _rope(lib, B=0) == OK


def _plan(lib, ctx=A, new=A + 256, free=A + 512, nf=4, cur=None, tab=A + 1024, ts=8, B=2, mp=8, page=16, cap=4,
          cu=A + 2048, kv=A + 2304, pos=A + 2560, slots=A + 4096, counts=A + 8192):
    return lib.fa_paged_plan(ctx, new, free, nf, cur, tab, ts, B, mp, page, cap, cu, kv, pos, slots, counts, None)


def test_plan_codes(lib):
    for kw in (dict(ctx=None), dict(free=None), dict(nf=-1), dict(tab=None), dict(ts=7), dict(B=0), dict(mp=0),
               dict(page=8), dict(page=24), dict(page=2048), dict(cap=0), dict(slots=None)):
        assert _plan(lib, **kw) == INVALID, kw
    assert _plan(lib, slots=A + 4) == ALIGN and _plan(lib, cur=A + 1) == ALIGN
    for kw in (dict(cur=A + 8192 + 12), dict(ctx=A + 2304), dict(new=A + 2304 + 4), dict(free=A + 1024 + 28),
               dict(pos=A + 508), dict(counts=A + 4)):
        assert _plan(lib, **kw) == INVALID, kw
        assert "overlaps" in lib.fa_get_last_error().decode()


def test_plan_outputs_apart(lib):
    """Two outputs in one place would be written by different threads: refused, as an input is."""
    base = dict(cu=A + 2048, kv=A + 2304, pos=A + 2560, slots=A + 4096, counts=A + 8192, tab=A + 1024)
    size = dict(cu=12, kv=8, pos=16, slots=32, counts=16, tab=64)  # B = 2, 4 tokens, 8 pages a row
    for a in base:
        for b in base:
            if a == b:
                continue
            step = 8 if b == "slots" else 4
            for at in (base[a], base[a] + (size[a] - 1) // step * step):
                assert _plan(lib, **{b: at}) == INVALID, (a, b)
                assert "overlap" in lib.fa_get_last_error().decode()


def test_plan_outputs_between_the_tables_rows(lib):
    """A table that is the left part of a wider buffer leaves the space behind its rows to others."""
    wide = dict(tab=A + 1024, ts=64, mp=8)  # rows of 32 bytes, 256 apart: A + 1024 and A + 1280
    for name, n in (("counts", 16), ("kv", 8), ("cu", 12), ("pos", 16), ("ctx", 8), ("free", 16)):
        for at in (A + 1024 + 32, A + 1024 + 256 - n, A + 1280 + 32, A + 1024 - n):
            assert _plan(lib, **wide, **{name: at}) != INVALID, (name, at - A)
        for at in (A + 1024, A + 1024 + 28, A + 1280 - n + 4, A + 1280 + 28, A + 1024 - n + 4):
            assert _plan(lib, **wide, **{name: at}) == INVALID, (name, at - A)
            assert "overlap" in lib.fa_get_last_error().decode()


def _append(lib, q=A, k=A, qo=A + 4096, kc=A, slots=A, pos=A, f=A, T=2, H=2, H_kv=1, d=64, rot=64,
            st=(128, 64, 64, 64, 64, 64, 128, 64), kp=1024, vp=1024, page=16, pages=4, mag=1.0, opt=0, dtype=0):
    return lib.fa_paged_append(q, k, A, qo, kc, A, slots, pos, f, T, H, H_kv, d, rot, L8(*st), kp, vp, page, pages,
                               mag, opt, dtype, None)


def test_append_codes(lib):
    for kw in (dict(dtype=2), dict(opt=2), dict(page=17), dict(T=-1), dict(H=-1), dict(H_kv=0), dict(pages=0),
               dict(rot=65), dict(rot=0), dict(f=None), dict(pos=None), dict(mag=float("inf")), dict(kp=1000),
               dict(vp=1), dict(k=None), dict(kc=None), dict(slots=None), dict(q=None), dict(qo=None),
               dict(st=(128, 64, 64, 64, 64, 64, 0, 64)), dict(qo=A, st=(128, 64, 64, 64, 64, 64, 256, 64))):
        assert _append(lib, **kw) == INVALID, kw
    assert _append(lib, d=2048, rot=64, kp=1 << 20, vp=1 << 20) == UNSUPPORTED
    assert _append(lib, k=A + 1) == ALIGN and _append(lib, slots=A + 4) == ALIGN
    assert _append(lib, T=0) == OK


def _fwd(lib, q=A, kc=A, tab=A, o=A + 65536, lse=A + 131072, T=4, B=2, H=4, H_kv=2, d=64, qt=256, qh=64, kp=2048, vp=2048, ts=8,
         page=16, pages=4, mp=8, scale=0.125, dtype=0, ws=A, wsb=1 << 30):
    return lib.fa_paged_fwd(q, kc, A, tab, A, A, o, lse, T, B, H, H_kv, d, qt, qh, kp, vp, ts, page, pages, mp, 1, scale, 1,
                            dtype, ws, wsb, None)


def test_fwd_codes(lib):
    for kw in (dict(q=None), dict(kc=None), dict(tab=None), dict(o=None), dict(lse=None), dict(T=-1), dict(B=0),
               dict(H_kv=3), dict(H_kv=0), dict(d=0), dict(scale=0.0), dict(scale=float("nan")), dict(dtype=5),
               dict(page=20), dict(pages=0), dict(mp=0), dict(ts=7), dict(kp=2047), dict(vp=0)):
        assert _fwd(lib, **kw) == INVALID, kw
    for kw in (dict(d=96, kp=1 << 20, vp=1 << 20), dict(d=256, dtype=1, kp=1 << 20, vp=1 << 20), dict(T=1 << 25),
               dict(mp=1 << 28, ts=1 << 28)):
        assert _fwd(lib, **kw) == UNSUPPORTED, kw
    for kw in (dict(o=A), dict(o=A + 2032), dict(lse=A + 16), dict(o=A + 131072)):
        assert _fwd(lib, **kw) == INVALID, kw
        assert "overlap" in lib.fa_get_last_error().decode()
    for kw in (dict(q=A + 8), dict(kc=A + 8), dict(o=A + 65540), dict(lse=A + 131076), dict(tab=A + 2), dict(qt=260),
               dict(qh=4), dict(kp=2052)):
        assert _fwd(lib, **kw) == ALIGN, kw
    for kw in (dict(ws=None), dict(wsb=64), dict(ws=A + 16)):
        assert _fwd(lib, **kw) == WORKSPACE, kw
    assert _fwd(lib, T=0) == OK


def test_workspace_size(lib):
    size = lib.fa_paged_workspace_size
    assert size(0, 1, 4, 2, 64) == 0 and size(1, 1, 4, 3, 64) == 0 and size(1, 1, 4, 2, 129) == 0
    assert 0 < size(1, 1, 4, 2, 64) <= size(64, 1, 4, 2, 64) <= size(4096, 1, 4, 2, 64) == size(1 << 20, 1, 4, 2, 64)
    assert size(1 << 20, 8, 64, 1, 128) < 64 << 20  # bounded whatever the batch


def test_plan_sizes_beyond_the_append(lib):
    # as the append and the attention, which take 2^24 tokens; a block's token range then fits 32 bits
    assert _plan(lib, cap=(1 << 24) + 1) == UNSUPPORTED and _plan(lib, cap=0x7fffffff) == UNSUPPORTED
    assert _plan(lib, B=(1 << 24) + 1) == UNSUPPORTED


def test_plan_reference_by_hand():
    """ctx 17 (pages 5, 6), 3 new: rows 1-3 of page 6.  ctx 0, 18 new: pages 9 and 2."""
    table = np.array([[5, 6, -1], [-1, -1, -1]], np.int32)
    r = plan_ref([17, 0], [3, 18], [9, 2, 4], table, 16, 23)
    assert r["cu_q"] == [0, 3, 21] and r["kv_len"] == [20, 18]
    assert r["positions"] == [17, 18, 19] + list(range(18)) + [0, 0]
    assert r["slots"] == [97, 98, 99] + [144 + i for i in range(16)] + [32, 33, -1, -1]
    assert r["table"].tolist() == [[5, 6, -1], [9, 2, -1]] and r["counts"] == [21, 2, 0, 2]


def test_binding_refuses_cpu_tensors():
    import torch
    x = torch.zeros((1, 1, 4, 64))
    f = torch.ones(32, dtype=torch.float64)
    c = torch.zeros((2, 1, 16, 64))
    i = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: fa.rope(x, f), lambda: fa.rope_bwd(x, f),
                 lambda: fa.paged_plan(i, i, i, i.view(2, 1), 16, 4),
                 lambda: fa.paged_append(x[0], x[0], c, c, torch.zeros(1, dtype=torch.int64)),
                 lambda: fa.paged_fwd(x[0], c, c, i.view(2, 1), i, torch.zeros(3, dtype=torch.int32))):
        with pytest.raises(fa.FaError):
            call()


def test_binding_constants_match_the_header():
    import os
    import re
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "fa.h")).read()
    vals = {k: int(v) for k, v in re.findall(r"\b(FA_ROPE_[A-Z]+)\s*=\s*(\d+)", text)}
    assert vals == {"FA_ROPE_INTERLEAVED": fa.ROPE_INTERLEAVED, "FA_ROPE_BACKWARD": fa.ROPE_BACKWARD}


def test_packed_calls(lib):
    """The packed forms refuse what their calls refuse, and a structure of another size."""
    A64 = A
    rope = [A64, A64 + 4096, 0, A64, 0, 512, 256, 64, 512, 256, 64, 0, 1, 2, 4, 64, 64, 0, 0, 1.0]
    plan = [A64, A64 + 256, A64 + 512, 0, A64 + 1024, A64 + 2048, A64 + 2304, A64 + 2560, A64 + 8192, A64 + 4096, 0, 8, 4,
            2, 8, 16, 4, 0]
    append = [A64, A64, A64, A64 + 4096, A64, A64, A64, A64, A64, 0, 128, 64, 64, 64, 64, 64, 128, 64, 1024, 1024,
              2, 2, 1, 64, 64, 16, 4, 0, 0, 1.0]
    fwd = [A64, A64, A64, A64, A64, A64, A64 + 65536, A64 + 131072, A64, 0, 1 << 30, 256, 64, 2048, 2048, 8, 4, 2, 4, 2, 64, 16, 4, 8, 1,
           1, 0, 0.125]
    for fn, st, ok, at, bad, code in (
            (lib.fa_rope_packed, fa._ROPE, rope, 16, 63, INVALID), (lib.fa_rope_packed, fa._ROPE, rope, 0, A + 1, ALIGN),
            (lib.fa_rope_packed, fa._ROPE, rope, 19, float("nan"), INVALID),
            (lib.fa_rope_packed, fa._ROPE, rope, 14, 1 << 25, UNSUPPORTED),
            (lib.fa_paged_plan_packed, fa._PLAN, plan, 15, 24, INVALID),
            (lib.fa_paged_plan_packed, fa._PLAN, plan, 16, 0, INVALID),
            (lib.fa_paged_plan_packed, fa._PLAN, plan, 9, A + 4, ALIGN),
            (lib.fa_paged_append_packed, fa._APPEND, append, 23, 2048, UNSUPPORTED),
            (lib.fa_paged_append_packed, fa._APPEND, append, 28, 2, INVALID),
            (lib.fa_paged_append_packed, fa._APPEND, append, 6, A + 4, ALIGN),
            (lib.fa_paged_append_packed, fa._APPEND, append, 29, float("inf"), INVALID),
            (lib.fa_paged_fwd_packed, fa._FWD, fwd, 27, 0.0, INVALID),
            (lib.fa_paged_fwd_packed, fa._FWD, fwd, 20, 96, UNSUPPORTED),
            (lib.fa_paged_fwd_packed, fa._FWD, fwd, 10, 64, WORKSPACE),
            (lib.fa_paged_fwd_packed, fa._FWD, fwd, 26, 5, INVALID), (lib.fa_paged_fwd_packed, fa._FWD, fwd, 11, 260, ALIGN)):
        values = list(ok)
        values[at] = bad
        if st is fa._FWD and at == 20:
            values[13] = values[14] = 1 << 20
        assert fn(st.pack(st.size, *values)) == code, (fn.__name__, at, bad)
        assert fn(st.pack(st.size + 8, *ok)) == INVALID and "bytes" in lib.fa_get_last_error().decode()
        assert fn(None) == INVALID
    none = list(fwd)
    none[16] = 0  # no token
    assert lib.fa_paged_fwd_packed(fa._FWD.pack(fa._FWD.size, *none)) == OK
