"""Plain 64-bit versions of the rotary and paged-cache operators, for their tests: numpy, one
request and one head at a time.  Beside each output of the attention stands a bound on a kernel's
error, from the arithmetic it may use."""
from __future__ import annotations

import numpy as np
import torch

U32 = 2.0 ** -24                       # half a step of fp32, relative
HALF = {"bf16": 2.0 ** -8, "f32": U32}  # half a step of the output type, relative
TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().to(torch.float64).numpy()


def rope_ref(x, inv_freq, pos, interleaved, magnitude=1.0, sign=1.0):
    """x [..., d] float64 whose second-last axis pairs with pos [tokens]."""
    h = len(inv_freq)
    a = sign * np.outer(np.asarray(pos, np.float64), inv_freq)
    c, s = magnitude * np.cos(a), magnitude * np.sin(a)
    y = x.copy()
    i = np.arange(h)
    i1, i2 = (2 * i, 2 * i + 1) if interleaved else (i, i + h)
    y[..., i1] = x[..., i1] * c - x[..., i2] * s
    y[..., i2] = x[..., i2] * c + x[..., i1] * s
    return y


def rope_bound(x, h, interleaved, magnitude, dtype):
    """Error bound of a rotation: the angle's cos and sin come within 2^-22 (the fp32 remainder of
    a quarter turn, a polynomial and the magnitude's product: under four half steps of 1), two
    products and a sum add three half steps, all relative to |x1| + |x2|; then one rounding to the
    output's type of a value of at most magnitude (|x1| + |x2|)."""
    i = np.arange(h)
    i1, i2 = (2 * i, 2 * i + 1) if interleaved else (i, i + h)
    b = np.zeros_like(x)
    size = magnitude * (np.abs(x[..., i1]) + np.abs(x[..., i2]))
    e = size * (8 * U32) + size * HALF[dtype]
    b[..., i1] = e
    b[..., i2] = e
    return b


def attend_ref(q, k, v, keep, scale, dtype):
    """One head: q [nq, d], k, v [nk, d] float64, keep [nq, nk] bool.  (o, lse, bound on |o error|,
    bound on |lse error|).  Scores: d products summed in fp32, scaled, in log2 units: at most
    (2 d + 4) half steps of sum |q k| scale (twice the d roundings: tensor-core sums may cut
    instead of round).  Exponentials: 2^-22 relative.  P rounded to the matrix type for the
    products with V in bf16.  Sums over nk terms: nk half steps at most."""
    nq, d = q.shape
    nk = k.shape[0]
    o = np.zeros((nq, d))
    lse = np.full(nq, -np.inf)
    bo, bl = np.zeros((nq, d)), np.zeros(nq)
    if nk == 0:
        return o, lse, bo, bl
    s = np.where(keep, (q @ k.T) * scale, -np.inf)
    size = np.where(keep, (np.abs(q) @ np.abs(k).T) * scale, 0.0)
    rows = keep.any(1)
    m = np.where(rows, s.max(1), 0.0)
    p = np.exp(s - m[:, None])
    l = p.sum(1)
    a = p / np.where(rows, l, 1.0)[:, None]
    av = np.where(keep.any(0)[:, None], v, 0.0)
    o[rows] = (a @ av)[rows]
    lse[rows] = (m + np.log(np.where(rows, l, 1.0)))[rows]
    es = (2 * d + 4) * U32 * size.max(1) + 2.0 ** -22 + 4 * U32 * np.abs(m)
    weight = (2 * es + 2 * nk * U32 + (HALF["bf16"] if dtype == "bf16" else 0.0))[:, None]
    bo = weight * (a @ np.abs(av)) + HALF[dtype] * np.abs(o) + 1e-30
    bl = es + nk * U32 + 4 * U32 * (np.abs(lse, where=rows, out=np.zeros(nq)) + np.log(nk) + 1)
    return o, lse, bo, bl


def paged_case(lens, H, H_kv, d, page, dtype="bf16", seed=0, pad=2, stale=True, split_cache=False,
               amp=1.0, extra_pages=3, strided_q=False):
    """A ragged batch on the CPU: lens = [(nq, nk)].  Every key row that no request owns is NaN with
    ``stale``.  Returns the tensors of fa.paged_fwd and the per-request dense K and V."""
    g = torch.Generator().manual_seed(seed)
    dt = TORCH[dtype]
    T = sum(n for n, _ in lens) + pad
    held = [-(-n // page) for _, n in lens]
    pages = sum(held) + extra_pages
    width = max(1, max(held))
    fill = float("nan") if stale else 0.0
    pool = torch.full((pages, 2, H_kv, page, d), fill, dtype=dt)
    kc, vc = (pool[:, 0], pool[:, 1]) if split_cache else (pool[:, 0].clone(), pool[:, 1].clone())
    order = torch.randperm(pages, generator=g)
    table = torch.full((len(lens), width), -7, dtype=torch.int32)
    dense = []
    at = 0
    for b, (_, nk) in enumerate(lens):
        k = (torch.randn((H_kv, nk, d), generator=g) * amp).to(dt)
        v = torch.randn((H_kv, nk, d), generator=g).to(dt)
        ids = order[at:at + held[b]]
        at += held[b]
        table[b, :held[b]] = ids.to(torch.int32)
        for i, pg in enumerate(ids.tolist()):
            n = min(page, nk - i * page)
            kc[pg, :, :n] = k[:, i * page:i * page + n]
            vc[pg, :, :n] = v[:, i * page:i * page + n]
        dense.append((f64(k), f64(v)))
    heads = H + 3 if strided_q else H
    q = (torch.randn((T, heads, d), generator=g) * amp).to(dt)[:, heads - H:]
    cu = np.concatenate([[0], np.cumsum([n for n, _ in lens])]).astype(np.int32)
    return dict(q=q, k_cache=kc, v_cache=vc, block_table=table,
                kv_len=torch.tensor([n for _, n in lens], dtype=torch.int32),
                cu_q=torch.from_numpy(cu), dense=dense, lens=lens, H=H, H_kv=H_kv, d=d, page=page,
                dtype=dtype, T=T)


def to_cuda(case):
    """The call's tensors on the GPU, with their strides."""
    out = {}
    for n in ("q", "k_cache", "v_cache", "block_table", "kv_len", "cu_q"):
        t = case[n]
        base = t._base if t._base is not None else t
        b = base.cuda()
        out[n] = torch.as_strided(b, t.shape, t.stride(), t.storage_offset())
    return out


def check_paged(case, o, lse, causal, scale, hidden=None, o_before=None, lse_before=None):
    """o, lse of a paged_fwd call against the plain version; hidden[b]: positions masked by bad
    pages.  Rows of no request must equal *_before."""
    o, lse = o.cpu(), lse.cpu()
    G = case["H"] // case["H_kv"]
    at = 0
    for b, (nq, nk) in enumerate(case["lens"]):
        if nq == 0:
            continue
        q = f64(case["q"][at:at + nq])
        keep = np.ones((nq, nk), bool)
        if causal:
            keep = np.arange(nk)[None, :] <= (nk - nq + np.arange(nq))[:, None]
        if hidden is not None and hidden[b] is not None:
            keep &= ~hidden[b][None, :]
        for h in range(case["H"]):
            k, v = (t[h // G] for t in case["dense"][b])
            ro, rl, bo, bl = attend_ref(q[:, h], k, v, keep, scale, case["dtype"])
            go, gl = f64(o[at:at + nq, h]), f64(lse[at:at + nq, h])
            assert np.array_equal(np.isneginf(gl), np.isneginf(rl)), f"request {b} head {h}: empty rows"
            live = ~np.isneginf(rl)
            assert np.all(go[~live] == 0.0), f"request {b} head {h}: rows without keys"
            err = np.abs(go - ro)
            assert np.all(err <= bo), \
                f"request {b} (nq {nq}, nk {nk}) head {h}: O off by {np.nanmax(err / bo):.2f} of the bound"
            el = np.abs(gl[live] - rl[live])
            assert np.all(el <= bl[live]), f"request {b} head {h}: lse off by {el.max():.3e}"
        at += nq
    if o_before is not None:
        assert torch.equal(o[at:], o_before.cpu()[at:]) and torch.equal(lse[at:], lse_before.cpu()[at:])


def plan_ref(ctx, new, free, table, page, max_tokens, cursor=0):
    """The plan, one token at a time."""
    table = table.copy()
    width = table.shape[1]
    cu, kv, pos, slots = [0], [], [], []
    want = taken = 0
    asked = sum(max(0, n) for n in new)
    for b, (c, n) in enumerate(zip(ctx, new)):
        c, n = max(0, c), max(0, n)
        n = min(n, max_tokens - cu[-1])
        for p in range(c, c + n):
            at = p // page
            pid = -1
            if at < width:
                if p % page == 0:
                    k = cursor + want
                    want += 1
                    table[b, at] = free[k] if k < len(free) else -1
                    taken += k < len(free)
                pid = int(table[b, at])
            pos.append(p)
            slots.append(-1 if pid < 0 else pid * page + p % page)
        cu.append(cu[-1] + n)
        kv.append(c + n)
    pos += [0] * (max_tokens - len(pos))
    slots += [-1] * (max_tokens - len(slots))
    return dict(cu_q=cu, kv_len=kv, positions=pos, slots=slots, table=table,
                counts=[asked, taken, want - taken, cursor + taken])
