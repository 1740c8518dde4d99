"""Measured cases of the rotary-position and paged-cache operators.

``run`` computes each operator in plain torch operations, or, with ``own`` set, through this
package's entry points.  Four operators:

  rope    rotary positions on query or key tensors, forward and backward (bf16, fp32)
  plan    lengths of a batch of requests -> token offsets, positions, cache slots, block table
  append  new keys (rotated) and values into the paged cache, and the queries' rotation
  attend  attention of each request's new tokens over its paged cache: output and log-sum-exp
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------------- cases
def listed():
    return [
        # the GPT-2-shaped training batch of the benchmark, pairs interleaved
        dict(name="rope_train_d64", op="rope", B=8, H=12, N=1024, d=64, rot=64, dtype="bf16",
             interleaved=True, backward=False, packed=False, scaling="none", far=0),
        # the gradient of the long-context queries, frequencies scaled by parts for a 4x context
        dict(name="rope_grad_long_d128", op="rope", B=1, H=16, N=16384, d=128, rot=128,
             dtype="bf16", interleaved=False, backward=True, packed=False, scaling="by_parts",
             far=0),
        # a ragged token batch cut out of a fused projection, part of the head, far positions
        dict(name="rope_packed_f32_d80", op="rope", B=1, H=5, N=4099, d=80, rot=48, dtype="f32",
             interleaved=False, backward=False, packed=True, scaling="linear", far=1000000),
        # one decode step of a full server batch: every request has one new token
        dict(name="plan_decode_b256", op="plan", B=256, ctx=32768, new=1, page=16, pad=0),
        # a step of prompt chunks of all lengths, with room left for more tokens
        dict(name="plan_chunks_b64", op="plan", B=64, ctx=8192, new=1000, page=64, pad=300),
        # keys, values and queries of one decode step
        dict(name="append_decode_t64", op="append", T=64, H=32, H_kv=8, d=128, rot=128, page=16,
             dtype="bf16", interleaved=False, pad=0),
        # keys, values and queries of prompt chunks, the last tokens being padding
        dict(name="append_chunk_t8201", op="append", T=8201, H=16, H_kv=4, d=64, rot=32, page=64,
             dtype="bf16", interleaved=True, pad=9),
        # one request, one new token: the latency of a single user's decode step
        dict(name="attend_decode_one", op="attend", B=1, q_lo=1, q_hi=1, chunks=0, kv_lo=2000,
             kv_hi=2000, H=32, H_kv=8, d=128, page=16, dtype="bf16", causal=True),
        # a decode step of a server batch with contexts of all lengths
        dict(name="attend_decode_b64", op="attend", B=64, q_lo=1, q_hi=1, chunks=0, kv_lo=1,
             kv_hi=16384, H=32, H_kv=8, d=128, page=64, dtype="bf16", causal=True),
        # decode steps and prompt chunks in one batch
        dict(name="attend_mixed_b32", op="attend", B=32, q_lo=1, q_hi=1, chunks=4, kv_lo=100,
             kv_hi=8192, H=16, H_kv=4, d=64, page=16, dtype="bf16", causal=True),
        # a chunk of a long prompt over what has been cached of it
        dict(name="attend_chunk_long", op="attend", B=1, q_lo=2048, q_hi=2048, chunks=0,
             kv_lo=32768, kv_hi=32768, H=16, H_kv=4, d=128, page=64, dtype="bf16", causal=True),
        # fp32, an odd head dimension, every length from none upwards
        dict(name="attend_f32_d80", op="attend", B=7, q_lo=0, q_hi=130, chunks=0, kv_lo=0,
             kv_hi=2500, H=6, H_kv=2, d=80, page=16, dtype="f32", causal=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "plan", "append", "attend", "attend"])
    if op == "rope":
        dtype = rng.choice(["bf16", "f32"])
        d = rng.choice([32, 64, 64, 80, 96, 128, 128])
        packed = rng.random() < 0.5
        H = rng.randint(1, 24)
        B = 1 if packed else rng.randint(1, 8)
        N = _log_int(rng, 1, max(2, 12000000 // (B * H * d)))
        return dict(op="rope", B=B, H=H, N=N, d=d, rot=rng.choice([d, d, 2 * rng.randint(1, d // 2)]),
                    dtype=dtype, interleaved=rng.random() < 0.5, backward=rng.random() < 0.5,
                    packed=packed, scaling=rng.choice(["none", "linear", "ntk", "by_parts"]),
                    far=rng.choice([0, 5000, 1000000]))
    if op == "plan":
        new = _log_int(rng, 1, 1000)
        return dict(op="plan", B=_log_int(rng, 1, min(1024, 60000 // new)), ctx=_log_int(rng, 16, 32768),
                    new=new, page=rng.choice([16, 32, 64, 128]), pad=rng.choice([0, 7, 300]))
    if op == "append":
        d = rng.choice([64, 128])
        H_kv = rng.choice([1, 2, 4, 8])
        return dict(op="append", T=_log_int(rng, 1, 8201), H=H_kv * rng.choice([1, 2, 3, 4]), H_kv=H_kv, d=d,
                    rot=rng.choice([d, d // 2]), page=rng.choice([16, 32, 64, 128]),
                    dtype=rng.choice(["bf16", "bf16", "f32"]), interleaved=rng.random() < 0.5,
                    pad=rng.choice([0, 5]))
    H_kv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 8])
    page = rng.choice([16, 32, 64, 128])
    if rng.random() < 0.2:
        return dict(op="attend", B=rng.randint(1, 8), q_lo=0, q_hi=_log_int(rng, 1, 130), chunks=0, kv_lo=0,
                    kv_hi=_log_int(rng, 1, 2500), H=2 * group, H_kv=2, d=rng.choice([32, 64, 80, 128]),
                    page=page, dtype="f32", causal=rng.random() < 0.7)
    kind = rng.choice(["decode", "few", "chunk", "mixed"])
    d = rng.choice([64, 128])
    base = dict(op="attend", H=H_kv * group, H_kv=H_kv, d=d, page=page, dtype="bf16",
                causal=rng.random() < 0.85, chunks=0)
    if kind == "decode":
        B = _log_int(rng, 1, 64)
        return dict(base, B=B, q_lo=1, q_hi=1, kv_lo=1, kv_hi=_log_int(rng, 16, 16384))
    if kind == "few":
        return dict(base, B=rng.randint(1, 24), q_lo=1, q_hi=rng.randint(2, 9), kv_lo=0,
                    kv_hi=_log_int(rng, 64, 8192))
    if kind == "chunk":
        q = _log_int(rng, 16, 1024)
        return dict(base, B=rng.randint(1, 4), q_lo=1, q_hi=q, kv_lo=0, kv_hi=_log_int(rng, q, 16384))
    return dict(base, B=rng.randint(3, 32), q_lo=1, q_hi=1, chunks=rng.randint(1, 2), kv_lo=100,
                kv_hi=_log_int(rng, 512, 8192))


# ------------------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 7919 + 13)


def _randn(g, shape, dtype):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(DTYPES[dtype])


def _i32(values):
    return torch.tensor(np.asarray(values, dtype=np.int32), device=DEV)


def _scaling(kind):
    """(base, factor, original length, beta_fast, beta_slow) of the scaled frequencies."""
    return dict(base=10000.0, factor=4.0 if kind != "none" else 1.0, original_length=4096,
                beta_fast=32.0, beta_slow=1.0)


def _plain_frequencies(rot, kind):
    s = _scaling(kind)
    i = torch.arange(rot // 2, dtype=torch.float64)
    base = s["base"]
    if kind == "ntk" and rot > 2:
        base = base * s["factor"] ** (rot / (rot - 2.0))
    f = torch.pow(torch.tensor(base, dtype=torch.float64), -2.0 * i / rot)
    magnitude = 1.0
    if kind == "linear":
        f = f / s["factor"]
    if kind == "by_parts":
        turns = s["original_length"] * f / (2.0 * math.pi)
        keep = ((turns - s["beta_slow"]) / (s["beta_fast"] - s["beta_slow"])).clamp(0.0, 1.0)
        f = f * keep + f / s["factor"] * (1.0 - keep)
        magnitude = 0.1 * math.log(s["factor"]) + 1.0
    return f.to(DEV), magnitude


def _frequencies(rot, kind):
    if own:
        import exact_io_aware_98_b200 as fa
        s = _scaling(kind)
        return fa.rope_frequencies(rot, base=s["base"], scaling=None if kind == "none" else kind,
                                   factor=s["factor"], original_length=s["original_length"],
                                   beta_fast=s["beta_fast"], beta_slow=s["beta_slow"], device=DEV)
    return _plain_frequencies(rot, kind)


def _attend_lengths(case):
    """Query and key lengths of the requests, on the host as a scheduler holds them (of the case
    alone, so that the work is the same whatever the seed)."""
    rng = np.random.default_rng([case["B"], case["kv_hi"], case["q_hi"], 5])
    B = case["B"]
    kv = rng.integers(case["kv_lo"], case["kv_hi"] + 1, size=B)
    q = rng.integers(case["q_lo"], case["q_hi"] + 1, size=B)
    if case["chunks"]:
        who = rng.permutation(B)[:case["chunks"]]
        q[who] = np.maximum(1, kv[who] // rng.integers(2, 9, size=len(who)))
    q = np.minimum(q, kv) if case["kv_lo"] > 0 else q  # a server's new tokens are in the cache
    return [int(x) for x in q], [int(x) for x in kv]


def _plan_lengths(case):
    rng = np.random.default_rng([case["B"], case["ctx"], case["new"], 6])
    ctx = rng.integers(0, case["ctx"] + 1, size=case["B"])
    new = np.ones(case["B"], np.int64) if case["new"] == 1 else rng.integers(0, case["new"] + 1, size=case["B"])
    return [int(x) for x in ctx], [int(x) for x in new]


def prepare(case, seed):
    g = _gen(seed)
    st = {"case": dict(case)}
    if case["op"] == "rope":
        B, H, N, d = case["B"], case["H"], case["N"], case["d"]
        st["inv_freq"], st["magnitude"] = _frequencies(case["rot"], case["scaling"])
        if case["packed"]:
            fused = _randn(g, (N, (H + 2) * d), case["dtype"])  # queries, one key, one value
            st["x"] = fused[:, :H * d].view(N, H, d)
        else:
            st["x"] = _randn(g, (B, H, N, d), case["dtype"])
        st["positions"] = None
        if case["far"]:
            st["positions"] = torch.randint(0, case["far"], (N,), generator=g, device=DEV, dtype=torch.int32)
        st["y"] = torch.empty(st["x"].shape, dtype=st["x"].dtype, device=DEV)
        return st
    if case["op"] == "plan":
        ctx, new = _plan_lengths(case)
        page = case["page"]
        held = [-(-c // page) for c in ctx]
        need = sum(-(-(c + n) // page) for c, n in zip(ctx, new))
        pages = torch.randperm(need + 32, generator=g, device=DEV).to(torch.int32)
        width = max(-(-(c + n) // page) for c, n in zip(ctx, new)) + 1
        table = torch.full((case["B"], width), -1, dtype=torch.int32)
        ids = pages.cpu()
        at = 0
        for b, h in enumerate(held):
            table[b, :h] = ids[at:at + h]
            at += h
        st.update(ctx=ctx, new=new, ctx_len=_i32(ctx), new_len=_i32(new), table=table.to(DEV),
                  free=pages[at:].clone(), max_tokens=max(1, sum(new) + case["pad"]))
        if own:
            import exact_io_aware_98_b200 as fa
            st["plan"] = fa.PagedPlan.empty(case["B"], st["max_tokens"], DEV)
        return st
    if case["op"] == "append":
        T, H, H_kv, d, page = case["T"], case["H"], case["H_kv"], case["d"], case["page"]
        fused = _randn(g, (T, (H + 2 * H_kv) * d), case["dtype"])
        st["q"] = fused[:, :H * d].view(T, H, d)
        st["k"] = fused[:, H * d:(H + H_kv) * d].view(T, H_kv, d)
        st["v"] = fused[:, (H + H_kv) * d:].view(T, H_kv, d)
        pages = -(-T // page) + 5
        st["k_cache"] = _randn(g, (pages, H_kv, page, d), case["dtype"])
        st["v_cache"] = _randn(g, (pages, H_kv, page, d), case["dtype"])
        slots = torch.randperm(pages * page, generator=g, device=DEV)[:T].to(torch.int64)
        if case["pad"] and T > case["pad"]:
            slots[T - case["pad"]:] = -1
        st["slots"] = slots
        st["positions"] = torch.randint(0, 32768, (T,), generator=g, device=DEV, dtype=torch.int32)
        st["inv_freq"], st["magnitude"] = _frequencies(case["rot"], "none")
        st["q_out"] = torch.empty((T, H, d), dtype=st["q"].dtype, device=DEV)
        return st
    q_len, kv_len = _attend_lengths(case)
    B, H, H_kv, d, page = case["B"], case["H"], case["H_kv"], case["d"], case["page"]
    T = sum(q_len) + 3  # three rows of padding behind the last request
    held = [-(-n // page) for n in kv_len]
    pages = sum(held) + 4
    width = max(1, max(held))
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table = torch.zeros((B, width), dtype=torch.int32)
    ids = order.cpu()
    at = 0
    for b, h in enumerate(held):
        table[b, :h] = ids[at:at + h]
        at += h
    st.update(q_len=q_len, kv_lens=kv_len, table=table.to(DEV), kv_len=_i32(kv_len),
              cu_q=_i32(np.concatenate([[0], np.cumsum(q_len)])), max_q=max(1, max(q_len)))
    st["q"] = _randn(g, (T, H, d), case["dtype"])
    st["k_cache"] = _randn(g, (pages, H_kv, page, d), case["dtype"])
    st["v_cache"] = _randn(g, (pages, H_kv, page, d), case["dtype"])
    st["out"] = torch.zeros((T, H, d), dtype=st["q"].dtype, device=DEV)
    st["lse"] = torch.zeros((T, H), dtype=torch.float32, device=DEV)
    if own:
        import exact_io_aware_98_b200 as fa
        st["workspace"] = torch.empty(fa.paged_workspace_size(T, B, H, H_kv, d), dtype=torch.uint8, device=DEV)
    return st


# ------------------------------------------------------------------------------------- passes
def run(st):
    return {"rope": _rope, "plan": _plan, "append": _append, "attend": _attend}[st["case"]["op"]](st)


def _rotate(x32, angles, rot, interleaved, sign, magnitude):
    """Plain rotation of the first ``rot`` columns; ``angles`` broadcasts over x32[..., :rot/2]."""
    cos = (torch.cos(angles) * magnitude).to(torch.float32)
    sin = (torch.sin(angles) * (magnitude * sign)).to(torch.float32)
    h = rot // 2
    y = x32.clone()
    if interleaved:
        a, b = x32[..., 0:rot:2], x32[..., 1:rot:2]
        y[..., 0:rot:2] = a * cos - b * sin
        y[..., 1:rot:2] = b * cos + a * sin
    else:
        a, b = x32[..., :h], x32[..., h:rot]
        y[..., :h] = a * cos - b * sin
        y[..., h:rot] = b * cos + a * sin
    return y


def _rope(st):
    c = st["case"]
    if own:
        import exact_io_aware_98_b200 as fa
        call = fa.rope_bwd if c["backward"] else fa.rope
        return call(st["x"], st["inv_freq"], positions=st["positions"], interleaved=c["interleaved"],
                    magnitude=st["magnitude"], out=st["y"])
    pos = st["positions"] if st["positions"] is not None else torch.arange(c["N"], device=DEV)
    ang = pos.to(torch.float64)[:, None] * st["inv_freq"][None, :]
    if c["packed"]:
        ang = ang[:, None, :]
    y = _rotate(st["x"].to(torch.float32), ang, c["rot"], c["interleaved"],
                -1.0 if c["backward"] else 1.0, st["magnitude"])
    return y.to(st["x"].dtype)


def _plan(st):
    c = st["case"]
    if own:
        import exact_io_aware_98_b200 as fa
        p = fa.paged_plan(st["ctx_len"], st["new_len"], st["free"], st["table"], c["page"], st["max_tokens"],
                          out=st["plan"])
        return [p.cu_q, p.kv_len, p.positions, p.slots, st["table"], p.counts]
    page, B, cap = c["page"], c["B"], st["max_tokens"]
    ctx, new = st["ctx_len"].long(), st["new_len"].long()
    cu = torch.zeros(B + 1, dtype=torch.int64, device=DEV)
    cu[1:] = torch.cumsum(new, 0)
    first = (ctx + page - 1) // page
    pages = (ctx + new + page - 1) // page - first
    base = torch.cumsum(pages, 0) - pages
    t = torch.arange(cap, device=DEV)
    req = torch.searchsorted(cu, t, right=True) - 1
    live = t < cu[B]
    req = req.clamp(0, B - 1)
    pos = ctx[req] + t - cu[req]
    at = pos // page
    fresh = at >= first[req]
    pick = (base[req] + at - first[req]).clamp(0, st["free"].numel() - 1)
    old = st["table"].long()[req, at.clamp(0, st["table"].shape[1] - 1)]
    ids = torch.where(fresh, st["free"].long()[pick], old)
    slots = torch.where(live, ids * page + pos % page, torch.full_like(ids, -1))
    opens = live & fresh & (pos % page == 0)
    st["table"][req[opens], at[opens]] = ids[opens].to(torch.int32)
    total = pages.sum()
    counts = torch.stack([cu[B], total, torch.zeros_like(total), total]).to(torch.int32)
    return [cu.to(torch.int32), (ctx + new).to(torch.int32),
            torch.where(live, pos, torch.zeros_like(pos)).to(torch.int32), slots, st["table"], counts]


def _append(st):
    c = st["case"]
    if own:
        import exact_io_aware_98_b200 as fa
        q = fa.paged_append(st["k"], st["v"], st["k_cache"], st["v_cache"], st["slots"],
                            positions=st["positions"], inv_freq=st["inv_freq"],
                            interleaved=c["interleaved"], magnitude=st["magnitude"], q=st["q"],
                            q_out=st["q_out"])
        return [q, st["k_cache"], st["v_cache"]]
    ang = (st["positions"].to(torch.float64)[:, None] * st["inv_freq"][None, :])[:, None, :]
    k = _rotate(st["k"].to(torch.float32), ang, c["rot"], c["interleaved"], 1.0, st["magnitude"])
    q = _rotate(st["q"].to(torch.float32), ang, c["rot"], c["interleaved"], 1.0, st["magnitude"])
    live = st["slots"] >= 0
    s = st["slots"][live]
    pg, off = s // c["page"], s % c["page"]
    st["k_cache"][pg, :, off] = k[live].to(st["k_cache"].dtype)
    st["v_cache"][pg, :, off] = st["v"][live]
    st["q_out"].copy_(q)
    return [st["q_out"], st["k_cache"], st["v_cache"]]


def _attend(st):
    c = st["case"]
    scale = float(np.float32(1.0 / math.sqrt(c["d"])))
    if own:
        import exact_io_aware_98_b200 as fa
        o, lse = fa.paged_fwd(st["q"], st["k_cache"], st["v_cache"], st["table"], st["kv_len"], st["cu_q"],
                              scale=scale, causal=c["causal"], max_q=st["max_q"], out=st["out"],
                              lse=st["lse"], workspace=st["workspace"])
        return [o, lse]
    o, lse = st["out"], st["lse"]
    H, H_kv, d, page = c["H"], c["H_kv"], c["d"], c["page"]
    G = H // H_kv
    at = 0
    for b, (nq, nk) in enumerate(zip(st["q_len"], st["kv_lens"])):
        if nq == 0:
            continue
        rows = slice(at, at + nq)
        at += nq
        if nk == 0:
            o[rows] = 0
            lse[rows] = -math.inf
            continue
        ids = st["table"][b, :-(-nk // page)].long()
        k = st["k_cache"][ids].transpose(0, 1).reshape(H_kv, -1, d)[:, :nk].to(torch.float32)
        v = st["v_cache"][ids].transpose(0, 1).reshape(H_kv, -1, d)[:, :nk].to(torch.float32)
        hide = None
        if c["causal"] and nq > 1:
            i = torch.arange(nq, device=DEV)[:, None] + (nk - nq)
            hide = torch.arange(nk, device=DEV)[None, :] > i
        for j in range(H_kv):
            q = st["q"][rows, j * G:(j + 1) * G].transpose(0, 1).to(torch.float32)
            s = torch.matmul(q, k[j].t()) * scale
            if hide is not None:
                s.masked_fill_(hide, -math.inf)
            m = s.amax(-1, keepdim=True)
            m = torch.where(m == -math.inf, torch.zeros_like(m), m)
            s.sub_(m).exp_()
            l = s.sum(-1, keepdim=True)
            r = torch.matmul(s, v[j])
            r = torch.where(l > 0, r / l, torch.zeros_like(r))
            o[rows, j * G:(j + 1) * G] = r.transpose(0, 1).to(o.dtype)
            lse[rows, j * G:(j + 1) * G] = (m + torch.log(l))[..., 0].t()
    return [o, lse]


# ------------------------------------------------------------------------------------- work
def work(case):
    es = 2 if case.get("dtype") == "bf16" else 4
    if case["op"] == "rope":
        n = case["B"] * case["H"] * case["N"] * case["d"]
        rotated = case["B"] * case["H"] * case["N"] * case["rot"]
        return {"bytes": 2 * n * es + 4 * case["N"] * (1 if case["far"] else 0), "flops": 3 * rotated}
    if case["op"] == "plan":
        ctx, new = _plan_lengths(case)
        tokens = sum(new) + case["pad"]
        fresh = sum(-(-(c + n) // case["page"]) - -(-c // case["page"]) for c, n in zip(ctx, new))
        return {"bytes": 16 * case["B"] + 4 + 12 * tokens + 8 * fresh, "flops": 4 * tokens}
    if case["op"] == "append":
        per = (case["H"] + 2 * case["H_kv"]) * case["d"] * es
        return {"bytes": case["T"] * (2 * per + 12), "flops": 3 * case["T"] * (case["H"] + case["H_kv"]) * case["rot"]}
    q_len, kv_len = _attend_lengths(case)
    pairs = 0
    read = 0
    for nq, nk in zip(q_len, kv_len):
        if nq == 0:
            continue
        read += nk
        pairs += sum(max(0, nk - nq + 1 + i) for i in range(nq)) if case["causal"] else nq * nk
    H, H_kv, d = case["H"], case["H_kv"], case["d"]
    return {"bytes": 2 * sum(q_len) * H * d * es + 4 * sum(q_len) * H + 2 * read * H_kv * d * es
            + 4 * read // case["page"], "flops": 4 * d * H * pairs}


# ------------------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    """The outputs of ``run`` from the definitions, in 64 bits."""
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    return {"rope": _exact_rope, "plan": _exact_plan, "append": _exact_append,
            "attend": _exact_attend}[case["op"]](st)


def _exact_turn(x, pos, st, sign=1.0):
    """Rotation as a complex product e^{i a} (x1 + i x2), x [tokens, heads, d] in float64."""
    c = st["case"]
    rot, x = c["rot"], x.double()
    w = torch.polar(torch.full((pos.numel(), rot // 2), st["magnitude"], dtype=torch.float64, device=DEV),
                    sign * torch.outer(pos.double(), st["inv_freq"]))[:, None, :]
    if c["interleaved"]:
        z = torch.complex(x[..., 0:rot:2].contiguous(), x[..., 1:rot:2].contiguous()) * w
        head = torch.stack([z.real, z.imag], -1).flatten(-2)
    else:
        z = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous()) * w
        head = torch.cat([z.real, z.imag], -1)
    return torch.cat([head, x[..., rot:]], -1)


def _exact_rope(st):
    c = st["case"]
    pos = st["positions"] if st["positions"] is not None else torch.arange(c["N"], device=DEV)
    sign = -1.0 if c["backward"] else 1.0
    if c["packed"]:
        return _exact_turn(st["x"], pos, st, sign)
    return torch.stack([_exact_turn(xb.transpose(0, 1), pos, st, sign).transpose(0, 1) for xb in st["x"]])


def _exact_plan(st):
    c = st["case"]
    page, cap = c["page"], st["max_tokens"]
    table = st["table"].cpu().numpy().copy()
    free = [int(x) for x in st["free"].cpu()]
    cu, pos, slots, taken = [0], [], [], 0
    for b, (h, n) in enumerate(zip(st["ctx"], st["new"])):
        for p in range(h, h + n):
            if p % page == 0:
                table[b, p // page] = free[taken]
                taken += 1
            pos.append(p)
            slots.append(int(table[b, p // page]) * page + p % page)
        cu.append(cu[-1] + n)
    pos += [0] * (cap - len(pos))
    slots += [-1] * (cap - len(slots))
    return [_i32(cu), _i32([h + n for h, n in zip(st["ctx"], st["new"])]), _i32(pos),
            torch.tensor(slots, dtype=torch.int64, device=DEV), _i32(table), _i32([cu[-1], taken, 0, taken])]


def _exact_append(st):
    c = st["case"]
    k, v = st["k_cache"].double(), st["v_cache"].double()
    rows = torch.arange(c["T"], device=DEV)[st["slots"] >= 0]
    s = st["slots"][rows]
    turned = _exact_turn(st["k"], st["positions"], st)
    for j in range(c["H_kv"]):
        kj, vj = k[:, j].flatten(0, 1), v[:, j].flatten(0, 1)  # copies: slots in order
        kj[s] = turned[rows, j]
        vj[s] = st["v"][rows, j].double()
        k[:, j], v[:, j] = kj.view_as(k[:, j]), vj.view_as(v[:, j])
    return [_exact_turn(st["q"], st["positions"], st), k, v]


def _exact_attend(st):
    c = st["case"]
    H, d, page, G = c["H"], c["d"], c["page"], c["H"] // c["H_kv"]
    scale = float(np.float32(1.0 / math.sqrt(d)))
    o, lse = st["out"].double(), st["lse"].double()
    start = 0
    for b, (nq, nk) in enumerate(zip(st["q_len"], st["kv_lens"])):
        j = torch.arange(nk, device=DEV)
        slot_page, slot_off = st["table"][b].long()[j // page], j % page
        for h in range(H):
            if nq == 0:
                break
            k = st["k_cache"][slot_page, h // G, slot_off].double()
            v = st["v_cache"][slot_page, h // G, slot_off].double()
            for i0 in range(0, nq, 1024):
                i = torch.arange(i0, min(nq, i0 + 1024), device=DEV)
                logits = scale * (st["q"][start + i, h].double() @ k.T)
                if c["causal"]:
                    logits = torch.where(j[None, :] <= (nk - nq + i)[:, None], logits,
                                         torch.full_like(logits, -math.inf))
                z = torch.logsumexp(logits, -1) if nk else torch.full((i.numel(),), -math.inf, dtype=torch.float64, device=DEV)
                lse[start + i, h] = z
                p = torch.exp(logits - torch.where(torch.isinf(z), torch.zeros_like(z), z)[:, None])
                o[start + i, h] = p @ v
        start += nq
    return [o, lse]
