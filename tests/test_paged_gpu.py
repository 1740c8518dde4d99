"""The paged cache on the GPU: the plan, the append and the attention over pages, each against a
64-bit (or one-token-at-a-time) version, at the lengths, layouts and masks where they can go
wrong; and the three run together step after step."""
import numpy as np
import pytest
import torch

import synthetic as syn
from paged_util import (TORCH, check_paged, f64, paged_case, plan_ref, rope_bound, rope_ref, to_cuda)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------------ the plan
def _plan(fa, ctx, new, free, table, page, cap, cursor=None):
    i = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    tab = i(table)
    p = fa.paged_plan(i(ctx), i(new), i(free), tab, page, cap,
                      cursor=None if cursor is None else i([cursor]))
    return p, tab


def _check_plan(fa, ctx, new, free, table, page, cap, cursor=None):
    p, tab = _plan(fa, ctx, new, free, table, page, cap, cursor)
    r = plan_ref(ctx, new, free, np.array(table, np.int32), page, cap, cursor or 0)
    for name in ("cu_q", "kv_len", "positions", "slots", "counts"):
        assert getattr(p, name).cpu().tolist() == list(r[name]), name
    assert np.array_equal(tab.cpu().numpy(), r["table"])
    return p, tab


@pytest.mark.parametrize("B,page,hi,seed", [(1, 16, 40, 0), (7, 32, 90, 1), (256, 16, 1, 2), (300, 64, 9, 3),
                                            (1100, 16, 3, 4), (3, 128, 700, 5)])
def test_plan_random_batches(cuda_lib, B, page, hi, seed):
    rng = np.random.default_rng(seed)
    ctx = [int(x) for x in rng.integers(0, 5 * page, B)]
    new = [int(x) for x in rng.integers(0, hi + 1, B)]
    width = max(-(-(c + n) // page) for c, n in zip(ctx, new)) + 1
    ids = [int(x) for x in rng.permutation(B * width + 50)]
    table = [[-1] * width for _ in range(B)]
    at = 0
    for b, c in enumerate(ctx):
        for j in range(-(-c // page)):
            table[b][j] = ids[at]
            at += 1
    _check_plan(cuda_lib, ctx, new, ids[at:], table, page, max(1, sum(new) + seed))
    _check_plan(cuda_lib, ctx, new, ids, table, page, max(1, sum(new) + 300), cursor=at)


def test_plan_edges(cuda_lib):
    fa = cuda_lib
    wide = [[9, 8, 7, -1, -1]]
    _check_plan(fa, [0], [1], [3, 4], [[-1]], 16, 1)
    _check_plan(fa, [0], [0], [3], [[-1]], 16, 4)                        # nothing new
    _check_plan(fa, [-5, 3], [4, -2], [3, 5], [[-1, -1], [2, -1]], 16, 9)  # negative lengths count as 0
    _check_plan(fa, [16], [16], [5, 6], [[4, -1]], 16, 16)               # a page exactly filled
    _check_plan(fa, [31, 40], [20, 20], [5], [[4, 3, -1, -1], [0, 1, 2, -1]], 16, 40)  # pages run out
    _check_plan(fa, [0, 0], [5, 5], [], [[-1], [-1]], 16, 10)            # no page at all
    _check_plan(fa, [40], [60], list(range(20, 30)), wide, 16, 60)       # beyond the table's width
    _check_plan(fa, [10, 20, 30], [30, 30, 30], list(range(50, 70)),
                [[1, -1, -1, -1], [2, 3, -1, -1], [4, 5, -1, -1]], 16, 47)  # more than max_tokens
    _check_plan(fa, [0], [3], [-4, 7], [[-1]], 16, 3)                    # a negative page id
    _check_plan(fa, [0], [40], [3, 4], [[-1, -1, -1]], 16, 40, cursor=9)  # the cursor past the list
    p, _ = _plan(fa, [0] * 3, [2 ** 31 - 1] * 3, [1], [[-1]] * 3, 1024, 5)
    assert p.counts.cpu().tolist()[0] == 2 ** 31 - 1 and p.cu_q.cpu().tolist() == [0, 5, 5, 5]


def test_plan_chains_through_the_cursor(cuda_lib):
    """Step after step with the cursor fed back on the device gives what one long step gives."""
    fa = cuda_lib
    free = torch.randperm(64, generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
    table = torch.full((3, 8), -1, dtype=torch.int32, device="cuda")
    cursor = torch.zeros(1, dtype=torch.int32, device="cuda")
    ctx = torch.zeros(3, dtype=torch.int32, device="cuda")
    new = torch.tensor([17, 1, 9], dtype=torch.int32, device="cuda")
    plan = None
    for _ in range(6):
        plan = fa.paged_plan(ctx, new, free, table, 16, 30, cursor=cursor, out=plan)
        ctx.copy_(plan.kv_len)
        cursor.copy_(plan.counts[3:4])
    assert ctx.cpu().tolist() == [102, 6, 54]
    t = table.cpu().numpy()
    used = t[t >= 0]
    assert len(used) == 7 + 1 + 4 == len(set(used)) == int(cursor)
    assert set(used) == set(free[:12].cpu().tolist())


# ------------------------------------------------------------------------------------ the append
@pytest.mark.parametrize("T,H,H_kv,d,rot,page,dtype,il", [
    (1, 4, 2, 64, 64, 16, "bf16", False), (37, 8, 8, 128, 64, 32, "bf16", True),
    (300, 3, 1, 64, 0, 64, "bf16", False), (65, 5, 5, 80, 40, 16, "bf16", False),
    (129, 6, 2, 20, 10, 128, "f32", True), (50, 2, 1, 7, 4, 16, "f32", False),
    (2000, 32, 8, 128, 128, 1024, "f32", False)])
def test_append_stores_rotated_rows(cuda_lib, T, H, H_kv, d, rot, page, dtype, il):
    fa = cuda_lib
    g = torch.Generator().manual_seed(T)
    fused = torch.randn((T, (H + 2 * H_kv) * d), generator=g).to(TORCH[dtype])
    cut = lambda t: (t[:, :H * d].view(T, H, d), t[:, H * d:(H + H_kv) * d].view(T, H_kv, d),
                     t[:, (H + H_kv) * d:].view(T, H_kv, d))
    pages = -(-T // page) + 2
    pool = torch.randn((pages, 2, H_kv, page, d), generator=g).to(TORCH[dtype])  # one pool for k and v
    slots = torch.randperm(pages * page, generator=g)[:T]
    slots[T // 2] = -1
    if T > 3:
        slots[1], slots[2] = pages * page, 2 ** 40      # past the cache: not stored
    pos = torch.randint(0, 100000, (T,), generator=g, dtype=torch.int32)
    fi, m = fa.rope_frequencies(rot) if rot else (None, 1.0)
    dev = pool.cuda()
    q, k, v = cut(fused.cuda())
    out = fa.paged_append(k, v, dev[:, 0], dev[:, 1], slots.cuda(), positions=pos.cuda() if rot else None,
                          inv_freq=fi, interleaved=il, q=q)
    got = dev.cpu()
    fr = fi.cpu().numpy() if rot else np.zeros(0)
    qr, kr, vr = (t.transpose(0, 1) for t in cut(fused))
    for t, y in ((qr, out.cpu().transpose(0, 1)),):
        err = np.abs(f64(y) - rope_ref(f64(t), fr, pos, il))
        assert np.all(err <= rope_bound(f64(t), len(fr), il, 1.0, dtype))
    want_k, bound_k = rope_ref(f64(kr), fr, pos, il), rope_bound(f64(kr), len(fr), il, 1.0, dtype)
    untouched = torch.ones((pages, page), dtype=torch.bool)
    for t in range(T):
        s = int(slots[t])
        if not 0 <= s < pages * page:
            continue
        pg, off = s // page, s % page
        untouched[pg, off] = False
        assert np.all(np.abs(f64(got[pg, 0, :, off]) - want_k[:, t]) <= bound_k[:, t])
        assert torch.equal(got[pg, 1, :, off], vr[:, t])
    keep = untouched[:, None, None, :, None].expand_as(pool)
    assert torch.equal(got[keep], pool[keep]), "a row that no token names changed"
    z = q.clone()
    fa.paged_append(k, v, dev[:, 0], dev[:, 1], slots.cuda(), positions=pos.cuda() if rot else None,
                    inv_freq=fi, interleaved=il, q=z, q_out=z)
    assert torch.equal(z, out)
    # without queries the cache is the same
    dev2 = pool.cuda()
    assert fa.paged_append(k, v, dev2[:, 0], dev2[:, 1], slots.cuda(),
                           positions=pos.cuda() if rot else None, inv_freq=fi, interleaved=il) is None
    assert torch.equal(dev2, dev)


def test_append_equals_rope(cuda_lib):
    """The append's rotation is fa_rope's, bit for bit, for aligned and unaligned rows."""
    fa = cuda_lib
    fi, m = fa.rope_frequencies(64, scaling="by_parts", factor=4.0, original_length=2048)
    g = torch.Generator().manual_seed(5)
    pos = torch.randint(0, 1 << 20, (70,), generator=g, dtype=torch.int32).cuda()
    for off in (0, 1):
        flat = torch.randn(70 * 2 * 96 + 1, generator=g).to(torch.bfloat16).cuda()
        k = flat[off:off + 70 * 2 * 96].view(70, 2, 96)
        kc = torch.zeros((5, 2, 16, 96), dtype=torch.bfloat16, device="cuda")
        slots = torch.arange(70, device="cuda")
        q = fa.paged_append(k, k, kc, torch.zeros_like(kc), slots, positions=pos, inv_freq=fi, magnitude=m, q=k)
        want = fa.rope(k, fi, positions=pos, magnitude=m)
        assert torch.equal(q, want)
        assert torch.equal(kc.transpose(1, 2).reshape(80, 2, 96)[:70], want)


# ------------------------------------------------------------------------------------ the attention
def _run(fa, case, causal=True, max_q=None, ws=None):
    t = to_cuda(case)
    scale = syn.scale_for(case["d"])
    o = torch.full(case["q"].shape, 3.5, dtype=TORCH[case["dtype"]], device="cuda")
    lse = torch.full(case["q"].shape[:2], 7.25, device="cuda")
    o0, l0 = o.clone(), lse.clone()
    if ws is None:  # scratch that holds anything
        ws = torch.full((fa.paged_workspace_size(case["T"], len(case["lens"]), case["H"], case["H_kv"], case["d"]),),
                        255, dtype=torch.uint8, device="cuda")
    fa.paged_fwd(t["q"], t["k_cache"], t["v_cache"], t["block_table"], t["kv_len"], t["cu_q"], scale=scale,
                 causal=causal, max_q=max_q, out=o, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    assert fa.device_status() == 0
    return t, o, lse, o0, l0, scale


DECODE = [(1, 1), (1, 2), (1, 15), (1, 16), (1, 17), (1, 63), (1, 64), (1, 65), (1, 127), (1, 128), (1, 129),
          (1, 700), (1, 2049), (0, 50), (1, 0), (0, 0)]
RAGGED = [(1, 1), (5, 5), (0, 9), (33, 200), (130, 130), (1, 777), (64, 65), (9, 4), (3, 0), (200, 1031)]
LONG = [(3, 9000)]
CASES = [
    # lens, H, H_kv, d, page, dtype, causal, max_q
    (DECODE, 8, 2, 128, 16, "bf16", True, 1),
    (DECODE, 8, 8, 64, 32, "bf16", True, 1),
    (DECODE, 6, 2, 64, 64, "bf16", True, 1),
    (DECODE, 5, 1, 128, 128, "bf16", False, 1),
    (DECODE, 24, 2, 128, 16, "bf16", True, 1),       # 12 heads a group
    (DECODE, 33, 1, 64, 16, "bf16", True, 1),        # 33 heads a group
    (RAGGED, 4, 2, 64, 16, "bf16", True, 200),
    (RAGGED, 3, 1, 128, 32, "bf16", True, 200),
    (RAGGED, 4, 4, 128, 64, "bf16", True, 200),
    (RAGGED, 2, 1, 64, 1024, "bf16", True, 200),
    (RAGGED, 10, 2, 128, 128, "bf16", False, 200),
    (RAGGED, 3, 3, 128, 16, "bf16", True, 1),        # the hint is wrong
    (DECODE, 8, 2, 128, 16, "bf16", True, 999),      # and the other way
    (RAGGED, 71, 1, 64, 256, "bf16", True, 200),     # 71 heads a group
    (LONG, 8, 2, 128, 16, "bf16", True, 3),          # one request over all SMs
    (LONG, 4, 1, 64, 64, "bf16", True, 3),
    (LONG, 40, 2, 128, 64, "bf16", True, None),
    ([(1, 20000)] * 6, 2, 2, 128, 64, "bf16", True, 1),  # many key tiles per SM
    ([(1, 30000)] * 6, 4, 2, 64, 16, "bf16", True, 1),
    ([(2, 9000), (1, 1)] * 9, 16, 4, 128, 32, "bf16", True, 2),
    ([(300, 4000), (1, 3000), (40, 41)], 8, 2, 128, 16, "bf16", True, 300),
    ([(257, 513)], 2, 2, 64, 16, "bf16", True, 257),
    ([(1, 300)] * 300, 2, 1, 64, 16, "bf16", True, 1),  # many small requests
    ([(0, 5)] * 40 + [(2, 3)] * 600, 1, 1, 64, 16, "bf16", True, 2),
    ([(1, 3)] * 9000, 1, 1, 64, 16, "bf16", True, 1),   # more row tiles than a CTA lists at a time
    ([(1, 3), (2, 2), (0, 7)] * 3000, 2, 2, 64, 16, "bf16", True, 99),
    ([(40, 900)] * 3, 8, 2, 128, 64, "bf16", True, 40),
    ([(12, 900), (3, 40)], 8, 2, 64, 64, "bf16", True, 12),  # 48 rows over a small cache
    ([(1, 2)] * 9000, 1, 1, 8, 16, "f32", True, 1),
    (DECODE, 6, 2, 80, 16, "f32", True, 1),
    (RAGGED, 4, 2, 80, 16, "f32", True, 200),
    (RAGGED, 3, 1, 33, 32, "f32", False, 200),       # odd head dimension
    (RAGGED, 2, 2, 1, 16, "f32", True, 1),
    (DECODE, 20, 1, 128, 64, "f32", True, 1),
    (LONG, 4, 2, 128, 16, "f32", True, 3),
    ([(70, 2000), (1, 900)], 40, 1, 64, 16, "f32", True, 70),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_paged_attention(cuda_lib, case):
    lens, H, H_kv, d, page, dtype, causal, max_q = CASES[case]
    c = paged_case(lens, H, H_kv, d, page, dtype, seed=case)
    _, o, lse, o0, l0, scale = _run(cuda_lib, c, causal, max_q)
    check_paged(c, o, lse, causal, scale, o_before=o0, lse_before=l0)


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("f32", 48)])
@pytest.mark.parametrize("max_q", [1, 500])
def test_paged_layouts_and_large_scores(cuda_lib, dtype, d, max_q):
    """One pool for K and V (page stride of both), queries inside a fused projection, scores of
    size 8 and more."""
    c = paged_case(RAGGED, 4, 2, d, 16, dtype, seed=77, split_cache=True, strided_q=True, amp=3.0)
    _, o, lse, o0, l0, scale = _run(cuda_lib, c, True, max_q)
    check_paged(c, o, lse, True, scale, o_before=o0, lse_before=l0)


@pytest.mark.parametrize("dtype,d,page", [("bf16", 64, 16), ("bf16", 128, 64), ("f32", 40, 16)])
@pytest.mark.parametrize("max_q", [1, 500])
def test_bad_pages_are_masked(cuda_lib, dtype, d, page, max_q):
    """Block-table entries outside the cache hide their keys; a request of bad pages only has
    empty rows; lengths past the table are cut to it."""
    fa = cuda_lib
    lens = [(1, 300), (40, 300), (7, 130), (1, 20)]
    c = paged_case(lens, 4, 2, d, page, dtype, seed=5, extra_pages=4)
    n_pages = c["k_cache"].shape[0]
    hidden = [np.zeros(n, bool) for _, n in lens]
    for b, j, bad in ((0, 1, -1), (0, 3, n_pages), (1, 0, 2 ** 31 - 1), (1, 2, -2 ** 31), (3, 0, n_pages + 5),
                      (3, 1, -9)):
        if j * page < lens[b][1]:
            c["block_table"][b, j] = bad
            hidden[b][j * page:(j + 1) * page] = True
    _, o, lse, o0, l0, scale = _run(fa, c, True, max_q)
    check_paged(c, o, lse, True, scale, hidden=hidden, o_before=o0, lse_before=l0)


@pytest.mark.parametrize("max_q", [1, 500])
def test_lengths_out_of_range_are_clamped(cuda_lib, max_q):
    """kv_len past the table and negative, cu_q past T and falling: in bounds, and the requests with
    sound lengths keep their results."""
    fa = cuda_lib
    lens = [(3, 64), (2, 48), (4, 33)]
    c = paged_case(lens, 2, 1, 64, 16, "bf16", seed=6, pad=0, stale=False)
    t = to_cuda(c)
    good = fa.paged_fwd(t["q"], t["k_cache"], t["v_cache"], t["block_table"], t["kv_len"], t["cu_q"], max_q=max_q)
    kv = torch.tensor([10 ** 9, -3, 33], dtype=torch.int32, device="cuda")
    o, lse = fa.paged_fwd(t["q"], t["k_cache"], t["v_cache"], t["block_table"], kv, t["cu_q"], max_q=max_q)
    assert torch.equal(o[5:], good[0][5:]) and torch.equal(o[:3], good[0][:3])  # 64 positions are the table's
    assert torch.all(o[3:5] == 0) and torch.all(torch.isinf(lse[3:5]))
    cu = torch.tensor([-4, 3, 1, 999], dtype=torch.int32, device="cuda")  # the second request: 3 .. 1
    o = torch.zeros_like(t["q"])
    fa.paged_fwd(t["q"], t["k_cache"], t["v_cache"], t["block_table"], t["kv_len"], cu, out=o, max_q=max_q)
    torch.cuda.synchronize()
    assert fa.device_status() == 0


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f32", 64)])
def test_captured_call_follows_the_lengths(cuda_lib, dtype, d):
    """A captured call, replayed after the lengths, table and queries changed on the device, equals a
    fresh call; two graphs may share a workspace; repeated calls agree bit for bit."""
    fa = cuda_lib
    a = paged_case([(1, 900), (60, 300), (1, 5)], 8, 2, d, 16, dtype, seed=1, pad=20, extra_pages=40)
    t = to_cuda(a)
    wide = torch.zeros((3, 80), dtype=torch.int32, device="cuda")
    wide[:, :t["block_table"].shape[1]] = t["block_table"]
    ws = torch.empty(fa.paged_workspace_size(a["T"], 3, 8, 2, d), dtype=torch.uint8, device="cuda")
    outs = [(torch.zeros_like(t["q"]), torch.zeros(t["q"].shape[:2], device="cuda")) for _ in range(2)]
    calls = [lambda i=i: fa.paged_fwd(t["q"], t["k_cache"], t["v_cache"], wide, t["kv_len"], t["cu_q"],
                                      max_q=(1, 60)[i], out=outs[i][0], lse=outs[i][1], workspace=ws)
             for i in range(2)]
    for c in calls:
        c()
    torch.cuda.synchronize()
    graphs = []
    for c in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c()
        graphs.append(g)
    pages = t["k_cache"].shape[0]
    for kv, cu in (([900, 300, 5], [0, 1, 61, 62]), ([77, 0, 1200], [0, 30, 31, 80]), ([1, 1, 1], [0, 0, 0, 1])):
        t["kv_len"].copy_(torch.tensor(kv, dtype=torch.int32))
        t["cu_q"].copy_(torch.tensor(cu, dtype=torch.int32))
        wide.copy_(torch.randint(0, pages, (3, 80), dtype=torch.int32))
        t["k_cache"].nan_to_num_()
        t["v_cache"].nan_to_num_()
        for o, l in outs:
            o.zero_()
            l.zero_()
        for _ in range(2):
            for g in graphs:
                g.replay()
        torch.cuda.synchronize()
        for i in range(2):
            o2, l2 = torch.zeros_like(outs[i][0]), torch.zeros_like(outs[i][1])
            fa.paged_fwd(t["q"], t["k_cache"], t["v_cache"], wide, t["kv_len"], t["cu_q"], max_q=(1, 60)[i], out=o2,
                         lse=l2)
            assert torch.equal(o2, outs[i][0]) and torch.equal(l2, outs[i][1])
    assert fa.device_status() == 0


def test_two_streams_at_once(cuda_lib):
    """Calls on two streams, each with its workspace, do not disturb one another."""
    fa = cuda_lib
    cases = [paged_case([(1, 3000)] * 6, 8, 2, 128, 16, seed=3), paged_case([(200, 1500)], 8, 2, 64, 64, seed=4)]
    ts = [to_cuda(c) for c in cases]
    args = [(t["q"], t["k_cache"], t["v_cache"], t["block_table"], t["kv_len"], t["cu_q"]) for t in ts]
    want = [fa.paged_fwd(*x) for x in args]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(8):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(fa.paged_fwd(*args[i]))
    torch.cuda.synchronize()
    for i in range(2):
        n = sum(q for q, _ in cases[i]["lens"])
        for o, lse in got[i]:
            assert torch.equal(o[:n], want[i][0][:n]) and torch.equal(lse[:n], want[i][1][:n])


@pytest.mark.parametrize("dtype,d,max_q", [("bf16", 64, 1), ("bf16", 64, 500), ("bf16", 128, 1), ("bf16", 128, 500),
                                           ("f32", 20, 1), ("f32", 20, 500)])
def test_offsets_beyond_32_bits(cuda_lib, dtype, d, max_q):
    """The pages of a cache of more than 2^31 elements, at its far end: append, then attention.  All
    other rows of the cache hold whatever the allocation held."""
    fa = cuda_lib
    page, H, H_kv = 16, 2, 1
    n_pages = (1 << 31) // (H_kv * page * d) + 40
    g = torch.Generator().manual_seed(d)
    dt = TORCH[dtype]
    kc = torch.empty((n_pages, H_kv, page, d), dtype=dt, device="cuda")
    vc = torch.empty_like(kc)
    lens = [(2, 50), (30, 77)]
    c = paged_case(lens, H, H_kv, d, page, dtype, seed=d)
    table = torch.tensor([[n_pages - 1 - i for i in range(10)], [n_pages - 20 - i for i in range(10)]],
                         dtype=torch.int32, device="cuda")
    for b, (_, nk) in enumerate(lens):
        k, v = (torch.from_numpy(x).to(dt).transpose(0, 1).contiguous().cuda() for x in c["dense"][b])
        pos = torch.arange(nk, device="cuda")
        slots = table[b].long()[pos // page] * page + pos % page
        assert int(slots.min()) * H_kv * d > (1 << 31) - 40 * page * d
        fa.paged_append(k, v, kc, vc, slots)
    q = c["q"].cuda()
    o, lse = fa.paged_fwd(q, kc, vc, table, c["kv_len"].cuda(), c["cu_q"].cuda(), scale=syn.scale_for(d), max_q=max_q)
    torch.cuda.synchronize()
    assert fa.device_status() == 0
    check_paged(c, o, lse, True, syn.scale_for(d))


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("f32", 7), ("f32", 64)])
@pytest.mark.parametrize("max_q", [1, 500])
def test_outputs_at_any_allowed_alignment(cuda_lib, dtype, d, max_q):
    """o, lse, q and the caches 16-byte aligned and no more."""
    fa = cuda_lib
    c = paged_case([(3, 70), (20, 40), (1, 300)], 4, 2, d, 16, dtype, seed=8)
    t = to_cuda(c)
    es = 2 if dtype == "bf16" else 4

    def shifted(x, step):
        flat = torch.empty(x.numel() + step, dtype=x.dtype, device="cuda")
        y = flat[step:].view(x.shape)
        y.copy_(x)
        assert y.data_ptr() % 32 == 16
        return y
    q, k, v = (shifted(t[n].contiguous(), 16 // es) for n in ("q", "k_cache", "v_cache"))
    o = shifted(torch.full(c["q"].shape, 2.0, dtype=TORCH[dtype]), 16 // es)
    lse = shifted(torch.full(c["q"].shape[:2], 2.0), 4)
    o0, l0 = o.clone(), lse.clone()
    fa.paged_fwd(q, k, v, t["block_table"], t["kv_len"], t["cu_q"], scale=syn.scale_for(d), max_q=max_q, out=o, lse=lse)
    check_paged(c, o, lse, True, syn.scale_for(d), o_before=o0, lse_before=l0)


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("f32", 33)])
@pytest.mark.parametrize("max_q", [1, 500])
def test_a_bad_request_stays_alone(cuda_lib, dtype, d, max_q):
    """NaN and infinities in one request's keys, values and queries change no other request."""
    fa = cuda_lib
    c = paged_case([(1, 200), (5, 90), (1, 40), (9, 300)], 4, 2, d, 16, dtype, seed=12, stale=False)
    t = to_cuda(c)
    args = lambda: (t["q"], t["k_cache"], t["v_cache"], t["block_table"], t["kv_len"], t["cu_q"])
    want, wl = fa.paged_fwd(*args(), max_q=max_q)
    bad = t["block_table"][1][:6].long()
    t["k_cache"][bad[1]] = float("nan")
    t["k_cache"][bad[3]] = float("inf")
    t["v_cache"][bad[2]] = float("nan")
    t["q"][1:6, 0] = float("nan")
    got, gl = fa.paged_fwd(*args(), max_q=max_q)
    for rows in (slice(0, 1), slice(6, 16)):
        assert torch.equal(got[rows], want[rows]) and torch.equal(gl[rows], wl[rows])
    assert torch.isnan(got[1:6]).any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_captured_step_serves(cuda_lib, dtype):
    """Plan, append and attention captured as one graph of fixed capacity, replayed while lengths,
    tokens, cursor and tables live on the device, against the same calls one by one."""
    fa = cuda_lib
    H, H_kv, d, page, cap = 4, 2, 64, 16, 48
    dt = TORCH[dtype]
    g = torch.Generator().manual_seed(3)
    fi, m = fa.rope_frequencies(d)
    steps = [[40, 0, 3], [1, 1, 1], [1, 30, 1], [0, 1, 17], [1, 1, 1]]
    xs = [torch.randn((cap, (H + 2 * H_kv) * d), generator=g).to(dt).cuda() for _ in steps]
    free = torch.randperm(40, generator=g).to(torch.int32).cuda()

    def fresh():
        s = dict(kc=torch.zeros((40, H_kv, page, d), dtype=dt, device="cuda"), ctx=torch.zeros(3, dtype=torch.int32, device="cuda"),
                 new=torch.zeros(3, dtype=torch.int32, device="cuda"), cursor=torch.zeros(1, dtype=torch.int32, device="cuda"),
                 table=torch.full((3, 8), -1, dtype=torch.int32, device="cuda"), x=torch.zeros_like(xs[0]),
                 plan=fa.PagedPlan.empty(3, cap), o=torch.zeros((cap, H, d), dtype=dt, device="cuda"),
                 lse=torch.zeros((cap, H), device="cuda"), q=torch.empty((cap, H, d), dtype=dt, device="cuda"),
                 ws=torch.empty(fa.paged_workspace_size(cap, 3, H, H_kv, d), dtype=torch.uint8, device="cuda"))
        s["vc"] = torch.zeros_like(s["kc"])
        return s

    def step(s):
        p = fa.paged_plan(s["ctx"], s["new"], free, s["table"], page, cap, cursor=s["cursor"], out=s["plan"])
        q, k, v = (t.view(cap, -1, d) for t in s["x"].split([H * d, H_kv * d, H_kv * d], 1))
        fa.paged_append(k, v, s["kc"], s["vc"], p.slots, positions=p.positions, inv_freq=fi, q=q, q_out=s["q"])
        fa.paged_fwd(s["q"], s["kc"], s["vc"], s["table"], p.kv_len, p.cu_q, max_q=cap, out=s["o"], lse=s["lse"],
                     workspace=s["ws"])
        s["ctx"].copy_(p.kv_len)
        s["cursor"].copy_(p.counts[3:4])

    a, b = fresh(), fresh()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):  # every kernel once before the capture, and not on the default stream
        step(b)
        b["ctx"].zero_()
        b["cursor"].zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(b)
    for n, x in zip(steps, xs):
        for s in (a, b):
            s["new"].copy_(torch.tensor(n, dtype=torch.int32))
            s["x"].copy_(x)
            s["o"].zero_()
            s["lse"].zero_()
        step(a)
        graph.replay()
        torch.cuda.synchronize()
        for k in ("o", "lse", "kc", "vc", "table", "ctx", "cursor"):
            assert torch.equal(a[k], b[k]), k
    assert a["ctx"].cpu().tolist() == [43, 33, 23] and fa.device_status() == 0


def test_empty_batch_and_refusals(cuda_lib):
    fa = cuda_lib
    c = paged_case([(2, 20)], 4, 2, 64, 16, seed=1, stale=False)
    t = to_cuda(c)
    call = lambda **kw: fa.paged_fwd(**{**dict(q=t["q"], k_cache=t["k_cache"], v_cache=t["v_cache"],
                                               block_table=t["block_table"], kv_len=t["kv_len"],
                                               cu_q=t["cu_q"]), **kw})
    call()
    o, lse = call(q=t["q"][:0])
    assert o.shape == (0, 4, 64) and lse.shape == (0, 4)
    three = torch.zeros((4, 3, 64), dtype=torch.bfloat16, device="cuda")
    for kw in (dict(q=t["q"].float()), dict(q=three), dict(v_cache=t["v_cache"][:-1]),
               dict(k_cache=t["k_cache"][:, :, :8], v_cache=t["v_cache"][:, :, :8]),
               dict(k_cache=t["k_cache"].transpose(1, 2)), dict(kv_len=t["kv_len"].long()),
               dict(cu_q=t["cu_q"][:1]), dict(block_table=t["block_table"].float()),
               dict(block_table=t["block_table"].cpu()), dict(scale=0.0), dict(scale=float("nan")), dict(scale=1e300), dict(max_q=1 << 40), dict(scale="x"),
               dict(out=torch.empty((3, 4, 64), dtype=torch.bfloat16, device="cuda")),
               dict(lse=torch.empty((4, 4), dtype=torch.bfloat16, device="cuda")),
               dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(fa.FaError):
            call(**kw)
    k = t["k_cache"]
    with pytest.raises(fa.FaError):  # a head dimension the bf16 kernels lack
        fa.paged_fwd(t["q"][..., :32].contiguous(), k[..., :32].contiguous(), k[..., :32].contiguous(),
                     t["block_table"], t["kv_len"], t["cu_q"])
    x = torch.zeros((3, 2, 64), dtype=torch.bfloat16, device="cuda")
    s = torch.zeros(3, dtype=torch.int64, device="cuda")
    fi, _ = fa.rope_frequencies(64)
    for kw in (dict(slots=s.int()), dict(slots=s[:2]), dict(v=x[:, :1]), dict(inv_freq=fi),
               dict(q=x[:2]), dict(q_out=x), dict(k=x.float(), v=x.float()), dict(k=x.cpu(), v=x.cpu())):
        with pytest.raises(fa.FaError):
            fa.paged_append(**{**dict(k=x, v=x, k_cache=k, v_cache=k.clone(), slots=s), **kw})
    i = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    for a in ((i(1), i(1, 2), i(3), i(1).view(1, 1), 16, 4), (i(1), i(1), i(3), i(1), 16, 4),
              (i(1), i(1), i(3), i(1).view(1, 1), 24, 4), (i(1), i(1), i(3), i(1).view(1, 1), 16, 0),
              (i(1), i(1).long(), i(3), i(1).view(1, 1), 16, 4)):
        with pytest.raises(fa.FaError):
            fa.paged_plan(*a)
    assert fa.paged_workspace_size(0, 1, 4, 2, 64) == 0 and fa.paged_workspace_size(4, 1, 4, 3, 64) == 0


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("f32", 64)])
def test_served_steps_match_dense_attention(cuda_lib, dtype, d):
    """Two sequences prefilled in chunks and then decoded -- plan, append with rotation, attention,
    step after step -- give what rope and the causal fwd give on the whole sequences.  Both sides
    round rotated keys and O once to the type and P (bf16) once, so they differ by at most the sum
    of two such bounds: 2 (2^-8 A|V| + 2^-8 |O|) in bf16, and 1e-5 in fp32 as elsewhere."""
    fa = cuda_lib
    H, H_kv, page, N = 4, 2, 16, 150
    g = torch.Generator().manual_seed(11)
    dt = TORCH[dtype]
    seq = [torch.randn((n, (H + 2 * H_kv) * d), generator=g).to(dt).cuda() for n in (N, 67)]
    fi, m = fa.rope_frequencies(d, scaling="ntk", factor=2.0)
    cut = lambda t: (t[:, :H * d].view(-1, H, d), t[:, H * d:(H + H_kv) * d].view(-1, H_kv, d),
                     t[:, (H + H_kv) * d:].view(-1, H_kv, d))
    kc = torch.full((20, H_kv, page, d), float("nan"), dtype=dt, device="cuda")
    vc = kc.clone()
    table = torch.full((2, 10), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(20, generator=g).to(torch.int32).cuda()
    cursor = torch.zeros(1, dtype=torch.int32, device="cuda")
    ctx = torch.zeros(2, dtype=torch.int32, device="cuda")
    done = [0, 0]
    got = [[], []]
    plan = None
    for step in ([70, 1], [1, 40], [60, 0], [1, 1], [1, 25], [17, 0]):
        new = torch.tensor(step, dtype=torch.int32, device="cuda")
        plan = fa.paged_plan(ctx, new, free, table, page, 80, cursor=cursor, out=plan)
        x = torch.zeros((80, (H + 2 * H_kv) * d), dtype=dt, device="cuda")
        at = 0
        for i, n in enumerate(step):
            x[at:at + n] = seq[i][done[i]:done[i] + n]
            done[i] += n
            at += n
        q, k, v = cut(x)
        q = fa.paged_append(k, v, kc, vc, plan.slots, positions=plan.positions, inv_freq=fi, magnitude=m, q=q)
        o, lse = fa.paged_fwd(q, kc, vc, table, plan.kv_len, plan.cu_q, max_q=max(step))
        at = 0
        for i, n in enumerate(step):
            got[i].append((o[at:at + n].clone(), lse[at:at + n].clone()))
            at += n
        ctx.copy_(plan.kv_len)
        cursor.copy_(plan.counts[3:4])
    assert done == [N, 67] and int(plan.counts[2]) == 0
    for i in range(2):
        q, k, v = (t.transpose(0, 1)[None] for t in cut(seq[i]))
        q, k = fa.rope(q, fi, magnitude=m), fa.rope(k, fi, magnitude=m)
        o, lse = fa.fwd(q, k, v.contiguous(), causal=True)
        av, _ = fa.fwd(q.float(), k.float(), v.float().abs().contiguous(), causal=True)  # A|V|
        mine_o = torch.cat([x for x, _ in got[i]]).transpose(0, 1)[None]
        mine_l = torch.cat([x for _, x in got[i]]).t()[None]
        tol = 2 * 2.0 ** -8 * (av + o.float().abs()) if dtype == "bf16" else torch.full_like(av, 1e-5)
        assert torch.all((mine_o.float() - o.float()).abs() <= tol + 1e-6)
        assert (mine_l - lse).abs().max() <= 1e-3 if dtype == "bf16" else 1e-5


# ------------- 17 to 32 rows of a K/V head: more than the decoding kernel's, few for the chunk kernel
FEW = [(1, 1), (2, 2), (3, 64), (5, 65), (8, 700), (7, 3), (4, 0), (0, 9), (1, 2049), (8, 128), (6, 6)]
BETWEEN = [
    # lens, H, H_kv, d, page, causal, max_q
    (FEW, 8, 2, 128, 16, True, 8),                      # 32 rows
    (FEW, 8, 2, 64, 32, False, 8),
    (FEW, 6, 2, 128, 64, True, 8),                      # three heads a group, 24 rows
    (FEW, 10, 2, 64, 16, True, 4),                      # five: 20 rows
    (DECODE, 32, 1, 128, 16, True, 1),                  # 32 heads a group
    (DECODE, 40, 2, 64, 64, True, 1),                   # 20
    (DECODE, 17, 1, 128, 128, False, 1),                # 17
    (RAGGED, 4, 1, 64, 16, True, 5),                    # longer than the hint
    (RAGGED, 3, 1, 128, 32, True, 6),
    ([(8, 20000)] * 6, 8, 2, 128, 64, True, 8),         # the ring goes round
    ([(6, 30000), (1, 70)] * 5, 8, 2, 64, 16, True, 6),
    ([(2, 9000), (1, 1)] * 9, 36, 2, 128, 32, True, 1),
    ([(5, 300), (1, 7)] * 300, 4, 1, 64, 16, True, 5),  # many small requests
    ([(1, 3), (7, 7), (0, 7)] * 3000, 3, 1, 128, 16, True, 7),
]


@pytest.mark.parametrize("case", range(len(BETWEEN)))
def test_paged_attention_between_the_kernels(cuda_lib, case):
    lens, H, H_kv, d, page, causal, max_q = BETWEEN[case]
    assert 16 < max_q * (H // H_kv) <= 32
    c = paged_case(lens, H, H_kv, d, page, "bf16", seed=100 + case)
    _, o, lse, o0, l0, scale = _run(cuda_lib, c, causal, max_q)
    check_paged(c, o, lse, causal, scale, o_before=o0, lse_before=l0)


@pytest.mark.parametrize("d,page", [(64, 16), (128, 64)])
def test_between_the_kernels_as_the_others(cuda_lib, d, page):
    """Two heads a group and a hint of 12 new tokens: 24 rows."""
    test_bad_pages_are_masked(cuda_lib, "bf16", d, page, 12)
    test_paged_layouts_and_large_scores(cuda_lib, "bf16", d, 12)
    test_outputs_at_any_allowed_alignment(cuda_lib, "bf16", d, 12)
    test_a_bad_request_stays_alone(cuda_lib, "bf16", d, 12)
    test_offsets_beyond_32_bits(cuda_lib, "bf16", d, 12)
    test_lengths_out_of_range_are_clamped(cuda_lib, 12)
