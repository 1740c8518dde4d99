"""Paged-cache and rotary paths that only unusual sizes reach: groups of heads larger than a row
tile, batches beyond a grid's second dimension, offsets that are cut to the batch, queries in any
order of strides, and the served chain's log-sum-exp in fp32."""
import numpy as np
import pytest
import torch

import synthetic as syn
from paged_util import TORCH, attend_ref, check_paged, f64, paged_case, rope_bound, rope_ref, to_cuda

pytestmark = pytest.mark.gpu


def _run(fa, c, causal=True, max_q=None):
    t = to_cuda(c)
    o = torch.full(c["q"].shape, 3.5, dtype=TORCH[c["dtype"]], device="cuda")
    lse = torch.full(c["q"].shape[:2], 7.25, device="cuda")
    o0, l0 = o.clone(), lse.clone()
    fa.paged_fwd(t["q"], t["k_cache"], t["v_cache"], t["block_table"], t["kv_len"], t["cu_q"],
                 scale=syn.scale_for(c["d"]), causal=causal, max_q=max_q, out=o, lse=lse)
    torch.cuda.synchronize()
    assert fa.device_status() == 0
    check_paged(c, o, lse, causal, syn.scale_for(c["d"]), o_before=o0, lse_before=l0)


@pytest.mark.parametrize("dtype,d,H,H_kv", [("bf16", 64, 257, 1), ("bf16", 128, 300, 1), ("bf16", 64, 600, 2),
                                            ("bf16", 128, 514, 2), ("f32", 64, 71, 1), ("f32", 40, 130, 2),
                                            ("f32", 128, 65, 1)])
@pytest.mark.parametrize("causal", [True, False])
def test_groups_larger_than_a_row_tile(cuda_lib, dtype, d, H, H_kv, causal):
    """The chunk kernels deal such a group out over tiles, the last of which is short and overhangs
    into the next group or past the last head.  One request's items are cut and joined."""
    c = paged_case([(3, 70), (1, 900), (2, 0), (2, 5000), (5, 4)], H, H_kv, d, 16, dtype, seed=H + d)
    _run(cuda_lib, c, causal, 5)


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("f32", 24)])
@pytest.mark.parametrize("max_q", [1, 500])
@pytest.mark.parametrize("order", ["heads first", "padded tokens", "heads first, padded"])
def test_queries_in_any_order_of_strides(cuda_lib, dtype, d, max_q, order):
    """[H][T][d] memory seen as [T][H][d], rows further apart than d, and both."""
    c = paged_case([(1, 300), (40, 90), (3, 3)], 6, 2, d, 16, dtype, seed=d)
    T, H = c["T"], c["H"]
    q = c["q"]
    if order == "padded tokens":
        pool = torch.full((T, H * d + 40), float("nan"), dtype=q.dtype)
        view = pool[:, :H * d].view(T, H, d)
    else:
        pool = torch.full((H, T + (3 if "padded" in order else 0), d + (8 if "padded" in order else 0)),
                          float("nan"), dtype=q.dtype)
        view = pool[:, :T, :d].transpose(0, 1)
    view.copy_(q)
    c["q"] = view
    t = to_cuda(c)
    base = pool.cuda()
    t["q"] = torch.as_strided(base, view.shape, view.stride(), view.storage_offset())
    o = torch.full((T, H, d), 3.5, dtype=q.dtype, device="cuda")
    lse = torch.full((T, H), 7.25, device="cuda")
    o0, l0 = o.clone(), lse.clone()
    cuda_lib.paged_fwd(t["q"], t["k_cache"], t["v_cache"], t["block_table"], t["kv_len"], t["cu_q"],
                       scale=syn.scale_for(d), max_q=max_q, out=o, lse=lse)
    check_paged(c, o, lse, True, syn.scale_for(d), o_before=o0, lse_before=l0)


@pytest.mark.parametrize("B", [65535, 65536, 65537, 70000])
@pytest.mark.parametrize("per_batch", [False, True])
def test_rope_batches_beyond_65535(cuda_lib, B, per_batch):
    """Such a batch is folded into two grid dimensions: each element has its positions, in place too."""
    fa = cuda_lib
    fi, m = fa.rope_frequencies(4)
    fr = fi.cpu().numpy()
    g = torch.Generator().manual_seed(B)
    x = torch.randn((B, 1, 2, 8), generator=g)
    pos = torch.randint(0, 9999, (B, 2), generator=g, dtype=torch.int32) if per_batch else \
        torch.tensor([5, 70], dtype=torch.int32)
    y = fa.rope(x.cuda(), fi, positions=pos.cuda())
    flat = pos.reshape(-1).numpy() if per_batch else np.tile(pos.numpy(), B)
    ref = rope_ref(f64(x).reshape(-1, 8), fr, flat, False, m)
    assert np.all(np.abs(f64(y).reshape(-1, 8) - ref) <= rope_bound(f64(x).reshape(-1, 8), 2, False, m, "f32") + 1e-30)
    z = x.cuda()
    fa.rope(z, fi, positions=pos.cuda(), out=z)
    assert torch.equal(z, y)


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("f32", 48)])
@pytest.mark.parametrize("max_q", [1, 12, 500])
def test_offsets_cut_to_the_batch(cuda_lib, dtype, d, max_q):
    """cu_q below 0 and past T is cut; a request whose end lies before its start has no row; the rows of
    no request stay as they were."""
    fa = cuda_lib
    c = paged_case([(3, 64), (2, 48), (4, 33)], 2, 1, d, 16, dtype, seed=6, pad=0)
    t = to_cuda(c)

    def call(cu):
        o = torch.full(c["q"].shape, 3.5, dtype=TORCH[dtype], device="cuda")
        lse = torch.full(c["q"].shape[:2], 7.25, device="cuda")
        fa.paged_fwd(t["q"], t["k_cache"], t["v_cache"], t["block_table"], t["kv_len"],
                     torch.tensor(cu, dtype=torch.int32, device="cuda"), scale=syn.scale_for(d), max_q=max_q,
                     out=o, lse=lse)
        torch.cuda.synchronize()
        assert fa.device_status() == 0
        return o.cpu(), lse.cpu()
    for cut, sound in (([-4, 3, 3, 999], [0, 3, 3, 9]), ([-2 ** 31, 3, 5, 2 ** 31 - 1], [0, 3, 5, 9]),
                       ([-9, -1, 4, 20], [0, 0, 4, 9])):
        (o, lse), (so, sl) = call(cut), call(sound)
        assert torch.equal(o, so) and torch.equal(lse, sl)
        lens = [(sound[b + 1] - sound[b], nk) for b, (_, nk) in enumerate(c["lens"])]
        check_paged({**c, "lens": lens}, o, lse, True, syn.scale_for(d))
    o, lse = call([0, 3, 1, 1])  # the second request would own 3 .. 1: no row
    check_paged({**c, "lens": [(3, 64)]}, o, lse, True, syn.scale_for(d),
                o_before=torch.full_like(o, 3.5), lse_before=torch.full_like(lse, 7.25))
    o, lse = call([20, 30, 40, 999])  # every request behind the batch
    assert torch.all(o == 3.5) and torch.all(lse == 7.25)


@pytest.mark.parametrize("d", [64, 128])
def test_served_lse_in_fp32(cuda_lib, d):
    """Plan, append with rotation and attention in steps, against the causal fwd on the whole sequence.
    Both compute the lse in fp32 from the same rotated rows, so they differ by at most the sum of two
    bounds of attend_ref."""
    fa = cuda_lib
    H, H_kv, page, N = 4, 2, 16, 150
    g = torch.Generator().manual_seed(11)
    seq = torch.randn((N, (H + 2 * H_kv) * d), generator=g).cuda()
    cut = lambda x: (x[:, :H * d].view(-1, H, d), x[:, H * d:(H + H_kv) * d].view(-1, H_kv, d),
                     x[:, (H + H_kv) * d:].view(-1, H_kv, d))
    fi, m = fa.rope_frequencies(d, scaling="ntk", factor=2.0)
    kc = torch.full((12, H_kv, page, d), float("nan"), device="cuda")
    vc = kc.clone()
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    table = torch.full((1, 10), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(12, generator=g).to(torch.int32).cuda()
    cursor, ctx, at, got = i32(0), i32(0), 0, []
    for n in (70, 1, 60, 1, 1, 17):
        plan = fa.paged_plan(ctx, i32(n), free, table, page, n, cursor=cursor)
        q, k, v = cut(seq[at:at + n])
        q = fa.paged_append(k, v, kc, vc, plan.slots, positions=plan.positions, inv_freq=fi, magnitude=m, q=q)
        got.append(fa.paged_fwd(q, kc, vc, table, plan.kv_len, plan.cu_q, max_q=n)[1])
        at += n
        ctx.copy_(plan.kv_len)
        cursor.copy_(plan.counts[3:4])
    assert at == N
    q, k, v = (x.transpose(0, 1)[None] for x in cut(seq))
    q, k = fa.rope(q, fi, magnitude=m), fa.rope(k, fi, magnitude=m)
    lse = f64(fa.fwd(q, k, v.contiguous(), causal=True)[1])[0]
    mine = f64(torch.cat(got)).T
    keep = np.tril(np.ones((N, N), bool))
    for h in range(H):
        _, rl, _, bl = attend_ref(f64(q[0, h]), f64(k[0, h // 2]), f64(v[0, h // 2]), keep, syn.scale_for(d), "f32")
        assert np.all(np.abs(mine[h] - rl) <= bl) and np.all(np.abs(mine[h] - lse[h]) <= 2 * bl)
