"""Paged attention of values that are not finite: NaN in a row's scores stays in that row's O and lse,
however the batch is divided over the GPU, and a row that sees no key is empty whatever V holds."""
import numpy as np
import pytest
import torch

import synthetic as syn
from paged_util import TORCH, attend_ref, f64, paged_case, to_cuda

pytestmark = pytest.mark.gpu

KERNELS = [("bf16", 64, 1), ("bf16", 64, 500), ("bf16", 128, 1), ("bf16", 128, 500),
           ("f32", 33, 1), ("f32", 33, 500), ("f32", 64, 1), ("f32", 128, 1), ("f32", 128, 500)]  # dtype, d, max_q


def _call(fa, t, max_q):
    o = torch.full(t["q"].shape, 3.5, dtype=t["q"].dtype, device="cuda")
    lse = torch.full(t["q"].shape[:2], 7.25, device="cuda")
    fa.paged_fwd(t["q"], t["k_cache"], t["v_cache"], t["block_table"], t["kv_len"], t["cu_q"],
                 scale=syn.scale_for(t["q"].shape[2]), max_q=max_q, out=o, lse=lse)
    torch.cuda.synchronize()
    assert fa.device_status() == 0
    return o.cpu(), lse.cpu()


def _check(c, t, o, lse):
    """Every row of the causal call against the 64-bit form: a visible score that is NaN makes the
    row NaN, a row without keys is 0 and -inf, the others are within attend_ref's bound."""
    G, page = c["H"] // c["H_kv"], c["page"]
    at = 0
    kc, vc, q = f64(t["k_cache"]), f64(t["v_cache"]), f64(t["q"])
    for b, (nq, nk) in enumerate(c["lens"]):
        pos = np.arange(nk)
        ids = t["block_table"][b].cpu().numpy()[pos // page]
        keep = pos[None, :] <= (nk - nq + np.arange(nq))[:, None]
        for h in range(c["H"]):
            k, v = kc[ids, h // G, pos % page], vc[ids, h // G, pos % page]
            qh, go, gl = q[at:at + nq, h], f64(o[at:at + nq, h]), f64(lse[at:at + nq, h])
            bad_q, bad_k = np.isnan(qh).any(1), np.isnan(k).any(1)
            nan = (keep & (bad_q[:, None] | bad_k[None, :])).any(1)
            empty = ~keep.any(1)
            where = f"request {b} (nq {nq}, nk {nk}) head {h}"
            assert np.isnan(go[nan]).all(), f"{where}: O of {(~np.isnan(go[nan]).all(1)).sum()} rows of NaN scores"
            assert np.isnan(gl[nan]).all(), f"{where}: lse of rows of NaN scores: {gl[nan][~np.isnan(gl[nan])][:4]}"
            assert np.all(go[empty] == 0.0) and np.all(np.isneginf(gl[empty])), f"{where}: rows without keys"
            live = ~nan & ~empty
            if not live.any() or not np.isfinite(v).all():
                continue
            clean_q, clean_k = np.where(np.isnan(qh), 0.0, qh), np.where(np.isnan(k), 0.0, k)
            ro, rl, bo, bl = attend_ref(clean_q, clean_k, v, keep, syn.scale_for(c["d"]), c["dtype"])
            assert np.all(np.abs(go - ro)[live] <= bo[live]), f"{where}: O of finite rows"
            assert np.all(np.abs(gl[live] - rl[live]) <= bl[live]), f"{where}: lse of finite rows"
        at += nq


# the request in question alone (cut between many CTAs) and among others (mostly whole)
BATCHES = [[(4, 6000)], [(4, 6000)] + [(1, 40)] * 5, [(4, 60)] + [(2, 70)] * 400]


@pytest.mark.parametrize("batch", range(len(BATCHES)))
@pytest.mark.parametrize("dtype,d,max_q", KERNELS)
def test_nan_queries(cuda_lib, dtype, d, max_q, batch):
    """Query rows of NaN: their O and lse are NaN, the rows beside them are not touched."""
    c = paged_case(BATCHES[batch], 4, 2, d, 16, dtype, seed=31 + batch)
    t = to_cuda(c)
    t["q"][1, 0] = float("nan")
    t["q"][2, 3] = float("nan")
    t["q"][3, :, 1] = float("nan")  # a single column is enough
    _check(c, t, *_call(cuda_lib, t, max_q))


# ranges that end inside a key tile, and (the last four) ranges of whole tiles: no part is mixed
@pytest.mark.parametrize("first,last", [(0, 3000), (0, 1), (5998, 5999), (256, 1500), (0, 2944), (2944, 6000),
                                        (1280, 1408), (0, 5888)])
@pytest.mark.parametrize("dtype,d,max_q", KERNELS)
def test_nan_keys(cuda_lib, dtype, d, max_q, first, last):
    """Keys [first, last) of NaN: whole parts of a cut item have no other score, the others are finite."""
    c = paged_case([(4, 6000), (1, 3), (2, 130)], 4, 2, d, 16, dtype, seed=41)
    t = to_cuda(c)
    pos = torch.arange(first, last, device="cuda")
    t["k_cache"][t["block_table"][0, pos // 16].long(), 1, pos % 16] = float("nan")  # one of two K/V heads
    _check(c, t, *_call(cuda_lib, t, max_q))


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("dtype,d,max_q", KERNELS)
def test_rows_without_keys_beside_bad_values(cuda_lib, dtype, d, max_q, value):
    """More new tokens than cached keys: the first rows see no key and are empty, although the values
    that later rows of their tile see are not finite.  So is a part of which a row sees no key."""
    c = paged_case([(6, 3), (70, 40), (300, 200), (9, 2)], 4, 2, d, 16, dtype, seed=51)
    t = to_cuda(c)
    t["v_cache"].fill_(value)
    o, lse = _call(cuda_lib, t, max_q)
    _check(c, t, o, lse)
    at = 0
    for nq, nk in c["lens"]:
        assert torch.isfinite(lse[at + nq - nk:at + nq]).all() and not torch.isfinite(o[at + nq - 1]).any()
        at += nq


@pytest.mark.parametrize("dtype,d,max_q", KERNELS)
def test_nan_does_not_depend_on_the_division(cuda_lib, dtype, d, max_q):
    """The same request alone and among 300 others: NaN in the same places."""
    found = []
    for others in (0, 300):
        c = paged_case([(3, 2500)] + [(1, 900)] * others, 4, 2, d, 16, dtype, seed=61, stale=False)
        t = to_cuda(c)
        t["q"][1, 2] = float("nan")
        pos = torch.arange(640, 1920, device="cuda")
        t["k_cache"][t["block_table"][0, pos // 16].long(), 0, pos % 16] = float("nan")
        o, lse = _call(cuda_lib, t, max_q)
        found.append((torch.isnan(o[:3]), torch.isnan(lse[:3])))
        assert torch.isfinite(o[3:3 + others]).all() and torch.isfinite(lse[3:3 + others]).all()
    assert torch.equal(found[0][0], found[1][0]) and torch.equal(found[0][1], found[1][1])
    assert found[0][1][:, :2].all() and found[0][1][1, 2] and not found[0][1][0, 2:].any()
