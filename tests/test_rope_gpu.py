"""Rotary positions (fa_rope) against a 64-bit rotation: layouts, types, strides, far positions,
the gradient as the transposed map and against differences."""
import numpy as np
import pytest
import torch

from paged_util import TORCH, f64, rope_bound, rope_ref

pytestmark = pytest.mark.gpu


def _freqs(fa, rot, **kw):
    f, m = fa.rope_frequencies(rot, **kw)
    return f, m, f.cpu().numpy()


def _check(y, x, fr, pos, il, mag, dtype, sign=1.0, axis_tokens=-2):
    ref = rope_ref(f64(x), fr, pos, il, mag, sign)
    err = np.abs(f64(y) - ref)
    rot = 2 * len(fr)
    bound = rope_bound(f64(x), len(fr), il, mag, dtype)
    assert np.all(err[..., :rot] <= bound[..., :rot] + 1e-30), (err - bound)[..., :rot].max()
    assert torch.equal(y[..., rot:].cpu(), x[..., rot:].cpu()), "pass-through columns changed"


CASES = [
    # B, H, N, d, rot, dtype, interleaved, backward
    (1, 1, 1, 64, 64, "bf16", False, False),
    (2, 3, 129, 64, 64, "bf16", True, False),
    (2, 12, 257, 128, 128, "bf16", False, True),
    (3, 5, 77, 80, 48, "f32", False, False),      # part of the head
    (1, 4, 33, 80, 40, "bf16", True, True),       # rot/2 not a multiple of 8: the element path
    (2, 2, 50, 7, 4, "f32", False, False),        # odd head dimension
    (1, 3, 31, 7, 6, "f32", True, True),
    (70, 1, 3, 32, 2, "bf16", False, False),      # a single pair
    (1, 33, 5, 256, 256, "f32", True, False),
    (1, 2, 3, 1024, 1024, "bf16", False, False),  # the widest head
    (1, 40, 2500, 64, 32, "bf16", False, False),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_rope_matches_the_rotation(cuda_lib, case):
    B, H, N, d, rot, dtype, il, back = CASES[case]
    fa = cuda_lib
    fi, m, fr = _freqs(fa, rot)
    x = torch.randn((B, H, N, d), generator=torch.Generator().manual_seed(case)).to(TORCH[dtype]).cuda()
    call = fa.rope_bwd if back else fa.rope
    y = call(x, fi, interleaved=il)
    _check(y, x, fr, np.arange(N), il, m, dtype, -1.0 if back else 1.0)
    z = x.clone()
    assert call(z, fi, interleaved=il, out=z) is z  # in place
    assert torch.equal(z, y)


@pytest.mark.parametrize("kind", ["linear", "ntk", "by_parts"])
def test_rope_scaled_far_positions(cuda_lib, kind):
    """Positions up to 2^31 - 1 and per-batch positions; the frequencies are the method's own."""
    fa = cuda_lib
    rot, factor, L = 64, 8.0, 4096
    fi, m, fr = _freqs(fa, rot, scaling=kind, factor=factor, original_length=L)
    base = 10000.0 ** (-np.arange(0, rot, 2) / rot)
    if kind == "linear":
        want = base / factor
    elif kind == "ntk":
        want = (10000.0 * factor ** (rot / (rot - 2))) ** (-np.arange(0, rot, 2) / rot)
    else:
        g = np.clip((L * base / (2 * np.pi) - 1.0) / 31.0, 0, 1)
        want = base * g + base / factor * (1 - g)
        assert m == pytest.approx(0.1 * np.log(factor) + 1.0, rel=1e-15)
    np.testing.assert_allclose(fr, want, rtol=1e-13)
    pos = torch.tensor([[0, 1, 2 ** 31 - 1, 1000003], [5, 123456789, 7, 2 ** 30]], dtype=torch.int32)
    x = torch.randn((2, 3, 4, rot), generator=torch.Generator().manual_seed(9))
    y = fa.rope(x.cuda(), fi, positions=pos.cuda(), magnitude=m)
    for b in range(2):
        # the angle itself is formed in fp64: position times frequency is off by 2^-53 relative,
        # 2^31 radians 2^-53 is below 3e-7, which the reference's own cos shares
        ref = rope_ref(f64(x[b]), fr, pos[b].numpy(), False, m)
        err = np.abs(f64(y[b]) - ref)
        assert np.all(err <= rope_bound(f64(x[b]), rot // 2, False, m, "f32") + 2 * 3e-7 * np.abs(f64(x[b])).max())


def test_rope_strides_and_packed(cuda_lib):
    """A slice of a fused projection (packed), [B, N, H, d] memory, broadcast input, unaligned rows."""
    fa = cuda_lib
    fi, m, fr = _freqs(fa, 64)
    g = torch.Generator().manual_seed(3)
    fused = torch.randn((37, 9 * 64), generator=g).to(torch.bfloat16).cuda()
    x = fused[:, 64:6 * 64].view(37, 5, 64)
    pos = torch.randint(0, 9999, (37,), generator=g, dtype=torch.int32)
    y = fa.rope(x, fi, positions=pos.cuda())
    _check(y.transpose(0, 1), x.transpose(0, 1), fr, pos.numpy(), False, m, "bf16")
    before = fused.clone()
    fa.rope(x, fi, positions=pos.cuda(), out=x)      # in place inside the projection
    assert torch.equal(x, y)
    assert torch.equal(fused[:, :64], before[:, :64]) and torch.equal(fused[:, 384:], before[:, 384:])
    xt = torch.randn((2, 21, 3, 64), generator=g).to(torch.bfloat16).cuda().transpose(1, 2)
    yt = fa.rope(xt, fi)
    assert torch.equal(yt, fa.rope(xt.contiguous(), fi))
    one = torch.randn((2, 1, 21, 64), generator=g).cuda().expand(2, 4, 21, 64)
    assert torch.equal(fa.rope(one, fi), fa.rope(one.contiguous(), fi))
    flat = torch.randn(2 * 3 * 21 * 65 + 1, generator=g).cuda()
    odd = flat[1:].view(2, 3, 21, 65)[..., :64]      # rows 65 elements apart, 4-byte aligned only
    assert torch.equal(fa.rope(odd, fi, interleaved=True), fa.rope(odd.contiguous(), fi, interleaved=True))
    assert fa.rope(torch.empty((0, 3, 64), device="cuda"), fi).shape == (0, 3, 64)


def test_rope_gradient_against_differences(cuda_lib):
    """<g, rope(x + h e) - rope(x - h e)> / 2h against rope_bwd(g); the map is linear, so the
    difference has no truncation error: what is left is fp32 rounding, 2^-22 of values of size
    h-scaled 1 over 2h = 2 per output, two outputs a coordinate."""
    fa = cuda_lib
    fi, m, _ = _freqs(fa, 6)
    x = torch.randn((1, 2, 5, 8), generator=torch.Generator().manual_seed(1)).cuda()
    gy = torch.randn((1, 2, 5, 8), generator=torch.Generator().manual_seed(2)).cuda()
    for il in (False, True):
        gx = fa.rope_bwd(gy, fi, interleaved=il, magnitude=1.25)
        for idx in [(0, 0, 0, 0), (0, 1, 4, 5), (0, 0, 3, 2), (0, 1, 2, 7)]:
            e = torch.zeros_like(x)
            e[idx] = 1.0
            d = (fa.rope(x + e, fi, interleaved=il, magnitude=1.25).double()
                 - fa.rope(x - e, fi, interleaved=il, magnitude=1.25).double()) / 2
            if idx[-1] >= 6:
                d = (x + e).double() / 2 - (x - e).double() / 2
            size = float(x.abs().max()) + 1
            got, want = float(gx[idx]), float((gy.double() * d).sum())
            assert abs(got - want) <= 8 * 1.25 * size * float(gy.abs().max()) * 2.0 ** -21


def test_rope_special_values_stay_in_their_pair(cuda_lib):
    fa = cuda_lib
    fi, _, _ = _freqs(fa, 64)
    x = torch.randn((1, 1, 4, 64), generator=torch.Generator().manual_seed(4)).cuda()
    clean = fa.rope(x, fi)
    x[0, 0, 2, 5] = float("nan")
    y = fa.rope(x, fi)
    bad = torch.isnan(y)
    assert bad.sum() == 2 and bad[0, 0, 2, 5] and bad[0, 0, 2, 37]
    assert torch.equal(y[~bad], clean[~bad])


def test_rope_refusals(cuda_lib):
    fa = cuda_lib
    fi, _, _ = _freqs(fa, 64)
    x = torch.zeros((1, 2, 4, 64), device="cuda")
    for bad in (lambda: fa.rope(x[..., :32].contiguous(), fi),          # rotary_dim > d
                lambda: fa.rope(x.double(), fi),
                lambda: fa.rope(x, fi.float()),
                lambda: fa.rope(x, fi, positions=torch.zeros(3, dtype=torch.int32, device="cuda")),
                lambda: fa.rope(x, fi, positions=torch.zeros(4, dtype=torch.int64, device="cuda")),
                lambda: fa.rope(x, fi, out=torch.zeros((1, 1, 4, 64), device="cuda").expand(1, 2, 4, 64)),
                lambda: fa.rope(x.transpose(2, 3), fi),
                lambda: fa.rope(x, fi, magnitude=float("inf")),
                lambda: fa.rope(x[0, 0], fi),
                lambda: fa.rope(x, fi.cpu()),
                lambda: fa.rope_frequencies(7), lambda: fa.rope_frequencies(8, scaling="other"),
                lambda: fa.rope_frequencies(8, scaling="by_parts", factor=2.0),
                lambda: fa.rope_frequencies(8, factor=0.5)):
        with pytest.raises(fa.FaError):
            bad()
