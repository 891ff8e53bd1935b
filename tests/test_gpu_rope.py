"""Rotary positions on the GPU against a 64-bit restatement.

Bound: |error| <= 2^-8 |y| (one rounding to bf16) + 2^-19 m (|a| + |b|).  The second term covers
the fp32 arithmetic: the angle's 24-bit conversion moves it by at most 2^-24 half turns = 1.9e-7
rad, the frequency's fp64 rounding at 2^31 positions by 4.8e-7 (and the restatement's own fp64
angle by 2.4e-7), sincospif, the factor and two products by 4 x 2^-23: together below 2^-19."""
import numpy as np
import pytest
import torch

from mla_latent_kv_17_gb300 import ops
import step_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from mla_latent_kv_17_gb300 import build
    build.build()
    ops.lib()


def check(x, pos, freqs, layout, mscale, got_pass, got_rot, d_pass):
    xs = x.double().cpu().numpy()
    y, pair = step_ref.rotate(xs[..., d_pass:], pos.cpu().numpy(), freqs.cpu().numpy(), layout, mscale)
    err = np.abs(got_rot.double().cpu().numpy() - y)
    bound = 2.0 ** -8 * np.abs(y) + 2.0 ** -19 * abs(mscale) * pair * (1 + 2.0 ** -8)
    assert (err <= bound).all(), (err - bound).max()
    if got_pass is not None:
        assert torch.equal(got_pass, x[..., :d_pass])


CASES = [  # tokens, heads, passing, rotated
    (1, 1, 128, 64), (1, 128, 128, 64), (7, 3, 128, 64), (300, 16, 128, 64), (33, 128, 64, 128), (5, 2, 0, 16),
    (9, 5, 8, 2), (4, 3, 3, 6), (2, 2, 5, 64), (6, 1, 512, 64), (3, 7, 16, 24), (2, 1, 0, 2048),
    (1500, 1, 512, 64), (5000, 2, 0, 64), (3, 2, 1003, 10), (2, 130, 24, 16)]


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("n,h,dp,dr", CASES)
def test_rope(n, h, dp, dr, layout):
    g = torch.Generator().manual_seed(n * 1000 + h * 10 + dr)
    x = torch.randn(n, h, dp + dr, generator=g).to(torch.bfloat16).cuda()
    pos = torch.randint(0, 2 ** 31 - 1, (n,), generator=g).to(torch.int32).cuda()
    pos[0] = 0
    freqs, m = ops.rope_frequencies(dr, scaling="yarn", factor=16.0)
    p, r = ops.rope(x, pos, freqs, layout=layout, mscale=m)
    assert (p is None) == (dp == 0) and r.shape == (n, h, dr)
    check(x, pos, freqs, layout, m, p, r, dp)
    if n > 1:  # position 0 turns nothing
        assert torch.equal(ops.rope(x[:1], pos[:1], freqs, layout=layout)[1], x[:1, :, dp:])


@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_rope_strides_in_place_and_backwards(layout):
    g = torch.Generator().manual_seed(3)
    freqs, _ = ops.rope_frequencies(64)
    pos = torch.randint(0, 100000, (40,), generator=g).to(torch.int32).cuda()
    wide = torch.randn(40, 4 * 192 + 56, generator=g).to(torch.bfloat16).cuda()
    for cut in (0, 8, 1):  # aligned rows, another aligned start, rows of odd alignment (single values)
        x = wide[:, cut:cut + 4 * 192].unflatten(1, (4, 192))
        p, r = ops.rope(x, pos, freqs, layout=layout)
        check(x, pos, freqs, layout, 1.0, p, r, 128)
    # heads outermost in memory, and in place
    y = torch.randn(4, 40, 192, generator=g).to(torch.bfloat16).cuda()
    x = y.transpose(0, 1)
    before = x.clone()
    p, r = ops.rope(x, pos, freqs, layout=layout, out_rot=x[..., 128:], copy_pass=False)
    assert p is None and r.data_ptr() == x[..., 128:].data_ptr()
    check(before, pos, freqs, layout, 1.0, None, r, 128)
    assert torch.equal(x[..., :128], before[..., :128])
    # turning back by the negated positions: two roundings to bf16 (2^-8 each) and the angle
    back = ops.rope(x, -pos, freqs, layout=layout)[1].double().cpu()
    a = before[..., 128:].double().cpu()
    pair = step_ref.rotate(a.numpy(), pos.cpu().numpy(), freqs.cpu().numpy(), layout, 1.0)[1]
    assert ((back - a).abs().numpy() <= 2.0 ** -7 * (1 + 2.0 ** -8) * pair + 2.0 ** -18 * pair).all()


def test_rope_empty_and_refusals():
    freqs, _ = ops.rope_frequencies(64)
    p, r = ops.rope(torch.zeros(0, 4, 192, dtype=torch.bfloat16, device="cuda"),
                    torch.zeros(0, dtype=torch.int32, device="cuda"), freqs)
    assert p.shape == (0, 4, 128) and r.shape == (0, 4, 64)
    x = torch.zeros(2, 4, 192, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(2, dtype=torch.int32, device="cuda")
    for bad in (dict(layout="x"), dict(layout=0), dict(out_rot=x), dict(mscale=float("nan")),
                dict(out_pass=torch.zeros(2, 4, 128, device="cuda"))):
        with pytest.raises((ValueError, ops.MlaError)):
            ops.rope(x, pos, freqs, **bad)
    with pytest.raises(ValueError):
        ops.rope(x, pos.long(), freqs)
    with pytest.raises(ValueError):
        ops.rope(x, pos, freqs.float())
    with pytest.raises(ValueError):
        ops.rope(x.transpose(1, 2)[:, :192, :].transpose(0, 1)[:, :2], pos, freqs)
