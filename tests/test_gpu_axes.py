"""Rotary positions with several axes on the GPU, of queries and of keys on their way into the cache,
against a 64-bit restatement.

Bound: |error| <= 2^-8 |y| (one rounding to bf16) + 2^-19 m (|a| + |b|), as for one axis: the angle's
24-bit conversion (1.9e-7 rad), the frequency's fp64 rounding at 2^31 positions (4.8e-7), the
restatement's own fp64 angle (2.4e-7), sincospif, the factor and two products (4 x 2^-23)."""
import numpy as np
import pytest
import torch

from mla_latent_kv_17_gb300 import ops
import prompt_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from mla_latent_kv_17_gb300 import build
    build.build()
    ops.lib()


def check_rot(x, pos, sections, order, freqs, layout, mscale, got):
    y, pair = prompt_ref.rotate(x.double().cpu().numpy(), pos.cpu().numpy(), prompt_ref.axis_of_pair(sections, order),
                                freqs.cpu().numpy(), layout, mscale)
    err = np.abs(got.double().cpu().numpy() - y)
    bound = 2.0 ** -8 * np.abs(y) + 2.0 ** -19 * abs(mscale) * pair * (1 + 2.0 ** -8)
    assert (err <= bound).all(), (err - bound).max()


def split(pairs, axes):
    """Pairs of each axis, uneven."""
    counts = [pairs // axes] * axes
    counts[-1] += pairs - sum(counts)
    if axes > 2 and counts[0] > 1:
        counts[0] -= 1
        counts[1] += 1
    return counts


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("order", ["blocks", "interleaved"])
@pytest.mark.parametrize("n,h,dp,dr,axes", [
    (1, 1, 128, 64, 3), (7, 3, 128, 64, 3), (300, 16, 128, 64, 4), (33, 128, 64, 128, 3), (5, 2, 0, 16, 2),
    (9, 5, 8, 6, 3), (2, 2, 5, 64, 3), (1500, 1, 512, 64, 3), (3, 7, 16, 24, 3), (2, 1, 0, 512, 4), (4, 130, 24, 16, 1)])
def test_rope_axes(n, h, dp, dr, axes, order, layout):
    g = torch.Generator().manual_seed(n * 1000 + h * 10 + dr)
    x = torch.randn(n, h, dp + dr, generator=g).to(torch.bfloat16).cuda()
    pos = torch.randint(-2 ** 31, 2 ** 31 - 1, (axes, n), generator=g).to(torch.int32).cuda()
    freqs, m = ops.rope_frequencies(dr, scaling="yarn", factor=16.0)
    counts = split(dr // 2, axes)
    for p in (pos.t(), pos.t().contiguous()):  # an axis's positions together, or a token's
        passed, r = ops.rope(x, p, freqs, layout=layout, mscale=m, axes=ops.rope_axes(counts, order))
        check_rot(x[..., dp:], p, counts, order, freqs, layout, m, r)
        assert passed is None and dp == 0 or torch.equal(passed, x[..., :dp])


@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_equal_positions_turn_as_one(layout):
    # text: the same position on every axis; strides, heads outermost, in place, odd alignment
    g = torch.Generator().manual_seed(3)
    freqs, _ = ops.rope_frequencies(64)
    pos = torch.randint(0, 100000, (40,), generator=g).to(torch.int32).cuda()
    axes = ops.rope_axes((8, 12, 12), "interleaved")
    wide = torch.randn(40, 4 * 192 + 56, generator=g).to(torch.bfloat16).cuda()
    for cut in (0, 8, 1):
        x = wide[:, cut:cut + 4 * 192].unflatten(1, (4, 192))
        for p in (pos.unsqueeze(1).expand(40, 3), pos.repeat(5, 1).t()[:, 1:4]):
            got, one = ops.rope(x, p, freqs, layout=layout, axes=axes), ops.rope(x, pos, freqs, layout=layout)
            assert torch.equal(got[0], one[0]) and torch.equal(got[1], one[1])
    y = torch.randn(4, 40, 192, generator=g).to(torch.bfloat16).cuda().transpose(0, 1)
    want = ops.rope(y, pos, freqs, layout=layout)[1]
    ops.rope(y, pos.unsqueeze(1).expand(40, 3), freqs, layout=layout, out_rot=y[..., 128:], copy_pass=False, axes=axes)
    assert torch.equal(y[..., 128:], want)


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("n,axes,norm", [(1, 3, False), (5, 2, True), (67, 3, True), (333, 4, False), (1001, 1, True)])
def test_cache_write_axes(n, axes, norm, kv, layout):
    g = torch.Generator().manual_seed(n)
    pages = n // 64 + 3
    table = torch.randperm(pages, generator=g).to(torch.int32).view(1, pages).cuda()
    req = torch.zeros(n, dtype=torch.int32, device="cuda")
    slot = torch.randperm(pages * 64, generator=g)[:n].to(torch.int32)
    slot[n // 2] = -1 if n > 1 else slot[0]  # a skipped token
    slot = slot.cuda()
    pos = torch.randint(0, 2 ** 31 - 1, (n, axes), generator=g).to(torch.int32).cuda()
    rows = torch.randn(n, 576 + 8, generator=g).to(torch.bfloat16).cuda()[:, :576]
    weight = (1 + 0.1 * torch.randn(512, generator=g)).to(torch.bfloat16).cuda() if norm else None
    freqs, m = ops.rope_frequencies(64, scaling="yarn", factor=4.0)
    width = 576 if kv == "bf16" else 656
    new = lambda: torch.full((pages, 64, width), 7, dtype=torch.bfloat16 if kv == "bf16" else torch.uint8, device="cuda")
    counts = split(32, axes)
    for order in ("blocks", "interleaved"):
        cache, one = new(), new()
        kw = dict(freqs=freqs, layout=layout, mscale=m, norm_weight=weight)
        ops.cache_write(cache, table, req, slot, rows, rope_positions=pos, axes=ops.rope_axes(counts, order), **kw)
        # all but the key is what the write with one axis gives, bit for bit; rows without a token stay
        ops.cache_write(one, table, req, slot, rows, rope_positions=pos[:, 0].contiguous(), **kw)
        flat, flat1 = cache.view(-1, width), one.view(-1, width)
        split_at = 512 if kv == "bf16" else 528
        assert torch.equal(flat[:, :split_at], flat1[:, :split_at])
        live = slot >= 0
        at = table[0].long()[slot[live].long() // 64] * 64 + slot[live].long() % 64
        untouched = torch.ones(pages * 64, dtype=torch.bool, device="cuda")
        untouched[at] = False
        assert bool((flat[untouched] == 7).all())
        key = flat[at][:, split_at:].contiguous().view(torch.bfloat16)
        check_rot(rows[live][:, 512:], pos[live], counts, order, freqs, layout, m, key)
    # equal positions: the write with one
    cache, one = new(), new()
    ops.cache_write(cache, table, req, slot, rows, rope_positions=pos[:, :1].expand(n, axes), axes=ops.rope_axes(counts), **kw)
    ops.cache_write(one, table, req, slot, rows, rope_positions=pos[:, 0].contiguous(), **kw)
    assert torch.equal(cache, one)


def test_far_rows_need_64_bits():
    # positions past 2^31 elements from their base, and an axis stride of that size
    n, far = 3, 2 ** 31 + 5
    buf = torch.zeros(2 * far + 16, dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(1)
    pos = buf.as_strided((n, 3), (1, far))
    pos.copy_(torch.randint(0, 100000, (n, 3), generator=g).to(torch.int32))
    x = torch.randn(n, 4, 192, generator=g).to(torch.bfloat16).cuda()
    freqs, _ = ops.rope_frequencies(64)
    got = ops.rope(x, pos, freqs, axes=ops.rope_axes((8, 12, 12)))[1]
    check_rot(x[..., 128:], pos, (8, 12, 12), "blocks", freqs, "interleaved", 1.0, got)


def test_empty_and_refusals():
    freqs, _ = ops.rope_frequencies(64)
    axes = ops.rope_axes((8, 12, 12))
    none = torch.zeros(0, 3, dtype=torch.int32, device="cuda")
    p, r = ops.rope(torch.zeros(0, 4, 192, dtype=torch.bfloat16, device="cuda"), none, freqs, axes=axes)
    assert p.shape == (0, 4, 128) and r.shape == (0, 4, 64)
    x = torch.zeros(2, 4, 192, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    for bad in (dict(axes=ops.rope_axes((8, 12))), dict(axes=list(axes)), dict(axes=ops.rope_axes((8, 8, 8, 8)))):
        with pytest.raises((ValueError, ops.MlaError)):
            ops.rope(x, pos, freqs, **bad)
    for bad in (pos[:, 0], pos.long(), pos[:1], pos[:, :0], torch.zeros(2, 5, dtype=torch.int32, device="cuda")[:, :2]):
        with pytest.raises((ValueError, ops.MlaError)):
            ops.rope(x, bad, freqs, axes=axes)
    cache = torch.zeros(1, 64, 576, dtype=torch.bfloat16, device="cuda")
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    one = torch.zeros(2, dtype=torch.int32, device="cuda")
    kv = torch.zeros(2, 576, dtype=torch.bfloat16, device="cuda")
    for kw in (dict(axes=axes), dict(axes=axes, freqs=freqs), dict(axes=axes, rope_positions=pos),
               dict(axes=axes, freqs=freqs, rope_positions=one), dict(axes=axes[:31], freqs=freqs, rope_positions=pos),
               dict(axes=axes, freqs=freqs, rope_positions=pos[:, :2])):
        with pytest.raises((ValueError, ops.MlaError)):
            ops.cache_write(cache, table, one, one, kv, **kw)
