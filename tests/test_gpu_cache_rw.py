"""Cache write and read of many tokens on the GPU: bytes against the CPU oracle's append where
nothing is computed but the record, 64-bit restatements with derived bounds where the norm and
the rotation join in."""
import numpy as np
import pytest
import torch

import oracle
from mla_latent_kv_17_gb300 import ops
import step_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from mla_latent_kv_17_gb300 import build
    build.build()
    ops.lib()


def _pool(fp8, pages, seed):
    g = torch.Generator().manual_seed(seed)
    raw = torch.randint(0, 256, (pages, 64, 656 if fp8 else 1152), dtype=torch.uint8, generator=g)
    return raw if fp8 else raw.view(torch.bfloat16)


def _case(n, b, seed, stride=576):
    """n tokens of b requests at distinct places of a shuffled pool."""
    g = torch.Generator().manual_seed(seed)
    max_pages = max(2, (n // b + 64) // 64 + 1)
    pages = b * max_pages
    bt = torch.randperm(pages, generator=g)[:b * max_pages].reshape(b, max_pages).to(torch.int32)
    at = torch.randperm(b * max_pages * 64, generator=g)[:n]
    req, pos = (at // (max_pages * 64)).to(torch.int32), (at % (max_pages * 64)).to(torch.int32)
    mag = torch.tensor([1.0, 1e-3, 300.0, 0.0]).repeat_interleave(128)
    kv = torch.cat([torch.randn(n, 512, generator=g) * mag, torch.randn(n, 64, generator=g)], 1).to(torch.bfloat16)
    wide = torch.zeros(n, stride, dtype=torch.bfloat16)
    wide[:, :576] = kv
    return bt, pages, req, pos, wide[:, :576]


def _bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n,b,stride", [(1, 1, 576), (9, 3, 576), (200, 5, 640), (3001, 7, 1024)])
def test_write_equals_append_bytes_and_reads_back(fp8, n, b, stride):
    bt, pages, req, pos, kv = _case(n, b, 100 + n, stride)
    pool = _pool(fp8, pages, 7)
    # the oracle appends one token per request: give it each token as a request of its own
    ref, err = oracle.append(pool.contiguous().view(torch.uint8).reshape(-1).numpy(), fp8, bt[req.long()].numpy(),
                             pos.numpy(), _bits(kv[:, :512]), _bits(kv[:, 512:]))
    assert err == 0
    wide = torch.zeros(n, stride, dtype=torch.bfloat16, device="cuda")
    wide[:, :576] = kv.cuda()
    cache = pool.clone().cuda()
    ops.cache_write(cache, bt.cuda(), req.cuda(), pos.cuda(), wide[:, :576])
    assert np.array_equal(cache.cpu().contiguous().view(torch.uint8).reshape(-1).numpy(), ref)
    got = ops.cache_read(cache, bt.cuda(), req.cuda(), pos.cuda())
    if not fp8:
        assert torch.equal(got.cpu().view(torch.int16), kv.contiguous().view(torch.int16))
        return
    rows = (bt[req.long(), (pos // 64).long()] * 64 + pos % 64).long()
    rec = cache.cpu().reshape(-1, 656)[rows]
    x = rec[:, :512].contiguous().view(torch.float8_e4m3fn).double() \
        * rec[:, 512:528].contiguous().view(torch.float32).double().repeat_interleave(128, 1)
    err = (got[:, :512].cpu().double() - x).abs()
    # code x scale in fp32 (2^-24), then bf16 (2^-8)
    assert bool((err <= (2.0 ** -8 + 2.0 ** -23) * x.abs()).all())
    assert torch.equal(got[:, 512:].cpu().view(torch.int16), kv[:, 512:].contiguous().view(torch.int16))


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n", [1, 37, 2500])
def test_write_with_norm_and_rotation(n, fp8, layout):
    bt, pages, req, pos, kv = _case(n, 3, 300 + n)
    g = torch.Generator().manual_seed(n)
    w = (1 + 0.3 * torch.randn(512, generator=g)).to(torch.bfloat16)
    freqs, m = ops.rope_frequencies(64, scaling="yarn", factor=40.0)
    rpos = torch.randint(0, 10 ** 6, (n,), generator=g).to(torch.int32)
    cache = _pool(fp8, pages, 8).cuda()
    before = cache.clone()
    ops.cache_write(cache, bt.cuda(), req.cuda(), pos.cuda(), kv.cuda(), freqs=freqs, rope_positions=rpos.cuda(),
                    layout=layout, mscale=m, norm_weight=w.cuda(), norm_eps=1e-5)
    rows = (bt[req.long(), (pos // 64).long()] * 64 + pos % 64).long()
    flat = cache.cpu().reshape(pages * 64, -1)
    untouched = torch.ones(pages * 64, dtype=torch.bool)
    untouched[rows] = False
    assert torch.equal(flat[untouched].view(torch.uint8), before.cpu().reshape(pages * 64, -1)[untouched].view(torch.uint8))
    got = flat[rows]
    x = kv.double().numpy()
    y = x[:, :512] / np.sqrt((x[:, :512] ** 2).mean(1, keepdims=True) + 1e-5) * w.double().numpy()
    k, pair = step_ref.rotate(x[:, 512:], rpos.numpy(), freqs.cpu().numpy(), layout, m)
    if fp8:
        key = got[:, 528:].contiguous().view(torch.bfloat16).double().numpy()
        s = got[:, 512:528].contiguous().view(torch.float32).double().numpy()
        code = got[:, :512].contiguous().view(torch.float8_e4m3fn).double().numpy()
        amax = np.abs(y).reshape(n, 4, 128).max(2)
        want = np.where(amax > 0, amax / 448, 1.0)
        # fp32: 21 additions of squares, a root (2 ulp), three products, a division: below 2^-19
        assert (np.abs(s - want) <= 2.0 ** -19 * want).all()
        sr = np.repeat(s, 128, 1)
        # e4m3: half a step is 2^-4 of the value, or 2^-10 of the scale below the normal range
        assert (np.abs(code * sr - y) <= (2.0 ** -4 + 2.0 ** -18) * np.abs(y) + 2.0 ** -10 * sr).all()
    else:
        key = got[:, 512:].double().numpy()
        assert (np.abs(got[:, :512].double().numpy() - y) <= (2.0 ** -8 + 2.0 ** -19) * np.abs(y)).all()
    assert (np.abs(key - k) <= 2.0 ** -8 * np.abs(k) + 2.0 ** -19 * m * pair * (1 + 2.0 ** -8)).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_skipped_and_unmapped_tokens(fp8):
    bt, pages, req, pos, kv = _case(8, 2, 11)
    mp = bt.shape[1]
    bt = bt.clone()
    bt[1, 1] = pages + 3                                     # a page id outside the pool
    req = torch.tensor([0, 0, 1, 1, 0, 2, -1, 0], dtype=torch.int32)
    pos = torch.tensor([0, -1, 5, 64, 64 * mp, 3, 3, 63], dtype=torch.int32)  # skip; bad page; past the table; bad requests
    good = [0, 2, 7]
    pool = _pool(fp8, pages, 9)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cache = pool.clone().cuda()
    ops.cache_write(cache, bt.cuda(), req.cuda(), pos.cuda(), kv.cuda(), device_status=status)
    assert int(status) == 5  # MLA_ERR_INDEX
    ref, _ = oracle.append(pool.contiguous().view(torch.uint8).reshape(-1).numpy(), fp8, bt[req[good].long()].numpy(),
                           pos[good].numpy(), _bits(kv[good][:, :512]), _bits(kv[good][:, 512:]))
    assert np.array_equal(cache.cpu().contiguous().view(torch.uint8).reshape(-1).numpy(), ref)
    status.zero_()
    rows = torch.full((8, 640), 3.0, dtype=torch.bfloat16, device="cuda")
    ops.cache_read(cache, bt.cuda(), req.cuda(), pos.cuda(), entries=rows[:, :576], device_status=status)
    assert int(status) == 5
    bad = [1, 3, 4, 5, 6]
    assert bool((rows[bad] == 3.0).all()) and bool((rows[:, 576:] == 3.0).all())
    assert torch.equal(rows[good][:, 512:576].cpu().view(torch.int16), kv[good][:, 512:].contiguous().view(torch.int16))
    # only skips: nothing recorded, nothing written
    status.zero_()
    again = cache.clone()
    ops.cache_write(cache, bt.cuda(), req.cuda(), torch.full_like(pos, -1).cuda(), kv.cuda(), device_status=status)
    assert int(status) == 0 and torch.equal(cache.view(torch.uint8), again.view(torch.uint8))


def test_no_requests_given_means_one_token_each():
    bt, pages, _, _, kv = _case(4, 4, 12)
    pos = torch.tensor([1, 70, -1, 0], dtype=torch.int32).cuda()
    a, b = _pool(True, pages, 1).cuda(), _pool(True, pages, 1).cuda()
    ops.cache_write(a, bt.cuda(), None, pos, kv.cuda())
    ops.cache_append(b, bt.cuda(), pos, kv[:, :512].contiguous().cuda(), kv[:, 512:].contiguous().cuda())
    assert torch.equal(a, b)
    with pytest.raises(ops.MlaError):
        ops.cache_write(a, bt[:3].contiguous().cuda(), None, pos, kv.cuda())


def test_long_cache_offsets_and_empty_calls():
    # a row 5 GB into the pool: byte offsets beyond 32 bits
    cache = torch.empty(70000, 64, 576, dtype=torch.bfloat16, device="cuda")
    bt = torch.tensor([[69999, 1]], dtype=torch.int32, device="cuda")
    kv = torch.randn(2, 576, device="cuda").to(torch.bfloat16)
    pos = torch.tensor([63, 64], dtype=torch.int32, device="cuda")
    req = torch.zeros(2, dtype=torch.int32, device="cuda")
    ops.cache_write(cache, bt, req, pos, kv)
    assert torch.equal(cache[69999, 63], kv[0]) and torch.equal(cache[1, 0], kv[1])
    assert torch.equal(ops.cache_read(cache, bt, req, pos), kv)
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    ops.cache_write(cache, bt, none, none, kv[:0])
    assert ops.cache_read(cache, bt, none, none).shape == (0, 576)


def test_norm_weights_that_underflow_leave_zero_blocks():
    # x * weight near fp32's smallest values: max / 448 rounds to 0, which is no scale to divide by
    bt, pages, req, pos, kv = _case(6, 2, 30)
    kv = kv.contiguous()
    kv[:, :512] = (kv[:, :512].double() * 1e-20).to(torch.bfloat16)
    w = torch.full((512,), 1e-24, dtype=torch.bfloat16)
    w[128:256] = 0.0
    w[256:384] = 1e-16
    w[384:] = 1.0
    cache = _pool(True, pages, 3).cuda()
    ops.cache_write(cache, bt.cuda(), req.cuda(), pos.cuda(), kv.cuda(), norm_weight=w.cuda(), norm_eps=1e-6)
    got = ops.cache_read(cache, bt.cuda(), req.cuda(), pos.cuda())[:, :512].double().cpu()
    x = kv[:, :512].double()
    y = x / (x.pow(2).mean(1, keepdim=True) + 1e-6).sqrt() * w.double()
    assert bool((got[:, :256] == 0).all())
    # the others are ordinary blocks: half a step of e4m3 (2^-4, or 2^-10 of the scale), then bf16 (2^-8)
    s = y.view(-1, 4, 128).abs().amax(2).repeat_interleave(128, 1) / 448
    tol = (2.0 ** -4 + 2.0 ** -7) * y.abs() + 2.0 ** -9 * s
    assert bool(((got - y).abs()[:, 256:] <= tol[:, 256:]).all())
    assert bool(torch.isfinite(got).all())


def test_records_of_extreme_values_equal_the_oracle():
    # blocks from the smallest bf16 values to the largest: scales below and above the range in
    # which the quotient's Newton step is exact, subnormal ones among them
    n = 260
    bt, pages, req, pos, kv = _case(n, 2, 21)
    kv = kv.contiguous()
    g = torch.Generator().manual_seed(22)
    e = torch.linspace(-133, 127, n).round()
    kv[:, :512] = (torch.rand(n, 512, generator=g).double() * 1.99 - 0.99).mul(2.0 ** e.double()[:, None]).to(torch.bfloat16)
    pool = _pool(True, pages, 3)
    ref, err = oracle.append(pool.reshape(-1).numpy(), True, bt[req.long()].numpy(), pos.numpy(),
                             _bits(kv[:, :512]), _bits(kv[:, 512:]))
    assert err == 0
    cache = pool.clone().cuda()
    ops.cache_write(cache, bt.cuda(), req.cuda(), pos.cuda(), kv.cuda())
    assert np.array_equal(cache.cpu().reshape(-1).numpy(), ref)
