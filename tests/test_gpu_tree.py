"""Tree attention on the GPU against its 64-bit definition, with bounds derived in tree_ref."""
import math

import numpy as np
import pytest
import torch

from guards import Guarded
from mla_latent_kv_17_gb300 import inputs, ops
from planview import parse
import tree_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from mla_latent_kv_17_gb300 import build
    build.build()
    ops.lib()


def make(B, T, H, contexts, lens=None, kv="bf16", seed=0, chain=False, q_scale=1.0):
    """Requests of contexts[b] committed tokens and lens[b] drafted ones, shuffled pages, NaN behind
    each request's last token, a random tree per request."""
    g = torch.Generator().manual_seed(seed)
    lens = torch.full((B,), T, dtype=torch.int32) if lens is None else torch.tensor(lens, dtype=torch.int32)
    seq = torch.tensor(contexts, dtype=torch.int32) + lens
    c = inputs.make_case(B, 1, seq, seed=seed + 1, kv_dtype=kv, device="cuda", extra_pages=3)
    qn = (torch.randn(B, T, H, 512, generator=g) * q_scale).to(torch.bfloat16).cuda()
    qr = (torch.randn(B, T, H, 64, generator=g) * q_scale).to(torch.bfloat16).cuda()
    mask = np.zeros((B, T), dtype=np.uint64)
    for b in range(B):
        for i in range(T):
            par = i - 1 if chain else int(torch.randint(-1, i, (1,), generator=g)) if i else -1
            mask[b, i] = (mask[b, par] if par >= 0 else np.uint64(0)) | np.uint64(1) << np.uint64(i)
    mask = torch.from_numpy(mask.view(np.int64)).cuda()
    return dict(qn=qn, qr=qr, cache=c.cache, bt=c.block_table, seq=seq.cuda(), lens=lens.cuda(), mask=mask)


def run(d, out_dtype=torch.float32, with_lse=True, kv=None, num_sms=0):
    B, T, H, _ = d["qn"].shape
    ws = ops.TreeWorkspace(B, T, H)
    guard = Guarded(ws.nbytes)
    guard.inner[:256].zero_()
    ws.buf = guard.inner
    ops.plan_tree(ws, d["seq"], d["lens"], kv_dtype="fp8" if d["cache"].dtype == torch.uint8 else "bf16", num_sms=num_sms)
    go, gl = Guarded(B * T * H * 512 * (4 if out_dtype == torch.float32 else 2)), Guarded(B * T * H * 4)
    out = go.inner.view(out_dtype).view(B, T, H, 512).fill_(7.0)
    lse = gl.inner.view(torch.float32).view(B, T, H).fill_(7.0) if with_lse else None
    ops.decode_tree(ws, d["qn"], d["qr"], d["cache"], d["bt"], d["seq"], d["lens"], d["mask"], tree_ref.SCALE, out=out,
                    lse=lse, with_lse=with_lse)
    st = ops.status(ws)
    for x, n in ((guard, "workspace"), (go, "out"), (gl, "lse")):
        x.check(n)
    return out, lse, st, ws


def both(d, out_dtype=torch.float32, what="", **kw):
    out, lse, st, ws = run(d, out_dtype, **kw)
    assert st == 0, what
    tree_ref.check(out, lse, tree_ref.tree(d["qn"], d["qr"], d["cache"], d["bt"], d["seq"], d["lens"], d["mask"]), what)
    return out, lse, ws


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("T,H", [(1, 1), (1, 128), (2, 128), (3, 48), (5, 16), (8, 16), (64, 2), (13, 10)])
def test_tree_shapes(T, H, kv):
    both(make(3, T, H, [200, 0, 65], seed=T * 100 + H, kv=kv), torch.float32, f"T {T} H {H} {kv}")


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_tree_ragged(kv, out_dtype):
    # trees of different sizes, one empty request, one without drafted tokens, borders of pages and tiles
    contexts = [0, 63, 64, 127, 128, 60, 1000, 0, 300, 1]
    lens = [7, 1, 7, 2, 5, 7, 3, 0, 0, 6]
    d = make(10, 7, 24, contexts, lens, kv, seed=5)
    out, lse, _ = both(d, out_dtype, f"ragged {kv}")
    assert bool((out[7:9] == 0).all()) and bool(torch.isneginf(lse[7:9]).all())
    assert bool((out[1, 1:] == 0).all())


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_tree_splits(kv):
    # few requests with long contexts are cut into pieces over the units, and merged
    d = make(2, 3, 128, [9000, 20000], kv=kv, seed=6)
    _, _, ws = both(d, torch.bfloat16, f"split {kv}")
    d = make(1, 4, 16, [30001], kv=kv, seed=7)
    both(d, torch.float32, f"split {kv}, one tile")
    both(make(2, 40, 16, [5000, 77], kv=kv, seed=8), torch.bfloat16, f"split {kv}, five tiles", with_lse=False)


@pytest.mark.parametrize("kv,out_dtype", [("bf16", torch.float32), ("bf16", torch.bfloat16), ("fp8", torch.bfloat16)])
def test_many_empty_row_tiles(kv, out_dtype):
    # eight row tiles per request, most of them past the drafted tokens: written as zeros, by all units
    lens = [1, 0, 2, 16, 3, 0, 1, 1, 9, 2, 0, 4]
    d = make(12, 16, 64, [150, 20, 0, 700, 64, 0, 3, 127, 40, 1, 300, 90], lens, kv, seed=16)
    out, lse, _ = both(d, out_dtype, "empty tiles")
    for b, n in enumerate(lens):
        assert bool((out[b, n:] == 0).all()) and bool(torch.isneginf(lse[b, n:]).all())


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_plans_and_calls_in_a_row_on_one_workspace(kv):
    # the merge reads its plan while the attention before it still runs: plans of other lengths that
    # follow one another without a pause must never mix
    d = make(3, 4, 64, [9000, 20000, 400], kv=kv, seed=17)
    other = d["seq"].clone()
    other[1] = 700
    ws = ops.TreeWorkspace(3, 4, 64)
    lens = {False: d["seq"], True: other}
    outs = [torch.zeros(3, 4, 64, 512, device="cuda") for _ in range(24)]

    def step(k, out):
        seq = lens[k % 3 == 1]
        ops.plan_tree(ws, seq, d["lens"], kv_dtype=kv)
        ops.decode_tree(ws, d["qn"], d["qr"], d["cache"], d["bt"], seq, d["lens"], d["mask"], tree_ref.SCALE, out=out)

    want = [torch.zeros_like(outs[0]) for _ in range(2)]
    for k in range(2):
        step(k, want[k])
        assert ops.status(ws) == 0
    for k, out in enumerate(outs):
        step(k, out)
    assert ops.status(ws) == 0
    for k, out in enumerate(outs):
        assert torch.equal(out, want[k % 3 == 1]), k


def test_peaked_scores():
    both(make(2, 4, 32, [500, 1300], seed=9, q_scale=8.0), torch.float32, "peaked")


def test_chain_of_one_equals_plain_decode():
    # T = 1 attending itself is the single-token decode: the same kernels and items, the same bits
    d = make(5, 1, 128, [100, 64, 4000, 0, 511], seed=10)
    out, lse, st, _ = run(d)
    ws = ops.Workspace(5, 128)
    ops.plan(ws, d["seq"])
    o, l = ops.decode(ws, d["qn"].view(5, 128, 512), d["qr"].view(5, 128, 64), d["cache"], d["bt"], d["seq"], tree_ref.SCALE)
    assert torch.equal(out.view(5, 128, 512), o) and torch.equal(lse.view(5, 128), l)


def test_chain_equals_decode_of_each_prefix():
    d = make(2, 6, 16, [150, 58], seed=11, chain=True)
    out, lse, _, _ = run(d)
    for i in range(6):
        seq = (d["seq"] - 5 + i).contiguous()
        ws = ops.Workspace(2, 16)
        ops.plan(ws, seq)
        o, l = ops.decode(ws, d["qn"][:, i].contiguous(), d["qr"][:, i].contiguous(), d["cache"], d["bt"], seq, tree_ref.SCALE)
        ref = tree_ref.tree(d["qn"], d["qr"], d["cache"], d["bt"], d["seq"], d["lens"], d["mask"])
        assert bool(((out[:, i] - o).double().abs() <= 2 * ref[2][:, i]).all())
        assert bool(((lse[:, i] - l).double().abs() <= 2 * ref[3][:, i]).all())


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_split_pieces_of_padded_rows(kv):
    # few real rows in a split tile: the padded ones have no partial results and come out empty
    d = make(2, 8, 16, [30000, 12000], lens=[3, 1], kv=kv, seed=16)
    d["qn"][0, 3:], d["qr"][0, 3:] = float("nan"), float("nan")
    out, lse, ws = both(d, torch.bfloat16, f"padded {kv}")
    assert bool((out[0, 3:] == 0).all()) and bool(torch.isneginf(lse[1, 1:]).all())


def test_one_plan_serves_several_calls():
    # the layers of a model share lengths: one plan, other queries and caches
    d, e = (make(3, 4, 32, [900, 64, 3000], seed=s) for s in (17, 18))
    ws = ops.TreeWorkspace(3, 4, 32)
    ops.plan_tree(ws, d["seq"], d["lens"])
    got = [ops.decode_tree(ws, x["qn"], x["qr"], x["cache"], x["bt"], x["seq"], x["lens"], x["mask"], tree_ref.SCALE)
           for x in (d, e, d)]
    assert ops.status(ws) == 0
    for x, (o, l) in zip((d, e), got):
        tree_ref.check(o, l, tree_ref.tree(x["qn"], x["qr"], x["cache"], x["bt"], x["seq"], x["lens"], x["mask"]))
    assert torch.equal(got[0][0], got[2][0]) and torch.equal(got[0][1], got[2][1])


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_masks_that_leave_a_row_empty(kv):
    d = make(3, 5, 20, [0, 0, 70], kv=kv, seed=12)
    d["mask"][0] = 0                     # no context and no ancestors: nothing is attended
    d["mask"][1, 2] = 0
    d["mask"][2, 3] = 0                  # only the context
    d["mask"][1, 4] = -1                 # every bit set, those behind the tree too
    out, lse, _ = both(d, torch.float32, "empty rows")
    assert bool((out[0] == 0).all()) and bool(torch.isneginf(lse[0]).all())
    assert bool((out[1, 2] == 0).all()) and bool(torch.isneginf(lse[1, 2]).all())


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("context", [0, 61, 500, 12000])
def test_bad_values_reach_only_the_rows_that_attend_them(kv, context):
    d = make(1, 6, 40, [context], kv=kv, seed=13)
    bits = np.array([1, 2, 4, 8 | 1, 16 | 2, 32 | 16 | 2], dtype=np.uint64)  # token 2 is attended by itself only
    d["mask"][0] = torch.from_numpy(bits.view(np.int64)).cuda()
    want = run(d, torch.bfloat16)
    at = context + 2
    page, row = int(d["bt"][0, at // 64]), at % 64
    if kv == "bf16":
        d["cache"][page, row, 3::7] = float("nan")
        d["cache"][page, row, 100] = float("inf")
    else:
        d["cache"][page, row, 3:500:7] = 0x7F  # the NaN code
    out, lse, st, _ = run(d, torch.bfloat16)
    keep = [0, 1, 3, 4, 5]
    assert torch.equal(out[0, keep], want[0][0, keep]) and torch.equal(lse[0, keep], want[1][0, keep])
    assert bool(torch.isnan(out[0, 2]).all()) and bool(torch.isnan(lse[0, 2]).all())


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("contexts", [[100, 30], [20000, 30]])
def test_queries_of_padded_tokens_may_hold_anything(kv, contexts):
    d = make(2, 9, 16, contexts, lens=[3, 0], kv=kv, seed=15)  # two row tiles, the second all padding
    want = both(d, torch.float32, "finite padding")
    for q in (d["qn"], d["qr"]):
        q[0, 3:] = float("nan")
        q[0, 4::2] = float("inf")
        q[1] = -1e30
    out, lse, st, _ = run(d)
    assert st == 0 and torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_device_errors_are_reported():
    d = make(2, 4, 16, [100, 200], seed=14)
    d["lens"][0] = 9                     # above T: clamped
    assert run(d)[2] == 5
    d["lens"][0] = -1
    out, _, st, _ = run(d)
    assert st == 5 and bool((out[0] == 0).all())
    d = make(2, 4, 16, [100, 200], seed=14)
    d["seq"][0] = 2                      # fewer entries than drafted tokens
    assert run(d)[2] == 5
    d = make(2, 4, 16, [100, 200], seed=14)
    d["bt"][1, 1] = 10 ** 6              # a page outside the pool
    assert run(d)[2] == 5
    # a plan of another shape, and no plan
    d = make(2, 4, 16, [100, 200], seed=14)
    ws = ops.TreeWorkspace(2, 4, 16)
    args = (d["qn"], d["qr"], d["cache"], d["bt"], d["seq"], d["lens"], d["mask"], tree_ref.SCALE)
    ops.decode_tree(ws, *args)
    assert ops.status(ws) == 3
    other = ops.TreeWorkspace(2, 2, 32)  # the same number of row tiles
    ops.plan_tree(other, d["seq"], None)
    ws.buf = other.buf
    ops.decode_tree(ws, *args)
    assert ops.status(ws) == 3


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_device_plan_equals_host_plan(kv):
    for B, T, H, hi in ((3, 5, 16, 3000), (40, 16, 128, 3000), (1, 64, 128, 90000), (300, 2, 128, 400)):
        g = torch.Generator().manual_seed(B)
        lens = torch.randint(0, T + 1, (B,), generator=g, dtype=torch.int32)
        seq = torch.randint(0, hi, (B,), generator=g, dtype=torch.int32) + lens
        ws = ops.TreeWorkspace(B, T, H)
        ops.plan_tree(ws, seq.cuda(), lens.cuda(), kv_dtype=kv)
        sms = torch.cuda.get_device_properties(0).multi_processor_count
        host = ops.plan_tree_host(seq, lens, B, T, H, num_sms=sms, kv_dtype=kv)
        entries = B * ((T * H + 127) // 128)
        a, b = parse(ws.buf.cpu().numpy(), entries, 128), parse(host, entries, 128)
        for k in ("unit_begin", "items", "num_splits", "split_base", "split_list", "n_partials", "per"):
            assert np.array_equal(a[k], b[k]), k


def test_stall_is_reported_and_the_workspace_stays_usable():
    d = make(2, 3, 32, [700, 90], seed=15)
    want = run(d)
    ops.set_wait_limit(2_000_000)
    ops.inject_stall(True)
    try:
        assert run(d)[2] == 6  # MLA_ERR_TIMEOUT
    finally:
        ops.inject_stall(False)
        ops.set_wait_limit(0)
    got = run(d)
    assert got[2] == 0 and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("scale", [2.0 ** -14, 2.0 ** -3, 40.0])
def test_fp8_scales_of_other_magnitudes(scale):
    # record scales below, inside and at the top of the range in which they are split into fp16
    # parts, and a batch that mixes them
    d = make(2, 3, 20, [300, 90], kv="fp8", seed=19)
    s = d["cache"][..., 512:528].view(torch.float32)
    s.mul_(scale * 448 / 3)              # (about max |x| / 448 = 3 / 448 before)
    d["qn"] = (d["qn"].float() / max(1.0, scale * 100)).to(torch.bfloat16)
    both(d, torch.float32, f"scale {scale}")
    s[:, ::3] *= 2.0 ** -9
    both(d, torch.float32, f"mixed {scale}")


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("tree", [True, False])
def test_replayed_plans_follow_the_lengths(kv, tree):
    # a captured run of plans and calls whose lengths, and so split requests, change from step to
    # step: every merge has to use the plan of its own step
    T, H = (4, 64) if tree else (1, 128)
    d = make(3, T, H, [9000, 20000, 400], kv=kv, seed=24)
    kinds = [d["seq"].clone() for _ in range(3)]
    kinds[1][1], kinds[2][0] = 700, 64
    ws = ops.TreeWorkspace(3, T, H) if tree else ops.Workspace(3, H)
    seq = d["seq"].clone()
    shape = (3, T, H, 512) if tree else (3, H, 512)

    def step(lens, out):
        seq.copy_(lens)
        if tree:
            ops.plan_tree(ws, seq, d["lens"], kv_dtype=kv)
            ops.decode_tree(ws, d["qn"], d["qr"], d["cache"], d["bt"], seq, d["lens"], d["mask"], tree_ref.SCALE, out=out)
        else:
            ops.plan(ws, seq, kv_dtype=kv)
            ops.decode(ws, d["qn"].view(3, H, 512), d["qr"].view(3, H, 64), d["cache"], d["bt"], seq, tree_ref.SCALE, out=out)

    want = [torch.zeros(shape, device="cuda") for _ in kinds]
    for lens, out in zip(kinds, want):
        step(lens, out)
        assert ops.status(ws) == 0
    outs = [torch.zeros(shape, device="cuda") for _ in range(12)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            for k, out in enumerate(outs):
                step(kinds[k % 3], out)
        for _ in range(5):
            for out in outs:
                out.fill_(7.0)
            graph.replay()
            s.synchronize()
            assert ops.status(ws, stream=s) == 0
            for k, out in enumerate(outs):
                assert torch.equal(out, want[k % 3]), k


def _behind(d):
    """(page, first row) of what lies behind each request's last token in its last page."""
    return [(int(d["bt"][b, int(n) // 64]), int(n) % 64) for b, n in enumerate(d["seq"]) if int(n) % 64]


@pytest.mark.parametrize("contexts", [[300, 90, 17], [20000, 60, 1]])
def test_fp8_bits_do_not_depend_on_what_lies_behind_the_last_token(contexts):
    # the same inputs, whatever the last pages' unused rows held before: zeros of a fresh pool, old
    # records of any scale, NaN
    d = make(3, 5, 24, contexts, kv="fp8", seed=20)
    want = None
    for scale, code in ((0.0, 0), (3.0 / 448, 0x35), (2.0 ** -20, 0x11), (1e30, 0x7E), (float("nan"), 0x7F), (None, None)):
        for k, (page, row) in enumerate(_behind(d)):
            rec = d["cache"][page, row:]
            if scale is None:  # every other row another scale
                rec[:, 512:528].view(torch.float32)[::2] = 2.0 ** -12
                continue
            rec[:, :512] = code
            rec[:, 512:528].view(torch.float32).fill_(scale)
            rec[:, 528:] = code
        out, lse, st, _ = run(d)
        assert st == 0
        want = want or (out, lse)
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1]), (scale, code)


@pytest.mark.parametrize("context", [0, 40, 61, 12000])
def test_fp8_scales_of_a_masked_token_leave_the_other_rows_bits(context):
    d = make(1, 6, 40, [context], kv="fp8", seed=21)
    bits = np.array([1, 2, 4, 8 | 1, 16 | 2, 32 | 16 | 2], dtype=np.uint64)  # token 2 is attended by itself only
    d["mask"][0] = torch.from_numpy(bits.view(np.int64)).cuda()
    for page, row in _behind(d):  # ordinary records
        d["cache"][page, row:] = d["cache"][int(d["bt"][0, 0]), 0]
    at, want, keep = context + 2, run(d), [0, 1, 3, 4, 5]
    rec = d["cache"][int(d["bt"][0, at // 64]), at % 64]
    for scale in (2.0 ** -16, 2.0 ** -11, 0.0, 130.0):
        rec[512:528].view(torch.float32).fill_(scale)
        out, lse, st, _ = run(d)
        assert st == 0
        assert torch.equal(out[0, keep], want[0][0, keep]) and torch.equal(lse[0, keep], want[1][0, keep]), scale


@pytest.mark.parametrize("T", [1, 2])
def test_fp8_values_enter_rounded_as_documented(T):
    # one token attended with weight 1: the output is the fp16 value its code x scale became.  One
    # rounding (2^-11, or 2^-25 below fp16's normal range) of code x scale, the scale held to 2^-15.
    B = 256
    g = torch.Generator().manual_seed(23)
    scales = (2.0 ** (torch.rand(B, 4, generator=g).double() * 21 - 14)).float()  # 2^-14 .. 2^7
    edges = [2.0 ** -10, 2.0 ** -9, 2.0 ** -8, 2.0 ** -7, 0.0010438, 3.0 / 448, 1.0, 127.9, 128.0, 145.0]
    for k, s in enumerate(edges):
        scales[k] = torch.tensor([s, s * (1 - 2.0 ** -24), s * (1 + 2.0 ** -23), s * 1.0037], dtype=torch.float64).float()
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8)
    codes[codes & 0x7F == 0x7F] = 0
    codes = torch.cat([codes, codes.flip(0)]).view(4, 128)
    cache = torch.zeros(B, 64, 656, dtype=torch.uint8)
    at = torch.arange(B)
    for r in range(2):  # every scale meets all codes: the blocks change places
        for k in range(4):
            cache[at, r, 128 * k:128 * (k + 1)] = codes[(at[:, None] + k + r) % 4].reshape(B, -1)
        cache[at, r, 512:528] = scales[at].contiguous().view(torch.uint8).view(B, 16)
    cache[:, 2:] = cache[:, :1]  # (what lies behind the last token is like the tokens)
    d = dict(qn=torch.zeros(B, T, 1, 512, dtype=torch.bfloat16, device="cuda"),
             qr=torch.zeros(B, T, 1, 64, dtype=torch.bfloat16, device="cuda"), cache=cache.cuda(),
             bt=torch.randperm(B, generator=g).to(torch.int32).view(B, 1).cuda(),
             seq=torch.full((B,), T, dtype=torch.int32, device="cuda"),
             lens=torch.full((B,), T, dtype=torch.int32, device="cuda"),
             mask=(1 << torch.arange(T, dtype=torch.int64)).repeat(B, 1).cuda())
    out, lse, st, _ = run(d)
    assert st == 0 and bool((lse == 0).all())
    rec = cache[d["bt"].cpu().long().view(-1)][:, :T]
    x = rec[..., :512].contiguous().view(torch.float8_e4m3fn).double() \
        * rec[..., 512:528].contiguous().view(torch.float32).double().repeat_interleave(128, -1)
    err = (out.view(B, T, 512).cpu().double() - x).abs()
    bound = torch.where(x.abs() >= 2.0 ** -14, 2.0 ** -11 * (1 + 2.0 ** -4) * x.abs(), 2.0 ** -25 + 2.0 ** -15 * x.abs())
    assert bool((err <= bound).all()), float((err / x.abs().clamp(min=2.0 ** -14) * 2.0 ** 11).max())


@pytest.mark.parametrize("kv,channel", [("bf16", 100), ("bf16", 400), ("bf16", 530), ("fp8", 530)])
@pytest.mark.parametrize("value", [float("inf"), float("-inf")])
@pytest.mark.parametrize("context", [0, 61, 126, 500, 12000])
def test_one_infinity_shows_in_every_row_that_attends_it(kv, channel, value, context):
    # whichever sign it gives the score: a weight of 0 must not hide the token
    d = make(1, 6, 40, [context], kv=kv, seed=22)
    bits = np.array([1, 2, 4, 8 | 1, 16 | 2, 32 | 4], dtype=np.uint64)  # token 2: by itself and by token 5
    d["mask"][0] = torch.from_numpy(bits.view(np.int64)).cuda()
    want = run(d)
    at = context + 2
    rec = d["cache"][int(d["bt"][0, at // 64]), at % 64]
    if kv == "bf16":
        rec[channel] = value
        q = d["qn"][0, 2, :, channel] if channel < 512 else d["qr"][0, 2, :, channel - 512]
    else:
        rec[528:].view(torch.bfloat16)[channel - 512] = value
        q = d["qr"][0, 2, :, channel - 512]
    assert bool((q > 0).any()) and bool((q < 0).any())  # scores of both signs
    for dtype in (torch.float32, torch.bfloat16):
        out, lse, st, _ = run(d, dtype)
        keep = [0, 1, 3, 4]
        assert st == 0
        assert torch.equal(out[0, keep], want[0][0, keep].to(dtype)) and torch.equal(lse[0, keep], want[1][0, keep])
        for i in (2, 5):
            assert bool(torch.isnan(out[0, i]).all()) and bool(torch.isnan(lse[0, i]).all()), i
