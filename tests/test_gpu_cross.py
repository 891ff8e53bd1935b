"""Attention to key runs of another length on the GPU against a 64-bit restatement.

Bounds (u = 2^-24).  A score is a sum of d = 128 or 192 exact products in fp32: off by at most
d u scale sum |q k| =: e (absolute, in nats), and by 3 u of itself more for its factors.  A weight is
off by 2 e + 2^-21 relative (its score, the row's maximum, the exponential) and by the rounding of
the probability to bf16, 2^-8; the sum of weights by the same without the rounding, and by
(128 / 4 + 8 + tiles) u for its additions.  So out is off by 2^-8 E|v| + (4 e + 2^-20 + K u) E|v| with
E|v| the mean of |v| under the weights and K = 60 + keys (PV's additions), and lse by e + (K u + 2^-20),
and 4 u |lse|.  A part in bf16 output adds 2^-8 |out|."""
import numpy as np
import pytest
import torch

from guards import Guarded
from mla_latent_kv_17_gb300 import ops
import prompt_ref

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from mla_latent_kv_17_gb300 import build
    build.build()
    ops.lib()


class Case:
    """Packed runs; rows before, between and behind them hold NaN (q, k, entries, v)."""

    def __init__(self, q_lens, k_lens, H, positions, seed, spread=1.0, pad=0, before=False, device="cpu"):
        g = torch.Generator(device=device).manual_seed(seed)
        randn = lambda *s: torch.randn(*s, generator=g, device=device).to(BF)
        self.B, self.H, self.positions = len(q_lens), H, positions
        self.cu_q = np.concatenate([[pad], pad + np.cumsum(q_lens)]).astype(np.int32)
        self.cu_k = np.concatenate([[pad], pad + np.cumsum(k_lens)]).astype(np.int32)
        self.nq, self.nk = int(self.cu_q[-1]) + pad, int(self.cu_k[-1]) + pad
        self.q_nope, self.q_rope = randn(self.nq, H, 128), randn(self.nq, H, 64)
        self.q_nope, self.q_rope = (t * spread for t in (self.q_nope, self.q_rope))
        self.k_nope, self.v, self.entries = randn(H, self.nk, 128), randn(H, self.nk, 128), randn(self.nk, 576)
        self.scale = float(np.float32(1 / np.sqrt(192 if positions else 128)))
        self.before = None
        if before:
            lse = 2 + 2 * torch.randn(self.nq, H, generator=g, device=device)
            out = torch.randn(self.nq, H, 128, generator=g, device=device)
            gone = torch.rand(self.nq, H, generator=g, device=device) < 0.2
            lse[gone] = -torch.inf
            out[gone] = torch.nan
            self.before = (out, lse)
        if pad:
            for t in (self.q_nope, self.q_rope):
                t[:pad], t[-pad:] = torch.nan, torch.nan
            self.entries[:pad], self.entries[-pad:] = torch.nan, torch.nan
            for t in (self.k_nope, self.v):
                t[:, :pad], t[:, -pad:] = torch.nan, torch.nan

    def cuda(self):
        for n in ("q_nope", "q_rope", "k_nope", "v", "entries"):
            setattr(self, n, getattr(self, n).cuda())
        self.d_cu = torch.from_numpy(self.cu_q).cuda(), torch.from_numpy(self.cu_k).cuda()
        if self.before is not None:
            self.before = tuple(t.cuda() for t in self.before)
        return self

    def run(self, causal=False, ws=None, **kw):
        if ws is None:
            ws = ops.CrossWorkspace(self.B, self.H, self.nq)
        ops.plan_cross(ws, *self.d_cu, self.nk, causal=causal, stream=kw.get("stream"))
        q_rope, entries = (self.q_rope, self.entries) if self.positions else (None, None)
        got = ops.cross_attention(ws, self.q_nope, q_rope, entries, self.k_nope, self.v, self.scale, before=self.before, **kw)
        self.ws = ws
        return got

    def check(self, got, causal=False, heads=None):
        """Against the definition, all heads or the given ones."""
        assert ops.status(self.ws) == 0
        h = slice(None) if heads is None else torch.tensor(heads, device="cuda")
        num = lambda t: t.double().cpu().numpy()
        q, k, v = num(self.q_nope[:, h]), num(self.k_nope[h]), num(self.v[h])
        if self.positions:
            q = np.concatenate([q, num(self.q_rope[:, h])], -1)
            k = np.concatenate([k, np.broadcast_to(num(self.entries)[None, :, 512:], (len(k), self.nk, 64))], -1)
        before = None if self.before is None else tuple(num(t[:, h]) for t in self.before)
        got = (got[0][:, h], None if got[1] is None else got[1][:, h])
        out, lse, mean, dot = prompt_ref.cross(q, k, v, self.cu_q, self.cu_k, self.scale, causal, before)
        r = slice(self.cu_q[0], self.cu_q[-1])
        out, lse, mean, dot = out[r], lse[r], mean[r], dot[r]
        e = q.shape[-1] * U * self.scale * dot
        K = 60 + int(np.diff(self.cu_k).max(initial=0))
        go, gl = num(got[0])[r], got[1] if got[1] is None else num(got[1])[r]
        bound = (2.0 ** -8 + 4 * e[..., None] + 2.0 ** -20 + K * U) * mean
        if got[0].dtype == BF:
            bound = bound + 2.0 ** -8 * (np.abs(out) + bound)
        assert np.isfinite(go).all()
        err = np.abs(go - out)
        assert (err <= bound + 1e-30).all(), ("out", (err - bound).max(), np.argwhere(err > bound)[:4])
        if gl is not None:
            same = (gl == lse)
            with np.errstate(invalid="ignore"):
                ok = same | (np.abs(gl - lse) <= e + K * U + 2.0 ** -20 + 4 * U * np.abs(lse))
            assert ok.all(), ("lse", gl[~ok][:4], lse[~ok][:4])


@pytest.mark.parametrize("positions", [True, False])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("q_lens,k_lens,H", [
    ([1], [1], 1), ([5], [3], 2), ([1], [300], 3), ([1, 1, 1], [128, 129, 127], 16), ([128], [128], 2),
    ([129], [257], 2), ([256, 256], [512, 100], 3), ([257], [640], 9), ([300, 1, 77], [1000, 50, 129], 4),
    ([700], [701], 10), ([0, 5, 0, 130], [40, 0, 0, 260], 3), ([40, 0], [0, 0], 2), ([3] * 20, list(range(0, 400, 20)), 5)])
def test_cross(q_lens, k_lens, H, causal, positions):
    c = Case(q_lens, k_lens, H, positions, sum(q_lens) + sum(k_lens) + H).cuda()
    c.check(c.run(causal), causal)


# where the keys and values of all heads take 192 MB and more, a pair of query tiles shares them
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("q_lens,k_lens,positions,pad", [
    ([129], [3300], True, 0), ([256], [16000], True, 0), ([400], [3400], False, 0), ([700, 300], [3500, 3100], True, 29),
    ([1024, 0], [4000, 50], True, 0), ([1000, 24], [3301, 127], True, 0), ([200, 824], [5000, 17], False, 5),
    ([1, 1023], [9000, 1025], True, 0), ([500, 500, 536], [0, 9000, 100], True, 0), ([385, 639], [100, 5000], True, 0)])
def test_pairs_of_query_tiles(q_lens, k_lens, positions, pad, causal):
    c = Case(q_lens, k_lens, 128, positions, sum(q_lens) + sum(k_lens), pad=pad, before=sum(q_lens) % 2 == 1, device="cuda").cuda()
    got = c.run(causal)
    assert int(c.ws.buf[24:28].view(torch.int32)) == 256  # rows per item
    c.check(got, causal, heads=[0, 77, 127])
    for _ in range(2):
        again = c.run(causal, ws=c.ws)
        r = slice(c.cu_q[0], c.cu_q[-1])
        assert torch.equal(got[0][r], again[0][r]) and torch.equal(got[1][r], again[1][r])


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("positions", [True, False])
@pytest.mark.parametrize("q_len,k_lo,k_hi,B,H", [(1, 1, 700, 40, 16), (3, 130, 300, 64, 16), (150, 1, 500, 9, 128),
                                                 (90, 100, 200, 10, 64)])
def test_many_units_for_each_sm(q_len, k_lo, k_hi, B, H, causal, positions):
    k_lens = [k_lo + (k_hi - k_lo) * ((i * 37) % B) // (B - 1) for i in range(B)]
    c = Case([q_len] * B, k_lens, H, positions, B).cuda()
    got = c.run(causal)
    c.check(got, causal)
    for _ in range(4):
        again = c.run(causal, ws=c.ws)
        assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("q_lens,k_lens,H", [
    ([1], [20000], 1), ([1], [9000], 8), ([2, 1, 7], [100, 5000, 30], 4), ([130], [6000], 2), ([257], [9001], 1),
    ([1, 1], [64, 16384], 3), ([400, 3], [3000, 7000], 2)])
def test_keys_cut_into_pieces(q_lens, k_lens, H, causal):
    c = Case(q_lens, k_lens, H, True, sum(k_lens)).cuda()
    got = c.run(causal)
    assert int(c.ws.buf[36:40].view(torch.int32)) > 0  # some item is cut
    c.check(got, causal)
    again = c.run(causal, ws=c.ws)  # tickets and units are back where they were
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("q_lens,k_lens,H", [([5, 3], [100, 61], 3), ([1, 200], [7000, 333], 2), ([300, 260], [0, 500], 2)])
@pytest.mark.parametrize("dtype", [torch.float32, BF])
def test_joined_with_an_earlier_part(q_lens, k_lens, H, causal, dtype):
    c = Case(q_lens, k_lens, H, True, 17 + H, before=True).cuda()
    got = c.run(causal, out_dtype=dtype)
    c.check(got, causal)
    if dtype == torch.float32:  # in place
        want = got
        out, lse = c.before
        got = c.run(causal, out=out, lse=lse)
        assert got[0].data_ptr() == out.data_ptr()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_parts_of_the_keys_one_after_the_other():
    # keys in three calls, each joined with those before, against one call: the same formula's bounds
    c = Case([150, 20], [900, 300], 4, True, 5).cuda()
    cuts = [np.array([0, 0]), np.array([100, 300]), np.array([500, 300]), np.array([900, 300])]
    state = None
    for lo, hi in zip(cuts, cuts[1:]):
        part = Case([150, 20], list(hi - lo), 4, True, 5)
        pick = np.concatenate([np.arange(a, b) + off for a, b, off in zip(lo, hi, (0, 900))])
        for n in ("k_nope", "v"):
            setattr(part, n, getattr(c, n)[:, pick].contiguous())
        part.entries, part.q_nope, part.q_rope = c.entries[pick].contiguous(), c.q_nope, c.q_rope
        part.before = state
        state = part.cuda().run()
    c.ws = part.ws
    c.check(state)


@pytest.mark.parametrize("dtype", [torch.float32, BF])
def test_rows_outside_the_runs(dtype):
    # what lies before and behind the runs holds NaN and is neither used nor written
    for q_lens, k_lens in (([3, 9], [70, 200]), ([300, 40], [150, 5])):
        c = Case(q_lens, k_lens, 3, True, 8, pad=37).cuda()
        out = torch.full((c.nq, 3, 128), 5.0, dtype=dtype, device="cuda")
        lse = torch.full((c.nq, 3), 5.0, device="cuda")
        c.check(c.run(out=out, lse=lse))
        for t in (out, lse):
            assert bool((t[:37] == 5).all()) and bool((t[-37:] == 5).all())


def test_peaked_scores_and_no_lse():
    c = Case([200, 6], [3000, 900], 3, True, 12, spread=8.0).cuda()
    got = c.run(True, with_lse=False, out_dtype=BF)
    assert got[1] is None
    c.check(got, True)
    rising = Case([140], [1500], 2, False, 13).cuda()  # scores that grow along the keys: the reference moves
    rising.q_nope.fill_(0.25)
    rising.k_nope.copy_((torch.arange(1500, device="cuda") / 40.0).view(1, -1, 1).expand(2, 1500, 128).to(BF))
    rising.check(rising.run())


def test_no_write_outside_the_arrays():
    for q_lens, k_lens, H in (([1, 2], [9000, 30], 3), ([300], [700], 2)):
        c = Case(q_lens, k_lens, H, True, 3).cuda()
        ws = ops.CrossWorkspace(c.B, H, c.nq)
        g = [Guarded(ws.nbytes), Guarded(c.nq * H * 512), Guarded(c.nq * H * 4)]
        ws.buf = g[0].inner
        got = c.run(ws=ws, out=g[1].inner.view(torch.float32).view(c.nq, H, 128), lse=g[2].inner.view(torch.float32).view(c.nq, H))
        c.check(got)
        for b in g:
            b.check("cross attention")


def test_plan_serves_several_calls_and_a_captured_one():
    c = Case([5, 300, 1], [400, 900, 4000], 4, True, 31).cuda()
    want = c.run()
    c.check(want)
    call = lambda: ops.cross_attention(c.ws, c.q_nope, c.q_rope, c.entries, c.k_nope, c.v, c.scale)
    for _ in range(3):
        got = call()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.plan_cross(c.ws, *c.d_cu, c.nk)
        got = call()
    # other runs of the same rows, replayed
    for q_lens, k_lens in (([5, 300, 1], [400, 900, 4000]), ([100, 0, 206], [5000, 300, 0]), ([306, 0, 0], [1, 2, 5297])):
        c.cu_q = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
        c.cu_k = np.concatenate([[0], np.cumsum(k_lens)]).astype(np.int32)
        c.d_cu[0].copy_(torch.from_numpy(c.cu_q))
        c.d_cu[1].copy_(torch.from_numpy(c.cu_k))
        graph.replay()
        c.check(got)


def test_two_streams():
    a, b = Case([4, 260], [3000, 512], 4, True, 1).cuda(), Case([1, 1], [8000, 90], 16, False, 2).cuda()
    want = [c.run() for c in (a, b)]  # (workspaces are made, and zeroed, on the current stream)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        gb = b.run(ws=b.ws, stream=side)
        ga = a.run(ws=a.ws)
        torch.cuda.synchronize()
        for got, w in zip((ga, gb), want):
            assert torch.equal(got[0], w[0]) and torch.equal(got[1], w[1])


def test_runs_that_fall_or_lie_outside_are_recorded():
    c = Case([50, 60], [90, 100], 2, True, 3).cuda()
    for cu_q, cu_k in (([0, 50, 40], [0, 90, 190]), ([-3, 50, 110], [0, 90, 190]), ([0, 50, 400], [0, 90, 190]),
                       ([0, 50, 110], [0, 90, 5000]), ([0, 2 ** 31 - 1, -2 ** 31], [2 ** 31 - 1, -5, 190]),
                       ([110, 0, 110], [190, 0, 190])):
        ws = ops.CrossWorkspace(2, 2, c.nq)
        ops.plan_cross(ws, torch.tensor(cu_q, dtype=torch.int32, device="cuda"),
                       torch.tensor(cu_k, dtype=torch.int32, device="cuda"), c.nk)
        ops.cross_attention(ws, c.q_nope, c.q_rope, c.entries, c.k_nope, c.v, c.scale)
        assert ops.status(ws) == 5
    c.check(c.run())


def test_a_workspace_without_a_matching_plan():
    c = Case([50, 60], [90, 100], 2, True, 3).cuda()
    ws = ops.CrossWorkspace(2, 2, c.nq)
    with pytest.raises(ValueError, match="no plan"):
        ops.cross_attention(ws, c.q_nope, c.q_rope, c.entries, c.k_nope, c.v, c.scale)
    ws.total_k = c.nk
    ops.cross_attention(ws, c.q_nope, c.q_rope, c.entries, c.k_nope, c.v, c.scale)
    assert ops.status(ws) == 3
    ops.plan_cross(ws, *c.d_cu, c.nk + 1)
    ws.total_k = c.nk
    ops.cross_attention(ws, c.q_nope, c.q_rope, c.entries, c.k_nope, c.v, c.scale)
    assert ops.status(ws) == 3


def test_empty_and_refusals():
    c = Case([50, 60], [90, 100], 2, True, 3).cuda()
    ws = ops.CrossWorkspace(2, 2, 0)
    zero = torch.zeros(3, dtype=torch.int32, device="cuda")
    ops.plan_cross(ws, zero, c.d_cu[1], c.nk)
    out, lse = ops.cross_attention(ws, c.q_nope[:0], c.q_rope[:0], c.entries, c.k_nope, c.v, c.scale)
    assert out.shape == (0, 2, 128) and ops.status(ws) == 0
    ws = ops.CrossWorkspace(2, 2, c.nq)  # no key at all
    ops.plan_cross(ws, c.d_cu[0], zero, 0, causal=True)
    out, lse = ops.cross_attention(ws, c.q_nope, c.q_rope, c.entries[:0], c.k_nope[:, :0].contiguous(),
                                   c.v[:, :0].contiguous(), c.scale)
    assert bool((out == 0).all()) and bool((lse == -torch.inf).all()) and ops.status(ws) == 0
    c.run()
    good = dict(q_nope=c.q_nope, q_rope=c.q_rope, entries=c.entries, k_nope=c.k_nope, v=c.v, softmax_scale=c.scale)
    o32, l32 = torch.zeros(c.nq, 2, 128, device="cuda"), torch.zeros(c.nq, 2, device="cuda")
    for bad in (dict(q_rope=None), dict(entries=None), dict(q_nope=c.q_nope.float()), dict(v=c.v[:, :-1]),
                dict(k_nope=c.k_nope.transpose(0, 1)), dict(softmax_scale=0.0), dict(softmax_scale=float("inf")),
                dict(before=(o32, None)), dict(before=(o32.to(BF), l32)), dict(before=(o32, l32[:-1])),
                dict(out=o32.half()), dict(out=o32[:-1]), dict(lse=l32.to(BF)), dict(out_dtype=torch.float16),
                dict(q_nope=c.q_nope.cpu())):
        with pytest.raises((ValueError, ops.MlaError)):
            ops.cross_attention(c.ws, **{**good, **bad})
    for bad in ((c.d_cu[0][:-1], c.d_cu[1]), (c.d_cu[0].long(), c.d_cu[1]), (c.d_cu[0].cpu(), c.d_cu[1])):
        with pytest.raises(ValueError):
            ops.plan_cross(c.ws, *bad, c.nk)


@pytest.mark.parametrize("q_lens,k_lens,H,causal", [([1024], [1024], 19, False), ([1024], [2048], 19, False),
                                                    ([256], [8192], 128, True), ([128] * 9, [640] * 9, 16, True)])
def test_items_that_fill_the_sms_stay_whole(q_lens, k_lens, H, causal):
    c = Case(q_lens, k_lens, H, True, 9 + H, device="cuda").cuda()
    got = c.run(causal)
    assert int(c.ws.buf[36:40].view(torch.int32)) == 0  # cut items
    c.check(got, causal, heads=[0, H // 2, H - 1])


@pytest.mark.parametrize("sms", [1, 7, 76, 1000])
def test_plans_for_other_numbers_of_sms(sms):
    c = Case([130, 1, 300], [6000, 9000, 700], 4, True, 40, before=True).cuda()
    ws = ops.CrossWorkspace(c.B, c.H, c.nq, num_sms=sms)
    c.check(c.run(True, ws=ws), True)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("B", [511, 513, 1025, 3000])
def test_many_runs(B, causal):
    g = np.random.default_rng(B)
    q_lens, k_lens = g.integers(0, 4, B), g.integers(0, 90, B)
    q_lens[B // 2], k_lens[B // 3], k_lens[B // 2] = 300, 3000, 5000
    c = Case(q_lens, k_lens, 2, True, B, pad=3).cuda()
    c.check(c.run(causal), causal)


def test_far_keys_and_far_queries():
    # keys, values, queries and results whose places pass 2^31 elements: the last head's, and the last rows'
    c = Case([3, 130], [139_000, 1300], 128, True, 41, device="cuda").cuda()
    assert c.k_nope.numel() > 2 ** 31
    c.check(c.run(True), True, heads=[0, 127])
    del c
    c = Case([131_500, 130], [40, 200], 128, False, 42, device="cuda").cuda()
    assert c.q_nope.numel() > 2 ** 31
    got = c.run(True)
    assert ops.status(c.ws) == 0
    last = Case([130], [200], 128, False, 43, device="cuda").cuda()  # the last run by itself
    last.q_nope, last.k_nope = c.q_nope[-130:].contiguous(), c.k_nope[:, -200:].contiguous()
    last.v = c.v[:, -200:].contiguous()
    want = last.run(True)
    last.check(want, True, heads=[0, 127])
    assert torch.equal(got[0][-130:], want[0]) and torch.equal(got[1][-130:], want[1])
    assert bool((got[1][:100] == -torch.inf).all()) and bool((got[0][:100] == 0).all())  # they see no key


def test_two_graphs_share_a_workspace():
    a = Case([5, 300], [4000, 900], 4, True, 44).cuda()
    b = Case([300, 5], [30, 5000], 4, True, 45).cuda()
    a.run()
    ws = a.ws
    b.run(ws=ws)
    graphs, got = [], []
    for c, causal in ((a, False), (b, True)):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            got.append(c.run(causal, ws=ws))
    for i in (0, 1, 1, 0, 1, 0, 0):
        graphs[i].replay()
        (a, b)[i].check(got[i], causal=i == 1)


@pytest.mark.parametrize("q_lens,k_lens,H,causal,sms,pays", [
    ([512] * 5, [3000] * 5, 32, False, 0, True), ([1001], [9193], 128, True, 0, True), ([512], [4096], 40, True, 0, True),
    ([130, 129], [2000, 2000], 16, False, 7, True), ([300], [5000], 3, True, 2, True),
    # 11 units of 24 + 2 key tiles: three rounds on 4 SMs end at 78, in pieces they would at 71.5 + 5 + 8
    ([1], [3000], 11, True, 4, False)])
def test_the_first_heads_stay_whole(q_lens, k_lens, H, causal, sms, pays):
    c = Case(q_lens, k_lens, H, True, 50 + H, before=H < 100, device="cuda").cuda()
    ws = ops.CrossWorkspace(c.B, H, c.nq, num_sms=sms)
    got = c.run(causal, ws=ws)
    whole, cut = int(ws.buf[48:52].view(torch.int32)), int(ws.buf[36:40].view(torch.int32))
    assert 0 < whole < H and cut > 0 if pays else whole == H and cut == 0
    c.check(got, causal, heads=sorted({0, whole - 1, min(whole, H - 1), H - 1}))
    again = c.run(causal, ws=ws)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


@pytest.mark.parametrize("causal", [False, True])
def test_more_pieces_than_are_put_in_order(causal):
    c = Case([1] * 24, [48_000 + 16 * i for i in range(24)], 1, False, 51, device="cuda").cuda()
    ws = ops.CrossWorkspace(c.B, c.H, c.nq, num_sms=2000)
    got = c.run(causal, ws=ws)
    assert int(ws.buf[32:36].view(torch.int32)) > 2048  # pieces
    c.check(got, causal)


def test_no_queries_in_any_run():
    c = Case([0, 0], [300, 5], 2, True, 52).cuda()
    ws = ops.CrossWorkspace(2, 2, 7)  # seven rows that no run has
    ops.plan_cross(ws, *c.d_cu, c.nk)
    q = torch.full((7, 2, 192), torch.nan, dtype=BF, device="cuda")
    out, lse = torch.full((7, 2, 128), 5.0, device="cuda"), torch.full((7, 2), 5.0, device="cuda")
    ops.cross_attention(ws, q[..., :128].contiguous(), q[..., 128:].contiguous(), c.entries, c.k_nope, c.v, c.scale, out=out,
                        lse=lse)
    assert ops.status(ws) == 0 and bool((out == 5).all()) and bool((lse == 5).all())


@pytest.mark.parametrize("q_lens,k_lens,H,causal", [([256] * 9, [2000] * 9, 16, False), ([2048], [8192], 16, True),
                                                    ([512, 700, 300, 536], [3000, 2400, 3600, 3000], 16, True)])
def test_pairs_of_query_tiles_that_end_sooner(q_lens, k_lens, H, causal):
    c = Case(q_lens, k_lens, H, True, 53 + H, before=causal, device="cuda").cuda()
    got = c.run(causal)
    assert int(c.ws.buf[24:28].view(torch.int32)) == 256  # rows per item
    c.check(got, causal, heads=[0, H // 2, H - 1])


@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("q,k,H", [(600, 13, 40), (257, 130, 64), (130, 1, 128)])
def test_joined_many_queries_few_keys(q, k, H, dtype):
    c = Case([q, 1, q, 0, q + 7, q], [k, k, 0, k, k + 1, k], H, True, 54 + q, before=True, device="cuda").cuda()
    got = c.run(out_dtype=dtype)
    c.check(got, heads=[0, H // 2, H - 1])
    if dtype == torch.float32:  # in place
        want, (out, lse) = got, c.before
        got = c.run(out=out, lse=lse)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_a_workspace_of_any_content():
    # the first plan in a workspace sets its status word up, whatever the memory held; later ones keep an unread error
    c = Case([5, 200], [3000, 129], 3, True, 60).cuda()
    want = c.run(True)
    c.check(want, True)
    bad = torch.tensor([0, 150, 40], dtype=torch.int32, device="cuda")
    call = lambda ws: ops.cross_attention(ws, c.q_nope, c.q_rope, c.entries, c.k_nope, c.v, c.scale)
    for fill in (0xFF, 0x01, 0x7F):
        ws = ops.CrossWorkspace(c.B, c.H, c.nq)
        ws.buf.fill_(fill)
        got = c.run(True, ws=ws)
        assert ops.status(ws) == 0
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        ws.buf.fill_(fill)
        ops.plan_cross(ws, bad, c.d_cu[1], c.nk, causal=True)
        call(ws)
        got = c.run(True, ws=ws)  # another plan, and its call, before anybody asks
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert ops.status(ws) == 5 and ops.status(ws) == 0
        c.run(True, ws=ws)
        assert ops.status(ws) == 0
        ops.plan_cross(ws, bad, c.d_cu[1], c.nk, causal=True)
        assert ops.status(ws) == 5


@pytest.mark.parametrize("q,k,H,rows", [(19456, 16384, 1, 128), (4864, 65536, 8, 256)])
def test_waits_for_long_units_have_longer_limits(q, k, H, rows):
    # one role waits for as long as another one's unit takes: 128 key tiles of some 2,000 cycles, 512 of 3,600, while
    # the limit by itself is 50,000
    c = Case([q], [k], H, False, 61, device="cuda").cuda()
    want = c.run()
    assert int(c.ws.buf[24:28].view(torch.int32)) == rows and int(c.ws.buf[36:40].view(torch.int32)) == 0  # none is cut
    ops.set_wait_limit(50_000)
    try:
        got = c.run(ws=c.ws)
        assert ops.status(c.ws) == 0
    finally:
        ops.set_wait_limit(0)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("q_lens,k_lens,H,causal,before,kind", [
    ([5, 200], [3000, 129], 3, True, False, "cut"), ([70, 1], [100, 0], 2, False, True, "whole"),
    ([1001], [3400], 128, True, False, "pairs"), ([512], [16384], 128, False, True, "pairs")])
def test_a_wait_that_runs_out(q_lens, k_lens, H, causal, before, kind):
    # the MMA warps wait for a barrier that nothing completes: the call is recorded, its kernels return and write inside
    # their arrays, and the plan has to be made again
    c = Case(q_lens, k_lens, H, True, 62, before=before, device="cuda").cuda()
    want = c.run(causal)
    assert ops.status(c.ws) == 0
    assert (int(c.ws.buf[24:28].view(torch.int32)) == 256) == (kind == "pairs")
    assert kind != "cut" or int(c.ws.buf[36:40].view(torch.int32)) > 0
    ws = ops.CrossWorkspace(c.B, H, c.nq)
    g = [Guarded(ws.nbytes), Guarded(c.nq * H * 512), Guarded(c.nq * H * 4)]
    ws.buf = g[0].inner
    out, lse = g[1].inner.view(torch.float32).view(c.nq, H, 128), g[2].inner.view(torch.float32).view(c.nq, H)
    ops.plan_cross(ws, *c.d_cu, c.nk, causal=causal)
    call = lambda: ops.cross_attention(ws, c.q_nope, c.q_rope, c.entries, c.k_nope, c.v, c.scale, before=c.before, out=out, lse=lse)
    ops.set_wait_limit(2_000_000)  # about a millisecond
    ops.inject_stall(True)
    try:
        call()
        assert ops.status(ws) == 6
    finally:
        ops.inject_stall(False)
        ops.set_wait_limit(0)
    out.fill_(5)
    lse.fill_(5)
    call()  # without a new plan: refused, and nothing written
    assert ops.status(ws) == 3
    assert bool((out == 5).all()) and bool((lse == 5).all())
    for _ in range(2):
        got = c.run(causal, ws=ws, out=out, lse=lse)
        assert ops.status(ws) == 0 and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for b in g:
        b.check("after a wait that ran out")


def test_the_plan_says_how_many_sms_may_be_used():
    # 320 units of one length take 3 rounds of 152 SMs, and 40 of 8
    c = Case([2560], [1024], 16, True, 63, device="cuda").cuda()
    want = c.run()

    def took(sms):
        ws = ops.CrossWorkspace(c.B, c.H, c.nq, num_sms=sms)
        c.check(c.run(ws=ws), heads=[0, 15])
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        times = []
        for _ in range(3):
            a.record()
            ops.cross_attention(ws, c.q_nope, c.q_rope, c.entries, c.k_nope, c.v, c.scale, out=want[0], lse=want[1])
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b))
        return min(times)

    assert took(8) > 4 * took(0)


def test_the_largest_limit_of_a_wait():
    c = Case([5, 200], [3000, 129], 3, True, 64).cuda()
    ops.set_wait_limit(2 ** 63 - 1)
    try:
        c.check(c.run())
    finally:
        ops.set_wait_limit(0)
