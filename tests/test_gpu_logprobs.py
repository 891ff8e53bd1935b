"""Token log probabilities on the GPU against a 64-bit restatement; ranks and alternatives have to be
equal.

Bounds (u = 2^-24).  A thread adds at most K = ceil(V / 256) + 16 of the row's terms one after the
other (a unit's 8 at most beyond its even share), 13 joins follow (5 shuffles, 8 warps, 3 of them
again for a cluster's 8 CTAs), each a factor and a sum of both sides: (K + 64) u of the sum.  A term
2^t has the approximation's 2^-22 and t's own error: the difference, two roundings of its factor and
the product, 4 u |t|, weighted by p: 4 u ln 2 E|t|, with E|t| the mean distance below the maximum.  So
the sum is off by r = (K + 64) u + 2^-22 + 4 u B relative (B: E|t| in nats), and
  log p   by r + 2 u (token's distance below the maximum) + 4 u ln s + u |log p| <= r + 8 u (|log p| + ln s),
  entropy by r + B (2 r + 4 u) + 4 u (ln s + B): w has the sum's errors once more, then the quotient."""
import numpy as np
import pytest
import torch

from guards import Guarded
from mla_latent_kv_17_gb300 import ops
import prompt_ref

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from mla_latent_kv_17_gb300 import build
    build.build()
    ops.lib()


def check(x, tok, top, scale, got):
    N, V = x.shape
    lp, h, rank, ids, alt, below, logs = prompt_ref.logprobs(x.double().cpu().numpy(), tok.cpu().numpy(), scale, top)
    r = (-(-V // 256) + 16 + 64) * U + 2.0 ** -22 + 4 * U * below
    num = lambda t: t.double().cpu().numpy()

    def near(a, want, bound, what):
        same = (a == want) | (np.isnan(a) & np.isnan(want))
        with np.errstate(invalid="ignore"):
            ok = same | (np.abs(a - want) <= bound)
        assert ok.all(), (what, a[~ok][:4], want[~ok][:4])

    fin = lambda v: np.where(np.isfinite(v), np.abs(v), 0.0)
    near(num(got[0]), lp, r + 8 * U * (fin(lp) + logs), "logprob")
    near(num(got[1]), h, r + below * (2 * r + 4 * U) + 4 * U * (logs + below), "entropy")
    assert np.array_equal(got[2].cpu().numpy(), rank), "rank"
    if top == 0:
        assert got[3] is None and got[4] is None
        return
    assert np.array_equal(got[3].cpu().numpy(), ids), "top tokens"
    near(num(got[4]), alt, r[:, None] + 8 * U * (fin(alt) + logs[:, None]), "top logprobs")


def make(n, v, dtype, seed, spread=3.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (spread * torch.randn(n, v, generator=g, device="cuda")).to(TYPES[dtype])
    tok = torch.randint(0, v, (n,), generator=g, device="cuda").to(torch.int32)
    best = x.float().argmax(1).to(torch.int32)
    return x, torch.where(torch.arange(n, device="cuda") % 3 == 1, best, tok)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("n,v,top", [(1, 1, 1), (3, 2, 2), (2, 7, 5), (5, 8, 64), (4, 9, 3), (3, 127, 20), (70, 1000, 64),
                                     (2, 4099, 5), (3, 32001, 20), (400, 1531, 0), (1, 131072, 20), (20, 131072, 5),
                                     (2, 262147, 64), (330, 8193, 7), (1, 600000, 1)])
def test_logprobs(n, v, top, dtype):
    x, tok = make(n, v, dtype, n * 7 + v)
    check(x, tok, top, 1.0, ops.token_logprobs(x, tok, top=top))


@pytest.mark.parametrize("scale", [0.01, 0.5, 1.7, 40.0])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_scales(dtype, scale):
    x, tok = make(4, 5003, dtype, 3)
    check(x, tok, 10, float(np.float32(scale)), ops.token_logprobs(x, tok, top=10, scale=scale))


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_ties(dtype):
    # a few different values only, equal ones to the lower token; signed zeros are equal; all the same
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randint(-2, 3, (6, 9001), generator=g, device="cuda").to(TYPES[dtype])
    x[1] = 0.5
    x[2] = torch.where(torch.rand(9001, generator=g, device="cuda") < 0.5, 0.0, -0.0).to(TYPES[dtype])
    x[3, 4000:] = 7.0
    x[4] = torch.arange(9001, device="cuda").div(64).floor().to(TYPES[dtype])  # rising
    x[5] = -x[4]
    tok = torch.tensor([5, 0, 9000, 4001, 8999, 3], dtype=torch.int32, device="cuda")
    for top in (1, 20, 64):
        check(x, tok, top, 1.0, ops.token_logprobs(x, tok, top=top))
    one = torch.full((2, 140001), -3.0, device="cuda", dtype=TYPES[dtype])  # shared by a cluster
    tok = torch.tensor([140000, 70000], dtype=torch.int32, device="cuda")
    check(one, tok, 9, 1.0, ops.token_logprobs(one, tok, top=9))


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("v", [40, 5000, 131072])
def test_masked(dtype, v):
    x, tok = make(8, v, dtype, v)
    g = torch.Generator(device="cuda").manual_seed(2)
    x[0, torch.rand(v, generator=g, device="cuda") < 0.5] = -torch.inf
    x[1, 3:] = -torch.inf             # fewer tokens left than alternatives asked for
    x[2] = -torch.inf                 # none left
    x[3, 1:] = -torch.inf             # one left
    x[4, :v - 1] = -torch.inf         # the last one
    x[5, tok[5].long()] = -torch.inf  # the given token
    x[6] = -torch.inf
    x[6, v // 2] = 1.0
    tok[1], tok[2], tok[3], tok[4], tok[6] = 7, 5, 0, v - 1, v // 2 + 1
    check(x, tok, 20, 1.0, ops.token_logprobs(x, tok, top=20))


def test_the_types_lowest_and_largest_values():
    for dtype in TYPES.values():
        big = torch.finfo(dtype).max
        x = torch.full((3, 3000), -big, dtype=dtype, device="cuda")  # masks of the lowest value
        x[0, 17] = 2.0
        x[1, 2000:2010] = torch.arange(10, device="cuda").to(dtype)
        x[2, 5] = big if dtype == torch.float16 else 1e30
        tok = torch.tensor([17, 2009, 5], dtype=torch.int32, device="cuda")
        got = ops.token_logprobs(x, tok, top=3)
        check(x[:2], tok[:2], 3, 1.0, [t[:2] for t in got])
        assert got[0][2] == 0 and got[1][2] == 0 and got[2][2] == 0
        assert got[3][2].tolist() == [5, 0, 1]
    for dtype in TYPES.values():
        # the lowest value and -inf together; values so large that 160 below them is not a value of the type
        low, inf = torch.finfo(dtype).min, torch.inf
        x = torch.full((2, 6000), -inf, dtype=dtype, device="cuda")
        x[0, 1000:1007] = low
        x[1, 50:53] = 6e4 if dtype == torch.float16 else 1e12
        tok = torch.tensor([1003, 52], dtype=torch.int32, device="cuda")
        check(x, tok, 10, 1.0, ops.token_logprobs(x, tok, top=10))
    x = torch.zeros(1, 50000, device="cuda")  # nearly certain: both terms of the entropy are small
    x[0, 33333] = 30.0
    tok = torch.tensor([33333], dtype=torch.int32, device="cuda")
    check(x, tok, 2, 1.0, ops.token_logprobs(x, tok, top=2))


def test_rows_without_a_token_and_bad_tokens():
    x, tok = make(5, 700, "bf16", 9)
    tok[1], tok[2], tok[4] = -1, 700, 2 ** 31 - 1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = ops.token_logprobs(x, tok, top=4, device_status=status)
    check(x, tok, 4, 1.0, got)
    assert int(status) == 5 and got[0][1] == 0 and bool(got[0][2].isnan()) and got[2].tolist()[1:3] == [-1, -1]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_strides(dtype):
    wide, _ = make(6, 40050, dtype, 11)
    tok = torch.tensor([0, 1, 39999, 20000, 5, 39990], dtype=torch.int32, device="cuda")
    for lo in (0, 1, 3, 4, 7, 8, 33):  # rows that start anywhere
        x = wide[:, lo:lo + 40000]
        check(x, tok, 6, 1.0, ops.token_logprobs(x, tok, top=6))
        check(x[::2], tok[::2].contiguous(), 6, 1.0, ops.token_logprobs(x[::2], tok[::2].contiguous(), top=6))
    x = wide[2:3].expand(6, 40050)  # one row, several tokens
    check(x, tok, 6, 1.0, ops.token_logprobs(x, tok, top=6))


def test_far_rows():
    # row offsets past 2^31 elements
    far = 2 ** 31 + 24
    buf = torch.empty(far + 5000, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((2, 5000), (far, 1))
    y, tok = make(2, 5000, "bf16", 4)
    x.copy_(y)
    check(y, tok, 8, 1.0, ops.token_logprobs(x, tok, top=8))


def test_no_write_outside_the_outputs():
    N, V, top = 3, 1001, 5
    x, tok = make(N, V, "bf16", 21)
    bufs = [Guarded(n) for n in (4 * N, 4 * N, 4 * N, 4 * N * top, 4 * N * top)]
    st = ops.lib().mla_token_logprobs(x.data_ptr(), 0, V, N, V, tok.data_ptr(), 1.0, top, *[b.inner.data_ptr() for b in bufs],
                                      0, torch.cuda.current_stream().cuda_stream)
    assert st == 0
    torch.cuda.synchronize()
    for b in bufs:
        b.check("token_logprobs")
    i, f = torch.int32, torch.float32
    got = [b.inner.view(t) for b, t in zip(bufs, (f, f, i, i, f))]
    check(x, tok, top, 1.0, got[:3] + [t.view(N, top) for t in got[3:]])
    # what may be left out is left out
    only = torch.empty(N, device="cuda")
    st = ops.lib().mla_token_logprobs(x.data_ptr(), 0, V, N, V, tok.data_ptr(), 1.0, 0, only.data_ptr(), 0, 0, 0, 0, 0,
                                      torch.cuda.current_stream().cuda_stream)
    assert st == 0 and torch.equal(only, got[0])


def test_captured_on_a_stream_and_empty():
    x, tok = make(9, 33000, "bf16", 5)
    want = ops.token_logprobs(x, tok, top=7)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    on_side = ops.token_logprobs(x, tok, top=7, stream=side)
    side.synchronize()
    for a, b in zip(on_side, want):  # the same bits wherever it runs
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = ops.token_logprobs(x, tok, top=7)
    for seed in (6, 7):
        y, t = make(9, 33000, "bf16", seed)
        x.copy_(y)
        tok.copy_(t)
        graph.replay()
        check(y, t, 7, 1.0, got)
    e = ops.token_logprobs(x[:0], tok[:0].contiguous(), top=7)
    assert e[0].shape == (0,) and e[3].shape == (0, 7)


def test_refusals():
    x, tok = make(2, 100, "fp32", 5)
    for bad in (dict(top=65), dict(top=-1), dict(scale=0.0), dict(scale=float("nan")), dict(scale=float("inf")),
                dict(scale=-1.0)):
        with pytest.raises((ValueError, ops.MlaError)):
            ops.token_logprobs(x, tok, **bad)
    for a, b in ((x.double(), tok), (x.t(), tok), (x[0], tok), (x, tok.long()), (x, tok[:1]), (x, tok.cpu())):
        with pytest.raises(ValueError):
            ops.token_logprobs(a, b)
