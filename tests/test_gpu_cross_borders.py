"""Attention to key runs of another length: no key lost or counted twice at the borders of key tiles, pieces, runs and
causal limits, against 64 bits.

The products of the scores are whole numbers here, so a score d is exact, and a log-sum-exp is off by (u = 2^-24)
  4 u S: the factor's two roundings (relative to the score), one of the exponent's (it lies within 2 S nats of the
         reference), S the largest |score|;
  2^-22 + (40 + 2 tiles) u: the exponential, the additions of a thread's 128 / 8 pairs, of its sums and of the tiles;
  2^-21 + groups (2^-22 + 2 u) + 4 u |lse|: joined parts (their own lse's rounding twice, a factor per group of
         four parts), with groups <= tiles / 16 + 2, as parts have at least four key tiles;
  6 u |lse|: log2, the sum with the reference, ln 2 and the product.
A missing key moves it by its weight: about 1.5 bounds for one of 20,000 alike, far more at the borders below."""
import pytest
import torch

from mla_latent_kv_17_gb300 import ops
from test_gpu_cross import Case, U

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from mla_latent_kv_17_gb300 import build
    build.build()
    ops.lib()


def bound(keys, largest, lse):
    tiles = -(-keys // 128)
    groups = tiles / 16 + 2
    return (4 * U * largest + 2.0 ** -22 + (40 + 2 * tiles) * U + 2.0 ** -21 + groups * (2.0 ** -22 + 2 * U)
            + 10 * U * torch.where(lse.isfinite(), lse.abs(), 0.0))


def near(got, want, by, what):
    ok = (got == want) | ((got - want).abs() <= by)
    assert bool(ok.all()), (what, got[~ok][:4], want[~ok][:4])


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("q_lens,k_lens,H,positions", [
    ([1], [20000], 1, True), ([1], [9000], 8, False), ([2, 1, 7], [100, 5000, 30], 4, True), ([130], [6000], 2, True),
    ([257], [9001], 1, True), ([1, 1], [64, 16384], 3, False), ([400, 3], [3000, 7000], 2, True),
    ([300, 129], [4000, 2500], 96, True), ([150, 3, 700], [1000, 40, 900], 5, False)])
def test_sums_of_weights(q_lens, k_lens, H, positions, causal):
    c = Case(q_lens, k_lens, H, positions, 70 + H, device="cuda").cuda()
    for t in (c.q_nope, c.q_rope, c.k_nope, c.entries):  # -1, 0 and 1
        t.copy_(t.sign() * (t.abs() > 0.5))
    out, lse = c.run(causal)
    c.check((out, lse), causal, heads=sorted({0, H - 1}))
    for b in range(c.B):
        rows, keys = slice(c.cu_q[b], c.cu_q[b + 1]), slice(c.cu_k[b], c.cu_k[b + 1])
        n, m = q_lens[b], k_lens[b]
        hidden = torch.ones(n, m, dtype=torch.bool, device="cuda").triu(m - n + 1) if causal else None
        for h in range(H):
            d = c.q_nope[rows, h].double() @ c.k_nope[h, keys].double().T
            if positions:
                d += c.q_rope[rows, h].double() @ c.entries[keys, 512:].double().T
            d *= c.scale
            largest = float(d.abs().max())
            if hidden is not None:
                d[hidden] = -torch.inf
            want = d.logsumexp(1)
            near(lse[rows, h].double(), want, bound(m, largest, want), (b, h))


@pytest.mark.parametrize("q_lens,k_lens,H,causal,rows,cut", [
    ([3, 130], [9001, 5000], 16, False, 128, True), ([3, 130], [9001, 5000], 16, True, 128, True),
    ([1], [16384], 8, False, 128, True), ([2048], [8192], 16, True, 256, None), ([256] * 3, [2000] * 3, 16, True, 128, None),
    ([300], [5003], 32, True, 128, True)])
def test_weight_on_the_keys_at_borders(q_lens, k_lens, H, causal, rows, cut):
    # Each head's weight lies on one key at a border (e^20 against 1), and e^10 on another for all heads: a tile's first
    # or last key, a run's, or a query's last one
    c = Case(q_lens, k_lens, H, True, 80 + H, device="cuda").cuda()
    c.scale = 20 / 128  # (exact)
    for t in (c.q_nope, c.q_rope):
        t.fill_(1)
    most = max(k_lens)
    at = sorted({k for t in range(0, most + 1, 128) for k in (t - 1, t)} | {most - 1, most - 2})
    at += [m - 1 for m in k_lens] + [m - n + i for n, m in zip(q_lens, k_lens) for i in (0, n // 2, n - 1)]
    at = sorted({k for k in at if 0 <= k < most})
    for i in range(0, len(at), H):
        c.k_nope.zero_()
        c.entries[:, 512:].zero_()
        mine = [at[(i + h) % len(at)] for h in range(H)]
        for b in range(c.B):
            k0, m = int(c.cu_k[b]), k_lens[b]
            for h, k in enumerate(mine):
                c.k_nope[h, k0 + k % m] = 1
            c.entries[k0 + at[(i + 5) % len(at)] % m, 512:] = 1
        out, lse = c.run(causal)
        assert ops.status(c.ws) == 0 and int(c.ws.buf[24:28].view(torch.int32)) == rows
        if cut is not None:
            assert (int(c.ws.buf[36:40].view(torch.int32)) > 0) == cut
        for b in range(c.B):
            n, m = q_lens[b], k_lens[b]
            r, keys = slice(c.cu_q[b], c.cu_q[b + 1]), slice(c.cu_k[b], c.cu_k[b + 1])
            s = c.scale * (c.k_nope[:, keys].double().sum(2) + c.entries[keys, 512:].double().sum(1))
            last = torch.arange(n, device="cuda") + m - n if causal else torch.full((n,), m - 1, device="cuda")
            some = last >= 0
            want = torch.where(some, s.logcumsumexp(1)[:, last.clamp(min=0)], -torch.inf).T
            near(lse[r].double(), want, bound(m, 30.0, want), (b, i))
            # the weighted values: sums over the seen keys, under the largest score of all (e^30 / e^0: no underflow)
            v = c.v[:, keys].double()
            w = (s - 30).exp().unsqueeze(2)
            total = w.cumsum(1)[:, last.clamp(min=0)]
            mean = ((w * v).cumsum(1)[:, last.clamp(min=0)] / total).transpose(0, 1)
            size = ((w * v.abs()).cumsum(1)[:, last.clamp(min=0)] / total).transpose(0, 1)
            some = some.view(-1, 1, 1)
            near(out[r].double(), torch.where(some, mean, 0.0),
                 torch.where(some, (2.0 ** -8 + 2.0 ** -20 + (60 + m) * U + 4 * U * 30) * size, 0.0), (b, i, "out"))
