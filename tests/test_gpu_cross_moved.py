"""Attention to key runs of another length whose starts fall or lie outside: the error is recorded, the runs are moved
up or in as documented, and nothing is written outside them."""
import numpy as np
import pytest
import torch

from guards import Guarded
from mla_latent_kv_17_gb300 import ops
from test_gpu_cross import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from mla_latent_kv_17_gb300 import build
    build.build()
    ops.lib()


def moved(cu, total):
    """Where starts that fall or lie outside are taken to be."""
    return np.maximum.accumulate(np.clip(cu.astype(np.int64), 0, total)).astype(np.int32)


def run_moved(c, cu_q, cu_k, causal):
    nq, nk, H = c.nq, c.nk, c.H
    c.cu_q, c.cu_k = moved(cu_q, nq), moved(cu_k, nk)
    assert (c.cu_q != cu_q).any() or (c.cu_k != cu_k).any()
    c.d_cu = torch.from_numpy(cu_q).cuda(), torch.from_numpy(cu_k).cuda()
    ws = ops.CrossWorkspace(c.B, H, nq)
    g = [Guarded(ws.nbytes), Guarded(nq * H * 512), Guarded(nq * H * 4)]
    ws.buf = g[0].inner
    out, lse = g[1].inner.view(torch.float32).view(nq, H, 128).fill_(5), g[2].inner.view(torch.float32).view(nq, H).fill_(5)
    got = c.run(causal, ws=ws, out=out, lse=lse)
    assert ops.status(ws) == 5
    c.check(got, causal)
    for t in (out, lse):  # rows of no run
        assert bool((t[:c.cu_q[0]] == 5).all()) and bool((t[c.cu_q[-1]:] == 5).all())
    for b in g:
        b.check("runs that fall or lie outside")


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("cu_q,cu_k", [
    ([0, 50, 40], [0, 90, 190]), ([-3, 50, 110], [0, 90, 190]), ([0, 50, 400], [0, 90, 190]), ([0, 50, 110], [0, 90, 5000]),
    ([0, 2 ** 31 - 1, -2 ** 31], [2 ** 31 - 1, -5, 190]), ([110, 0, 110], [190, 0, 190]), ([20, 90, 60], [150, 30, 170]),
    ([5, 105, 110], [7, -9, 130])])
def test_two_runs_that_fall_or_lie_outside(cu_q, cu_k, causal):
    c = Case([50, 60], [90, 100], 2, True, 3).cuda()
    run_moved(c, np.array(cu_q, np.int32), np.array(cu_k, np.int32), causal)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("B", [513, 700, 1100])
def test_many_runs_that_fall_or_lie_outside(B, causal):
    # a fall in the first 512 runs (the plan takes that many at a time), across their end, and behind it
    g = np.random.default_rng(B)
    q_lens, k_lens = g.integers(0, 5, B), g.integers(0, 60, B)
    q_lens[B // 2], k_lens[B // 3], k_lens[512] = 300, 3000, 700
    c = Case(q_lens, k_lens, 2, True, B).cuda()
    good = c.cu_q.copy(), c.cu_k.copy()

    def case(edit):
        q, k = good[0].copy(), good[1].copy()
        edit(q, k)
        run_moved(c, q, k, causal)

    def early(q, k):
        q[100], k[200] = q[130], k[260]

    def across(q, k):  # the largest start of the first 512 runs reaches into the next
        q[511], k[510] = q[min(B, 540)], k[min(B, 515)]

    def late(q, k):
        q[B - 3], k[B - 2], k[B] = -7, c.nk + 9, 0

    def all_of_it(q, k):
        early(q, k)
        across(q, k)
        late(q, k)
        q[512], k[512] = 2 ** 31 - 1, -2 ** 31

    for edit in (early, across, late, all_of_it):
        case(edit)
