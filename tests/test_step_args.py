"""Refusals of the speculative step's calls: what the C ABI and the binding reject before
anything is enqueued (no GPU needed)."""
import ctypes
import math

import pytest
import torch

from mla_latent_kv_17_gb300 import build as mbuild
from mla_latent_kv_17_gb300 import ops

P = ctypes.c_void_p
OK, INVALID, UNSUPPORTED = 0, 1, 2
A = 0x10000  # a 16-byte-aligned address; nothing is read in a refused call


@pytest.fixture(scope="module", autouse=True)
def _built():
    mbuild.build()


def _rope(**kw):
    d = dict(x=A, xt=192 * 4, xh=192, N=3, H=4, dp=128, dr=64, layout=0, pos=A, freqs=A, m=1.0, op=A, pt=512, ph=128,
             orr=A, rt=256, rh=64)
    d.update(kw)
    return ops.lib().mla_rope(P(d["x"]), d["xt"], d["xh"], d["N"], d["H"], d["dp"], d["dr"], d["layout"], P(d["pos"]),
                              P(d["freqs"]), d["m"], P(d["op"]), d["pt"], d["ph"], P(d["orr"]), d["rt"], d["rh"], P(0))


@pytest.mark.parametrize("kw", [dict(x=0), dict(pos=0), dict(freqs=0), dict(orr=0), dict(N=-1), dict(H=0), dict(dp=-8),
                                dict(dr=0), dict(dr=63), dict(layout=2), dict(m=math.nan), dict(m=math.inf),
                                dict(x=A + 1), dict(op=A + 1), dict(orr=A + 3)])
def test_rope_refuses(kw):
    assert _rope(**kw) == INVALID


def test_rope_limits():
    assert _rope(dr=2050) == UNSUPPORTED and _rope(dp=8200) == UNSUPPORTED
    assert _rope(N=0, x=0, pos=0) == OK  # nothing to do


def _write(**kw):
    d = dict(cache=A, kind=0, pages=4, bt=A, B=2, mp=2, req=A, pos=A, kv=A, stride=576, N=5, w=0, eps=1e-6, freqs=0,
             rp=0, layout=0, m=1.0)
    d.update(kw)
    return ops.lib().mla_cache_write(P(d["cache"]), d["kind"], d["pages"], P(d["bt"]), d["B"], d["mp"], P(d["req"]),
                                     P(d["pos"]), P(d["kv"]), d["stride"], d["N"], P(d["w"]), d["eps"], P(d["freqs"]),
                                     P(d["rp"]), d["layout"], d["m"], P(0), P(0))


@pytest.mark.parametrize("kw", [dict(cache=0), dict(bt=0), dict(pos=0), dict(kv=0), dict(kind=2), dict(pages=0),
                                dict(B=0), dict(mp=0), dict(N=-1), dict(stride=575), dict(stride=580), dict(kv=A + 2),
                                dict(cache=A + 8), dict(req=0), dict(w=A + 2), dict(w=A, eps=-1.0),
                                dict(w=A, eps=math.nan), dict(layout=7), dict(m=math.inf)])
def test_cache_write_refuses(kw):  # (req=0: five tokens, two requests)
    assert _write(**kw) == INVALID


def test_cache_write_of_nothing():
    assert _write(N=0, kv=0, pos=0) == OK


def _read(**kw):
    d = dict(cache=A, kind=1, pages=4, bt=A, B=2, mp=2, req=A, pos=A, N=5, e=A, stride=576)
    d.update(kw)
    return ops.lib().mla_cache_read(P(d["cache"]), d["kind"], d["pages"], P(d["bt"]), d["B"], d["mp"], P(d["req"]),
                                    P(d["pos"]), d["N"], P(d["e"]), d["stride"], P(0), P(0))


@pytest.mark.parametrize("kw", [dict(cache=0), dict(bt=0), dict(pos=0), dict(e=0), dict(kind=-1), dict(pages=0),
                                dict(B=0), dict(mp=0), dict(N=-1), dict(stride=512), dict(stride=578), dict(e=A + 4),
                                dict(req=0)])
def test_cache_read_refuses(kw):
    assert _read(**kw) == INVALID


def _verify(**kw):
    d = dict(t=A, d=A, tok=A, u=A, B=2, T=4, V=10, n=A, dep=A, nx=A)
    d.update(kw)
    return ops.lib().mla_verify_draft(P(d["t"]), P(d["d"]), P(d["tok"]), P(0), P(0), P(d["u"]), d["B"], d["T"], d["V"],
                                      P(d["n"]), P(d["dep"]), P(d["nx"]), P(0), P(0))


@pytest.mark.parametrize("kw", [dict(t=0), dict(tok=0), dict(u=0), dict(n=0), dict(dep=0), dict(nx=0), dict(B=-1),
                                dict(T=0), dict(V=0)])
def test_verify_refuses(kw):
    assert _verify(**kw) == INVALID


def test_verify_limits():
    assert _verify(T=65) == UNSUPPORTED and _verify(V=(1 << 20) + 1) == UNSUPPORTED
    assert _verify(B=0, t=0) == OK


def test_binding_refuses_host_tensors_and_wrong_types():
    f = torch.zeros(32, dtype=torch.float64)
    with pytest.raises(ValueError, match="x must be a CUDA tensor"):
        ops.rope(torch.zeros(2, 3, 192, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32), f)
    with pytest.raises(ValueError, match="bf16"):
        ops.rope(torch.zeros(2, 3, 192), torch.zeros(2, dtype=torch.int32), f)
    with pytest.raises(ValueError, match="per head"):
        ops.rope(torch.zeros(2, 3, 32, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32), f)
    cache = torch.zeros(2, 64, 576, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="cache must be a CUDA tensor"):
        ops.cache_write(cache, i.view(1, 2), i, i, torch.zeros(2, 576, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="cache must be a CUDA tensor"):
        ops.cache_read(cache, i.view(1, 2), i, i)
    with pytest.raises(ValueError, match="target_probs must be a CUDA tensor"):
        ops.verify_draft(torch.zeros(1, 2, 5), None, i.view(1, 2)[:, :1], torch.zeros(1, 2))


def test_rope_frequencies():
    f, m = ops.rope_frequencies(64, device="cpu")
    assert f.dtype == torch.float64 and m == 1.0
    assert torch.equal(f, 10000.0 ** (-2.0 * torch.arange(32, dtype=torch.float64) / 64))
    assert torch.equal(ops.rope_frequencies(64, scaling="linear", factor=4.0, device="cpu")[0], f / 4)
    n, _ = ops.rope_frequencies(64, scaling="ntk", factor=4.0, device="cpu")
    assert n[0] == 1.0 and abs(float(n[-1] * 4 / f[-1]) - 1) < 1e-12
    y, m = ops.rope_frequencies(64, scaling="yarn", factor=40.0, device="cpu")
    # j turns 4096 f_j / (2 pi) times: above 32 turns kept, below 1 divided by 40, between in order
    turns = 4096 * f / (2 * math.pi)
    assert torch.equal(y[turns > 33], f[turns > 33])
    assert torch.allclose(y[turns < 0.9], f[turns < 0.9] / 40, rtol=1e-12)
    ratio = y / f
    assert bool((ratio[1:] <= ratio[:-1] + 1e-12).all()) and abs(m - (0.1 * math.log(40) + 1)) < 1e-12
    for kw in (dict(d_rot=63), dict(base=1.0), dict(factor=0.5), dict(scaling="x"), dict(scaling="yarn", beta_fast=1.0)):
        with pytest.raises(ValueError):
            ops.rope_frequencies(**{**dict(d_rot=64, device="cpu"), **kw})


def test_no_tokens_are_nothing_to_do_whatever_the_batch():
    # a step without requests: no table, no pages, no rows
    none = dict(N=0, cache=0, bt=0, req=0, pos=0, pages=0, B=0, mp=0)
    assert _write(**none, kv=0) == OK and _write(**none, kv=0, kind=1, w=A, freqs=A) == OK
    assert _read(**none, e=0) == OK
    # what does not depend on the batch is checked all the same
    assert _write(**none, kv=0, kind=2) == INVALID and _write(**none, kv=0, layout=5) == INVALID
    assert _read(**none, e=0, stride=512) == INVALID
