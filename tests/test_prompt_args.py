"""Refusals of the calls for prompts of text and images: what the C ABI and the binding reject before
anything is enqueued (no GPU needed), and the helpers that need none."""
import ctypes
import math

import numpy as np
import pytest
import torch

from mla_latent_kv_17_gb300 import build as mbuild
from mla_latent_kv_17_gb300 import ops
import prompt_ref

P = ctypes.c_void_p
OK, INVALID, UNSUPPORTED = 0, 1, 2
A = 0x10000  # a 16-byte-aligned address; nothing is read in a refused call
AXES = bytes([0] * 8 + [1] * 12 + [2] * 12)


@pytest.fixture(scope="module", autouse=True)
def _built():
    mbuild.build()


def _rope(**kw):
    d = dict(x=A, N=3, H=4, dp=128, dr=64, layout=0, pos=A, ts=3, xs=1, n=3, axes=AXES, freqs=A, m=1.0, op=A, orr=A)
    d.update(kw)
    return ops.lib().mla_rope_axes(P(d["x"]), 768, 192, d["N"], d["H"], d["dp"], d["dr"], d["layout"], P(d["pos"]), d["ts"],
                                   d["xs"], d["n"], d["axes"], P(d["freqs"]), d["m"], P(d["op"]), 512, 128, P(d["orr"]),
                                   256, 64, P(0))


@pytest.mark.parametrize("kw", [dict(x=0), dict(pos=0), dict(freqs=0), dict(orr=0), dict(N=-1), dict(H=0), dict(dp=-8),
                                dict(dr=0), dict(dr=63), dict(layout=2), dict(m=math.nan), dict(x=A + 1), dict(n=0),
                                dict(axes=None), dict(n=2), dict(axes=AXES[:-1] + b"\x03")])
def test_rope_axes_refuses(kw):
    assert _rope(**kw) == INVALID


def test_rope_axes_limits():
    assert _rope(n=5) == UNSUPPORTED and _rope(dr=514, axes=bytes(257)) == UNSUPPORTED
    assert _rope(N=0, x=0, pos=0) == OK  # nothing to do


def _write(**kw):
    d = dict(cache=A, kind=0, pages=4, bt=A, B=2, mp=2, req=A, pos=A, kv=A, stride=576, N=5, w=0, eps=1e-6, freqs=A,
             rp=A, ts=3, xs=1, n=3, axes=AXES, layout=0, m=1.0)
    d.update(kw)
    return ops.lib().mla_cache_write_axes(P(d["cache"]), d["kind"], d["pages"], P(d["bt"]), d["B"], d["mp"], P(d["req"]),
                                          P(d["pos"]), P(d["kv"]), d["stride"], d["N"], P(d["w"]), d["eps"],
                                          P(d["freqs"]), P(d["rp"]), d["ts"], d["xs"], d["n"], d["axes"], d["layout"],
                                          d["m"], P(0), P(0))


@pytest.mark.parametrize("kw", [dict(cache=0), dict(bt=0), dict(pos=0), dict(kv=0), dict(kind=2), dict(pages=0),
                                dict(N=-1), dict(stride=575), dict(kv=A + 2), dict(req=0), dict(w=A, eps=-1.0),
                                dict(layout=7), dict(m=math.inf), dict(freqs=0), dict(rp=0), dict(n=0), dict(n=2),
                                dict(axes=None), dict(axes=bytes([3] * 32))])
def test_cache_write_axes_refuses(kw):
    assert _write(**kw) == INVALID


def test_cache_write_axes_limits():
    assert _write(n=5) == UNSUPPORTED
    assert _write(N=0, kv=0, pos=0, freqs=0, rp=0) == OK


def test_rope_axes_helper():
    assert ops.rope_axes((8, 12, 12)) == AXES
    for sections in ((8, 12, 12), (24, 20, 20), (1, 0, 5), (3,), (2, 2), (0, 0, 0, 7), (1, 2, 3, 4)):
        for order in ("blocks", "interleaved"):
            assert np.array_equal(np.frombuffer(ops.rope_axes(sections, order), np.uint8),
                                  prompt_ref.axis_of_pair(sections, order))
    for bad in ((), (1, 2, 3, 4, 5), (-1, 3), (0, 0), (1.5, 2)):
        with pytest.raises(ValueError):
            ops.rope_axes(bad)
    with pytest.raises(ValueError):
        ops.rope_axes((8, 12, 12), "x")


def test_binding_refuses_host_tensors():
    f = torch.zeros(32, dtype=torch.float64)
    with pytest.raises(ValueError, match="x must be a CUDA tensor"):
        ops.rope(torch.zeros(2, 3, 192, dtype=torch.bfloat16), torch.zeros(2, 3, dtype=torch.int32), f, axes=AXES)


def _score(**kw):
    d = dict(x=A, kind=0, stride=100, N=3, V=100, tok=A, scale=1.0, top=4, lp=A, h=A, r=A, ids=A, alt=A)
    d.update(kw)
    return ops.lib().mla_token_logprobs(P(d["x"]), d["kind"], d["stride"], d["N"], d["V"], P(d["tok"]), d["scale"], d["top"],
                                        P(d["lp"]), P(d["h"]), P(d["r"]), P(d["ids"]), P(d["alt"]), P(0), P(0))


@pytest.mark.parametrize("kw", [dict(x=0), dict(tok=0), dict(lp=0), dict(ids=0), dict(alt=0), dict(kind=3), dict(kind=-1),
                                dict(stride=-1), dict(N=-1), dict(V=0), dict(top=-1), dict(scale=0.0), dict(scale=-1.0),
                                dict(scale=math.nan), dict(scale=math.inf), dict(scale=1e-7), dict(x=A + 1),
                                dict(kind=2, x=A + 2)])
def test_token_logprobs_refuses(kw):
    assert _score(**kw) == INVALID


def test_token_logprobs_limits():
    assert _score(top=65) == UNSUPPORTED and _score(V=(1 << 28) + 1) == UNSUPPORTED
    assert _score(N=0, x=0, tok=0, lp=0) == OK


def _plan(**kw):
    d = dict(q=A, k=A, B=2, H=4, nq=10, nk=20, causal=0, sms=152, ws=A, bytes=1 << 40)
    d.update(kw)
    return ops.lib().mla_cross_plan(P(d["q"]), P(d["k"]), d["B"], d["H"], d["nq"], d["nk"], d["causal"], d["sms"], P(d["ws"]),
                                    d["bytes"], P(0))


@pytest.mark.parametrize("kw", [dict(q=0), dict(k=0), dict(B=0), dict(H=0), dict(nq=-1), dict(nk=-1), dict(sms=-1),
                                dict(sms=5000), dict(ws=0), dict(ws=A + 4)])
def test_cross_plan_refuses(kw):
    assert _plan(**kw) == INVALID


def test_cross_plan_limits():
    assert _plan(H=129) == UNSUPPORTED and _plan(B=(1 << 20) + 1) == UNSUPPORTED
    assert _plan(nq=(1 << 24) + 1) == UNSUPPORTED and _plan(nk=2 ** 31) == UNSUPPORTED
    need = ops.lib().mla_cross_workspace_size(2, 4, 10, 152)
    assert need > 0 and _plan(bytes=need - 1) == 3  # MLA_ERR_WORKSPACE
    for bad in ((0, 4, 10, 152), (2, 0, 10, 152), (2, 129, 10, 152), (2, 4, -1, 152), (2, 4, 10, -1), (2, 4, 1 << 25, 152)):
        assert ops.lib().mla_cross_workspace_size(*bad) == 0


def _cross(**kw):
    d = dict(ws=A, bytes=1 << 40, qn=A, qr=A, e=A, k=A, v=A, B=2, H=4, nq=10, nk=20, scale=0.1, bo=0, bl=0, out=A, dt=0, lse=A)
    d.update(kw)
    return ops.lib().mla_cross_attention(P(d["ws"]), d["bytes"], P(d["qn"]), P(d["qr"]), P(d["e"]), P(d["k"]), P(d["v"]),
                                         d["B"], d["H"], d["nq"], d["nk"], d["scale"], P(d["bo"]), P(d["bl"]), P(d["out"]),
                                         d["dt"], P(d["lse"]), P(0))


@pytest.mark.parametrize("kw", [dict(ws=0), dict(qn=0), dict(qr=0), dict(e=0), dict(k=0), dict(v=0), dict(B=0), dict(H=0),
                                dict(nq=-1), dict(nk=-1), dict(scale=0.0), dict(scale=-1.0), dict(scale=math.nan),
                                dict(scale=math.inf), dict(bo=A), dict(bl=A), dict(out=0), dict(dt=2), dict(qn=A + 2),
                                dict(k=A + 8), dict(v=A + 4), dict(e=A + 2), dict(out=A + 4), dict(ws=A + 8),
                                dict(bo=A + 16, bl=A), dict(out=A + 16)])
def test_cross_attention_refuses(kw):
    assert _cross(**kw) == INVALID


def test_cross_attention_limits():
    assert _cross(H=129) == UNSUPPORTED and _cross(nk=2 ** 31) == UNSUPPORTED
    assert _cross(bytes=256) == 3
    assert _cross(nq=0, qn=0, out=0) == OK
