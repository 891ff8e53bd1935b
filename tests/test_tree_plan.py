"""The tree planner (host twin of the device planner) and the refusals of the tree attention's
calls; CPU only."""
import ctypes
import math

import numpy as np
import pytest
import torch

from mla_latent_kv_17_gb300 import build as mbuild
from mla_latent_kv_17_gb300 import ops
from planview import parse

P = ctypes.c_void_p
A = 0x10000
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


@pytest.fixture(scope="module", autouse=True)
def _built():
    mbuild.build()


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("B,T,H,hi", [(1, 1, 1, 50), (1, 5, 16, 300), (4, 8, 128, 9000), (64, 8, 16, 8192),
                                      (2, 64, 128, 131072), (300, 3, 100, 700), (7, 13, 77, 0)])
def test_every_row_tile_attends_every_token_once(B, T, H, hi, kv):
    rng = np.random.default_rng(B * T + H)
    lens = rng.integers(0, T + 1, B)
    lens[0] = T
    seq = rng.integers(0, hi + 1, B) + lens
    units = 74
    R = (T * H + 127) // 128
    p = parse(ops.plan_tree_host(seq, lens, B, T, H, num_sms=2 * units, kv_dtype=kv), B * R, 128)
    assert p["topk"] == -1 and p["units"] == units and p["n_partials"] <= p["max_partials"] == 2 * units
    got = {}
    slots = []
    for e, t0, t1, slot in p["items"]:
        b, tile = int(e) & 0xFFFFFF, int(e) >> 24
        assert 0 <= b < B and 0 <= tile < R
        got.setdefault((b, tile), []).append((int(t0), int(t1)))
        if slot >= 0:
            slots.append(int(slot))
    assert sorted(slots) == list(range(p["n_partials"]))
    for b in range(B):
        for tile in range(R):
            need = int(seq[b]) if tile * 128 < lens[b] * H else 0
            at = 0
            for t0, t1 in got[b, tile]:
                assert t0 == at and t0 % 128 == 0
                at = t1
            assert at == need, (b, tile)
    cost = np.zeros(units)
    for u in range(units):
        for i in range(p["unit_begin"][u], p["unit_begin"][u + 1]):
            _, t0, t1, _ = p["items"][i]
            cost[u] += (t1 - t0 + 127) // 128 + (3 if kv == "fp8" else 2) if t1 > t0 else 0
    assert cost.max() <= p["per"] + 2 + 2 * 3


def _tree(**kw):
    d = dict(ws=A, n=1 << 30, qn=A, qr=A, cache=A, kind=0, pages=4, bt=A, mp=2, sl=A, mask=A, B=2, T=4, H=16,
             scale=0.07, out=A, od=0)
    d.update(kw)
    return ops.lib().mla_decode_tree(P(d["ws"]), d["n"], P(d["qn"]), P(d["qr"]), P(d["cache"]), d["kind"], d["pages"],
                                     P(d["bt"]), d["mp"], P(d["sl"]), P(0), P(d["mask"]), d["B"], d["T"], d["H"],
                                     d["scale"], P(d["out"]), d["od"], P(0), P(0))


@pytest.mark.parametrize("kw", [dict(ws=0), dict(qn=0), dict(qr=0), dict(cache=0), dict(bt=0), dict(sl=0), dict(mask=0),
                                dict(out=0), dict(kind=2), dict(od=2), dict(pages=0), dict(mp=0), dict(B=0), dict(T=0),
                                dict(H=0), dict(scale=0.0), dict(scale=-1.0), dict(scale=math.nan), dict(qn=A + 8),
                                dict(qr=A + 8), dict(cache=A + 8), dict(out=A + 8)])
def test_tree_refuses(kw):
    assert _tree(**kw) == INVALID


def test_tree_limits():
    assert _tree(T=65) == UNSUPPORTED and _tree(H=129) == UNSUPPORTED
    assert _tree(pages=1 << 40) == UNSUPPORTED and _tree(B=1 << 21) == UNSUPPORTED
    assert _tree(n=64) == WORKSPACE
    L = ops.lib()
    for B, T, H in ((0, 4, 16), (2, 0, 16), (2, 65, 16), (2, 4, 129), (1 << 21, 1, 1)):
        assert L.mla_decode_tree_workspace_size(B, T, H, 148) == 0
    assert L.mla_decode_tree_plan(P(0), P(0), 2, 4, 16, 0, 148, P(A), 1 << 30, P(0)) == INVALID
    assert L.mla_decode_tree_plan(P(A), P(0), 2, 4, 16, 3, 148, P(A), 1 << 30, P(0)) == INVALID
    assert L.mla_decode_tree_plan(P(A), P(0), 2, 65, 16, 0, 148, P(A), 1 << 30, P(0)) == UNSUPPORTED
    assert L.mla_decode_tree_plan(P(A), P(0), 2, 4, 16, 0, 148, P(A), 100, P(0)) == WORKSPACE


def test_binding_refuses_host_tensors():
    class Fake:
        B, T, H, nbytes, buf = 1, 2, 4, 10, torch.zeros(10, dtype=torch.uint8)
    z = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        ops.plan_tree(Fake(), z)
    with pytest.raises(ValueError, match="CUDA"):
        ops.decode_tree(Fake(), z, z, z, z, z, z, z, 0.1)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("B,T,H,hi,short", [(16, 64, 128, 300, 1), (16, 64, 128, 0, 0), (12, 16, 64, 700, 2), (40, 8, 128, 9000, 8),
                                            (64, 8, 16, 8192, 8), (5, 1, 128, 4000, 1), (1, 64, 128, 90000, 64)])
def test_units_share_the_cost_the_plan_states(B, T, H, hi, short, kv):
    # pieces at what the planner charges for them, and one tile for each row tile past the drafted
    # tokens (many of them in a row: none of them may fall to one unit)
    rng = np.random.default_rng(B + T + hi)
    lens = rng.integers(0, short + 1, B) if short else np.zeros(B, int)
    seq = rng.integers(0, hi + 1, B) + lens
    units = 74
    R = (T * H + 127) // 128
    p = parse(ops.plan_tree_host(seq, lens, B, T, H, num_sms=2 * units, kv_dtype=kv), B * R, 128)
    ovh, empty = (3 if kv == "fp8" else 2) + (T > 1), int(T > 1)
    cost, empties = np.zeros(units), np.zeros(units, int)
    for u in range(units):
        for i in range(p["unit_begin"][u], p["unit_begin"][u + 1]):
            _, t0, t1, _ = p["items"][i]
            cost[u] += (t1 - t0 + 127) // 128 + ovh if t1 > t0 else empty
            empties[u] += t1 <= t0
    # a unit's share, a tile folded in from either side, and the charge of a piece begun elsewhere
    most = p["per"] + 2 + ovh
    assert cost.max() <= most
    if T > 1:
        assert empties.max() <= most
    assert empties.sum() == sum(int(lens[b] * H <= t * 128 or seq[b] == 0) for b in range(B) for t in range(R))
