"""Verification of drafted trees on the GPU against a 64-bit restatement: the decisions and the
drawn tokens are whole numbers and have to be equal."""
import numpy as np
import pytest
import torch

from mla_latent_kv_17_gb300 import ops
import step_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from mla_latent_kv_17_gb300 import build
    build.build()
    ops.lib()


def make(B, T, V, seed, tree, probs, noise=0.7):
    g = torch.Generator(device="cuda").manual_seed(seed)
    at = torch.arange(T, device="cuda")
    back = torch.randint(1, 4, (B, T), generator=g, device="cuda") if tree else 1
    parents = (at - back).clamp(min=-1).expand(B, T).contiguous().to(torch.int32)
    logits = 2.5 * torch.randn(B, T + 1, V, generator=g, device="cuda")
    target = logits.softmax(-1)
    draft = (logits + noise * torch.randn(B, T + 1, V, generator=g, device="cuda")).softmax(-1)
    draft = draft.gather(1, (parents.long() + 1).unsqueeze(-1).expand(B, T, V)).contiguous()
    tok = torch.multinomial(draft.reshape(B * T, V), 1, generator=g).reshape(B, T).to(torch.int32)
    u = torch.rand(B, T + 1, generator=g, device="cuda")
    return target, draft if probs else None, tok, u, parents if tree else None


def run(target, draft, tok, u, parents, lens=None, status=None):
    got = ops.verify_draft(target, draft, tok, u, parents=parents, tree_lens=lens, device_status=status)
    num = lambda t: None if t is None else t.cpu().numpy()
    want = step_ref.verify(num(target), num(draft), num(tok), num(u), num(parents), num(lens))
    for g, w, name in zip(got, want, ("num_accepted", "depths", "next_token")):
        assert np.array_equal(g.cpu().numpy(), w), (name, g.cpu().numpy(), w)
    return got


@pytest.mark.parametrize("tree,probs", [(False, True), (False, False), (True, True), (True, False)])
@pytest.mark.parametrize("B,T,V", [(1, 1, 1), (3, 1, 2), (2, 5, 7), (4, 3, 127), (2, 64, 1000), (5, 8, 32001),
                                   (1, 4, 131072), (2, 2, 262147), (70, 6, 900)])
def test_verify(B, T, V, tree, probs):
    n = run(*make(B, T, V, B * 100 + T, tree, probs))[0]
    if probs and V >= 900 and B * T > 20:
        # some stand, some fall (without probabilities a whole batch may fall: u < p(x) alone)
        assert 0 < int(n.sum()) < B * T


@pytest.mark.parametrize("tree,probs", [(False, True), (True, True), (True, False)])
def test_the_largest_vocabulary_and_tree(tree, probs):
    target, draft, tok, u, parents = make(1, 64, 1 << 20, 29, tree, probs)
    run(target, draft, tok, u, parents)


def test_ragged_trees():
    target, draft, tok, u, parents = make(6, 7, 500, 4, True, True)
    lens = torch.tensor([0, 1, 7, 3, 2, 6], dtype=torch.int32, device="cuda")
    _, depths, _ = run(target, draft, tok, u, parents, lens)
    for b in range(6):
        assert bool((depths[b, int(lens[b]):] == -1).all())
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lens[0], lens[1] = -2, 99  # clamped and recorded
    run(target, draft, tok, u, parents, lens, status)
    assert int(status) == 5


def test_draft_equal_to_target_stands_and_the_bonus_is_drawn():
    target, _, tok, u, _ = make(4, 5, 3001, 9, False, True)
    n, depths, _ = run(target, target[:, :5].contiguous(), tok, u, None)
    assert bool((n == 5).all()) and torch.equal(depths[0].cpu(), torch.arange(5, dtype=torch.int32))


def test_siblings_are_tried_in_turn():
    # three candidates for the same place, two of them the same token: whichever stands is at depth 0
    V = 4000
    target, draft, tok, u, _ = make(40, 6, V, 12, False, True)
    parents = torch.tensor([-1, -1, -1, 0, 1, 2], dtype=torch.int32, device="cuda").repeat(40, 1)
    draft[:, 1] = draft[:, 0]
    draft[:, 2] = draft[:, 0]
    tok[:, 1] = tok[:, 0]
    _, depths, _ = run(target, draft, tok, u, parents)
    assert set(depths[:, :3].max(1).values.tolist()) <= {-1, 0}
    assert bool(((depths[:, :3] == 0).sum(1) <= 1).all())
    run(target, None, tok, u, parents)


def test_nothing_left_and_empty_rows():
    V = 300
    target = torch.full((3, 2, V), 1.0 / V, device="cuda")
    draft = 2 * target[:, :1].contiguous()          # covers all of the target
    target[2, 0] = 0.0                                # an empty row
    tok = torch.tensor([[5], [6], [7]], dtype=torch.int32, device="cuda")
    u = torch.tensor([[0.9, 0.5], [0.2, 0.5], [0.9, 0.5]], device="cuda")
    n, _, nxt = run(target, draft, tok, u, None)
    assert n.tolist() == [0, 1, 0] and nxt.tolist()[0] == 150 and nxt.tolist()[2] == -1


def test_odd_values():
    target, draft, tok, u, _ = make(3, 2, 700, 15, False, True)
    target[0, 0, 13] = float("nan")
    target[1, 0, 14] = -0.5
    draft[2, 0, 15] = float("nan")
    u[0, 2], u[1, 2], u[2, 2] = 0.0, 1.0 - 2 ** -24, 0.999
    run(target, draft, tok, u, None)
    # a token outside the vocabulary, a parent that comes later
    tok[0, 0], tok[1, 1] = 700, -1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    run(target, draft, tok, u, None, None, status)
    assert int(status) == 5
    parents = torch.tensor([[-1, 1], [5, 0], [-1, -2]], dtype=torch.int32, device="cuda")
    status.zero_()
    run(target, draft, tok.clamp(0, 699), u, parents, None, status)
    assert int(status) == 5


@pytest.mark.parametrize("sibling", [False, True])
@pytest.mark.parametrize("q,p,want", [(-0.5, 0.0, 0), (-0.5, 0.25, 1), (float("nan"), 0.25, 1), (2.0, 0.6, 1), (2.0, 0.4, 0),
                                      (float("inf"), 0.6, 1)])
def test_a_draft_probability_out_of_range_counts_as_clamped(q, p, want, sibling):
    # token x with u = 1/2: it stands where q/2 < p, for q clamped to [0, 1]; as a second sibling
    # what is left has the mass 1 - 2^-3 (the first one, certain, takes 2^-3 and nothing of x)
    V, x = 300, 17
    T = 2 if sibling else 1
    target, draft = torch.zeros(1, T + 1, V, device="cuda"), torch.zeros(1, T, V, device="cuda")
    target[:, :, 5] = 0.125
    target[:, :, x] = p
    target[:, :, 200] = 0.875 - p
    draft[0, -1, x] = q
    tok = torch.full((1, T), x, dtype=torch.int32, device="cuda")
    parents = torch.full((1, T), -1, dtype=torch.int32, device="cuda")
    if sibling:
        draft[0, 0, 5] = 1.0
        tok[0, 0] = 5
    u = torch.full((1, T + 1), 0.5, device="cuda")
    u[0, 0] = 0.5
    n, d, _ = run(target, draft, tok, u, parents)
    assert int(n[0]) == want and int(d[0, -1]) == want - 1


@pytest.mark.parametrize("V", [65, 5000, 131072])
def test_rows_that_overflow_the_sums_still_give_a_token(V):
    # every probability 1, or one in three: totals of 2^58 V wrap around
    target = torch.ones(40, 2, V, device="cuda")
    target[20:, :, 1::3] = 0.9
    target[20:, :, 2::3] = 0.0
    tok = torch.full((40, 1), V - 1, dtype=torch.int32, device="cuda")
    u = torch.rand(40, 2, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda")
    for lens in (None, torch.zeros(40, dtype=torch.int32, device="cuda")):
        torch.full((40,), 1 << 30, dtype=torch.int32, device="cuda")  # (freed: the outputs' memory)
        _, _, nxt = ops.verify_draft(target, None, tok, u, tree_lens=lens)
        assert bool(((nxt >= -1) & (nxt < V)).all())


def test_a_draw_next_to_a_border():
    # 2^18 equal tokens: u k / 2^18 lies on a border, the first token past it is drawn
    V = 1 << 18
    target = torch.full((64, 2, V), 1.0 / V, device="cuda")
    tok = torch.zeros(64, 1, dtype=torch.int32, device="cuda")
    k = torch.randint(0, V, (64,), generator=torch.Generator().manual_seed(1))
    u = torch.zeros(64, 2, device="cuda")
    u[:, 1] = (k.double() / V).float().cuda()
    _, _, nxt = ops.verify_draft(target, None, tok, u, tree_lens=torch.zeros(64, dtype=torch.int32, device="cuda"))
    assert torch.equal(nxt.cpu().long(), k)


def test_empty_batch():
    n, d, x = ops.verify_draft(torch.zeros(0, 3, 5, device="cuda"), None,
                               torch.zeros(0, 2, dtype=torch.int32, device="cuda"), torch.zeros(0, 3, device="cuda"))
    assert n.shape == (0,) and d.shape == (0, 2) and x.shape == (0,)


@pytest.mark.parametrize("total", [20.0, 40.0, 60.0])
def test_siblings_of_rows_that_add_up_to_less_than_64(total):
    # residuals of more than half the sums' range: what a second sibling covers is its share of all of it
    B, T, V = 60, 4, 200
    g = torch.Generator(device="cuda").manual_seed(31)
    target = torch.rand(B, T + 1, V, generator=g, device="cuda")
    target = (target / target.sum(-1, keepdim=True) * total).contiguous()
    draft = (3 * torch.randn(B, T, V, generator=g, device="cuda")).softmax(-1)
    tok = draft.argmax(-1).to(torch.int32)
    parents = torch.full((B, T), -1, dtype=torch.int32, device="cuda")
    u = 0.9 + 0.09 * torch.rand(B, T + 1, generator=g, device="cuda")
    u[:, T] = torch.rand(B, generator=g, device="cuda")
    n, _, _ = run(target, draft, tok, u, parents)
    assert int((n == 0).sum()) > 10  # all four fell
