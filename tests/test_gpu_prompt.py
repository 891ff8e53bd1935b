"""A prompt of text and images over a cached prefix, as a server would run it: its positions on three
axes, its entries written into the paged cache, its queries rotated, the prefix read back and
decompressed, attention to the prefix, to the prompt itself and to an encoder's states, joined, and
its tokens scored; eager, captured and replayed, on two streams."""
import math

import numpy as np
import pytest
import torch

from mla_latent_kv_17_gb300 import ops
import prompt_ref

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
H, V, D = 8, 3001, 256
SCALE = 1 / math.sqrt(192)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from mla_latent_kv_17_gb300 import build
    build.build()
    ops.lib()


def within(got, want, bound):
    off = np.abs(got - want) - bound
    return float(off.max(initial=-1.0)) <= 0


class Prompt:
    """What a server keeps (weights, cache, tables, workspaces) and one batch of prompts."""

    prefix, new, images = [130, 0, 61], [70, 33, 9], [64, 0, 150]

    def __init__(self, kv, seed):
        g = torch.Generator().manual_seed(seed)
        randn = lambda *s, d=1.0: (torch.randn(*s, generator=g) / math.sqrt(d)).to(BF).cuda()
        self.kv = kv
        width = 576 if kv == "bf16" else 656
        self.cache = torch.zeros(16, 64, width, dtype=BF if kv == "bf16" else torch.uint8, device="cuda")
        self.bt = torch.randperm(16, generator=g)[:12].reshape(3, 4).to(torch.int32).cuda()
        self.freqs, _ = ops.rope_frequencies(64)
        self.axes = ops.rope_axes((8, 12, 12), "interleaved")
        self.norm = (1 + 0.1 * torch.randn(512, generator=g)).to(BF).cuda()
        self.w_uk, self.w_uv = randn(H, 128, 512, d=512), randn(H, 128, 512, d=512)
        self.w_out = randn(H * 128, V, d=H * 16)
        runs = lambda n: torch.from_numpy(np.concatenate([[0], np.cumsum(n)]).astype(np.int32)).cuda()
        ints = lambda v: torch.tensor(np.concatenate(v).astype(np.int32)).cuda()
        both = [p + n for p, n in zip(self.prefix, self.new)]
        self.cu_q, self.cu_k, self.cu_i = runs(self.new), runs(both), runs(self.images)
        # the prefix's entries are in the cache already; then the prompt's own
        self.old_req, self.old_pos = ints([[b] * n for b, n in enumerate(self.prefix)]), ints([range(n) for n in self.prefix])
        self.req = ints([[b] * n for b, n in enumerate(self.new)])
        self.slot = ints([range(p, p + n) for p, n in zip(self.prefix, self.new)])
        self.all_req, self.all_pos = ints([[b] * n for b, n in enumerate(both)]), ints([range(n) for n in both])
        self.old_kv = randn(sum(self.prefix), 576)
        # text, then an image of rows of five, whose tokens share their time
        at = torch.arange(sum(self.new))
        image = at % 20 >= 5
        self.pos = torch.stack([torch.where(image, at // 20 * 20, at), torch.where(image, at // 20 * 20 + at % 20 // 5, at),
                                torch.where(image, at // 20 * 20 + at % 5, at)]).to(torch.int32).cuda().t()
        old = self.old_pos.unsqueeze(1).expand(-1, 3)
        ops.cache_write(self.cache, self.bt, self.old_req, self.old_pos, self.old_kv, freqs=self.freqs, rope_positions=old,
                        norm_weight=self.norm, axes=self.axes)
        n = sum(self.new)
        self.hidden = dict(q=randn(n, H, 192), kv=randn(n, 576), tokens=torch.randint(0, V, (n,), generator=g).to(torch.int32).cuda())
        self.i_entries = randn(sum(self.images), 576)
        self.ws, self.ws_i = ops.CrossWorkspace(3, H, n), ops.CrossWorkspace(3, H, n)

    def step(self, stream=None):
        k = dict(stream=stream)
        ops.cache_write(self.cache, self.bt, self.req, self.slot, self.hidden["kv"], freqs=self.freqs, rope_positions=self.pos,
                        norm_weight=self.norm, axes=self.axes, **k)
        q_nope, q_rope = ops.rope(self.hidden["q"], self.pos, self.freqs, axes=self.axes, **k)
        entries = ops.cache_read(self.cache, self.bt, self.all_req, self.all_pos, **k)
        k_nope, v = ops.prefill_decompress(entries, self.w_uk, self.w_uv, **k)
        ops.plan_cross(self.ws, self.cu_q, self.cu_k, entries.shape[0], causal=True, **k)
        first = ops.cross_attention(self.ws, q_nope, q_rope, entries, k_nope, v, SCALE, **k)
        # the images' states carry no positions
        ik, iv = ops.prefill_decompress(self.i_entries, self.w_uk, self.w_uv, **k)
        ops.plan_cross(self.ws_i, self.cu_q, self.cu_i, self.i_entries.shape[0], **k)
        out, lse = ops.cross_attention(self.ws_i, q_nope, None, None, ik, iv, SCALE, before=first, out_dtype=BF, **k)
        return q_nope, q_rope, entries, out, lse

    def score(self, out):
        logits = out.flatten(1) @ self.w_out
        return logits, ops.token_logprobs(logits, self.hidden["tokens"], top=5)

    def check(self, got):
        """The step's outputs against 64 bits, each from the bf16 tensors its call read."""
        q_nope, q_rope, entries, out, lse = got
        assert ops.status(self.ws) == 0 and ops.status(self.ws_i) == 0
        num = lambda t: t.double().cpu().numpy()
        # the queries: as test_gpu_axes bounds them
        axis = prompt_ref.axis_of_pair((8, 12, 12), "interleaved")
        y, pair = prompt_ref.rotate(num(self.hidden["q"])[..., 128:], self.pos.cpu().numpy(), axis, num(self.freqs), "interleaved")
        assert within(num(q_rope), y, 2.0 ** -8 * np.abs(y) + 2.0 ** -19 * pair)
        # the prompt's entries: norm, rotation and (FP8) the codes' half steps, 2^-4 of a value or of the smallest
        # normal code's step
        x = num(self.hidden["kv"])
        lat = x[:, :512] / np.sqrt((x[:, :512] ** 2).mean(1, keepdims=True) + 1e-6) * num(self.norm)
        mine = np.concatenate([np.arange(p, p + n) + o for p, n, o in zip(self.prefix, self.new, num(self.cu_k).astype(int))])
        e = num(entries)[mine]
        if self.kv == "bf16":
            tol = 2.0 ** -8 * 1.01 * np.abs(lat)
        else:
            block = np.abs(lat).reshape(len(lat), 4, 128).max(2).repeat(128, 1) / 448
            tol = 2.0 ** -4 * 1.01 * np.maximum(np.abs(lat), 2.0 ** -6 * block) + 2.0 ** -8 * np.abs(lat) * 1.1
        assert within(e[:, :512], lat, tol)
        y, pair = prompt_ref.rotate(x[:, 512:], self.pos.cpu().numpy(), axis, num(self.freqs), "interleaved")
        assert within(e[:, 512:], y, 2.0 ** -8 * np.abs(y) + 2.0 ** -19 * pair)
        # attention over the decompressed (bf16) keys and values
        q = np.concatenate([num(q_nope), num(q_rope)], -1)
        k_nope, v = (num(t) for t in ops.prefill_decompress(entries, self.w_uk, self.w_uv))
        k = np.concatenate([k_nope, np.broadcast_to(num(entries)[None, :, 512:], (H, len(num(entries)), 64))], -1)
        cu_q, cu_k, cu_i = (num(t).astype(int) for t in (self.cu_q, self.cu_k, self.cu_i))
        o1, l1, mean1, _ = prompt_ref.cross(q, k, v, cu_q, cu_k, SCALE, True)
        ik, iv = (num(t) for t in ops.prefill_decompress(self.i_entries, self.w_uk, self.w_uv))
        o, l, _, _ = prompt_ref.cross(num(q_nope), ik, iv, cu_q, cu_i, SCALE, False, (o1, l1))
        mean2 = prompt_ref.cross(num(q_nope), ik, iv, cu_q, cu_i, SCALE, False)[2]
        # each part is off by its probabilities' rounding to bf16, 2^-8 of its mean |v| (not of its |out|: the values
        # cancel in it); the parts' shares, then the output's own rounding; fp32 terms lie far below 2^-12 at
        # these sizes
        share = np.exp(l1 - l)[..., None]
        mean = share * mean1 + (1 - share) * mean2
        assert within(num(out), o, (2.0 ** -8 + 2.0 ** -12) * mean + 2.0 ** -8 * 1.01 * (np.abs(o) + 2.0 ** -7 * mean))
        assert within(num(lse), l, 2.0 ** -14 * (1 + np.abs(l)))


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_prompt(kv):
    p = Prompt(kv, 3)
    got = p.step()
    p.check(got)
    logits, scores = p.score(got[3])
    lp, h, rank, ids, alt, below, logs = prompt_ref.logprobs(logits.double().cpu().numpy(), p.hidden["tokens"].cpu().numpy(), 1.0, 5)
    assert np.array_equal(scores[2].cpu().numpy(), rank) and np.array_equal(scores[3].cpu().numpy(), ids)
    # (bounded in test_gpu_logprobs; 2^-14 covers (ceil(3001 / 256) + 80) u + 4 u B with room)
    for a, b in ((scores[0], lp), (scores[1], h), (scores[4], alt)):
        assert within(a.double().cpu().numpy(), b, 2.0 ** -14 * (1 + np.abs(b)))


def test_one_prompt_whole_equals_the_prefill():
    # a prompt from position 0 is what the prefill computes: within both's rounding of the probabilities
    g = torch.Generator().manual_seed(5)
    L = 300
    e = torch.randn(L, 576, generator=g).to(BF).cuda()
    q, r = torch.randn(L, H, 128, generator=g).to(BF).cuda(), torch.randn(L, H, 64, generator=g).to(BF).cuda()
    w = (torch.randn(H, 128, 512, generator=g) / 22).to(BF).cuda()
    k, v = ops.prefill_decompress(e, w, w)
    a, la = ops.prefill_attention(q, r, e, k, v, SCALE)
    ws = ops.CrossWorkspace(1, H, L)
    cu = torch.tensor([0, L], dtype=torch.int32, device="cuda")
    ops.plan_cross(ws, cu, cu, L, causal=True)
    b, lb = ops.cross_attention(ws, q, r, e, k, v, SCALE)
    assert float((la - lb).abs().max()) <= 2.0 ** -14 * (1 + float(la.abs().max()))
    assert float((a - b).abs().max()) <= 2 * 2.0 ** -8 * float(v.float().abs().max())


def test_captured_and_replayed():
    p = Prompt("bf16", 7)
    p.step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = p.step()
        logits, scores = p.score(got[3])
    g = torch.Generator().manual_seed(8)
    for _ in range(2):
        p.hidden["q"].copy_(torch.randn(p.hidden["q"].shape, generator=g).to(BF))
        p.hidden["kv"].copy_(torch.randn(p.hidden["kv"].shape, generator=g).to(BF))
        graph.replay()
        p.check(got)
        again = ops.token_logprobs(logits, p.hidden["tokens"], top=5)
        assert all(torch.equal(a, b) for a, b in zip(scores, again))


def test_on_two_streams():
    a, b = Prompt("bf16", 1), Prompt("fp8", 2)
    want = [[t.clone() for t in p.step()] for p in (a, b)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        gb, ga = b.step(stream=side), a.step()
        torch.cuda.synchronize()
        for got, w in ((ga, want[0]), (gb, want[1])):
            assert all(torch.equal(x, y) for x, y in zip(got, w))
