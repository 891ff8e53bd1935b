"""A whole speculative decoding step over the latent cache, as a server would run it: rotary
positions, cache write of the drafted tokens, absorption, tree attention, projection,
verification, and the accepted tokens' entries written again at their final positions; eager,
captured and replayed, and on two streams at once."""
import math

import numpy as np
import pytest
import torch

from mla_latent_kv_17_gb300 import inputs, ops
import step_ref
import tree_ref

pytestmark = pytest.mark.gpu
B, T, H, V = 3, 6, 16, 2000


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from mla_latent_kv_17_gb300 import build
    build.build()
    ops.lib()


class Step:
    """What a server keeps between steps (weights, cache, tables) and one step's inputs."""

    def __init__(self, kv, seed):
        g = torch.Generator().manual_seed(seed)
        self.kv = kv
        self.context = torch.tensor([130, 0, 61], dtype=torch.int32)
        width = 576 if kv == "bf16" else 656
        self.cache = torch.zeros(16, 64, width, dtype=torch.bfloat16 if kv == "bf16" else torch.uint8, device="cuda")
        self.bt = torch.randperm(16, generator=g)[:12].reshape(3, 4).to(torch.int32).cuda()
        self.freqs, self.mscale = ops.rope_frequencies(64, scaling="yarn", factor=4.0)
        self.w_uk = (torch.randn(H, 128, 512, generator=g) / math.sqrt(128)).to(torch.bfloat16).cuda()
        self.w_uv = (torch.randn(H, 128, 512, generator=g) / math.sqrt(512)).to(torch.bfloat16).cuda()
        self.norm = (1 + 0.1 * torch.randn(512, generator=g)).to(torch.bfloat16).cuda()
        # the committed tokens
        req = torch.cat([torch.full((int(n),), b, dtype=torch.int32) for b, n in enumerate(self.context)])
        pos = torch.cat([torch.arange(int(n), dtype=torch.int32) for n in self.context])
        prompt = torch.randn(len(req), 576, generator=g).to(torch.bfloat16)
        self.write(req.cuda(), pos.cuda(), prompt.cuda(), pos.cuda())
        # the tree: two branches; token i sits at depth depth[i] after the context
        self.parents = torch.tensor([[-1, -1, 0, 2, 1, 0]] * B, dtype=torch.int32)
        self.depth = torch.tensor([0, 0, 1, 2, 1, 1], dtype=torch.int32)
        bits = [0] * T
        for i in range(T):
            p = int(self.parents[0, i])
            bits[i] = (bits[p] if p >= 0 else 0) | 1 << i
        self.mask = torch.tensor([bits] * B, dtype=torch.int64).cuda()
        self.lens = torch.tensor([6, 6, 3], dtype=torch.int32).cuda()
        self.seq = (self.context.cuda() + self.lens).contiguous()
        self.req = torch.arange(B, dtype=torch.int32).repeat_interleave(T).cuda()
        ctx = self.context.repeat_interleave(T)
        at = torch.arange(T, dtype=torch.int32).repeat(B)
        self.slot = torch.where(at < self.lens.cpu().repeat_interleave(T), ctx + at, -1).to(torch.int32).cuda()
        self.rpos = (ctx + self.depth.repeat(B)).to(torch.int32).cuda()
        self.ws = ops.TreeWorkspace(B, T, H)
        self.x = {}
        self.draw(seed + 1)

    def write(self, req, pos, kv, rpos):
        ops.cache_write(self.cache, self.bt, req, pos, kv, freqs=self.freqs, rope_positions=rpos, mscale=self.mscale,
                        norm_weight=self.norm)

    def draw(self, seed):
        """New inputs of a step, into the same tensors."""
        g = torch.Generator().manual_seed(seed)
        logits = 2 * torch.randn(B, T + 1, V, generator=g)
        draft = (logits + 0.5 * torch.randn(B, T + 1, V, generator=g)).softmax(-1)
        draft = draft.gather(1, (self.parents.long() + 1).unsqueeze(-1).expand(B, T, V)).contiguous()
        new = dict(q=torch.randn(B * T, H, 192, generator=g).to(torch.bfloat16),
                   kv=torch.randn(B * T, 576, generator=g).to(torch.bfloat16), target=logits.softmax(-1), draft=draft,
                   tok=torch.multinomial(draft.view(-1, V), 1, generator=g).view(B, T).to(torch.int32),
                   u=torch.rand(B, T + 1, generator=g), parents=self.parents)
        for k, v in new.items():
            if k in self.x:
                self.x[k].copy_(v)
            else:
                self.x[k] = v.cuda()

    def run(self):
        x = self.x
        q_c, q_rope = ops.rope(x["q"], self.rpos, self.freqs, mscale=self.mscale)
        self.write(self.req, self.slot, x["kv"], self.rpos)
        q_nope = ops.absorb_query(q_c, self.w_uk)
        ops.plan_tree(self.ws, self.seq, self.lens, kv_dtype=self.kv)
        out, lse = ops.decode_tree(self.ws, q_nope.view(B, T, H, 512), q_rope.view(B, T, H, 64), self.cache, self.bt,
                                   self.seq, self.lens, self.mask, tree_ref.SCALE)
        y = ops.project_output(out.view(B * T, H, 512), self.w_uv)
        num, depths, nxt = ops.verify_draft(x["target"], x["draft"], x["tok"], x["u"], parents=x["parents"],
                                            tree_lens=self.lens)
        # the accepted tokens' entries, again, at context + depth (a rejected branch lay in between)
        ctx = (self.seq - self.lens).unsqueeze(1)
        final = torch.where(depths >= 0, ctx + depths, torch.full_like(depths, -1)).view(-1)
        self.write(self.req, final, x["kv"], self.rpos)
        return dict(q_nope=q_nope, q_rope=q_rope, out=out, lse=lse, y=y, num=num, depths=depths, nxt=nxt)


def check(st, before, r):
    """Every part of a step against 64 bits, on the step's own intermediate values."""
    x = {k: v.cpu() for k, v in st.x.items()}
    y, pair = step_ref.rotate(x["q"][..., 128:].double().numpy(), st.rpos.cpu().numpy(), st.freqs.cpu().numpy(),
                              "interleaved", st.mscale)
    e = np.abs(r["q_rope"].cpu().double().numpy() - y)
    assert (e <= 2.0 ** -8 * np.abs(y) + 2.0 ** -19 * st.mscale * pair * 1.01).all()
    qn = torch.einsum("nhk,hkc->nhc", x["q"][..., :128].double(), st.w_uk.cpu().double())
    assert bool(((r["q_nope"].cpu().double() - qn).abs() <= 2.0 ** -8 * qn.abs() + 1e-4).all())
    # the cache as the attention saw it: the drafted tokens' entries written over `before`
    mid = before.clone()
    ops.cache_write(mid, st.bt, st.req, st.slot, st.x["kv"], freqs=st.freqs, rope_positions=st.rpos, mscale=st.mscale,
                    norm_weight=st.norm)
    ref = tree_ref.tree(r["q_nope"].view(B, T, H, 512), r["q_rope"].view(B, T, H, 64), mid, st.bt, st.seq, st.lens, st.mask)
    tree_ref.check(r["out"], r["lse"], ref, "step")
    want = step_ref.verify(*(x[k].numpy() for k in ("target", "draft", "tok", "u", "parents")), st.lens.cpu().numpy())
    for k, w in zip(("num", "depths", "nxt"), want):
        assert np.array_equal(r[k].cpu().numpy(), w), k
    # the accepted path's entries lie one after another behind the context, bit for bit those of
    # its tokens; what is not overwritten stays
    flat, mf = st.cache.view(torch.uint8).view(16 * 64, -1), mid.view(torch.uint8).view(16 * 64, -1)
    row = lambda b, p: int(st.bt[b, p // 64]) * 64 + p % 64
    moved = set()
    for b in range(B):
        for i in range(T):
            d = int(want[1][b, i])
            if d >= 0:
                assert torch.equal(flat[row(b, int(st.context[b]) + d)], mf[row(b, int(st.context[b]) + i)]), (b, i)
                moved.add(row(b, int(st.context[b]) + d))
    keep = [k for k in range(16 * 64) if k not in moved]
    assert torch.equal(flat[keep], mf[keep])


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_step(kv):
    st = Step(kv, 1)
    total = 0
    for seed in (10, 11, 12):
        st.draw(seed)
        before = st.cache.clone()
        r = st.run()
        assert ops.status(st.ws) == 0
        check(st, before, r)
        total += int(r["num"].sum())
    assert total > 0


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_step_captured_and_replayed(kv):
    st = Step(kv, 2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        st.run()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            r = st.run()
        for seed in (20, 21):
            st.draw(seed)
            before = st.cache.clone()
            g.replay()
            s.synchronize()
            check(st, before, r)
            eager = Step(kv, 2)  # the same step run eagerly over the same cache
            eager.cache.copy_(before)
            eager.draw(seed)
            e = eager.run()
            for k in r:
                assert torch.equal(r[k], e[k]), k
            assert torch.equal(st.cache.view(torch.uint8), eager.cache.view(torch.uint8))


def test_two_steps_on_two_streams():
    # interleaved launches on two streams, each with its own workspace and cache
    a, b = Step("bf16", 3), Step("fp8", 4)
    ca, cb = a.cache.clone(), b.cache.clone()
    want = [a.run(), b.run()]
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    a.cache.copy_(ca)
    b.cache.copy_(cb)
    torch.cuda.synchronize()
    for _ in range(20):
        with torch.cuda.stream(sa):
            ra = a.run()
            a.cache.copy_(ca)
        with torch.cuda.stream(sb):
            rb = b.run()
            b.cache.copy_(cb)
    torch.cuda.synchronize()
    for r, w in zip((ra, rb), want):
        for k in r:
            assert torch.equal(r[k], w[k]), k


def test_calls_on_a_given_stream():
    st = Step("bf16", 5)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    x = st.x
    p, r = ops.rope(x["q"], st.rpos, st.freqs, stream=s)
    e = ops.cache_read(st.cache, st.bt, st.req, st.rpos, entries=torch.zeros(B * T, 576, dtype=torch.bfloat16, device="cuda"), stream=s)
    v = ops.verify_draft(x["target"], x["draft"], x["tok"], x["u"], parents=x["parents"], stream=s)
    s.synchronize()
    assert torch.equal(r, ops.rope(x["q"], st.rpos, st.freqs)[1])
    for a, b in zip(v, ops.verify_draft(x["target"], x["draft"], x["tok"], x["u"], parents=x["parents"])):
        assert torch.equal(a, b)
    assert e.shape == (B * T, 576)


def test_an_output_on_a_given_stream_takes_no_memory_still_in_use():
    # a tensor freed while work queued on the current stream has yet to read it; a call on another
    # stream, whose output has the same size, must not be given that memory
    n = 1 << 14
    x = torch.randn(n, 1, 576, device="cuda").to(torch.bfloat16)
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    freqs, _ = ops.rope_frequencies()
    s = torch.cuda.Stream()
    want = ops.rope(x, pos, freqs)
    torch.cuda.synchronize()
    # blocks of the outputs' two sizes, and no other free ones of those sizes
    held = [torch.full_like(t, 3.0) for t in want for _ in range(8)]
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)  # some 50 ms of the current stream
    copies = [t.clone() for t in held]
    del held[:]
    got = ops.rope(x, pos, freqs, stream=s)
    s.synchronize()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(bool((c == 3.0).all()) for c in copies)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_prefix_read_back_feeds_the_prefill(kv):
    # a prompt written into pages, read back as entries, decompressed: bit for bit what the
    # decompression of the same entries gives
    g = torch.Generator().manual_seed(6)
    L = 300
    prompt = torch.randn(L, 576, generator=g).to(torch.bfloat16).cuda()
    width = 576 if kv == "bf16" else 656
    cache = torch.zeros(8, 64, width, dtype=torch.bfloat16 if kv == "bf16" else torch.uint8, device="cuda")
    bt = torch.randperm(8, generator=g).view(1, 8).to(torch.int32).cuda()
    req, pos = torch.zeros(L, dtype=torch.int32, device="cuda"), torch.arange(L, dtype=torch.int32, device="cuda")
    ops.cache_write(cache, bt, req, pos, prompt)
    entries = ops.cache_read(cache, bt, req, pos)
    _, w_uk, w_uv, _ = inputs.projection_inputs(1, 2, seed=7, device="cuda")
    if kv == "bf16":
        assert torch.equal(entries, prompt)
    else:
        x = prompt[:, :512].double()
        s = x.view(L, 4, 128).abs().amax(2).repeat_interleave(128, 1) / 448
        # e4m3: half a step (2^-4, or 2^-10 of the scale), then bf16 (2^-8)
        assert bool(((entries[:, :512].double() - x).abs() <= (2.0 ** -4 + 2.0 ** -7) * x.abs() + 2.0 ** -9 * s).all())
    k, v = ops.prefill_decompress(entries, w_uk, w_uv)
    want = torch.einsum("hjc,tc->htj", w_uk.double(), entries[:, :512].double())
    assert bool(((k.double() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-3).all())


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_every_call_does_its_work_on_a_given_stream(kv):
    # the current stream is busy meanwhile: what a call queued there, or waited for there, would be
    # missing from its results
    st = Step(kv, 7)
    x, s = st.x, torch.cuda.Stream()
    q_nope = ops.absorb_query(ops.rope(x["q"], st.rpos, st.freqs)[0], st.w_uk).view(B, T, H, 512)
    q_rope = x["q"][..., 128:].contiguous().view(B, T, H, 64)

    def calls(cache, ws, given, stream=None):
        g = given
        p, r = ops.rope(x["q"], st.rpos, st.freqs, mscale=st.mscale, stream=stream)
        ops.rope(x["q"], st.rpos, st.freqs, out_pass=g["p"], out_rot=g["r"], stream=stream)
        ops.cache_write(cache, st.bt, st.req, st.slot, x["kv"], freqs=st.freqs, rope_positions=st.rpos,
                        mscale=st.mscale, norm_weight=st.norm, stream=stream)
        e = ops.cache_read(cache, st.bt, st.req, g["slot"], stream=stream)
        ops.cache_read(cache, st.bt, st.req, st.slot, entries=g["e"], stream=stream)
        ops.plan_tree(ws, st.seq, st.lens, kv_dtype=kv, stream=stream)
        args = (ws, q_nope, q_rope, cache, st.bt, st.seq, st.lens, st.mask, tree_ref.SCALE)
        o, l = ops.decode_tree(*args, out_dtype=torch.bfloat16, stream=stream)
        ops.decode_tree(*args, out=g["o"], lse=g["l"], stream=stream)
        v = ops.verify_draft(x["target"], x["draft"], x["tok"], x["u"], parents=x["parents"], tree_lens=st.lens, stream=stream)
        return [p, r, e, o, l, *v, *(g[k] for k in ("p", "r", "e", "o", "l")), cache.view(torch.uint8)]

    def buffers():
        new = lambda *shape, dtype=torch.bfloat16: torch.full(shape, 7.0, dtype=dtype, device="cuda")
        return dict(p=new(B * T, H, 128), r=new(B * T, H, 64), e=new(B * T, 576), o=new(B, T, H, 512, dtype=torch.float32),
                    l=new(B, T, H, dtype=torch.float32), slot=st.slot.clamp(min=0))

    want = calls(st.cache.clone(), ops.TreeWorkspace(B, T, H), buffers())
    runs = [(st.cache.clone(), ops.TreeWorkspace(B, T, H), buffers()) for _ in range(2)]
    torch.cuda.synchronize()
    calls(*runs[0], stream=s)  # (the allocator's blocks for this stream: an allocation may wait for the device)
    torch.cuda.synchronize()
    torch.cuda._sleep(400_000_000)  # some 200 ms of the current stream
    got = calls(*runs[1], stream=s)
    s.synchronize()
    assert not torch.cuda.current_stream().query()
    with torch.cuda.stream(s):
        same = [torch.equal(a, b) for a, b in zip(got, want)]
    assert all(same), same
    torch.cuda.synchronize()
    assert ops.status(runs[1][1]) == 0
