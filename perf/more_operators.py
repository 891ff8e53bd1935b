"""Cases, inputs and plain forms of the operators of a prompt of text and images that meets states which exist
already: a prefix in the cache, or an encoder's states.

The prompt's tokens have positions on several axes (time, height, width): their queries are rotated by them, and
their keys on the way into the paged cache.  Their queries attend key runs of another length than their own, a
ragged batch at a time (a cached prefix, a chunk over the prefix and itself, an encoder's states), and the result
may be joined with that of an earlier part of the keys.  At the end each prompt token is scored: its log
probability and rank, the row's entropy and best alternatives.

`run(state)` makes one call of one operator: with `own` false in its plain form (elementary torch operations in
32 bits, in 64 where 32 lose what matters, rounded once at the end), with `own` true through this library.
`exact` restates the operator in 64 bits.
"""
import math

import torch

own = False

PAGE, LATENT, ROPE, ENTRY, RECORD = 64, 512, 64, 576, 656
HEAD = 128  # per-head width of the keys' part without positions, and of the values
EPS = 1e-6
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # queries of the first few tokens of a prompt, a slice of a wider projection's output
        dict(name="rope_axes_few", op="rope", tokens=5, heads=16, d_pass=128, d_rot=64, layout="interleaved",
             order="interleaved", strided=True),
        # queries of a long prompt of images, all heads
        dict(name="rope_axes_images", op="rope", tokens=4096, heads=128, d_pass=128, d_rot=64, layout="half",
             order="blocks", strided=False),
        # one short prompt with an image joins a 16-bit cache
        dict(name="write_axes_bf16", op="write", kv="bf16", tokens=333, requests=1, layout="interleaved",
             order="blocks", norm=False),
        # the prompts of a batch join an FP8 cache straight from the down-projection
        dict(name="write_axes_fp8", op="write", kv="fp8", tokens=65536, requests=16, layout="half",
             order="interleaved", norm=True),
        # the smallest: a few tokens of one request over a short encoder run, no position parts
        dict(name="cross_small", op="cross", batch=1, heads=16, q_lo=5, q_hi=5, k_lo=256, k_hi=256, causal=False,
             positions=False, joined=False),
        # single tokens of a serving batch over encoder runs of different lengths, one of eight head shards
        dict(name="cross_single_b64", op="cross", batch=64, heads=16, q_lo=1, q_hi=1, k_lo=256, k_hi=2048,
             causal=False, positions=False, joined=False),
        # prompts of a batch over their images' states, lengths ragged on both sides
        dict(name="cross_batch_b8", op="cross", batch=8, heads=32, q_lo=200, q_hi=1024, k_lo=256, k_hi=2048,
             causal=False, positions=True, joined=False),
        # continued prompts over a part of their prefixes, joined with an earlier part's result
        dict(name="cross_joined_b4", op="cross", batch=4, heads=16, q_lo=256, q_hi=512, k_lo=1024, k_hi=8192,
             causal=False, positions=True, joined=True),
        # a chunk of a long prompt over 8,192 cached tokens and itself, all heads
        dict(name="cross_chunk_h128", op="cross", batch=1, heads=128, q_lo=1001, q_hi=1001, k_lo=9193, k_hi=9193,
             causal=True, positions=True, joined=False),
        # the tokens just sampled by a batch, with alternatives
        dict(name="logprobs_sampled", op="score", rows=16, vocab=131072, dtype="bf16", top=5, masked=0.0, scale=1.0),
        # an odd vocabulary in 32 bits, a third of it masked, at a temperature
        dict(name="logprobs_masked", op="score", rows=257, vocab=32001, dtype="fp32", top=20, masked=0.3, scale=1.25),
        # all tokens of a prompt
        dict(name="logprobs_prompt", op="score", rows=4096, vocab=131072, dtype="bf16", top=20, masked=0.0, scale=1.0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "write", "cross", "cross", "cross", "score", "score"])
    layout, order = rng.choice(["interleaved", "half"]), rng.choice(["interleaved", "blocks"])
    if op == "rope":
        heads = _log(rng, 1, 128)
        return dict(op=op, tokens=_log(rng, 1, 4096 * 128 // heads if heads > 16 else 32768), heads=heads,
                    d_pass=rng.choice([0, 8, 64, 128, 128]), d_rot=rng.choice([24, 64, 64, 128]) if heads < 32 else 64,
                    layout=layout, order=order, strided=rng.random() < 0.5 and heads <= 64)
    if op == "write":
        tokens = _log(rng, 1, 65536)
        return dict(op=op, kv=rng.choice(["bf16", "fp8"]), tokens=tokens, requests=_log(rng, 1, min(tokens, 64)),
                    layout=layout, order=order, norm=rng.random() < 0.5)
    if op == "cross":
        batch, heads = _log(rng, 1, 64), rng.choice([8, 16, 32, 64, 128])
        k_hi = _log(rng, 16, max(32, min(16384, 2000000 // (batch * heads))))  # keys and values: about a GB at most
        causal = rng.random() < 0.4
        # scores of the largest listed case; a causal chunk is part of its keys
        q_hi = _log(rng, 1, max(1, min(4096, k_hi if causal else 4096, 128 * 1001 * 9193 // (batch * heads * k_hi))))
        k_lo = max(1, k_hi // rng.choice([1, 3, 8]))
        return dict(op=op, batch=batch, heads=heads, q_lo=max(1, q_hi // rng.choice([1, 2, 5])), q_hi=q_hi,
                    k_lo=max(k_lo, q_hi) if causal else k_lo, k_hi=k_hi, causal=causal, positions=rng.random() < 0.7,
                    joined=rng.random() < 0.4)
    vocab, dtype = _log(rng, 1000, 262144), rng.choice(["bf16", "bf16", "fp16", "fp32"])
    rows = _log(rng, 1, max(1, min(8192, 4096 * 131072 // (vocab * (2 if dtype == "fp32" else 1)))))
    return dict(op="score", rows=rows, vocab=vocab, dtype=dtype, top=rng.choice([0, 1, 5, 20, 64]),
                masked=rng.choice([0.0, 0.0, 0.3, 0.999]), scale=rng.choice([1.0, 1.25, 0.5]))


# ---------------------------------------------------------------------------------------------- inputs
def _gen(case, seed):
    return torch.Generator(device=DEV).manual_seed(seed * 1000003 + len(repr(sorted(case.items()))))


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def _bf16(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)


def _freqs(d_rot):
    """Radians per position of each pair, 64 bits."""
    return (10000.0 ** (-2.0 * torch.arange(d_rot // 2, dtype=torch.float64) / d_rot)).to(DEV)


def _sections(d_rot):
    """How many pairs turn by time, height and width: a quarter, and halves of the rest."""
    pairs = d_rot // 2
    time = pairs // 4
    return time, (pairs - time + 1) // 2, (pairs - time) // 2


def _axis_of_pair(d_rot, order):
    """The axis of each pair: one axis after the other, or the axes in turn as long as each has pairs left."""
    counts = _sections(d_rot)
    axis = torch.repeat_interleave(torch.arange(3), torch.tensor(counts))
    if order == "interleaved":  # the i-th pair of an axis comes in round i
        turn = torch.cat([torch.arange(n) for n in counts])
        axis = axis[torch.argsort(turn * 3 + axis)]
    return axis.to(DEV)


def _grid_positions(g, n):
    """Positions [n, 3] of text and images in turn (stored axis by axis): text moves all axes, an image's tokens share
    their time and lie on a grid."""
    run = 64 + int(torch.randint(0, 400, (1,), generator=g, device=DEV))
    side = 1 + int(torch.randint(8, 40, (1,), generator=g, device=DEV))
    at = torch.arange(n, device=DEV)
    part, inside = at // run, at % run
    start = part * run + int(torch.randint(0, 100000, (1,), generator=g, device=DEV))
    image = part % 2 == 1
    pos = torch.stack([torch.where(image, start, start + inside), torch.where(image, start + inside // side, start + inside),
                       torch.where(image, start + inside % side, start + inside)])
    return pos.to(torch.int32).t()


def _ragged_tokens(g, tokens, requests):
    """Which request each of `tokens` tokens belongs to (every request has one), and its place among its tokens."""
    cuts = torch.randperm(tokens - 1, generator=g, device=DEV)[:requests - 1] + 1 if requests > 1 else torch.zeros(0, dtype=torch.int64, device=DEV)
    starts = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), cuts.sort().values])
    at = torch.arange(tokens, device=DEV)
    req = torch.searchsorted(starts, at, right=True) - 1
    return req.to(torch.int32), (at - starts[req]).to(torch.int32)


def _runs(g, batch, lo, hi):
    """Lengths spread over [lo, hi] in any order, and their starts and end [batch + 1]."""
    n = torch.linspace(hi, lo, batch, device=DEV).round().long()[torch.randperm(batch, generator=g, device=DEV)]
    return n, torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), n.cumsum(0)]).to(torch.int32)


def prepare(case, seed):
    g = _gen(case, seed)
    s = {"case": case}
    op = case["op"]
    if op == "rope":
        n, h, d = case["tokens"], case["heads"], case["d_pass"] + case["d_rot"]
        x = _bf16(g, n, h, d)
        if case["strided"]:  # the heads' part of a wider projection output
            x = torch.cat([x.reshape(n, h * d), _bf16(g, n, 64)], 1)[:, :h * d].unflatten(1, (h, d))
        s["x"], s["positions"], s["freqs"] = x, _grid_positions(g, n), _freqs(case["d_rot"])
    elif op == "write":
        n, b = case["tokens"], case["requests"]
        s["requests"], s["positions"] = _ragged_tokens(g, n, b)
        s["positions"] += torch.randint(0, 200, (b,), generator=g, device=DEV, dtype=torch.int32)[s["requests"].long()]
        s["rope_positions"], s["freqs"] = _grid_positions(g, n), _freqs(ROPE)
        last = torch.zeros(b, dtype=torch.int64, device=DEV).scatter_reduce(0, s["requests"].long(), s["positions"].long(), "amax")
        pages = last // PAGE + 1
        pool = n // PAGE + 6 * b  # enough for any split of the tokens
        perm = torch.randperm(pool, generator=g, device=DEV, dtype=torch.int32)
        column = torch.arange(int(pages.max()), device=DEV)
        s["block_table"] = perm[((pages.cumsum(0) - pages).unsqueeze(1) + column).clamp(max=pool - 1)].contiguous()
        fp8 = case["kv"] == "fp8"
        s["cache"] = torch.zeros(pool, PAGE, RECORD if fp8 else ENTRY, device=DEV, dtype=torch.uint8 if fp8 else torch.bfloat16)
        s["kv"] = (_randn(g, n, ENTRY) * (0.3 + 3 * torch.rand(n, 1, generator=g, device=DEV))).to(torch.bfloat16)
        s["weight"] = (1 + 0.2 * _randn(g, LATENT)).to(torch.bfloat16) if case["norm"] else None
    elif op == "cross":
        h = case["heads"]
        s["q_lens"], s["cu_q"] = _runs(g, case["batch"], case["q_lo"], case["q_hi"])
        s["k_lens"], s["cu_k"] = _runs(g, case["batch"], case["k_lo"], case["k_hi"])
        nq, nk = int(s["cu_q"][-1]), int(s["cu_k"][-1])
        s["q_nope"], s["k_nope"], s["v"] = _bf16(g, nq, h, HEAD), _bf16(g, h, nk, HEAD), _bf16(g, h, nk, HEAD)
        s["q_rope"], s["entries"] = (_bf16(g, nq, h, ROPE), _bf16(g, nk, ENTRY)) if case["positions"] else (None, None)
        # the result over an earlier part of the keys: some of its mass, and nothing for some rows
        s["before"] = None
        if case["joined"]:
            lse = 6.0 + 2.0 * _randn(g, nq, h)
            lse[torch.rand(nq, h, generator=g, device=DEV) < 0.02] = -math.inf
            s["before"] = (0.05 * _randn(g, nq, h, HEAD), lse)
        s["scale"] = 1.0 / math.sqrt(HEAD + (ROPE if case["positions"] else 0))
    else:
        n, v = case["rows"], case["vocab"]
        # rows between nearly uniform and nearly certain, as a language model's are
        logits = _randn(g, n, v).mul_(0.5 + 4 * torch.rand(n, 1, generator=g, device=DEV))
        if case["masked"]:
            logits.masked_fill_(torch.rand(n, v, generator=g, device=DEV) < case["masked"], -math.inf)
            logits[:, int(torch.randint(0, v, (1,), generator=g, device=DEV))] = 1.0  # (some token is always allowed)
        s["logits"] = logits.to(TYPES[case["dtype"]])
        # the sampled tokens: one of the likelier half of a few, none at a padded row
        few = torch.randint(0, v, (n, 8), generator=g, device=DEV)
        s["tokens"] = few.gather(1, s["logits"].float().gather(1, few).argmax(1, keepdim=True)).squeeze(1).to(torch.int32)
        s["tokens"][torch.rand(n, generator=g, device=DEV) < 0.03] = -1
    return s


# ---------------------------------------------------------------------------------------------- the calls
def run(s):
    if own:
        return _own(s)
    return {"rope": _rope, "write": _write, "cross": _cross, "score": _score}[s["case"]["op"]](s)


def _own(s):
    from mla_latent_kv_17_gb300 import ops
    case = s["case"]
    if case["op"] in ("rope", "write") and "axes" not in s:  # a program keeps the axes of its model's pairs
        s["axes"] = ops.rope_axes(_sections(case.get("d_rot", ROPE)), case["order"])
    if case["op"] == "rope":
        out = ops.rope(s["x"], s["positions"], s["freqs"], layout=case["layout"], axes=s["axes"])
        return out if case["d_pass"] else (s["x"][..., :0], out[1])  # (nothing passes: no output for it)
    if case["op"] == "write":
        ops.cache_write(s["cache"], s["block_table"], s["requests"], s["positions"], s["kv"], freqs=s["freqs"],
                        rope_positions=s["rope_positions"], layout=case["layout"], norm_weight=s["weight"],
                        norm_eps=EPS, axes=s["axes"])
        return _parts(s["cache"])
    if case["op"] == "cross":
        if "ws" not in s:  # a program keeps its workspace
            s["ws"] = ops.CrossWorkspace(case["batch"], case["heads"], s["q_nope"].shape[0])
        ops.plan_cross(s["ws"], s["cu_q"], s["cu_k"], s["v"].shape[1], causal=case["causal"])
        return ops.cross_attention(s["ws"], s["q_nope"], s["q_rope"], s["entries"], s["k_nope"], s["v"], s["scale"],
                                   before=s["before"], out_dtype=torch.bfloat16)
    got = ops.token_logprobs(s["logits"], s["tokens"], top=case["top"], scale=case["scale"])
    return got if case["top"] else got[:3]


def _parts(cache):
    """The cache's values: entries, or an FP8 cache's codes, scales and RoPE part (views)."""
    if cache.dtype == torch.bfloat16:
        return cache
    return (cache[..., :LATENT].view(torch.float8_e4m3fn), cache[..., LATENT:LATENT + 16].view(torch.float32),
            cache[..., LATENT + 16:].view(torch.bfloat16))


# ---------------------------------------------------------------------------------------------- plain forms
def _rotated(x, positions, freqs, case):
    """x [n, ..., d] in 32 bits, pair j turned by the position on its axis; the angles in 64 bits."""
    angle = positions.double()[:, _axis_of_pair(x.shape[-1], case["order"])] * freqs
    shape = (x.shape[0],) + (1,) * (x.dim() - 2) + (-1,)
    c, s = angle.cos().float().view(shape), angle.sin().float().view(shape)
    if case["layout"] == "interleaved":
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)
    a, b = x.chunk(2, -1)
    return torch.cat([a * c - b * s, a * s + b * c], -1)


def _rope(s):
    case, x = s["case"], s["x"]
    rot = _rotated(x[..., case["d_pass"]:].float(), s["positions"], s["freqs"], case)
    return x[..., :case["d_pass"]].contiguous(), rot.to(torch.bfloat16)


def _records(latent, rope):
    """FP8 records of cache entries: codes, scales, RoPE."""
    x = latent.float().reshape(-1, 4, 128)
    amax = x.abs().amax(-1, keepdim=True)
    s = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
    codes = (x / s).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).reshape(-1, LATENT).view(torch.uint8)
    return torch.cat([codes, s.reshape(-1, 4).view(torch.uint8), rope.to(torch.bfloat16).view(torch.uint8)], -1)


def _write(s):
    case, cache = s["case"], s["cache"]
    latent, rope = s["kv"][:, :LATENT].float(), s["kv"][:, LATENT:].float()
    if case["norm"]:
        latent = latent * (latent.square().mean(-1, keepdim=True) + EPS).rsqrt() * s["weight"].float()
    rope = _rotated(rope, s["rope_positions"], s["freqs"], case)
    req, pos = s["requests"].long(), s["positions"].long()
    at = s["block_table"].long()[req, pos // PAGE] * PAGE + pos % PAGE
    rows = torch.cat([latent, rope], -1).to(torch.bfloat16) if case["kv"] == "bf16" else _records(latent, rope)
    cache.view(-1, cache.shape[-1])[at] = rows
    return _parts(cache)


def _padded(lens, cu, most):
    """For a batch padded to `most`: each place's row among the packed ones, and whether it is one."""
    at = torch.arange(most, device=DEV)
    real = at < lens.unsqueeze(1)
    return torch.where(real, cu[:-1].long().unsqueeze(1) + at, torch.zeros_like(at)), real


def _cross(s):
    case = s["case"]
    q_at, q_real = _padded(s["q_lens"], s["cu_q"], case["q_hi"])
    k_at, k_real = _padded(s["k_lens"], s["cu_k"], case["k_hi"])
    q, k, v = s["q_nope"].float()[q_at].transpose(1, 2), s["k_nope"].float()[:, k_at], s["v"].float()[:, k_at]
    scores = torch.matmul(q, k.permute(1, 0, 3, 2))                                         # [b, h, q, k]
    if case["positions"]:
        q, k = s["q_rope"].float()[q_at].transpose(1, 2), s["entries"][:, LATENT:].float()[k_at]
        scores += torch.matmul(q, k.unsqueeze(1).transpose(2, 3))
    scores *= s["scale"]
    seen = k_real.unsqueeze(1)
    if case["causal"]:  # the last query sees all keys, the one before all but the last
        last = torch.arange(case["q_hi"], device=DEV) + (s["k_lens"] - s["q_lens"]).unsqueeze(1)
        seen = seen & (torch.arange(case["k_hi"], device=DEV) <= last.unsqueeze(2))
    scores.masked_fill_(~seen.unsqueeze(1), -math.inf)
    top = scores.amax(-1, keepdim=True)
    scores.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
    total = scores.sum(-1, keepdim=True)
    out = torch.matmul(scores, v.transpose(0, 1))
    out = torch.where(total > 0, out / total, torch.zeros_like(out)).transpose(1, 2)[q_real]
    lse = (total.log() + top).squeeze(-1).transpose(1, 2)[q_real]
    if case["joined"]:
        first, first_lse = s["before"]
        both = torch.logaddexp(first_lse, lse)
        out = first * (first_lse - both).exp().unsqueeze(-1) + out * (lse - both).exp().unsqueeze(-1)
        lse = both
    return out.to(torch.bfloat16), lse


def _ordered(x):
    """Whole numbers in the order of the floats x (-0 as 0)."""
    bits = (x.float() + 0.0).view(torch.int32).long()
    return torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits)


def _score(s):
    case = s["case"]
    y = s["logits"].float() * case["scale"]
    m = y.amax(1, keepdim=True)
    y -= torch.where(m == -math.inf, torch.zeros_like(m), m)
    e = y.exp()
    total = e.sum(1)
    given = s["tokens"] >= 0
    x = s["tokens"].long().clamp(min=0).unsqueeze(1)
    log_total = total.log()
    logprob = torch.where(given, y.gather(1, x).squeeze(1) - log_total, torch.zeros_like(total))
    entropy = log_total - torch.where(e > 0, e.mul_(y), torch.zeros_like(e)).sum(1) / total
    at = torch.arange(case["vocab"], device=DEV)
    mine = s["logits"].gather(1, x)
    ahead = (s["logits"] > mine) | ((s["logits"] == mine) & (at < x))
    rank = torch.where(given, ahead.sum(1), torch.full_like(x.squeeze(1), -1)).to(torch.int32)
    if not case["top"]:
        return logprob, entropy, rank
    # one whole number for each (logit, token): larger logits first, then lower tokens
    keys = (_ordered(s["logits"]) << 20) + (1 << 20) - 1 - at
    best = (1 << 20) - 1 - (keys.topk(case["top"], 1).values & ((1 << 20) - 1))
    alt = y.gather(1, best) - log_total.unsqueeze(1)
    best = torch.where(alt == -math.inf, torch.full_like(best, -1), best)
    return logprob, entropy, rank, best.to(torch.int32), alt


# ---------------------------------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op == "rope":
        n, d = case["tokens"] * case["heads"], case["d_pass"] + case["d_rot"]
        return {"bytes": 4.0 * n * d + 12 * case["tokens"], "flops": 3.0 * n * case["d_rot"]}
    if op == "write":
        row = ENTRY * 2 if case["kv"] == "bf16" else RECORD
        return {"bytes": case["tokens"] * (ENTRY * 2.0 + row + 24), "flops": case["tokens"] * 4.0 * LATENT}
    if op == "cross":
        b, h, width = case["batch"], case["heads"], HEAD + (ROPE if case["positions"] else 0)
        nq = case["q_hi"] if b == 1 else (case["q_lo"] + case["q_hi"]) / 2  # the means of the lengths
        nk = case["k_hi"] if b == 1 else (case["k_lo"] + case["k_hi"]) / 2
        pairs = nq * nk - (nq * nq / 2 if case["causal"] else 0)
        rows = h * nq * (2 * width + 2 * HEAD + 4 + (4 * HEAD + 4 if case["joined"] else 0))
        keys = nk * (h * 4 * HEAD + (2 * ROPE if case["positions"] else 0))
        return {"bytes": b * (rows + keys), "flops": 2.0 * b * h * pairs * (width + HEAD)}
    n = case["rows"]
    size = 4 if case["dtype"] == "fp32" else 2
    return {"bytes": n * (case["vocab"] * float(size) + 16 + 8 * case["top"]), "flops": 5.0 * n * case["vocab"]}


# ---------------------------------------------------------------------------------------------- in 64 bits
def _turned64(x, positions, freqs, case):
    half = x.shape[-1] // 2
    counts, i = _sections(2 * half), torch.arange(half, device=DEV)
    if case["order"] == "blocks":
        axis = (i >= counts[0]).long() + (i >= counts[0] + counts[1]).long()
    else:  # three in turn while time lasts, then height and width
        rest = i - 3 * counts[0]
        axis = torch.where(rest < 0, i % 3, 1 + rest % 2)
    first = 2 * i if case["layout"] == "interleaved" else i
    second = first + 1 if case["layout"] == "interleaved" else i + half
    angle = torch.gather(positions.double(), 1, axis.expand(x.shape[0], half)) * freqs
    z = torch.polar(torch.ones_like(angle), angle).view((x.shape[0],) + (1,) * (x.dim() - 2) + (half,))
    y = torch.complex(x[..., first], x[..., second]) * z
    out = torch.empty_like(x)
    out[..., first], out[..., second] = y.real, y.imag
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        x = s["x"].double()
        return x[..., :case["d_pass"]].contiguous(), _turned64(x[..., case["d_pass"]:].contiguous(), s["positions"], s["freqs"], case)
    if op == "write":
        kv, req, pos = s["kv"].double(), s["requests"].long(), s["positions"].long()
        rows = s["block_table"].long()[req, torch.div(pos, PAGE, rounding_mode="floor")] * PAGE + pos.remainder(PAGE)
        latent, rope = kv[:, :LATENT], _turned64(kv[:, LATENT:].contiguous(), s["rope_positions"], s["freqs"], case)
        if case["norm"]:
            latent = latent / ((latent ** 2).sum(1, keepdim=True) / LATENT + EPS).sqrt() * s["weight"].double()
        pages = s["cache"].shape[0]
        place = lambda v: torch.zeros(pages * PAGE, v.shape[1], dtype=torch.float64, device=DEV).index_copy_(0, rows, v).view(pages, PAGE, -1)
        if case["kv"] == "bf16":
            return place(torch.cat([latent, rope], 1))
        scale = latent.reshape(-1, 4, 128).abs().amax(2) / 448
        codes = (latent / scale.repeat_interleave(128, 1)).float().to(torch.float8_e4m3fn).double()  # what the codes stand for
        return place(codes), place(scale), place(rope)
    if op == "cross":
        nq, h = s["q_nope"].shape[:2]
        out, lse = torch.zeros(nq, h, HEAD, dtype=torch.float64, device=DEV), torch.zeros(nq, h, dtype=torch.float64, device=DEV)
        q0, k0 = s["cu_q"].tolist(), s["cu_k"].tolist()
        for b in range(case["batch"]):
            rows, keys = slice(q0[b], q0[b + 1]), slice(k0[b], k0[b + 1])
            n, m = q0[b + 1] - q0[b], k0[b + 1] - k0[b]
            hidden = torch.ones(n, m, dtype=torch.bool, device=DEV).triu(m - n + 1) if case["causal"] else None
            for i in range(h):
                x = s["q_nope"][rows, i].double() @ s["k_nope"][i, keys].double().T
                if case["positions"]:
                    x += s["q_rope"][rows, i].double() @ s["entries"][keys, LATENT:].double().T
                x *= s["scale"]
                if hidden is not None:
                    x[hidden] = -math.inf
                lse[rows, i] = x.logsumexp(1)
                out[rows, i] = (x - lse[rows, i].unsqueeze(1)).exp_() @ s["v"][i, keys].double()
        if case["joined"]:
            first, first_lse = s["before"][0].double(), s["before"][1].double()
            share = torch.sigmoid(lse - first_lse).unsqueeze(-1)  # the new part's
            return first * (1 - share) + out * share, torch.logsumexp(torch.stack([first_lse, lse]), 0)
        return out, lse
    n, top = case["rows"], case["top"]
    logprob, entropy = torch.zeros(n, dtype=torch.float64, device=DEV), torch.zeros(n, dtype=torch.float64, device=DEV)
    alt = torch.zeros(n, top, dtype=torch.float64, device=DEV)
    for i in range(0, n, 256):
        p = (s["logits"][i:i + 256].double() * case["scale"]).log_softmax(1)
        x = s["tokens"][i:i + 256].long()
        logprob[i:i + 256] = torch.where(x >= 0, p.gather(1, x.clamp(min=0).unsqueeze(1)).squeeze(1), 0.0)
        entropy[i:i + 256] = -(p.exp() * p.clamp(min=-1e4)).sum(1)
        if top:
            alt[i:i + 256] = p.topk(top, 1).values
    return (logprob, entropy, None, None, alt) if top else (logprob, entropy, None)
