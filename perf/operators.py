"""Cases, inputs and plain forms of the operators of one speculative decoding step over the latent cache.

A step takes T drafted tokens per request (a tree: each token has a parent among the earlier ones, or the
request's last committed token), rotates their queries and keys (rotary positions), writes their entries into
the paged cache (quantised where the cache is FP8), attends from every drafted token to the request's cache
and to the drafted tokens it descends from (tree attention), and decides from the target's and the draft's
probabilities which of them stand (verification).  A prefix that is to be prefilled against is read back from
the cache (cache read).

`run(state)` makes one call of one operator: with `own` false in its plain form (elementary torch operations in
32 bits, in 64 where 32 lose what matters, rounded once at the end), with `own` true through this library.
`exact` restates the operator in 64 bits.
"""
import math

import numpy as np
import torch

own = False

PAGE, LATENT, ROPE, ENTRY, RECORD = 64, 512, 64, 576, 656
HEAD = 128                      # per-head width of the query's part without positions
SCALE = 1.0 / math.sqrt(192.0)  # 1 / sqrt(128 + 64)
EPS = 1e-6
DEV = "cuda"

#: the tree attention's inputs and workspace of one state
_TREE = ("q_nope", "q_rope", "cache", "block_table", "seq_lens", "tree_lens", "mask")


# ---------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # queries of a few drafted tokens at far positions of a context stretched beyond its training length
        dict(name="rope_q_draft", op="rope", tokens=5, heads=16, d_pass=128, d_rot=64, layout="interleaved",
             far=1000000, yarn=40.0, strided=True),
        # queries of a long prefill, all heads
        dict(name="rope_q_prefill", op="rope", tokens=4096, heads=128, d_pass=128, d_rot=64, layout="half",
             far=4096, yarn=0.0, strided=False),
        # drafted tokens of a batch join a 16-bit cache: 64 requests, 8 tokens each
        dict(name="write_bf16_draft", op="write", kv="bf16", tokens=512, requests=64, layout="interleaved", norm=False),
        # the prompts of a batch join an FP8 cache straight from the down-projection
        dict(name="write_fp8_prompts", op="write", kv="fp8", tokens=65536, requests=16, layout="interleaved", norm=True),
        # a prefix read back for a continued prefill: an odd length of a 16-bit cache, and a long FP8 one
        dict(name="read_bf16_prefix", op="read", kv="bf16", tokens=1001, requests=3),
        dict(name="read_fp8_prefix", op="read", kv="fp8", tokens=65536, requests=4),
        # the smallest step: one request, five drafted tokens, a short context, few heads
        dict(name="tree_small", op="tree", kv="bf16", batch=1, heads=16, drafted=5, lo=256, hi=256, ragged=False),
        # a serving batch on one of eight head shards: 8 tokens x 16 heads fill one 128-row tile
        dict(name="tree_b64_h16", op="tree", kv="bf16", batch=64, heads=16, drafted=8, lo=1024, hi=8192, ragged=True),
        # all heads on one GPU: the products bound it
        dict(name="tree_b16_h128", op="tree", kv="bf16", batch=16, heads=128, drafted=8, lo=1024, hi=8192, ragged=True),
        # FP8 records, ragged contexts
        dict(name="tree_fp8_b32_h128", op="tree", kv="fp8", batch=32, heads=128, drafted=4, lo=1024, hi=8192, ragged=True),
        # a chain of drafted tokens with the draft's probabilities
        dict(name="verify_chain", op="verify", batch=64, drafted=4, vocab=131072, tree=False, probs=True),
        # a tree of candidates without probabilities (the draft's best ones), an odd vocabulary
        dict(name="verify_tree", op="verify", batch=3, drafted=12, vocab=32001, tree=True, probs=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "write", "read", "tree", "tree", "verify"])
    layout = rng.choice(["interleaved", "half"])
    kv = rng.choice(["bf16", "fp8"])
    if op == "rope":
        heads = _log(rng, 1, 128)
        return dict(op=op, tokens=_log(rng, 1, 4096 * 128 // heads if heads > 16 else 32768), heads=heads,
                    d_pass=rng.choice([0, 8, 64, 128, 128, 128]), d_rot=rng.choice([16, 64, 64, 64, 128]) if heads < 32 else 64,
                    layout=layout, far=_log(rng, 64, 4000000), yarn=rng.choice([0.0, 4.0, 40.0]),
                    strided=rng.random() < 0.5 and heads <= 64)
    if op == "write":
        tokens = _log(rng, 1, 65536)
        return dict(op=op, kv=kv, tokens=tokens, requests=_log(rng, 1, min(tokens, 128)), layout=layout,
                    norm=rng.random() < 0.5)
    if op == "read":
        tokens = _log(rng, 1, 65536)
        return dict(op=op, kv=kv, tokens=tokens, requests=_log(rng, 1, min(tokens, 128)))
    if op == "tree":
        heads, drafted, batch = rng.choice([8, 16, 32, 48, 64, 128]), _log(rng, 1, 64), _log(rng, 1, 64)
        # rows x tokens of the largest listed case, and a bounded score matrix
        most = min(16 * 128 * 8 * 4608 // (batch * heads * drafted), 65536)
        hi = max(drafted, _log(rng, max(16, most // 16), max(16, most)))
        lo = max(1, hi // rng.choice([1, 4, 16]))
        if kv == "fp8":
            lo, hi = max(lo, 64), max(hi, 64)
        return dict(op=op, kv=kv, batch=batch, heads=heads, drafted=drafted, lo=lo, hi=hi, ragged=rng.random() < 0.7)
    drafted, vocab = _log(rng, 1, 16), _log(rng, 1000, 131072)
    return dict(op="verify", batch=max(1, min(64, 64 * 4 * 131072 // (drafted * vocab), _log(rng, 1, 64))),
                drafted=drafted, vocab=vocab, tree=rng.random() < 0.5, probs=rng.random() < 0.6)


# ---------------------------------------------------------------------------------------------- inputs
def _gen(case, seed):
    return torch.Generator(device=DEV).manual_seed(seed * 1000003 + len(repr(sorted(case.items()))))


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def _freqs(d_rot, yarn):
    """Angular frequencies (radians per position, 64 bits) and the factor on the rotated values: base 10000,
    or with YaRN's ramp between kept and divided frequencies (factor `yarn`, trained length 4096)."""
    j = torch.arange(d_rot // 2, dtype=torch.float64)
    f = 10000.0 ** (-2.0 * j / d_rot)
    if not yarn:
        return f.to(DEV), 1.0
    at = lambda turns: d_rot * math.log(4096 / (turns * 2 * math.pi)) / (2 * math.log(10000.0))
    lo, hi = max(math.floor(at(32)), 0), min(math.ceil(at(1)), d_rot - 1)
    keep = 1.0 - ((j - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
    return (f / yarn * (1 - keep) + f * keep).to(DEV), 0.1 * math.log(yarn) + 1.0


def _records(latent, rope):
    """FP8 records of cache entries: codes, scales, RoPE."""
    x = latent.float().reshape(-1, 4, 128)
    amax = x.abs().amax(-1, keepdim=True)
    s = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
    codes = (x / s).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).reshape(-1, LATENT).view(torch.uint8)
    return torch.cat([codes, s.reshape(-1, 4).view(torch.uint8), rope.to(torch.bfloat16).view(torch.uint8)], -1)


def _filled(g, pages, kv):
    """A pool of pages of N(0, 1) entries."""
    if kv == "bf16":
        return _randn(g, pages, PAGE, ENTRY).to(torch.bfloat16)
    rows = [_records(_randn(g, n * PAGE, LATENT), _randn(g, n * PAGE, ROPE))
            for n in [min(1024, pages - p) for p in range(0, pages, 1024)]]
    return torch.cat(rows).reshape(pages, PAGE, RECORD)


def _tables(g, pages_each, pool=0):
    """A block table over a shuffled pool (of `pool` pages, or of those needed): pages_each pages per request."""
    perm = torch.randperm(max(pool, sum(pages_each)), generator=g, device=DEV, dtype=torch.int32)
    table = torch.zeros(len(pages_each), max(pages_each), dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(pages_each):
        table[b, :n] = perm[at:at + n]
        at += n
    return table


def _ragged_tokens(g, tokens, requests):
    """Which request each of `tokens` tokens belongs to (every request has one), and its place among its tokens."""
    cuts = torch.randperm(tokens - 1, generator=g, device=DEV)[:requests - 1] + 1 if requests > 1 else torch.zeros(0, dtype=torch.int64, device=DEV)
    starts = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), cuts.sort().values])
    at = torch.arange(tokens, device=DEV)
    req = torch.searchsorted(starts, at, right=True) - 1
    return req.to(torch.int32), (at - starts[req]).to(torch.int32)


def _tree(g, batch, drafted, chain):
    """Parents [batch, drafted] (-1: the last committed token) and each token's ancestors and itself as bits."""
    at = torch.arange(drafted, device=DEV)
    back = torch.randint(1, 4, (batch, drafted), generator=g, device=DEV)
    parents = (at - (1 if chain else back)).clamp(min=-1).expand(batch, drafted).contiguous()
    mask = torch.zeros(batch, drafted, dtype=torch.int64, device=DEV)
    one = torch.ones((), dtype=torch.int64, device=DEV)
    for i in range(drafted):
        up = mask.gather(1, parents[:, i:i + 1].clamp(min=0)).squeeze(1)
        mask[:, i] = torch.where(parents[:, i] >= 0, up, torch.zeros_like(up)) | (one << i)
    return parents.to(torch.int32), mask


def prepare(case, seed):
    g = _gen(case, seed)
    s = {"case": case}
    op = case["op"]
    if op == "rope":
        n, h, d = case["tokens"], case["heads"], case["d_pass"] + case["d_rot"]
        x = _randn(g, n, h, d).to(torch.bfloat16)
        if case["strided"]:  # the heads' part of a wider projection output
            x = torch.cat([x.reshape(n, h * d), _randn(g, n, 64).to(torch.bfloat16)], 1)[:, :h * d].unflatten(1, (h, d))
        s["x"] = x
        s["positions"] = torch.randint(0, case["far"], (n,), generator=g, device=DEV, dtype=torch.int32)
        s["freqs"], s["mscale"] = _freqs(case["d_rot"], case["yarn"])
    elif op in ("write", "read"):
        n, b = case["tokens"], case["requests"]
        s["requests"], s["positions"] = _ragged_tokens(g, n, b)
        if op == "write":  # each request has a prefix already
            s["positions"] += torch.randint(0, 200, (b,), generator=g, device=DEV, dtype=torch.int32)[s["requests"].long()]
        last = torch.zeros(b, dtype=torch.int64, device=DEV).scatter_reduce(0, s["requests"].long(), s["positions"].long(), "amax")
        pages = [int(p) // PAGE + 1 for p in last.tolist()]
        pool = n // PAGE + 6 * b  # enough for any split of the tokens
        s["block_table"] = _tables(g, pages, pool)
        if op == "read":
            s["cache"] = _filled(g, pool, case["kv"])
        else:
            width = ENTRY if case["kv"] == "bf16" else RECORD
            s["cache"] = torch.zeros(pool, PAGE, width, device=DEV,
                                     dtype=torch.bfloat16 if case["kv"] == "bf16" else torch.uint8)
            s["kv"] = (_randn(g, n, ENTRY) * (0.3 + 3 * torch.rand(n, 1, generator=g, device=DEV))).to(torch.bfloat16)
            s["weight"] = (1 + 0.2 * _randn(g, LATENT)).to(torch.bfloat16) if case["norm"] else None
            s["freqs"], s["mscale"] = _freqs(ROPE, 0.0)
    elif op == "tree":
        b, h, t = case["batch"], case["heads"], case["drafted"]
        context = torch.randint(case["lo"], case["hi"] + 1, (b,), generator=g, device=DEV, dtype=torch.int32)
        s["tree_lens"] = torch.randint(max(1, t // 2), t + 1, (b,), generator=g, device=DEV, dtype=torch.int32) if case["ragged"] else torch.full((b,), t, dtype=torch.int32, device=DEV)
        s["seq_lens"] = context + s["tree_lens"]
        pages = [(int(x) + PAGE - 1) // PAGE for x in s["seq_lens"].tolist()]
        s["block_table"] = _tables(g, pages)
        s["cache"] = _filled(g, sum(pages), case["kv"])
        s["q_nope"] = _randn(g, b, t, h, LATENT).to(torch.bfloat16)
        s["q_rope"] = _randn(g, b, t, h, ROPE).to(torch.bfloat16)
        s["mask"] = _tree(g, b, t, chain=False)[1]
    else:
        b, t, v = case["batch"], case["drafted"], case["vocab"]
        parents, _ = _tree(g, b, t, chain=not case["tree"])
        target = 3.0 * _randn(g, b, t + 1, v)
        draft = target + 0.7 * _randn(g, b, t + 1, v)
        target, draft = target.softmax(-1), draft.softmax(-1)
        draft = draft.gather(1, (parents.long() + 1).unsqueeze(-1).expand(b, t, v))  # what each token was drawn from
        noise = torch.rand(b, t, v, generator=g, device=DEV).clamp_(min=1e-20)
        s["tokens"] = (draft / -noise.log()).argmax(-1).to(torch.int32)
        s["target"], s["draft"] = target, draft if case["probs"] else None
        s["parents"] = parents if case["tree"] else None
        s["uniforms"] = torch.rand(b, t + 1, generator=g, device=DEV)
    return s


# ---------------------------------------------------------------------------------------------- the calls
def run(s):
    if own:
        return _own(s)
    return {"rope": _rope, "write": _write, "read": _read, "tree": _attend, "verify": _verify}[s["case"]["op"]](s)


def _own(s):
    from mla_latent_kv_17_gb300 import ops
    case = s["case"]
    if case["op"] == "rope":
        out = ops.rope(s["x"], s["positions"], s["freqs"], layout=case["layout"], mscale=s["mscale"])
        return out if case["d_pass"] else (s["x"][..., :0], out[1])  # (nothing passes: no output for it)
    if case["op"] == "write":
        ops.cache_write(s["cache"], s["block_table"], s["requests"], s["positions"], s["kv"], freqs=s["freqs"],
                        layout=case["layout"], mscale=s["mscale"], norm_weight=s["weight"], norm_eps=EPS)
        return _parts(s["cache"])
    if case["op"] == "read":
        return ops.cache_read(s["cache"], s["block_table"], s["requests"], s["positions"])
    if case["op"] == "tree":
        if "ws" not in s:  # a program keeps its workspace
            s["ws"] = ops.TreeWorkspace(case["batch"], case["drafted"], case["heads"])
        ops.plan_tree(s["ws"], s["seq_lens"], s["tree_lens"], kv_dtype=case["kv"])
        out, lse = ops.decode_tree(s["ws"], s["q_nope"], s["q_rope"], s["cache"], s["block_table"], s["seq_lens"],
                                   s["tree_lens"], s["mask"], SCALE, out_dtype=torch.bfloat16,
                                   with_lse=case["kv"] == "bf16")
        return (out, lse) if case["kv"] == "bf16" else out
    return ops.verify_draft(s["target"], s["draft"], s["tokens"], s["uniforms"], parents=s["parents"])


def _parts(cache):
    """The cache's values: entries, or an FP8 cache's codes, scales and RoPE part (views)."""
    if cache.dtype == torch.bfloat16:
        return cache
    return (cache[..., :LATENT].view(torch.float8_e4m3fn), cache[..., LATENT:LATENT + 16].view(torch.float32),
            cache[..., LATENT + 16:].view(torch.bfloat16))


# ---------------------------------------------------------------------------------------------- plain forms
def _rotated(x, positions, freqs, layout, mscale):
    """x [n, ..., d] in 32 bits, rotated by its token's position; the angles in 64 bits."""
    angle = positions.double().unsqueeze(-1) * freqs
    shape = (x.shape[0],) + (1,) * (x.dim() - 2) + (-1,)
    c, s = (mscale * angle.cos()).float().view(shape), (mscale * angle.sin()).float().view(shape)
    if layout == "interleaved":
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)
    a, b = x.chunk(2, -1)
    return torch.cat([a * c - b * s, a * s + b * c], -1)


def _rope(s):
    case, x = s["case"], s["x"]
    rot = _rotated(x[..., case["d_pass"]:].float(), s["positions"], s["freqs"], case["layout"], s["mscale"])
    return x[..., :case["d_pass"]].contiguous(), rot.to(torch.bfloat16)


def _row_of(s):
    req, pos = s["requests"].long(), s["positions"].long()
    return s["block_table"].long()[req, pos // PAGE] * PAGE + pos % PAGE


def _write(s):
    case, cache = s["case"], s["cache"]
    latent, rope = s["kv"][:, :LATENT].float(), s["kv"][:, LATENT:].float()
    if case["norm"]:
        latent = latent * (latent.square().mean(-1, keepdim=True) + EPS).rsqrt() * s["weight"].float()
    rope = _rotated(rope, s["positions"], s["freqs"], case["layout"], s["mscale"])
    if case["kv"] == "bf16":
        rows = torch.cat([latent, rope], -1).to(torch.bfloat16)
    else:
        rows = _records(latent, rope)
    cache.view(-1, cache.shape[-1])[_row_of(s)] = rows
    return _parts(cache)


def _entries(cache, rows):
    """Entries (latent | RoPE, 32 bits) of cache rows."""
    picked = cache.view(-1, cache.shape[-1])[rows]
    if cache.dtype == torch.bfloat16:
        return picked.float()
    codes, scales, rope = _parts(picked)
    return torch.cat([(codes.float().unflatten(-1, (4, 128)) * scales.unsqueeze(-1)).flatten(-2), rope.float()], -1)


def _read(s):
    return _entries(s["cache"], _row_of(s)).to(torch.bfloat16)


def _visible(s, at):
    """[b, t, l]: does drafted token t attend logical position at[l]?"""
    context = (s["seq_lens"] - s["tree_lens"]).long().view(-1, 1, 1)
    behind = at.view(1, 1, -1) - context
    bit = (s["mask"].unsqueeze(-1) >> behind.clamp(0, 63)) & 1
    seen = (behind < 0) | ((behind < s["tree_lens"].long().view(-1, 1, 1)) & (bit == 1))
    real = torch.arange(s["mask"].shape[1], device=DEV).view(1, -1, 1) < s["tree_lens"].view(-1, 1, 1)
    return seen & real


def _attend(s):
    b, t, h, _ = s["q_nope"].shape
    at = torch.arange(s["block_table"].shape[1] * PAGE, device=DEV)
    rows = s["block_table"].long()[:, at // PAGE] * PAGE + at % PAGE
    entries = _entries(s["cache"], rows)                                                     # [b, l, 576]
    q = torch.cat([s["q_nope"], s["q_rope"]], -1).float().view(b, t * h, ENTRY)
    scores = torch.bmm(q, entries.transpose(1, 2)).mul_(SCALE).view(b, t, h, -1)
    scores.masked_fill_(~_visible(s, at).unsqueeze(2), -math.inf)
    top = scores.amax(-1, keepdim=True)
    scores.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
    total = scores.sum(-1, keepdim=True)
    out = torch.bmm(scores.view(b, t * h, -1), entries[..., :LATENT]).view(b, t, h, LATENT)
    out = torch.where(total > 0, out / total, torch.zeros_like(out)).to(torch.bfloat16)
    lse = (total.log() + top).squeeze(-1)
    return (out, lse) if s["case"]["kv"] == "bf16" else out


def _verify(s):
    """Walks the drafted tokens in order: a token whose parent stands (and that no sibling has replaced) stands
    if u q < p; otherwise the target's remaining distribution loses what the draft's covers."""
    target, draft, tokens, u = s["target"], s["draft"], s["tokens"].long(), s["uniforms"].double()
    b, t = tokens.shape
    parents = s["parents"].long() if s["parents"] is not None else torch.arange(t, device=DEV).expand(b, t) - 1
    at = torch.full((b,), -1, dtype=torch.int64, device=DEV)
    depth = torch.zeros(b, dtype=torch.int64, device=DEV)
    depths = torch.full((b, t), -1, dtype=torch.int32, device=DEV)
    left, mass = target[:, 0].double(), torch.ones(b, dtype=torch.float64, device=DEV)
    for i in range(t):
        x = tokens[:, i:i + 1]
        if draft is None:
            q = torch.zeros_like(left).scatter_(1, x, 1.0)
        else:
            q = draft[:, i].double()
        live = parents[:, i] == at
        stands = live & (u[:, i] * q.gather(1, x).squeeze(1) * mass < left.gather(1, x).squeeze(1))
        rest = (left - mass.unsqueeze(1) * q).clamp(min=0)
        falls = live & ~stands
        left = torch.where(stands.unsqueeze(1), target[:, i + 1].double(), torch.where(falls.unsqueeze(1), rest, left))
        mass = torch.where(stands, torch.ones_like(mass), torch.where(falls, rest.sum(1), mass))
        depths[:, i] = torch.where(stands, depth, torch.full_like(depth, -1)).to(torch.int32)
        at = torch.where(stands, torch.full_like(at, i), at)
        depth = depth + stands
    # nothing left of the target's distribution (it equals the draft's): the target's own row
    own_row = target.gather(1, (at + 1).view(b, 1, 1).expand(b, 1, target.shape[2])).squeeze(1).double()
    left = torch.where((left.sum(1, keepdim=True) > 0), left, own_row)
    upto = left.cumsum(1)
    chosen = (upto <= u[:, t:] * upto[:, -1:]).sum(1)
    return depth.to(torch.int32), depths, chosen.to(torch.int32)


# ---------------------------------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op == "rope":
        n, d = case["tokens"] * case["heads"], case["d_pass"] + case["d_rot"]
        return {"bytes": 4.0 * n * d + 4 * case["tokens"], "flops": 3.0 * n * case["d_rot"]}
    if op in ("write", "read"):
        row = ENTRY * 2 if case["kv"] == "bf16" else RECORD
        n = case["tokens"]
        return {"bytes": n * (ENTRY * 2.0 + row + 12), "flops": n * (4.0 * LATENT if op == "write" else 1.0 * LATENT)}
    if op == "tree":
        b, h, t = case["batch"], case["heads"], case["drafted"]
        tokens = (case["lo"] + case["hi"]) / 2 + t * (0.75 if case["ragged"] else 1.0)  # the mean of the lengths drawn
        rows = h * t * (0.75 if case["ragged"] else 1.0)
        entry = ENTRY * 2 if case["kv"] == "bf16" else RECORD
        return {"bytes": b * (tokens * entry + h * t * (ENTRY * 2.0 + LATENT * 2 + 4)),
                "flops": 2.0 * b * rows * tokens * (ENTRY + LATENT)}
    # one rejection in the middle: a row of the target's and (where given) one of the draft's probabilities
    rows = 2 if case["probs"] else 1
    return {"bytes": case["batch"] * (4.0 * rows * case["vocab"] + 16 * case["drafted"]),
            "flops": 3.0 * case["batch"] * case["vocab"]}


# ---------------------------------------------------------------------------------------------- in 64 bits
def _turned64(x, positions, freqs, layout, mscale):
    half = x.shape[-1] // 2
    pair = (torch.arange(half, device=DEV) * 2, torch.arange(half, device=DEV) * 2 + 1) if layout == "interleaved" else (
        torch.arange(half, device=DEV), torch.arange(half, device=DEV) + half)
    z = torch.polar(torch.full_like(positions, mscale, dtype=torch.float64).unsqueeze(-1) * torch.ones_like(freqs),
                    positions.double().unsqueeze(-1) * freqs)
    z = z.view((x.shape[0],) + (1,) * (x.dim() - 2) + (half,))
    y = torch.complex(x[..., pair[0]], x[..., pair[1]]) * z
    out = torch.empty_like(x)
    out[..., pair[0]], out[..., pair[1]] = y.real, y.imag
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        x = s["x"].double()
        return x[..., :case["d_pass"]].contiguous(), _turned64(x[..., case["d_pass"]:], s["positions"], s["freqs"],
                                                              case["layout"], s["mscale"])
    if op in ("write", "read"):
        req, pos = s["requests"].long(), s["positions"].long()
        rows = s["block_table"].long()[req, torch.div(pos, PAGE, rounding_mode="floor")] * PAGE + pos.remainder(PAGE)
        flat = s["cache"].reshape(-1, s["cache"].shape[-1])
        if op == "read":
            got = flat.index_select(0, rows)
            if case["kv"] == "bf16":
                return got.double()
            scale = got[:, LATENT:LATENT + 16].contiguous().view(torch.float32).double().repeat_interleave(128, 1)
            return torch.cat([got[:, :LATENT].contiguous().view(torch.float8_e4m3fn).double() * scale,
                              got[:, LATENT + 16:].contiguous().view(torch.bfloat16).double()], 1)
        kv = s["kv"].double()
        latent, rope = kv[:, :LATENT], _turned64(kv[:, LATENT:].contiguous(), s["positions"], s["freqs"], case["layout"], s["mscale"])
        if case["norm"]:
            latent = latent / ((latent ** 2).sum(1, keepdim=True) / LATENT + EPS).sqrt() * s["weight"].double()
        shape = s["cache"].shape[:2]
        place = lambda v: torch.zeros(shape[0] * PAGE, v.shape[1], dtype=torch.float64, device=DEV).index_copy_(0, rows, v).view(*shape, -1)
        if case["kv"] == "bf16":
            return place(torch.cat([latent, rope], 1))
        scale = latent.reshape(-1, 4, 128).abs().amax(2) / 448
        codes = (latent / scale.repeat_interleave(128, 1)).float().to(torch.float8_e4m3fn).double()  # what the codes stand for
        return place(codes), place(scale), place(rope)
    if op == "verify":
        return None  # whole numbers
    b, t, h, _ = s["q_nope"].shape
    out = torch.zeros(b, t, h, LATENT, dtype=torch.float64, device=DEV)
    lse = torch.full((b, t, h), -math.inf, dtype=torch.float64, device=DEV)
    bits = s["mask"].cpu().numpy().astype(np.uint64)
    for i in range(b):
        total, n = int(s["seq_lens"][i]), int(s["tree_lens"][i])
        pages = s["block_table"][i, :(total + PAGE - 1) // PAGE].long()
        flat = s["cache"].index_select(0, pages).flatten(0, 1)[:total]
        if case["kv"] == "bf16":
            e = flat.double()
        else:
            scale = flat[:, LATENT:LATENT + 16].contiguous().view(torch.float32).double().repeat_interleave(128, 1)
            e = torch.cat([flat[:, :LATENT].contiguous().view(torch.float8_e4m3fn).double() * scale,
                           flat[:, LATENT + 16:].contiguous().view(torch.bfloat16).double()], 1)
        sees = np.ones((n, total), dtype=bool)
        sees[:, total - n:] = (bits[i, :n, None] >> np.arange(n, dtype=np.uint64)) & np.uint64(1) > 0
        q = torch.cat([s["q_nope"][i, :n], s["q_rope"][i, :n]], -1).double()
        x = (q.reshape(n * h, ENTRY) @ e.T).view(n, h, total) * SCALE
        x[~torch.from_numpy(sees).to(DEV).unsqueeze(1).expand(n, h, total)] = -math.inf
        lse[i, :n] = x.logsumexp(-1)
        out[i, :n] = ((x - lse[i, :n].unsqueeze(-1)).exp_().view(n * h, total) @ e[:, :LATENT]).view(n, h, LATENT)
    return (out, lse) if case["kv"] == "bf16" else out
