"""Tree attention in 64 bits (torch float64), and the bounds its bf16 / fp16 operands allow."""
import math

import torch

SCALE = 1.0 / math.sqrt(192.0)


def entries(cache, block_table, b, total):
    pages = block_table[b, :(total + 63) // 64].long()
    rows = cache[pages].reshape(-1, cache.shape[-1])[:total]
    if cache.dtype == torch.bfloat16:
        return rows.double()
    s = rows[:, 512:528].contiguous().view(torch.float32).double().repeat_interleave(128, 1)
    return torch.cat([rows[:, :512].contiguous().view(torch.float8_e4m3fn).double() * s,
                      rows[:, 528:].contiguous().view(torch.bfloat16).double()], 1)


def tree(qn, qr, cache, bt, seq, lens, mask, scale=SCALE):
    """-> out, lse (float64, as defined) and per output the error bounds.

    The kernel's scores are fp32 sums of 576 exact products: off by at most 576 x 2^-23 (its
    accumulator may cut instead of round) of scale sum |q||c|, d below; FP8 latents also enter as
    fp16 (2^-11 (1 + 2^-4) |x|: one rounding of code x scale, the scale held to 2^-15; 2^-25 below the
    normal range).  A weight is off by the factor e^2d (its score and the
    normaliser) and is rounded to bf16 (2^-8; fp16 for FP8 records 2^-11) when formed and once more when its page is
    rescaled; the values of FP8 records are rounded once (2^-11)."""
    B, T, H, _ = qn.shape
    fp8 = cache.dtype != torch.bfloat16
    half = 2.0 ** -11 if fp8 else 2.0 ** -8
    out = torch.zeros(B, T, H, 512, dtype=torch.float64, device=qn.device)
    lse = torch.full((B, T, H), -math.inf, dtype=torch.float64, device=qn.device)
    bo, bl = torch.zeros_like(out), torch.zeros(B, T, H, dtype=torch.float64, device=qn.device)
    for b in range(B):
        total, n = int(seq[b]), int(lens[b]) if lens is not None else T
        if total == 0 or n == 0:
            continue
        e = entries(cache, bt, b, total)
        for i in range(n):
            bits = int(mask[b, i]) & ((1 << 64) - 1)
            keep = list(range(total - n)) + [total - n + j for j in range(n) if bits >> j & 1]
            if not keep:
                continue
            k = e[keep]
            q = torch.cat([qn[b, i], qr[b, i]], -1).double()
            s = q @ k.T * scale
            lse[b, i] = s.logsumexp(-1)
            p = (s - lse[b, i, :, None]).exp()
            out[b, i] = p @ k[:, :512]
            d = (q.abs() @ k.T.abs()).amax(-1) * scale * 576 * 2.0 ** -23
            if fp8:
                d = d + (q[:, :512].abs() @ (2.0 ** -11 * (1 + 2.0 ** -4) * k[:, :512].abs() + 2.0 ** -25).T).amax(-1) * scale
            mean = p @ k[:, :512].abs()
            bo[b, i] = mean * (2 * half + (half * (1 + 2.0 ** -4) if fp8 else 0.0) + 2.1 * d[:, None]) * 1.01
            bl[b, i] = d + 2.0 ** -20 * (1 + lse[b, i].abs())
    return out, lse, bo, bl


def check(out, lse, ref, what=""):
    ro, rl, bo, bl = ref
    o = out.double()
    if out.dtype == torch.bfloat16:
        bo = bo + 2.0 ** -8 * (ro.abs() + bo)
    bad = ~((o - ro).abs() <= bo + 1e-30)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} outputs off, worst {float(((o - ro).abs() - bo).nan_to_num(9e9).max())}"
    if lse is not None:
        l = lse.double()
        empty = torch.isneginf(rl)
        assert torch.equal(torch.isneginf(l), empty), f"{what}: empty rows"
        bad = ~((l - rl).abs() <= bl) & ~empty
        assert not bool(bad.any()), f"{what}: {int(bad.sum())} lse off, worst {float(((l - rl).abs() - bl)[~empty].max())}"
