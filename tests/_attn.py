"""The attention operators and the 8-bit norm again, in 64 bits and from their definitions, and bounds on what 32-bit
arithmetic may lose."""
import math

import torch

HALF_BF16 = torch.finfo(torch.bfloat16).eps / 2
HALF_E4M3 = torch.finfo(torch.float8_e4m3fn).eps / 2
STEP = 2.0 ** -23   # a 32-bit sum may be cut to its last place by a matrix instruction
TINY_E4M3 = 2.0 ** -10  # half of the smallest e4m3 value


def rotated(x, positions, freq, axis, interleaved):
    """float64 [T, heads, D] of x with its first 2 len(freq) columns turned; positions [axes, T]."""
    out, n = x.double().clone(), len(freq)
    for i in range(n):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
        angle = positions[axis[i] if axis else 0].double() * freq[i]
        c, s = torch.cos(angle).unsqueeze(1), torch.sin(angle).unsqueeze(1)
        u, v = x[..., a].double(), x[..., b].double()
        out[..., a], out[..., b] = u * c - v * s, v * c + u * s
    return out


def rope_slack(x, freq, interleaved):
    """What the turned values may be off before they are rounded: the reduced angle, |2 pi frac| <= pi, is cut to 2^-32 of a
    turn and good to its last place (2^-24 of it), sincospi to 2^-22 with it; two products and a sum add 2^-23: together less
    than 2^-20 of |a| + |b|."""
    slack, n = torch.zeros_like(x, dtype=torch.float64), len(freq)
    cols = torch.arange(n, device=x.device)
    a, b = (2 * cols, 2 * cols + 1) if interleaved else (cols, cols + n)
    both = (x[..., a].double().abs() + x[..., b].double().abs()) * 2.0 ** -20
    slack[..., a], slack[..., b] = both, both
    return slack


def check_e4m3(code, want, slack, what):
    """code (float8) against unrounded values `want` (already divided by their scale): half a step, plus slack."""
    got = code.double()
    want = want.clamp(-448, 448)
    bound = torch.clamp(want.abs() * HALF_E4M3, min=TINY_E4M3) * (1 + 2.0 ** -20) + slack
    off = (got - want).abs()
    # a slack that carries a value over a border between two codes: the next code's half step
    assert bool((off <= bound * (1 + HALF_E4M3)).all()), f"{what}: {float((off / bound).max())} of the bound"


def attend(q, k, v, scale):
    """One sequence and key-value head: q [G, D], k, v [n, D] in 64 bits -> out [G, D], lse [G], and the bounds' parts:
    scores' error, weighted |v|."""
    z = (q @ k.t()) * scale
    lse = torch.logsumexp(z, 1)
    p = torch.softmax(z, 1)
    terms = (q.abs() @ k.abs().t()).amax(1) * abs(scale)
    return p @ v, lse, terms, p @ v.abs(), z.abs().amax(1)


def decode_ref(q, k, v, table, lengths, page, window, scale, ks=None, vs=None, eight=False):
    """(out, out's bound, lse, lse's bound) of ar_attn_decode.  k, v [pages, page, kv, D]; tokens on pages outside the cache
    are left out.

    Bounds: a score is a chain of D / 16 matrix instructions, each of which may lose a last place of the running sum of
    magnitudes, and its scaling and exponential lose 2^-22 of its size and 2^-21; each weight is then off by that share,
    and by its rounding to the products' operands (two bf16: 2^-17; one half: 2^-11); sums over n tokens lose at most
    n / 4 + 64 last places of the sum of magnitudes.  Weights and their sum both err: twice."""
    B, heads, D = q.shape
    kv = k.shape[2]
    G = heads // kv
    out = torch.zeros(B, heads, D, dtype=torch.float64, device=q.device)
    slack, lse = torch.zeros_like(out), torch.full((B, heads), float("-inf"), dtype=torch.float64, device=q.device)
    lse_slack = torch.zeros_like(lse)
    for b in range(B):
        n = max(0, min(int(lengths[b]), table.shape[1] * page))
        at = torch.arange(max(0, n - window) if window else 0, n, device=q.device)
        if at.numel() == 0:
            continue
        pages = table[b, at // page].long()
        good = (pages >= 0) & (pages < k.shape[0])
        at, pages = at[good], pages[good]
        if at.numel() == 0:
            continue
        for h in range(kv):
            rows = slice(h * G, (h + 1) * G)
            kk, vv = k[:, :, h][pages, at % page].double(), v[:, :, h][pages, at % page].double()
            if ks is not None:
                kk, vv = kk * ks[h].double(), vv * vs[h].double()
            o, l, terms, weighted, size = attend(q[b, rows].double(), kk, vv, scale)
            chain = (at.numel() / 4 + 64) * STEP
            score = terms * (D / 16 + 8) * STEP + size * 2.0 ** -22 + 2.0 ** -21
            weight = score + (2.0 ** -11 if eight else 2.0 ** -17)
            out[b, rows], lse[b, rows] = o, l
            slack[b, rows] = HALF_BF16 * o.abs() + (2 * weight + 2 * chain).unsqueeze(1) * weighted + 2.0 ** -134
            lse_slack[b, rows] = score + chain + l.abs() * 2.0 ** -22
    return out, slack * (1 + 2.0 ** -8), lse, lse_slack


def norm_q8_ref(partials, residual, gamma, weight_bias, eps, group, bf16_h=False):
    """(y, scale, h) in 64 bits; scale [T, groups]."""
    T, H = residual.shape
    h = residual.double()
    for p in partials:
        h = h + p.double()
    x = h.float().bfloat16().double() if bf16_h else h
    y = x / torch.sqrt((x * x).mean(1, keepdim=True) + eps) * (gamma.double() + weight_bias)
    scale = torch.stack([c.abs().amax(1) for c in y.split(group or H, dim=1)], 1) / 448.0
    return y, torch.where(scale == 0, 1.0, scale), h
