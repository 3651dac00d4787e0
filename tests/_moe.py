"""The few-token MoE operators again, in 64 bits and from their definitions, and bounds on what 32-bit sums may lose."""
import math

import torch

# A matrix instruction adds 16 products to a 32-bit sum and may cut, not round, each addend to the sum's last place:
# at most 17 * 2^-23 of the largest magnitude in it, so 2^-18 of the sum of magnitudes per instruction is generous,
# and what one instruction loses is relative to its own 16 products and the running sum.  A chain of n of them and the
# 16 warps' parts lose at most (n + 16) * 2^-23 of the sum of all magnitudes when each step loses one last place of it.
def gamma(cols):
    return (math.ceil(cols / 16) + 24) * 2.0 ** -23


HALF_BF16 = torch.finfo(torch.bfloat16).eps / 2


def w4_values(q, s):
    """float64 weights of packed codes and group scales (any leading shape)."""
    v = torch.empty(*q.shape[:-1], 2 * q.shape[-1], dtype=torch.float64, device=q.device)
    v[..., 0::2] = (q & 15).double() - 8
    v[..., 1::2] = (q >> 4).double() - 8
    return v * s.double().repeat_interleave(v.shape[-1] // s.shape[-1], dim=-1)


def make_w4(rows, cols, group, g, device="cpu"):
    q = torch.randint(0, 256, (*rows, cols // 2), dtype=torch.uint8, generator=g).to(device)
    s = ((torch.rand((*rows, cols // group), generator=g) + 0.5) / (4.6 * math.sqrt(cols))).bfloat16().to(device)
    return q, s


def route_ref(x, gate, bias, K, sigmoid, renorm, scale, n_group, topk_group, shared):
    l = x.double() @ gate.double().t()
    s = torch.sigmoid(l) if sigmoid else torch.softmax(l, dim=1)
    E = l.shape[1]
    ids = torch.empty(l.shape[0], K + shared, dtype=torch.int32)
    w = torch.ones(l.shape[0], K + shared, dtype=torch.float64)
    for t in range(l.shape[0]):
        c = (l if bias is None and n_group == 1 else s if bias is None else s + bias.double())[t].tolist()
        size = E // n_group
        score = [-sum(sorted(c[j * size:(j + 1) * size])[-2:]) for j in range(n_group)]
        kept = set(sorted(range(n_group), key=lambda j: (score[j], j))[:topk_group])
        order = sorted((e for e in range(E) if e // size in kept), key=lambda e: (-c[e], e))[:K]
        ids[t] = torch.tensor(order + list(range(E, E + shared)), dtype=torch.int32)
        v = s[t, order]
        if renorm:
            v = v / v.sum()
        w[t, :K] = v * scale
    return ids, w


def experts_ref(x, ids, weights, w13, w2):
    """(y, bound): the result in 64 bits and how far a bf16 result of 32-bit sums may be from it.  w13, w2: functions of
    an expert's index that return its float64 matrices."""
    T, H = x.shape
    xd = x.double()
    y = torch.zeros(T, H, dtype=torch.float64, device=x.device)
    lost = torch.zeros_like(y)
    for t in range(T):
        for k in range(ids.shape[1]):
            e = int(ids[t, k])
            if e < 0:
                continue
            a13, a2, w = w13(e), w2(e), float(weights[t, k])
            h, m = a13 @ xd[t], a13.abs() @ xd[t].abs()
            I = h.shape[0] // 2
            gt, up = h[:I], h[I:]
            a = gt * torch.sigmoid(gt) * up
            # |silu'| <= 1.1, |silu(g)| <= |g|; the activation's own evaluation: a few last places, and 2^-16 for
            # keeping it as two bf16 parts
            da = gamma(H) * (1.1 * m[:I] * up.abs() + gt.abs() * m[I:]) + a.abs() * (2.0 ** -16 + 2.0 ** -20)
            y[t] += w * (a2 @ a)
            lost[t] += abs(w) * (a2.abs() @ (da + gamma(I) * a.abs()))
    return y, lost + HALF_BF16 * (y.abs() + lost) + 1e-30


def close(got, ref, bound, what):
    err = (got.double() - ref).abs()
    bad = ~(err <= bound)
    assert not bool(bad.any()), (f"{what}: {int(bad.sum())} of {bad.numel()} outside the bound; first "
                                 f"{bad.nonzero()[:3].tolist()}, got {got[bad][:3].tolist()}, want {ref[bad][:3].tolist()}")
    # together: half a bf16 step of every value, and little more
    n = ref.norm()
    assert float((got.double() - ref).norm()) <= float(HALF_BF16 * n * 1.05) + 1e-30, what
