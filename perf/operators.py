"""Cases of the mixture-of-experts operators for a few tokens: the router, the experts' products (bf16 and 4-bit
weights) and the 4-bit matrix-vector product, each in its plain form and as a call of the framework.

    route       logits = x gate^T; scores = softmax or sigmoid; choice by score + bias (or by logit), optionally
                limited to the best expert groups; ids, weights of the top_k chosen, shared experts appended
    experts     y[t] = sum_k w[t,k] * W2_e ( silu(G_e x[t]) * (U_e x[t]) ),  e = ids[t,k],  W13_e = [G_e; U_e]
    experts_w4  the same with 4-bit weights: value = scale[row, k / group] * (code - 8), two codes a byte, low first
    matvec_w4   y[t] = W x[t] with such weights
"""
import math

import torch

own = False

# Sizes: hidden 7168 with 256 experts and top-8 (and 8192 with top-10) are this repository's decode configurations; an
# intermediate size of 256 is what one rank of eight holds of experts 2048 wide.
LISTED = [
    # one decoded token through the router of a large model: grouped choice by sigmoid and bias, a shared expert
    dict(name="route 1 token, groups", op="route", T=1, H=7168, E=256, K=8, scoring="sigmoid", bias=True, groups=8, top_groups=4, shared=1),
    # an ordinary decode batch: sigmoid and bias, no groups
    dict(name="route 16 tokens", op="route", T=16, H=6144, E=160, K=8, scoring="sigmoid", bias=True, groups=1, top_groups=1, shared=0),
    # the largest batch of the few-token path: softmax over the experts, no bias
    dict(name="route 64 tokens, softmax", op="route", T=64, H=4096, E=128, K=8, scoring="softmax", bias=False, groups=1, top_groups=1, shared=0),
    # the smallest layer: one token, two of eight narrow experts (latency counts)
    dict(name="experts 1 token, small", op="experts", T=1, H=1024, E=8, K=2, I=512, pad=0),
    # one decoded token on one rank of eight
    dict(name="experts 1 token, sliced", op="experts", T=1, H=7168, E=256, K=8, I=256, pad=0),
    # a speculative step of a few tokens over whole experts; odd widths, a padded row
    dict(name="experts 5 tokens, whole", op="experts", T=5, H=8192, E=32, K=10, I=1400, pad=1),
    # a full few-token batch on one rank of eight: nearly every expert is read
    dict(name="experts 64 tokens, sliced", op="experts", T=64, H=7168, E=256, K=8, I=256, pad=0),
    # one decoded token, whole experts in 4 bits
    dict(name="experts w4 1 token, whole", op="experts_w4", T=1, H=7168, E=64, K=8, I=2048, group=128, pad=0),
    # a decode batch in 4 bits on one rank, fine groups, padded rows
    dict(name="experts w4 16 tokens, sliced", op="experts_w4", T=16, H=7168, E=256, K=8, I=256, group=32, pad=3),
    # the attention output projection of one rank of eight, one token
    dict(name="matvec w4 1 token, sliced", op="matvec_w4", T=1, N=7168, H=2048, group=128),
    # a wide dense projection for one token
    dict(name="matvec w4 1 token, wide", op="matvec_w4", T=1, N=36864, H=7168, group=64),
    # the same kind of product for a decode batch, rows that divide by nothing
    dict(name="matvec w4 13 tokens, odd rows", op="matvec_w4", T=13, N=18431, H=8192, group=32),
]


def listed():
    return [dict(c) for c in LISTED]


def _log(rng, lo, hi, step=1):
    """A multiple of `step` between lo and hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step))


def draw(rng):
    op = rng.choice(["route", "experts", "experts_w4", "matvec_w4"])
    T = _log(rng, 1, 64)
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * _log(rng, max(2, 16 // groups), 256 // groups)
        top = rng.randint(1, groups)
        K = rng.randint(1, min(10, top * (E // groups)))
        return dict(op=op, T=T, H=_log(rng, 512, 8192, 8), E=E, K=K, scoring=rng.choice(["sigmoid", "softmax"]),
                    bias=rng.choice([True, False]), groups=groups, top_groups=top, shared=rng.choice([0, 0, 1, 2]))
    if op == "matvec_w4":
        group = rng.choice([32, 64, 128])
        return dict(op=op, T=T, N=_log(rng, 64, 16384), H=_log(rng, 512, 8192, group), group=group)
    step = 8 if op == "experts" else rng.choice([32, 64, 128])
    E, K = _log(rng, 8, 256), rng.randint(1, 8)
    while True:
        H, I = _log(rng, 512, 8192, step), _log(rng, 128, 2048, step)
        # weights and the plain form's gathered copies stay below the largest listed case's
        if E * H * I <= 256 * 7168 * 256 and T * K * H * I <= 512 * 7168 * 256:
            break
    c = dict(op=op, T=T, H=H, E=E, K=K, I=I, pad=rng.choice([0, 0, min(T - 1, 2)]))
    return dict(c, group=step) if op == "experts_w4" else c


def _codes(rows, k, group, g, dev):
    """Packed 4-bit codes [..., k/2] and bf16 scales [..., k/group] of weights with deviation about 1/sqrt(k)."""
    q = torch.randint(0, 256, (*rows, k // 2), dtype=torch.uint8, device=dev, generator=g)
    s = (torch.rand((*rows, k // group), device=dev, generator=g) + 0.5) / (4.6 * math.sqrt(k))
    return q, s.bfloat16()


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    op, T, H = case["op"], case["T"], case["H"]

    def normal(*shape, std=1.0):
        return torch.randn(shape, dtype=torch.bfloat16, device=dev, generator=g).mul_(std)

    s = dict(case, x=normal(T, H))
    if op == "matvec_w4":
        s["q"], s["s"] = _codes((case["N"],), H, case["group"], g, dev)
        s["out"] = torch.empty(T, case["N"], dtype=torch.bfloat16, device=dev)
        return s
    E, K = case["E"], case["K"]
    if op == "route":
        s["gate"] = normal(E, H, std=1.0 / math.sqrt(H))
        s["b"] = torch.randn(E, device=dev, generator=g) * 0.1 if case["bias"] else None
        s["ids"] = torch.empty(T, K + case["shared"], dtype=torch.int32, device=dev)
        s["w"] = torch.empty(T, K + case["shared"], dtype=torch.float32, device=dev)
    else:
        I = case["I"]
        logits = torch.randn(T, E, device=dev, generator=g)
        top, ids = torch.topk(torch.sigmoid(logits), min(K, E), dim=1)
        s["w"] = (top / top.sum(1, keepdim=True)).contiguous()
        s["ids"] = ids.int().contiguous()
        if case["pad"]:  # rows behind the batch: no experts
            s["ids"][T - case["pad"]:] = -1
        if op == "experts":
            s["w13"], s["w2"] = normal(E, 2 * I, H, std=1.0 / math.sqrt(H)), normal(E, H, I, std=1.0 / math.sqrt(I))
        else:
            s["q13"], s["s13"] = _codes((E, 2 * I), H, case["group"], g, dev)
            s["q2"], s["s2"] = _codes((E, H), I, case["group"], g, dev)
        s["out"] = torch.empty(T, H, dtype=torch.bfloat16, device=dev)
    if own:
        import tp_reduce_moe_gb300 as arf
        s["moe"] = arf.ar_moe_create(E, K, H, case.get("I", 0), T, shared=case.get("shared", 0))
    return s


def _values(q, s):
    """The weights that packed codes and scales stand for, in 32 bits."""
    code = torch.stack((q & 15, q >> 4), dim=-1).flatten(-2).float() - 8.0
    return (code.unflatten(-1, (s.shape[-1], -1)) * s.float().unsqueeze(-1)).flatten(-2)


def _choose(v, n):
    """Indices of the n largest of each row, the lowest index first among equals."""
    return torch.sort(v, dim=-1, descending=True, stable=True).indices[..., :n]


def _route(s):
    # 64 bits: two experts' scores next to each other must not change places
    T, E, K = s["T"], s["E"], s["K"]
    logits = s["x"].double() @ s["gate"].double().t()
    if s["scoring"] == "sigmoid":
        scores = 1.0 / (1.0 + torch.exp(-logits))
    else:
        e = torch.exp(logits - logits.amax(1, keepdim=True))
        scores = e / e.sum(1, keepdim=True)
    choice = logits if s["b"] is None and s["groups"] == 1 else scores if s["b"] is None else scores + s["b"].double()
    if s["groups"] > 1:
        by = choice.view(T, s["groups"], -1)
        two = by.sort(dim=-1, descending=True).values[..., :2].sum(-1)
        keep = torch.zeros(T, s["groups"], dtype=torch.bool, device=by.device).scatter_(1, _choose(two, s["top_groups"]), True)
        choice = torch.where(keep.unsqueeze(-1), by, float("-inf")).reshape(T, E)
    ids = _choose(choice, K)
    w = scores.gather(1, ids)
    w = 2.5 * w / w.sum(1, keepdim=True)
    more = torch.arange(E, E + s["shared"], device=ids.device).expand(T, -1)
    return torch.cat((ids, more), 1).int(), torch.cat((w.float(), torch.ones_like(more, dtype=torch.float32)), 1)


def _experts(s):
    T, K, H = s["T"], s["K"], s["H"]
    ids, there = s["ids"].flatten().long().clamp_min(0), s["ids"] >= 0
    if s["op"] == "experts":
        w13, w2 = s["w13"][ids].float(), s["w2"][ids].float()
    else:
        w13, w2 = _values(s["q13"][ids], s["s13"][ids]), _values(s["q2"][ids], s["s2"][ids])
    x = s["x"].float().repeat_interleave(s["ids"].shape[1], 0)
    gate, up = torch.bmm(w13, x.unsqueeze(-1)).squeeze(-1).chunk(2, dim=1)
    y = torch.bmm(w2, (gate / (1.0 + torch.exp(-gate)) * up).unsqueeze(-1)).view(T, -1, H)
    return (y * torch.where(there, s["w"], 0.0).unsqueeze(-1)).sum(1).bfloat16()


def run(state):
    s = state
    if own:
        import tp_reduce_moe_gb300 as arf
        if s["op"] == "route":
            return arf.ar_moe_route(s["moe"], s["x"], s["gate"], bias=s["b"],
                                    scoring=arf.AR_MOE_SIGMOID if s["scoring"] == "sigmoid" else arf.AR_MOE_SOFTMAX,
                                    renorm=True, scale=2.5, n_group=s["groups"], topk_group=s["top_groups"], ids=s["ids"], weights=s["w"])
        if s["op"] == "experts":
            return arf.ar_moe_experts(s["moe"], s["x"], s["ids"], s["w"], s["w13"], s["w2"], out=s["out"])
        if s["op"] == "experts_w4":
            return arf.ar_moe_experts_w4(s["moe"], s["x"], s["ids"], s["w"], s["q13"], s["s13"], s["q2"], s["s2"], s["group"], out=s["out"])
        return arf.ar_matvec_w4(s["x"], s["q"], s["s"], s["group"], out=s["out"])
    if s["op"] == "route":
        return _route(s)
    if s["op"] == "matvec_w4":
        return (s["x"].float() @ _values(s["q"], s["s"]).t()).bfloat16()
    return _experts(s)


def work(case):
    op, T, H = case["op"], case["T"], case["H"]
    if op == "route":
        E, k = case["E"], case["K"] + case["shared"]
        return {"bytes": 2 * E * H + 2 * T * H + 4 * E * case["bias"] + 8 * T * k, "flops": 2 * T * E * H}
    bits = 16 if op == "experts" else 4 + 16 / case["group"]
    if op == "matvec_w4":
        return {"bytes": case["N"] * H * bits / 8 + 2 * T * (H + case["N"]), "flops": 2 * T * case["N"] * H}
    n, E, K, I = T - case["pad"], case["E"], case["K"], case["I"]
    read = E * (1 - (1 - K / E) ** n)  # experts that n tokens reach, where all are as likely
    return {"bytes": read * 3 * H * I * bits / 8 + 4 * T * H + 8 * T * K, "flops": 6 * n * K * H * I}


def exact(case, seed):
    """The definitions again, in 64 bits and one token or expert slot at a time."""
    s = prepare(case, seed)
    x = s["x"].double()

    def weights(q, scale):
        v = torch.empty(q.shape[0], 2 * q.shape[1], dtype=torch.float64, device=q.device)
        v[:, 0::2], v[:, 1::2] = (q % 16).double() - 8, (q // 16).double() - 8
        return v * scale.double().repeat_interleave(case["group"], dim=1)

    if case["op"] == "matvec_w4":
        rows = zip(s["q"].split(4096), s["s"].split(4096))
        return torch.cat([weights(q, c) @ x.t() for q, c in rows], 0).t().contiguous()
    if case["op"] == "route":
        ids, ws = [], []
        rows = (x @ s["gate"].double().t()).cpu().tolist()
        b = s["b"].double().cpu().tolist() if case["bias"] else [0.0] * case["E"]
        for z in rows:
            top = max(z)
            p = [1 / (1 + math.exp(-v)) for v in z] if case["scoring"] == "sigmoid" else [math.exp(v - top) for v in z]
            total = 1.0 if case["scoring"] == "sigmoid" else math.fsum(p)
            p = [v / total for v in p]
            key = list(z) if not case["bias"] and case["groups"] == 1 else [u + v for u, v in zip(p, b)]
            size = case["E"] // case["groups"]
            best = sorted(range(case["groups"]), key=lambda g: (-sum(sorted(key[g * size:(g + 1) * size])[-2:]), g))[:case["top_groups"]]
            chosen = sorted((e for e in range(case["E"]) if case["groups"] == 1 or e // size in best), key=lambda e: (-key[e], e))[:case["K"]]
            norm = math.fsum(p[e] for e in chosen)
            ids.append(chosen + [case["E"] + j for j in range(case["shared"])])
            ws.append([2.5 * p[e] / norm for e in chosen] + [1.0] * case["shared"])
        return torch.tensor(ids, dtype=torch.int32), torch.tensor(ws, dtype=torch.float64)
    y = torch.zeros(case["T"], case["H"], dtype=torch.float64, device=x.device)
    for t, row in enumerate(s["ids"].tolist()):
        for k, e in enumerate(row):
            if e >= 0:
                w13 = s["w13"][e].double() if case["op"] == "experts" else weights(s["q13"][e], s["s13"][e])
                w2 = s["w2"][e].double() if case["op"] == "experts" else weights(s["q2"][e], s["s2"][e])
                h = w13 @ x[t]
                g, u = h[:case["I"]], h[case["I"]:]
                y[t] += s["w"][t, k].double() * (w2 @ (g * torch.sigmoid(g) * u))
    return y
