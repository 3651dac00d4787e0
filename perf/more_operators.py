"""Cases of the attention half of a decode layer: the norm with an 8-bit output, rotary positions with the write into the
paged key-value cache, and the attention of one new token over that cache, each in its plain form and as a call of the
framework.

    norm_q8  h = sum_r P_r + residual; y = h * rsqrt(mean(h^2) + eps) * gamma; per group of columns (or row)
             s = max|y| / 448, q = e4m3(y / s); h rounded to bf16
    append   rows of q, k, v heads; q and k heads rotated by pos[axis[i], t] * freq[i] in the pair of frequency i (first and
             second half of the rotated columns, or neighbours); q out, k and v into slots of the cache (bf16, or e4m3 of
             value / scale of the head); slot -1: not written
    attn     s_j = scale * q . k_j over the last `window` of `length` tokens, found through a page table;
             out = sum_j softmax(s)_j v_j, lse = log sum_j exp(s_j); no tokens: zeros and minus infinity
"""
import math

import torch

own = False

EPS = 1e-6
E4M3 = 448.0  # largest value of the 8-bit type

# Hidden sizes 6144, 7168 and 8192, two and eight partials and up to 8192 tokens are this repository's configurations;
# head layouts and cache sizes are generic.
LISTED = [
    # one decoded token between two layers, scales of 128 columns as an 8-bit product takes them (latency counts)
    dict(name="norm q8 1 token", op="norm_q8", T=1, R=2, H=7168, group=128),
    # a decode batch behind eight partials, one scale a token
    dict(name="norm q8 61 tokens, row", op="norm_q8", T=61, R=8, H=6144, group=0),
    # a prefill: memory alone counts; fine groups
    dict(name="norm q8 8192 tokens", op="norm_q8", T=8192, R=2, H=8192, group=32),
    # one decoded token on one rank of eight (latency counts)
    dict(name="append 1 token", op="append", T=1, heads=8, kv=1, D=128, rot=128, axes=1, near=False, page=16, kv8=False, pad=0, far=131072),
    # a decode batch with an 8-bit cache, half the columns rotated as neighbours, far positions, padded rows
    dict(name="append 48 tokens, 8 bits", op="append", T=48, heads=32, kv=8, D=128, rot=64, axes=1, near=True, page=64, kv8=True, pad=3, far=1000000),
    # a prefill of images and text: time, height and width
    dict(name="append 8192 tokens, 3 axes", op="append", T=8192, heads=64, kv=8, D=128, rot=128, axes=3, near=False, page=16, kv8=False, pad=0, far=32768),
    # one short conversation on one rank of eight (latency counts)
    dict(name="attn 1 short", op="attn", B=1, lo=500, hi=500, heads=8, kv=1, D=128, page=16, kv8=False, window=0, layout="token"),
    # one long conversation: the split over its length counts
    dict(name="attn 1 long", op="attn", B=1, lo=131071, hi=131071, heads=16, kv=2, D=128, page=64, kv8=False, window=0, layout="head"),
    # an ordinary batch of a server, lengths from short to long
    dict(name="attn 64 ragged", op="attn", B=64, lo=256, hi=8192, heads=32, kv=8, D=128, page=16, kv8=False, window=0, layout="token"),
    # an 8-bit cache, long contexts
    dict(name="attn 16, 8 bits", op="attn", B=16, lo=1000, hi=32768, heads=64, kv=8, D=128, page=64, kv8=True, window=0, layout="pair"),
    # narrow heads that share nothing, a sliding window, pages that end inside any tile, an empty row
    dict(name="attn 33 window", op="attn", B=33, lo=0, hi=16000, heads=16, kv=16, D=64, page=20, kv8=False, window=1024, layout="token"),
    # wide heads, a few sequences
    dict(name="attn 5 wide", op="attn", B=5, lo=1, hi=20001, heads=16, kv=2, D=256, page=32, kv8=False, window=0, layout="head"),
]


def listed():
    return [dict(c) for c in LISTED]


def _log(rng, lo, hi, step=1):
    """A multiple of `step` between lo and hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step))


def draw(rng):
    op = rng.choice(["norm_q8", "append", "attn", "attn"])
    if op == "norm_q8":
        while True:
            c = dict(op=op, T=_log(rng, 1, 8192), R=rng.choice([1, 2, 2, 3, 4, 8]), H=_log(rng, 512, 8192, 8), group=rng.choice([0, 32, 64, 128]))
            if c["T"] * c["H"] * c["R"] <= 8192 * 8192 * 2:
                return c
    D, kv8 = rng.choice([64, 128, 128, 256]), rng.choice([False, False, True])
    kv = rng.choice([1, 2, 4, 5, 8, 16])
    heads = kv * rng.choice([1, 2, 3, 4, 7, 8, 16, 20])
    page = rng.choice([1, 8, 16, 20, 32, 64, 128])
    if op == "append":
        axes, rot = rng.choice([1, 1, 2, 3]), 16 * rng.randint(1, D // 16)
        while True:
            T = _log(rng, 1, 8192)
            if T * (heads + 2 * kv) * D <= 8192 * 80 * 128:
                return dict(op=op, T=T, heads=heads, kv=kv, D=D, rot=rot, axes=axes, near=rng.choice([False, True]), page=page, kv8=kv8,
                            pad=rng.choice([0, 0, min(T - 1, 3)]), far=_log(rng, 1000, 4000000))
    while True:
        B, hi = _log(rng, 1, 128), _log(rng, 16, 131072)
        if B * hi * kv * D <= 64 * 8192 * 8 * 128 and B * hi * heads <= 64 * 8192 * 64:
            return dict(op=op, B=B, lo=rng.choice([0, 1, hi // 8 + 1, hi]), hi=hi, heads=heads, kv=kv, D=D, page=page, kv8=kv8,
                        window=rng.choice([0, 0, 1, 128, 1000]), layout=rng.choice(["token", "head", "pair"]))


def _lengths(case):
    """The sequences' lengths: hi, and the others spread from lo over their logarithm."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    return [hi if B == 1 or i == B - 1 else lo if i == 0 else round(max(lo, 1) * (hi / max(lo, 1)) ** (i / (B - 1))) for i in range(B)]


def _freq(case):
    """Radians a position for each pair, and the pair's axis."""
    n = case["rot"] // 2
    return [10000.0 ** (-i / n) for i in range(n)], [i * case["axes"] // n for i in range(n)]


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    op, s = case["op"], dict(case)

    def normal(*shape, std=1.0):
        return torch.randn(shape, dtype=torch.bfloat16, device=dev, generator=g).mul_(std)

    if op == "norm_q8":
        T, R, H = case["T"], case["R"], case["H"]
        s["partials"], s["residual"] = [normal(T, H) for _ in range(R)], normal(T, H)
        s["gamma"] = (torch.rand(H, device=dev, generator=g) + 0.5).bfloat16()
        s["q"] = torch.empty(T, H, dtype=torch.float8_e4m3fn, device=dev)
        s["scales"] = torch.empty(T, -(-H // (case["group"] or H)), device=dev)
        s["h"] = torch.empty(T, H, dtype=torch.bfloat16, device=dev)
        if own:
            import tp_reduce_moe_gb300 as arf
            s["ws"] = arf.ar_workspace_create(R, 0, H, T, EPS)
        return s

    heads, kv, D, page = case["heads"], case["kv"], case["D"], case["page"]
    tokens = [case["T"]] if op == "append" else _lengths(case)
    used = [-(-n // page) for n in tokens]
    pages = sum(used) + sum(used) // 8 + 2

    def cache(n):  # [n, pages, page, kv, D]: of the layout that the case names
        x = normal(pages, n, page, kv, D) if case.get("layout", "pair") == "pair" else None
        if x is None and case["layout"] == "head":
            x = normal(n, pages, kv, page, D).transpose(2, 3).transpose(0, 1)
        x = normal(n, pages, page, kv, D).transpose(0, 1) if x is None else x
        x = x.to(torch.float8_e4m3fn) if case["kv8"] else x
        return x[:, 0], x[:, 1]

    s["k"], s["v"] = cache(2)
    s["ks"] = torch.rand(kv, device=dev, generator=g) * 0.01 + 0.01 if case["kv8"] else None
    s["vs"] = torch.rand(kv, device=dev, generator=g) * 0.01 + 0.01 if case["kv8"] else None
    if case["kv8"] and op == "attn":
        s["ks"], s["vs"] = s["ks"] * 50, s["vs"] * 50
    order = torch.randperm(pages, device=dev, generator=g).int()
    if op == "append":
        T = case["T"]
        s["qkv"] = normal(T, (heads + 2 * kv) * D)
        s["pos"] = torch.randint(0, case["far"], (case["axes"], T), dtype=torch.int32, device=dev, generator=g)
        s["pos"][0] = s["pos"][0, 0] + torch.arange(T, dtype=torch.int32, device=dev)
        t = torch.arange(T, device=dev)
        s["slots"] = order[t // page] * page + (t % page).int()
        s["slots"][T - case["pad"]:] = -1
        s["out"] = torch.empty(T, heads, D, dtype=torch.bfloat16, device=dev)
        s["freq"], s["axis"] = _freq(case)
    else:
        B = case["B"]
        s["q"] = normal(B, heads, D)
        mixed = torch.randperm(B, generator=torch.Generator().manual_seed(seed)).tolist()
        table, at = torch.full((B, max(used + [1])), -1, dtype=torch.int32, device=dev), 0
        for row, i in enumerate(mixed):
            table[row, :used[i]] = order[at:at + used[i]]
            at += used[i]
        s["table"] = table
        s["lengths"] = torch.tensor([tokens[i] for i in mixed], dtype=torch.int32, device=dev)
        s["most"] = case["hi"]
        s["out"], s["lse"] = torch.empty_like(s["q"]), torch.empty(B, heads, device=dev)
    if own:
        import tp_reduce_moe_gb300 as arf
        s["attn"] = arf.ar_attn_create(heads, kv, D, page, case.get("B", 1))
        s["cache"] = arf.ar_kv_cache(s["k"], s["v"], s["ks"], s["vs"])
        if op == "append":
            arf.ar_attn_set_rope(s["attn"], s["freq"], axis=s["axis"], interleaved=case["near"])
    return s


def _norm_q8(s):
    # 64 bits: values next to a border between two 8-bit ones
    T, H, size = s["T"], s["H"], s["group"] or s["H"]
    h = s["residual"].double()
    for p in s["partials"]:
        h = h + p.double()
    y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * s["gamma"].double()
    y = torch.nn.functional.pad(y, (0, -H % size)).view(T, -1, size)
    top = y.abs().amax(2, keepdim=True)
    scale = torch.where(top > 0, top / E4M3, 1.0)
    q = (y / scale).clamp(-E4M3, E4M3).view(T, -1)[:, :H]
    return q.float().to(torch.float8_e4m3fn), scale.view(T, -1).float(), h.bfloat16()


def _append(s):
    T, heads, kv, D, n = s["T"], s["heads"], s["kv"], s["D"], s["rot"] // 2
    dev = s["qkv"].device
    # 64 bits: the angles of far positions
    axis = torch.tensor(s["axis"], device=dev)
    angle = s["pos"].double()[axis].t() * torch.tensor(s["freq"], dtype=torch.float64, device=dev)
    cos, sin = torch.cos(angle).float().unsqueeze(1), torch.sin(angle).float().unsqueeze(1)
    x = s["qkv"].float().view(T, heads + 2 * kv, D)
    turned, rest = x[:, :heads + kv, :2 * n], x[:, :heads + kv, 2 * n:]
    a, b = (turned[..., 0::2], turned[..., 1::2]) if s["near"] else (turned[..., :n], turned[..., n:])
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack((a, b), -1).flatten(-2) if s["near"] else torch.cat((a, b), -1)
    qk = torch.cat((turned, rest), -1)
    there = s["slots"] >= 0
    page, offset = s["slots"][there].long() // s["page"], s["slots"][there].long() % s["page"]
    for cache, scale, new in ((s["k"], s["ks"], qk[:, heads:]), (s["v"], s["vs"], x[:, heads + kv:])):
        new = new[there]
        new = new.bfloat16() if scale is None else (new / scale.view(1, -1, 1)).clamp(-E4M3, E4M3).to(torch.float8_e4m3fn)
        # moved as bytes: indexed writes do not know the 8-bit type
        kind = torch.uint8 if new.element_size() == 1 else torch.int16
        cache.view(kind)[page, offset] = new.view(kind)
    return qk[:, :heads].bfloat16(), s["k"], s["v"]


def _gathered(s, x, scale):
    """[B, tokens, kv, D] in 32 bits of a cache, the tokens of the longest sequence."""
    kind = torch.uint8 if x.element_size() == 1 else torch.int16
    x = x.view(kind)[s["table"].long().clamp_min(0)].flatten(1, 2)[:, :s["most"]].view(x.dtype).float()
    return x if scale is None else x * scale.view(1, 1, -1, 1)


def _attn(s):
    B, heads, kv, D = s["B"], s["heads"], s["kv"], s["D"]
    k = _gathered(s, s["k"], s["ks"])
    scores = torch.einsum("bhgd,bthd->bhgt", s["q"].float().view(B, kv, -1, D), k) / math.sqrt(D)
    del k
    at, n = torch.arange(scores.shape[-1], device=scores.device), s["lengths"].view(-1, 1)
    there = (at < n) & (at >= n - s["window"]) if s["window"] else at < n
    scores = torch.where(there.view(B, 1, 1, -1), scores, float("-inf"))
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == float("-inf"), 0.0, top)
    e = torch.exp(scores - top)
    total = e.sum(-1, keepdim=True)
    v = torch.where(there.view(B, -1, 1, 1), _gathered(s, s["v"], s["vs"]), 0.0)
    out = torch.einsum("bhgt,bthd->bhgd", e / torch.where(total > 0, total, 1.0), v)
    return out.reshape(B, heads, D).bfloat16(), (torch.log(total) + top).view(B, heads)


def run(state):
    s = state
    if own:
        import tp_reduce_moe_gb300 as arf
        if s["op"] == "norm_q8":
            return arf.ar_rmsnorm_q8(s["ws"], s["partials"], s["residual"], s["gamma"], 0.0, EPS, group=s["group"],
                                     q=s["q"], scales=s["scales"], residual_out=s["h"])
        if s["op"] == "append":
            q = arf.ar_attn_append(s["attn"], s["cache"], s["qkv"], s["pos"], s["slots"], q=s["out"])
            return q, s["k"], s["v"]
        return arf.ar_attn_decode(s["attn"], s["cache"], s["q"], s["table"], s["lengths"], window=s["window"], out=s["out"], lse=s["lse"])
    if s["op"] == "norm_q8":
        return _norm_q8(s)
    return _append(s) if s["op"] == "append" else _attn(s)


def work(case):
    op = case["op"]
    if op == "norm_q8":
        T, R, H = case["T"], case["R"], case["H"]
        return {"bytes": T * H * (2 * (R + 1) + 2 + 1) + 2 * H + 4 * T * -(-H // (case["group"] or H)), "flops": T * H * (R + 6)}
    heads, kv, D, size = case["heads"], case["kv"], case["D"], 1 if case["kv8"] else 2
    if op == "append":
        T, written = case["T"], case["T"] - case["pad"]
        return {"bytes": 2 * T * (heads + 2 * kv) * D + 2 * T * heads * D + size * written * 2 * kv * D + 4 * T * (case["axes"] + 1),
                "flops": 3 * T * (heads + kv) * case["rot"]}
    n = sum(min(x, case["window"] or x) for x in _lengths(case))
    return {"bytes": n * kv * D * 2 * size + 4 * case["B"] * heads * (D + 1) + 4 * n // case["page"], "flops": 4 * n * heads * D}


def exact(case, seed):
    """The definitions again, in 64 bits, a row or a sequence at a time; 8-bit values before they are rounded."""
    s = prepare(case, seed)
    if case["op"] == "norm_q8":
        qs, scales, hs = [], [], []
        for at in range(0, case["T"], 1024):
            rows = slice(at, at + 1024)
            h = torch.stack([p[rows].double() for p in s["partials"]] + [s["residual"][rows].double()]).sum(0)
            y = s["gamma"].double() * h / torch.sqrt(h.square().sum(1, keepdim=True) / case["H"] + EPS)
            parts = y.split(case["group"] or case["H"], dim=1)
            scale = torch.stack([p.abs().max(1).values for p in parts], 1) / E4M3
            qs.append(torch.cat([p / scale[:, i:i + 1] for i, p in enumerate(parts)], 1))
            scales.append(scale)
            hs.append(h)
        return torch.cat(qs), torch.cat(scales), torch.cat(hs)
    heads, kv, D = case["heads"], case["kv"], case["D"]
    if case["op"] == "append":
        freq, axis = _freq(case)
        n = len(freq)
        x = s["qkv"].double().view(case["T"], heads + 2 * kv, D)
        new = x.clone()
        for i in range(n):
            a, b = (2 * i, 2 * i + 1) if case["near"] else (i, i + n)
            z = torch.polar(torch.ones(case["T"], dtype=torch.float64, device=x.device), s["pos"][axis[i]].double() * freq[i])
            z = torch.complex(x[:, :heads + kv, a], x[:, :heads + kv, b]) * z.unsqueeze(1)
            new[:, :heads + kv, a], new[:, :heads + kv, b] = z.real, z.imag
        k, v, rows = s["k"].double(), s["v"].double(), (s["slots"] >= 0).nonzero().flatten()
        p, o = s["slots"][rows].long() // case["page"], s["slots"][rows].long() % case["page"]
        one = torch.ones(kv, dtype=torch.float64, device=x.device)
        k[p, o] = new[rows, heads:heads + kv] / (s["ks"].double() if case["kv8"] else one).view(1, -1, 1)
        v[p, o] = new[rows, heads + kv:] / (s["vs"].double() if case["kv8"] else one).view(1, -1, 1)
        return new[:, :heads], k, v
    out = torch.zeros(case["B"], heads, D, dtype=torch.float64, device=s["q"].device)
    lse = torch.full((case["B"], heads), float("-inf"), dtype=torch.float64, device=s["q"].device)
    group = heads // kv
    for b, n in enumerate(s["lengths"].tolist()):
        first = max(0, n - case["window"]) if case["window"] else 0
        if n == 0:
            continue
        at = torch.arange(first, n, device=s["q"].device)
        p, o = s["table"][b, at // case["page"]].long(), at % case["page"]
        for h in range(kv):
            k, v = (x[:, :, h].float()[p, o].double() for x in (s["k"], s["v"]))
            if case["kv8"]:
                k, v = k * s["ks"][h].double(), v * s["vs"][h].double()
            z = (s["q"][b, h * group:(h + 1) * group].double() @ k.t()) * D ** -0.5
            lse[b, h * group:(h + 1) * group] = torch.logsumexp(z, 1)
            out[b, h * group:(h + 1) * group] = torch.softmax(z, 1) @ v
    return out, lse
