"""The router where only exact sums or 64-bit scores decide: near ties, equal scores, undefined ones, scores near the end of
fp32's range (needs a GB300)."""
import math

import pytest
import torch

import tp_reduce_moe_gb300 as arf
from tests import _moe

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _built():
    from tp_reduce_moe_gb300 import build
    build.build()
    arf.load_library()
    torch.cuda.set_device(0)


def gen(seed):
    return torch.Generator().manual_seed(seed)


def scores(l, sigmoid):
    return torch.sigmoid(l) if sigmoid else torch.softmax(l, dim=-1)


def chosen(l, bias, K, sigmoid, n_group, topk_group, group_max=False):
    """The ids of one token's logits `l` (64 bits), undefined choice values last, the lowest index first among equals."""
    s = scores(l, sigmoid)
    c = (l if bias is None and n_group == 1 else s if bias is None else s + bias.double()).tolist()
    c = [-INF if v != v else v for v in c]
    nan = [v != v for v in (l if bias is None and n_group == 1 else s if bias is None else s + bias.double()).tolist()]
    size = len(c) // n_group
    best = [sum(sorted(c[j * size:(j + 1) * size])[-1 if group_max else -2:]) for j in range(n_group)]
    kept = set(sorted(range(n_group), key=lambda j: (-best[j], j))[:topk_group])
    return sorted((e for e in range(len(c)) if e // size in kept), key=lambda e: (nan[e], -c[e], e))[:K]


def check(x, gate, bias, K, sigmoid, n_group=1, topk_group=1, renorm=True, group_max=False):
    T, E = x.shape[0], gate.shape[0]
    l = x.double() @ gate.double().t()
    want = torch.tensor([chosen(l[t], bias, K, sigmoid, n_group, topk_group, group_max) for t in range(T)], dtype=torch.int32)
    m = arf.ar_moe_create(E, K, x.shape[1], 0, T, device=0)
    ids, w = arf.ar_moe_route(m, x.to(DEV), gate.to(DEV), None if bias is None else bias.to(DEV),
                              (arf.AR_MOE_SIGMOID if sigmoid else arf.AR_MOE_SOFTMAX) | (arf.AR_MOE_GROUP_MAX if group_max else 0),
                              renorm, 1.0, n_group, topk_group)
    ids, w = ids.cpu(), w.cpu().double()
    m.destroy()
    assert torch.equal(ids, want), [(t, ids[t].tolist(), want[t].tolist()) for t in range(T) if not torch.equal(ids[t], want[t])][:3]
    s = scores(l, sigmoid).gather(1, want.long())
    if renorm:
        s = torch.where(s.sum(1, keepdim=True) == 0, torch.zeros_like(s), s / s.sum(1, keepdim=True))
    assert torch.equal(torch.isnan(w), torch.isnan(s))
    # rounded once, from logits good to 2^-40; below fp32's normal numbers half a step of the subnormal ones
    known = ~torch.isnan(s)
    assert bool(((w - s).abs() <= s.abs() * 2.0 ** -23 + 2.0 ** -150)[known].all())
    return ids


def fp32_ids(x, gate, K):
    """The K largest logits of each token when they are 32-bit sums: even and odd columns apart in each of 256 threads (eight
    columns at a time), added up as a tree of 32 lanes, then over the warps in order."""
    p = x.float().unsqueeze(1) * gate.float()  # exact products [T, E, H]
    T, E, H = p.shape
    p = torch.nn.functional.pad(p, (0, -H % 2048)).view(T, E, -1, 256, 4, 2)
    lane = torch.zeros(T, E, 256, 2)
    for c in range(p.shape[2]):
        for i in range(4):
            lane = lane + p[:, :, c, :, i]
    v = (lane[..., 0] + lane[..., 1]).view(T, E, 8, 32)
    while v.shape[-1] > 1:
        v = v[..., :v.shape[-1] // 2] + v[..., v.shape[-1] // 2:]
    total = torch.zeros(T, E)
    for wp in range(8):
        total = total + v[:, :, wp, 0]
    return torch.sort(total, dim=1, descending=True, stable=True).indices[:, :K]


@pytest.mark.parametrize("T", [1, 2, 9])
def test_near_ties_with_terms_that_cancel(T):
    """Logits a few 2^-26 apart, under terms of up to 300 that cancel: 32-bit sums give other ids."""
    H, E, K, P = 4096, 64, 8, 32
    g = gen(40 + T)
    x = torch.randn(T, H, generator=g).bfloat16()
    gate = (torch.randn(1, H, generator=g) / math.sqrt(H)).bfloat16().repeat(E, 1)
    at = torch.randperm(H // 8, generator=g)[:2 * P + 1] * 8 + torch.randint(0, 8, (2 * P + 1,), generator=g)
    plus, minus, step = at[:P], at[P:2 * P], int(at[-1])
    big = (torch.randn(E, P, generator=g) * 300).bfloat16()
    x[:, minus] = x[:, plus]
    gate[:, plus], gate[:, minus] = big, -big
    x[:, step] = (torch.where(torch.arange(T) % 2 == 0, 1.0, -1.0) * 2.0 ** -26).bfloat16()
    gate[:, step] = torch.randperm(E, generator=g).bfloat16()  # whole numbers up to 63: one each
    l = x.double() @ gate.double().t()
    want = torch.sort(l, dim=1, descending=True, stable=True).indices[:, :K]
    gaps = torch.sort(l, dim=1).values.diff(dim=1)
    assert bool((gaps > 2.0 ** -28).all()) and bool((gaps < 2.0 ** -24).all())
    assert bool((fp32_ids(x, gate, K) != want).any(1).all())  # what 32-bit sums would choose
    check(x, gate, None, K, sigmoid=False)
    check(x, gate, torch.full((E,), 0.25), K, sigmoid=True)
    check(x, gate, None, K, sigmoid=True, n_group=8, topk_group=2)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("group_max", [False, True])
def test_groups_with_equal_and_undefined_choices(sigmoid, biased, renorm, group_max):
    """Four groups of six, two of them kept: what 64-bit scores decide, group by group."""
    H, E, K, G, keep = 256, 24, 5, 4, 2
    g = gen(50 + sigmoid + 2 * biased)
    x = torch.randn(7, H, generator=g).bfloat16()
    gate = (torch.randn(E, H, generator=g) / math.sqrt(H)).bfloat16()
    gate[13] = gate[12]          # twins in a group
    gate[18:24] = gate[12:18]    # a group as another
    x[1] = 0.0                   # every score the same
    x[2] = NAN                   # and none defined
    x[3] = x[0] * 4
    x[5, 7] = INF
    bias = None
    if biased:
        bias = torch.randn(E, generator=g) * 0.05
        bias[18:24] = bias[12:18]
        bias[13] = bias[12]
        bias[[0, 1, 2, 6]] = -INF  # half a group barred, and one of another
    check(x, gate, bias, K, sigmoid, G, keep, renorm, group_max)
    for t in range(7):  # alone, by the other split of the CTA's warps
        check(x[t:t + 1], gate, bias, K, sigmoid, G, keep, renorm, group_max)
    # the twin groups are the best two, then just one of them
    up = gate.clone()
    up[12:24] = (up[12:24].float() * 3).bfloat16()
    y = x.clone()
    y[0], y[4] = up[12] * 8, up[14] * 8
    check(y, up, bias, K, sigmoid, G, keep, renorm, group_max)
    check(y, up, bias, K, sigmoid, G, 1, renorm, group_max)
    # an expert whose logits are undefined
    up[14] = NAN
    check(y, up, bias, K, sigmoid, G, keep, renorm, group_max)
    check(y, up, None if bias is None else torch.full((E,), -INF), K, sigmoid, G, keep, renorm, group_max)


def logits_as(values, H=64):
    """(x, gate) with these logits: two bf16 terms each."""
    v = torch.tensor(values, dtype=torch.float64)
    gate = torch.zeros(len(values), H, dtype=torch.bfloat16)
    gate[:, 3] = v.bfloat16()
    gate[:, 44] = (v - gate[:, 3].double()).bfloat16()
    x = torch.zeros(1, H, dtype=torch.bfloat16)
    x[:, [3, 44]] = 1.0
    return x, gate


@pytest.mark.parametrize("T", [1, 4])
def test_scores_at_the_end_of_the_range(T):
    """Scores whose 32-bit form is zero, subnormal or coarse: the order is still that of 64-bit scores."""
    # two groups; by 32-bit sigmoids the other one's sum is larger: e^-88.875 is zero in them
    x, gate = logits_as([-88.0, -88.875, -88.5, -88.5625])
    assert check(x.repeat(T, 1), gate, None, 2, True, 2, 1)[0].tolist() == [0, 1]
    x, gate = logits_as([-88.5, -88.5625, -88.0, -88.875])
    assert check(x.repeat(T, 1), gate, None, 2, True, 2, 1)[0].tolist() == [2, 3]
    g = gen(60 + T)
    for sigmoid in (False, True):
        for low, high in ((-92.0, -86.0), (-106.0, -84.0), (-800.0, -700.0), (-120.0, 3.0), (60.0, 90.0)):
            x, gate = logits_as((torch.rand(48, generator=g, dtype=torch.float64) * (high - low) + low).tolist())
            if not sigmoid and low > -800:
                gate[5, 3], gate[5, 44] = 0.0, 0.0  # the largest: the others' exponentials are tiny
            x = x.repeat(T, 1)
            for bias in (None, torch.zeros(48), torch.full((48,), 1e-40)):
                for groups, keep in ((1, 1), (8, 3), (24, 4)):
                    check(x, gate, bias, 6, sigmoid, groups, keep)


@pytest.mark.parametrize("T,E,K,groups,keep", [(1, 160, 6, 8, 3), (3, 64, 4, 16, 2), (16, 256, 8, 8, 4), (33, 96, 6, 32, 5), (64, 160, 6, 8, 1)])
def test_groups_by_their_largest(T, E, K, groups, keep):
    """A group counts with its best expert: other groups than by the sums of two, for some tokens."""
    g = gen(70 + T)
    x = torch.randn(T, 1024, generator=g).bfloat16()
    gate = (torch.randn(E, 1024, generator=g) / 32).bfloat16()
    bias = torch.randn(E, generator=g) * 0.1
    other = 0
    for sigmoid in (False, True):
        for b in (None, bias):
            for renorm in (False, True):
                by_max = check(x, gate, b, K, sigmoid, groups, keep, renorm, True)
                other += int((by_max != check(x, gate, b, K, sigmoid, groups, keep, renorm, False)).any(1).sum())
            check(x, gate, b, K, sigmoid, 1, 1, True, True)  # without groups it says nothing
    assert T == 1 or other > 0
