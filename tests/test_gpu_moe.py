"""The few-token MoE layer and the 4-bit product against their definitions in 64 bits (needs a GB300)."""
import math

import pytest
import torch

import tp_reduce_moe_gb300 as arf
from tests import _moe

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    from tp_reduce_moe_gb300 import build
    build.build()
    arf.load_library()
    torch.cuda.set_device(0)


def gen(seed):
    return torch.Generator().manual_seed(seed)


def normal(shape, g, std=1.0):
    return (torch.randn(shape, generator=g) * std).bfloat16().to(DEV)


def guarded(shape, dtype):
    """A tensor with 64 guard values on both sides, and a check that they stand."""
    n = math.prod(shape)
    buf = torch.full((n + 128,), 77, dtype=dtype, device=DEV)
    return buf[64:64 + n].view(shape), lambda: bool((buf[:64] == 77).all()) and bool((buf[64 + n:] == 77).all())


# ------------------------------------------------------------------- router
ROUTES = [  # T, H, E, K, sigmoid, bias, groups, kept, shared, renorm
    (1, 7168, 256, 8, True, True, 8, 4, 1, True),
    (1, 8, 2, 1, False, False, 1, 1, 0, True),
    (2, 264, 5, 5, False, True, 1, 1, 0, False),
    (7, 1032, 33, 4, True, False, 1, 1, 2, True),
    (8, 2048, 512, 16, True, True, 1, 1, 0, True),
    (9, 2056, 64, 6, False, False, 32, 3, 0, True),
    (17, 4096, 100, 10, False, False, 5, 2, 1, False),
    (64, 6144, 160, 8, True, True, 1, 1, 0, True),
    (33, 16384, 31, 3, True, False, 1, 1, 0, True),
    (5, 512, 511, 15, False, True, 7, 7, 1, True),
]


@pytest.mark.parametrize("T,H,E,K,sigmoid,bias,groups,kept,shared,renorm", ROUTES)
def test_route(T, H, E, K, sigmoid, bias, groups, kept, shared, renorm):
    g = gen(T * 1000 + E)
    x, gate = normal((T, H), g), normal((E, H), g, 1 / math.sqrt(H))
    b = (torch.randn(E, generator=g) * 0.1).to(DEV) if bias else None
    ref_ids, ref_w = _moe.route_ref(x.cpu(), gate.cpu(), None if b is None else b.cpu(), K, sigmoid, renorm, 2.5, groups,
                                    kept, shared)
    m = arf.ar_moe_create(E, K, H, 0, T, shared=shared, device=0)
    ids, ok1 = guarded((T, K + shared), torch.int32)
    w, ok2 = guarded((T, K + shared), torch.float32)
    for _ in range(2):  # the second call finds the counters as the first left them
        ids.zero_()
        arf.ar_moe_route(m, x, gate, b, arf.AR_MOE_SIGMOID if sigmoid else arf.AR_MOE_SOFTMAX, renorm, 2.5, groups, kept,
                         ids=ids, weights=w)
        torch.cuda.synchronize()
        assert torch.equal(ids.cpu(), ref_ids)
        # 64-bit scores of logits good to 2^-40, rounded once
        assert bool(((w.cpu().double() - ref_w).abs() <= ref_w.abs() * 2.0 ** -23).all())
        assert ok1() and ok2()
    assert arf.ar_moe_device_error(m) == 0
    m.destroy()


def test_route_ties_and_masks():
    H, E, K = 256, 12, 4
    g = gen(3)
    x = normal((4, H), g)
    x[1] = 0.0                      # every logit the same
    x[2] = float("nan")
    gate = normal((E, H), g, 0.1)
    gate[7] = gate[2]               # two experts alike
    m = arf.ar_moe_create(E, K, H, 0, 4, device=0)
    ids, w = arf.ar_moe_route(m, x, gate, None, arf.AR_MOE_SOFTMAX)
    ref, ref_w = _moe.route_ref(x[:1].cpu(), gate.cpu(), None, K, False, True, 1.0, 1, 1, 0)
    assert torch.equal(ids[:1].cpu(), ref)
    assert ids[1].tolist() == [0, 1, 2, 3] and w[1].tolist() == [0.25] * 4
    assert sorted(set(ids[2].tolist())) == sorted(ids[2].tolist()) and all(0 <= i < E for i in ids[2].tolist())
    bias = torch.full((E,), float("-inf"), device=DEV)
    bias[[1, 4, 6, 9, 11]] = 0.0
    ids, w = arf.ar_moe_route(m, x, gate, bias)
    assert set(ids[0].tolist()) <= {1, 4, 6, 9, 11} and set(ids[3].tolist()) <= {1, 4, 6, 9, 11}
    assert bool(torch.isfinite(w[[0, 1, 3]]).all())
    assert ids[1].tolist() == [1, 4, 6, 9]
    assert ids[2].tolist() == [0, 1, 2, 3]  # all undefined: the lowest indices
    # groups: the barred ones never win over finite ones, and twins keep their order
    ids, _ = arf.ar_moe_route(m, x, gate, bias, n_group=3, topk_group=3)
    assert set(ids[0].tolist()) <= {1, 4, 6, 9, 11}
    with pytest.raises(arf.ArfuseError):
        arf.ar_moe_route(m, x, gate, bias, n_group=6, topk_group=1)
    m.destroy()


def test_route_near_ties_follow_the_exact_sums():
    # logits that differ by less than a 32-bit sum's error: large terms that cancel, and a small difference
    H, E = 4096, 64
    g = gen(4)
    x = normal((8, H), g, 30.0)
    gate = normal((1, H), g).repeat(E, 1)
    for e in range(E):  # one place of one weight apart
        gate[e, (37 * e) % H] = torch.nextafter(gate[e, (37 * e) % H].cpu(), torch.tensor(9.0, dtype=torch.bfloat16)).to(DEV)
    m = arf.ar_moe_create(E, 16, H, 0, 8, device=0)
    ids, _ = arf.ar_moe_route(m, x, gate, None, arf.AR_MOE_SOFTMAX)
    ref, _ = _moe.route_ref(x.cpu(), gate.cpu(), None, 16, False, True, 1.0, 1, 1, 0)
    assert torch.equal(ids.cpu(), ref)
    m.destroy()


# ------------------------------------------------------------------ experts
class Layer:
    """Weights of a layer in bf16 (group 0) or 4 bits, on the device, and as 64-bit matrices."""

    def __init__(self, E, H, I, group, g, device=DEV):
        self.group = group
        if group:
            self.t = [*_moe.make_w4((E, 2 * I), H, group, g, device), *_moe.make_w4((E, H), I, group, g, device)]
        else:
            self.t = [normal((E, 2 * I, H), g, 1 / math.sqrt(H)), normal((E, H, I), g, 1 / math.sqrt(I))]

    def w13(self, e):
        return _moe.w4_values(self.t[0][e], self.t[1][e]) if self.group else self.t[0][e].double()

    def w2(self, e):
        return _moe.w4_values(self.t[2][e], self.t[3][e]) if self.group else self.t[1][e].double()

    def run(self, m, x, ids, w, **kw):
        if self.group:
            return arf.ar_moe_experts_w4(m, x, ids, w, *self.t, self.group, **kw)
        return arf.ar_moe_experts(m, x, ids, w, *self.t, **kw)


def choice(T, E, K, g, spread=None):
    """Distinct experts per token (of the first `spread`), and weights of both signs."""
    ids = torch.stack([torch.randperm(spread or E, generator=g)[:K] for _ in range(T)]).int().to(DEV)
    return ids, (torch.randn(T, K, generator=g) * 0.4).to(DEV)


def check(m, layer, x, ids, w, what):
    out, ok = guarded((x.shape[0], x.shape[1]), torch.bfloat16)
    layer.run(m, x, ids, w, out=out)
    torch.cuda.synchronize()
    y, bound = _moe.experts_ref(x, ids, w, layer.w13, layer.w2)
    _moe.close(out, y, bound, what)
    assert ok(), what
    assert arf.ar_moe_device_error(m) == 0
    return out


SIZES = [  # T, H, E, K, I
    (1, 8, 1, 1, 8), (1, 264, 4, 2, 72), (1, 7168, 16, 8, 256), (2, 2048, 8, 8, 200), (3, 1032, 6, 3, 1000),
    (4, 512, 3, 2, 64), (5, 520, 9, 4, 136), (8, 4104, 8, 2, 96), (9, 1024, 5, 3, 264), (16, 2048, 32, 6, 128),
    (17, 776, 4, 4, 40), (31, 640, 64, 8, 80), (33, 1288, 7, 2, 520), (64, 1024, 128, 16, 32), (64, 152, 2, 1, 24),
    (1, 16384, 2, 2, 4096), (2, 64, 3, 2, 16384),
]


@pytest.mark.parametrize("T,H,E,K,I", SIZES)
def test_experts(T, H, E, K, I):
    g = gen(T + H + I)
    layer = Layer(E, H, I, 0, g)
    m = arf.ar_moe_create(E, K, H, I, T, device=0)
    check(m, layer, normal((T, H), g), *choice(T, E, K, g), f"{T} tokens")
    m.destroy()


W4_SIZES = [  # T, H, E, K, I, group
    (1, 32, 1, 1, 32, 32), (1, 7168, 12, 8, 256, 128), (2, 288, 4, 2, 96, 32), (3, 1056, 5, 2, 352, 32),
    (4, 192, 3, 3, 320, 64), (5, 832, 6, 4, 192, 64), (8, 384, 4, 2, 640, 128), (9, 1152, 8, 3, 128, 128),
    (13, 2048, 16, 8, 2048, 64), (17, 544, 4, 4, 32, 32), (33, 1024, 9, 2, 160, 32), (64, 896, 40, 8, 128, 128),
    (64, 128, 2, 2, 64, 64), (1, 2048, 8, 2, 4096, 32),
]


@pytest.mark.parametrize("T,H,E,K,I,group", W4_SIZES)
def test_experts_w4(T, H, E, K, I, group):
    g = gen(T + H + I + group)
    layer = Layer(E, H, I, group, g)
    m = arf.ar_moe_create(E, K, H, I, T, device=0)
    check(m, layer, normal((T, H), g), *choice(T, E, K, g), f"{T} tokens, groups of {group}")
    m.destroy()


@pytest.mark.parametrize("group", [0, 32, 128])
@pytest.mark.parametrize("T", [1, 6, 20, 64])
def test_experts_padding_duplicates_and_crowds(T, group):
    H, E, K, I = 640, 16, 4, 128
    g = gen(T)
    layer = Layer(E, H, I, group, g)
    m = arf.ar_moe_create(E, K, H, I, 64, device=0)
    x = normal((T, H), g)
    ids, w = choice(T, E, K, g)
    # every token at the same experts
    check(m, layer, x, ids[:1].repeat(T, 1).contiguous(), w, "a crowd")
    # an expert named twice and three times
    twice = ids.clone()
    twice[:, 3] = twice[:, 0]
    if T > 2:
        twice[2, 1:] = twice[2, 0]
    check(m, layer, x, twice, w, "duplicates")
    # holes and rows without experts, whose inputs are not numbers
    holes = ids.clone()
    holes[:, 1] = -1
    holes[T // 2:] = -1
    holes[0] = ids[0] if T > 1 else -1
    y = x.clone()
    y[T // 2 if T > 1 else 0:] = float("nan")
    z = w.clone()
    z[holes == -1] = float("nan")
    out = layer.run(m, y, holes, z)
    clean = torch.where(holes == -1, torch.zeros_like(w), w)
    ref, bound = _moe.experts_ref(torch.nan_to_num(y), holes, clean, layer.w13, layer.w2)
    _moe.close(out, ref, bound, "holes")
    assert bool((out[T // 2 if T > 1 else 0:] == 0).all())
    # nobody has an expert
    assert bool((layer.run(m, x, torch.full_like(ids, -1), w) == 0).all())
    assert arf.ar_moe_device_error(m) == 0
    # no such expert: skipped and said
    bad = ids.clone()
    bad[:, 0] = torch.tensor([E, -2, 2147483647, -2147483648], dtype=torch.int32, device=DEV).repeat(16)[:T]
    out = layer.run(m, x, bad, w)
    skip = torch.where((bad < 0) | (bad >= E), torch.full_like(bad, -1), bad)
    ref, bound = _moe.experts_ref(x, skip, w, layer.w13, layer.w2)
    _moe.close(out, ref, bound, "ids out of range")
    assert arf.ar_moe_device_error(m) == arf.AR_DEVERR_EXPERT_RANGE
    assert arf.ar_moe_device_error(m) == 0
    m.destroy()


def test_experts_infinite_weights_stay_with_their_tokens():
    """An infinite weight or scale reaches the tokens of its expert and row, no others."""
    H, E, K, I = 288, 4, 1, 96
    for group in (0, 32):
        g = gen(9)
        layer = Layer(E, H, I, group, g)
        m = arf.ar_moe_create(E, K, H, I, 8, device=0)
        x = normal((8, H), g)
        ids = (torch.arange(8, dtype=torch.int32, device=DEV) % E).view(8, 1).contiguous()
        w = torch.ones(8, 1, device=DEV)
        before = layer.run(m, x, ids, w)
        (layer.t[3] if group else layer.t[1])[2, 17, 0] = float("inf")
        after = layer.run(m, x, ids, w)
        hit = torch.zeros(8, H, dtype=torch.bool, device=DEV)
        hit[2::4, 17] = True
        assert torch.equal(after[~hit], before[~hit])
        assert not bool(torch.isfinite(after[hit]).any())
        m.destroy()


@pytest.mark.parametrize("group", [0, 64])
def test_experts_are_deterministic_and_independent_of_the_batch(group):
    H, E, K, I, T = 1024, 24, 4, 192, 40
    g = gen(11)
    layer = Layer(E, H, I, group, g)
    m = arf.ar_moe_create(E, K, H, I, 64, device=0)
    x = normal((T, H), g)
    ids, w = choice(T, E, K, g)
    first = layer.run(m, x, ids, w)
    for _ in range(5):
        assert torch.equal(layer.run(m, x, ids, w), first)
    # the same tokens in another order: the same results to within their bounds
    order = torch.randperm(T, generator=g).to(DEV)
    again = layer.run(m, x[order].contiguous(), ids[order].contiguous(), w[order].contiguous())
    y, bound = _moe.experts_ref(x, ids, w, layer.w13, layer.w2)
    _moe.close(again, y[order], bound[order], "another order")
    m.destroy()


@pytest.mark.parametrize("group", [0, 128])
def test_experts_offsets_beyond_32_bits(group):
    """Weights of more than 2^32 values (and, in 4 bits, more than 2^32 bytes); only the experts in use are filled."""
    H, I, K = 8192, 2048, 3
    E = 512 if group else 160
    g = gen(12)
    few = Layer(3, H, I, group, g)
    layer = Layer.__new__(Layer)
    layer.group = group
    use = [0, E // 2 + 1, E - 1]
    layer.t = []
    for t in few.t:
        big = torch.empty((E, *t.shape[1:]), dtype=t.dtype, device=DEV)
        for i, e in enumerate(use):
            big[e] = t[i]
        layer.t.append(big)
    assert layer.t[0].numel() > 2 ** 32
    m = arf.ar_moe_create(E, K, H, I, 2, device=0)
    ids = torch.tensor([use, use[::-1]], dtype=torch.int32, device=DEV)
    w = torch.tensor([[0.5, -1.0, 0.25], [1.0, 0.3, 0.7]], device=DEV)
    check(m, layer, normal((2, H), g), ids, w, "offsets")
    m.destroy()


# ------------------------------------------------------------- 4-bit product
MATVECS = [  # T, N, K, group
    (1, 1, 32, 32), (1, 7168, 2048, 128), (1, 151, 4096, 64), (2, 153, 96, 32), (3, 2049, 352, 32), (5, 1000, 128, 128),
    (8, 4097, 1152, 128), (9, 333, 832, 64), (13, 2431, 8192, 32), (16, 64, 16384, 128), (17, 500, 160, 32),
    (33, 305, 2048, 64), (64, 4864, 512, 32), (64, 7, 65536, 128),
]


@pytest.mark.parametrize("T,N,K,group", MATVECS)
def test_matvec_w4(T, N, K, group):
    g = gen(T + N + K)
    x = normal((T, K), g)
    q, s = _moe.make_w4((N,), K, group, g, DEV)
    W = _moe.w4_values(q, s)
    y, m = x.double() @ W.t(), x.double().abs() @ W.abs().t()
    lost = _moe.gamma(K) * m
    out, ok = guarded((T, N), torch.bfloat16)
    if out.data_ptr() % 16 == 0:
        arf.ar_matvec_w4(x, q, s, group, out=out)
        torch.cuda.synchronize()
        _moe.close(out, y, lost + _moe.HALF_BF16 * (y.abs() + lost), "bf16")
        assert ok()
    f = arf.ar_matvec_w4(x, q, s, group, out_fp32=True)
    assert f.dtype == torch.float32
    assert bool(((f.double() - y).abs() <= lost + 2.0 ** -24 * y.abs()).all())
    assert torch.equal(arf.ar_matvec_w4(x, q, s, group), f.bfloat16())  # one rounding
    # a token's result does not depend on the others
    if T <= 8:
        one = arf.ar_matvec_w4(x[T - 1:].contiguous(), q, s, group, out_fp32=True)
        assert torch.equal(one[0], f[T - 1])


def test_matvec_w4_zero_tokens_and_refusals():
    g = gen(1)
    q, s = _moe.make_w4((40,), 64, 32, g, DEV)
    x = normal((3, 64), g)
    assert arf.ar_matvec_w4(x[:0], q, s, 32).shape == (0, 40)
    with pytest.raises(ValueError):
        arf.ar_matvec_w4(x.cpu(), q, s, 32)
    with pytest.raises(ValueError):
        arf.ar_matvec_w4(x, q.cpu(), s, 32)
    with pytest.raises(arf.ArfuseError):
        arf.ar_matvec_w4(normal((65, 64), g), q, s, 32)


def test_matvec_w4_infinite_scale_stays_in_its_row():
    g = gen(2)
    N, K = 70, 96  # three groups of 32: the next row's scale shares a word with a row's last
    x = normal((2, K), g)
    q, s = _moe.make_w4((N,), K, 32, g, DEV)
    before = arf.ar_matvec_w4(x, q, s, 32, out_fp32=True)
    s[31] = float("inf")
    after = arf.ar_matvec_w4(x, q, s, 32, out_fp32=True)
    rows = torch.arange(N, device=DEV) != 31
    assert torch.equal(after[:, rows], before[:, rows])
    assert not bool(torch.isfinite(after[:, 31]).any())


# Shapes that take every way through the products: jobs of several rounds, activations that do not fit in one piece,
# groups of items, rows whose scales are copied in pieces of 16, 8, 4 and 2 bytes, last tiles of every height.
MORE_EXPERTS = [  # T, H, E, K, I
    (64, 256, 64, 4, 1024), (3, 64, 160, 10, 520),
]
MORE_W4 = [  # T, H, E, K, I, group
    (8, 16384, 4, 2, 64, 32), (16, 7168, 2, 2, 64, 64), (20, 7168, 16, 2, 64, 32), (12, 4096, 64, 4, 64, 32),
    (64, 256, 64, 4, 1024, 32), (40, 256, 16, 8, 1024, 64), (10, 192, 24, 4, 192, 32), (7, 768, 6, 3, 256, 64),
    (50, 1280, 60, 6, 256, 128), (1, 8192, 4, 4, 32, 32),
]
MORE_MATVECS = [  # T, N, K, group
    (3, 80000, 64, 32), (9, 80001, 64, 32), (1, 2888, 96, 32), (2, 3496, 4096, 64), (1, 4256, 224, 32), (4, 100, 256, 64),
    (2, 2900, 768, 64), (2, 33, 320, 64), (6, 3500, 1024, 128), (8, 300, 24576, 32), (12, 170, 7168, 64),
    (9, 1048576, 32, 32), (64, 300000, 128, 128),
]


@pytest.mark.parametrize("T,H,E,K,I", MORE_EXPERTS)
def test_experts_more(T, H, E, K, I):
    test_experts(T, H, E, K, I)


@pytest.mark.parametrize("T,H,E,K,I,group", MORE_W4)
def test_experts_w4_more(T, H, E, K, I, group):
    test_experts_w4(T, H, E, K, I, group)


@pytest.mark.parametrize("T,N,K,group", MORE_MATVECS)
def test_matvec_w4_more(T, N, K, group):
    g = gen(T + N + K)
    x = normal((T, K), g)
    q, s = _moe.make_w4((N,), K, group, g, DEV)
    W = _moe.w4_values(q, s)
    y, m = x.double() @ W.t(), x.double().abs() @ W.abs().t()
    f, ok = guarded((T, N), torch.float32)
    arf.ar_matvec_w4(x, q, s, group, out=f, out_fp32=True)
    torch.cuda.synchronize()
    assert bool(((f.double() - y).abs() <= _moe.gamma(K) * m + 2.0 ** -24 * y.abs()).all())
    assert ok()
    assert torch.equal(arf.ar_matvec_w4(x, q, s, group), f.bfloat16())


@pytest.mark.parametrize("group", [32, 64, 128])
def test_matvec_w4_range_of_activations(group):
    """Activations are scaled by powers of two inside, exactly, up to 2^101; beyond that a token's results are undefined."""
    g = gen(group)
    T, N, K = 5, 90, 1152
    x = normal((T, K), g)
    q, s = _moe.make_w4((N,), K, group, g, DEV)
    y = arf.ar_matvec_w4(x, q, s, group, out_fp32=True)
    for power in (-80, -30, 60, 95):
        z = arf.ar_matvec_w4((x.float() * 2.0 ** power).bfloat16(), q, s, group, out_fp32=True)
        assert torch.equal(z.double(), y.double() * 2.0 ** power), power
    assert bool((arf.ar_matvec_w4(torch.zeros_like(x), q, s, group) == 0).all())
    for value in (float("nan"), float("inf"), -float("inf"), 2.0 ** 101):
        bad = x.clone()
        bad[3, K - 1] = value
        z = arf.ar_matvec_w4(bad, q, s, group, out_fp32=True)
        assert bool(torch.isnan(z[3]).all())
        keep = [0, 1, 2, 4]
        assert torch.equal(z[keep], y[keep])


# ------------------------------------------------------------------ together
def layer_step(m, ws, layer, x, gate, bias, residual, gamma, bufs, stream=None):
    ids, w, y, out, res = bufs
    arf.ar_moe_route(m, x, gate, bias, n_group=4, topk_group=2, scale=2.5, ids=ids, weights=w, stream=stream)
    layer.run(m, x, ids, w, out=y, stream=stream)
    arf.ar_rmsnorm(ws, [y], residual, gamma, 0.0, 1e-6, out=out, residual_out=res, stream=stream)


@pytest.mark.parametrize("flags", [0, arf.AR_WS_PDL])
@pytest.mark.parametrize("group", [0, 64])
@pytest.mark.parametrize("T", [1, 12])
def test_layer_eager_and_captured(T, group, flags):
    """Router, experts with a shared one, residual norm: as a chain, eager and as a replayed graph on new inputs."""
    E, S, K, H, I = 32, 1, 4, 1024, 128
    g = gen(T + group)
    layer = Layer(E + S, H, I, group, g)
    gate, gamma = normal((E, H), g, 1 / math.sqrt(H)), normal((H,), g)
    bias = (torch.randn(E, generator=g) * 0.1).to(DEV)
    m = arf.ar_moe_create(E, K, H, I, T, shared=S, device=0, flags=flags)
    ws = arf.ar_workspace_create(1, 0, H, T, 1e-6, device=0, flags=flags)

    def fresh():
        return normal((T, H), g), normal((T, H), g)

    def bufs():
        return (torch.empty(T, K + S, dtype=torch.int32, device=DEV), torch.empty(T, K + S, device=DEV),
                *(torch.empty(T, H, dtype=torch.bfloat16, device=DEV) for _ in range(3)))

    def verify(x, residual, b, what):
        ids, w, y, out, res = b
        rid, rw = _moe.route_ref(x.cpu(), gate.cpu(), bias.cpu(), K, True, True, 2.5, 4, 2, S)
        assert torch.equal(ids.cpu(), rid), what
        ref, bound = _moe.experts_ref(x, rid, rw, layer.w13, layer.w2)
        # the weights' own rounding to 32 bits is far below the bound
        _moe.close(y, ref, bound, what)
        h = y.double() + residual.double()
        # h to half a bf16 step (its 32-bit sum of two values loses 2^-24 more)
        assert bool(((res.double() - h).abs() <= h.abs() * (_moe.HALF_BF16 + 2.0 ** -23)).all()), what
        n = h * torch.rsqrt((h * h).mean(1, keepdim=True) + 1e-6) * gamma.double()
        assert bool(((out.double() - n).abs() <= n.abs() * (_moe.HALF_BF16 + H * 2.0 ** -24) + 1e-30).all()), what

    x, residual = fresh()
    b = bufs()
    layer_step(m, ws, layer, x, gate, bias, residual, gamma, b)
    torch.cuda.synchronize()
    verify(x, residual, b, "eager")
    # back to back, two sets of inputs in flight on one stream
    x2, r2 = fresh()
    b2 = bufs()
    for _ in range(3):
        layer_step(m, ws, layer, x, gate, bias, residual, gamma, b)
        layer_step(m, ws, layer, x2, gate, bias, r2, gamma, b2)
    torch.cuda.synchronize()
    verify(x, residual, b, "first of a chain")
    verify(x2, r2, b2, "second of a chain")
    # captured on a side stream, replayed on other inputs
    sx, sr = x.clone(), residual.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    b3 = bufs()
    with torch.cuda.graph(graph, stream=side):
        layer_step(m, ws, layer, sx, gate, bias, sr, gamma, b3)
    for _ in range(3):
        nx, nr = fresh()
        sx.copy_(nx)
        sr.copy_(nr)
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        verify(nx, nr, b3, "replayed")
    assert arf.ar_moe_device_error(m) == 0
    m.destroy()
    ws.destroy()


def test_products_captured_with_forks_and_copies():
    """4-bit products captured behind a kernel, a copy, a fork and a join, replayed on new inputs."""
    T, N, K, group = 3, 700, 512, 64
    g = gen(41)
    q, s = _moe.make_w4((N,), K, group, g, DEV)
    W = _moe.w4_values(q, s)
    x, y = normal((T, K), g), torch.empty(T, K, dtype=torch.bfloat16, device=DEV)
    outs = [torch.empty(T, N, device=DEV) for _ in range(5)]

    def chain(main, side):
        y.copy_(x)                                                        # a copy before
        arf.ar_matvec_w4(y, q, s, group, out=outs[0], out_fp32=True)
        y.neg_()                                                          # a kernel before
        arf.ar_matvec_w4(y, q, s, group, out=outs[1], out_fp32=True)
        side.wait_stream(main)                                            # first on a forked stream
        arf.ar_matvec_w4(y, q, s, group, out=outs[2], out_fp32=True, stream=side)
        arf.ar_matvec_w4(x, q, s, group, out=outs[3], out_fp32=True)      # beside it
        main.wait_stream(side)                                            # behind both
        arf.ar_matvec_w4(x, q, s, group, out=outs[4], out_fp32=True)

    torch.cuda.synchronize()
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(main):
        chain(main, side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        chain(main, side)
    for _ in range(4):
        x.copy_(normal((T, K), g))
        graph.replay()
        torch.cuda.synchronize()
        ref, m = x.double() @ W.t(), x.double().abs() @ W.abs().t()
        for i, sign in enumerate((1, -1, -1, 1, 1)):
            assert bool(((outs[i].double() - sign * ref).abs() <= _moe.gamma(K) * m + 2.0 ** -24 * ref.abs()).all()), i


def test_two_handles_on_two_streams():
    E, K, H, I, T = 16, 4, 2048, 256, 4
    g = gen(21)
    layer = Layer(E, H, I, 0, g)
    pairs = []
    for _ in range(2):
        x = normal((T, H), g)
        ids, w = choice(T, E, K, g)
        m = arf.ar_moe_create(E, K, H, I, T, device=0)
        pairs.append((m, x, ids, w, torch.cuda.Stream(), torch.empty(T, H, dtype=torch.bfloat16, device=DEV)))
    torch.cuda.synchronize()
    for _ in range(20):
        for m, x, ids, w, s, out in pairs:
            layer.run(m, x, ids, w, out=out, stream=s)
    torch.cuda.synchronize()
    for m, x, ids, w, s, out in pairs:
        y, bound = _moe.experts_ref(x, ids, w, layer.w13, layer.w2)
        _moe.close(out, y, bound, "two streams")
        m.destroy()


def test_row_parallel_projection_feeds_the_norm():
    """Two ranks' 4-bit projections as the partials of the trailing all-reduce + norm."""
    T, H, K, group = 3, 1024, 512, 64
    g = gen(31)
    ws = arf.ar_workspace_create(2, 0, H, T, 1e-6, device=0)
    parts, refs = [], []
    for _ in range(2):
        x = normal((T, K), g)
        q, s = _moe.make_w4((H,), K, group, g, DEV)
        parts.append(arf.ar_matvec_w4(x, q, s, group))
        refs.append(x.double() @ _moe.w4_values(q, s).t())
    residual, gamma = normal((T, H), g), normal((H,), g)
    out, res = arf.ar_rmsnorm(ws, parts, residual, gamma, 0.0, 1e-6, residual_out_fp32=True)
    h = refs[0] + refs[1] + residual.double()
    slack = _moe.HALF_BF16 * (refs[0].abs() + refs[1].abs()) * 1.01 + 1e-3 * _moe.HALF_BF16
    assert bool(((res.double() - h).abs() <= slack + 2.0 ** -20 * h.abs()).all())
    ws.destroy()
