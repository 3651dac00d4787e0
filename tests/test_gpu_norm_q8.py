"""The norm with an 8-bit output against its definition in 64 bits (needs a GB300)."""
import pytest
import torch

import tp_reduce_moe_gb300 as arf
from tests import _attn
from tests.test_gpu_attn import DEV, gen, guarded, normal

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _built():
    from tp_reduce_moe_gb300 import build
    build.build()
    arf.load_library()
    torch.cuda.set_device(0)


def check(partials, residual, gamma, wb, eps, group, q, scales, h, out, bf16_h=False):
    """Bounds: h is a sum of R + 1 terms in fp32 (each step loses half a last place of the magnitudes summed); y is h times
    a root and a weight: 4 more last places and the root's, of a mean over H columns (2^-20 together, for its sum is over a
    tree).  With h rounded to bf16 a value next to a border may go either way: half a bf16 step, and the root with it."""
    y, scale, href = _attn.norm_q8_ref(partials, residual, gamma, wb, eps, group, bf16_h)
    R = len(partials)
    mags = residual.double().abs() + sum(p.double().abs() for p in partials)
    h_slack = mags * (R + 1) * 2.0 ** -24
    half = 2.0 ** -24 if h.dtype == torch.float32 else _attn.HALF_BF16
    assert bool(((h.double() - href).abs() <= href.abs() * half + h_slack * 1.01).all())
    per_h = (y / href).abs()  # what y makes of a change of h
    per_h = torch.where(torch.isfinite(per_h), per_h, 0.0)
    y_slack = per_h * h_slack + y.abs() * 2.0 ** -20 + (gamma.double() + wb).abs() * per_h.amax(1, keepdim=True) * 2.0 ** -60
    if bf16_h:
        near = (href.float().abs() * 0 + 1).double() * 2.0 ** -8  # every value may sit at a border
        y_slack = y_slack + y.abs() * near * 2
    size = group or y.shape[1]
    top = torch.stack([c.amax(1) for c in (y.abs() + y_slack).split(size, dim=1)], 1) / 448.0
    low = torch.stack([c.amax(1) for c in (y.abs() - y_slack).split(size, dim=1)], 1) / 448.0
    s = scales.double()
    zero = y.abs().split(size, dim=1)
    zero = torch.stack([c.amax(1) == 0 for c in zero], 1)
    assert bool(((s <= top * (1 + 2.0 ** -22)) | zero).all()) and bool(((s >= low * (1 - 2.0 ** -22)) | zero).all())
    assert bool((s[zero] == 1.0).all())
    spread = s.repeat_interleave(size, dim=1)[:, :y.shape[1]]
    _attn.check_e4m3(q, y / spread, y_slack / spread + (y / spread).abs() * 2.0 ** -22, "q")
    if out is not None:
        assert bool(((out.double() - y).abs() <= y.abs() * _attn.HALF_BF16 + y_slack * 1.01).all())


CASES = [  # T, R, H, group, fp32 residual, wb, with out
    (1, 2, 7168, 128, False, 0.0, False),
    (61, 8, 6144, 0, False, 0.0, True),
    (3, 1, 8, 0, True, 1.0, True),
    (3, 1, 8, 128, False, 0.0, True),
    (5, 3, 264, 32, True, 1.0, False),
    (7, 5, 1000, 64, False, 0.0, True),
    (2, 16, 8192, 32, False, 0.0, False),
    (9, 4, 8200, 128, True, 0.0, True),
    (4, 2, 16384, 0, False, 1.0, True),
    (4, 7, 16384, 32, True, 0.0, False),
    (700, 2, 1032, 128, False, 0.0, True),
    (2000, 1, 2048, 0, False, 0.0, False),
    (1500, 2, 4104, 64, True, 0.0, True),
    (333, 16, 512, 32, False, 0.0, False),
]


@pytest.mark.parametrize("T,R,H,group,fp32,wb,with_out", CASES)
def test_norm_q8(T, R, H, group, fp32, wb, with_out):
    g = gen(T + H)
    partials, residual = [normal((T, H), g) for _ in range(R)], normal((T, H), g)
    gamma = (torch.rand(H, device=DEV, generator=g) + 0.5 - wb).bfloat16()
    ws = arf.ar_workspace_create(R, 0, H, T, 1e-6, device=0)
    q8, ok0 = guarded((T, H), torch.uint8)
    scales, ok1 = guarded((T, -(-H // group) if group else 1), torch.float32)
    h, ok2 = guarded((T, H), torch.float32 if fp32 else torch.bfloat16)
    out, ok3 = guarded((T, H), torch.bfloat16)
    kept = None
    for _ in range(2):
        arf.ar_rmsnorm_q8(ws, partials, residual, gamma, wb, 1e-6, group=group, q=q8.view(F8), scales=scales, residual_out=h,
                          residual_out_fp32=fp32, out=out if with_out else None)
        torch.cuda.synchronize()
        check(partials, residual, gamma, wb, 1e-6, group, q8.view(F8), scales, h, out if with_out else None)
        assert ok0() and ok1() and ok2() and ok3()
        assert with_out or bool((out == 77).all())
        if kept is not None:
            assert torch.equal(kept[0], q8) and torch.equal(kept[1], scales) and torch.equal(kept[2], h)
        kept = q8.clone(), scales.clone(), h.clone()
    assert arf.ar_workspace_device_error(ws) == 0
    ws.destroy()


def test_out_is_that_of_the_plain_norm():
    g = gen(5)
    for T, R, H in ((4, 2, 7168), (300, 2, 1024)):
        partials, residual, gamma = [normal((T, H), g) for _ in range(R)], normal((T, H), g), normal((H,), g)
        ws = arf.ar_workspace_create(R, 0, H, T, 1e-6, device=0)
        want, h = arf.ar_rmsnorm(ws, partials, residual, gamma, 0.0, 1e-6)
        out = torch.empty_like(want)
        _, _, h8 = arf.ar_rmsnorm_q8(ws, partials, residual, gamma, 0.0, 1e-6, out=out)
        assert torch.equal(h, h8)
        # both are a rounding of values within some last places of each other
        assert bool(((out.double() - want.double()).abs() <= want.double().abs() * 2 * _attn.HALF_BF16).all())
        assert float((out != want).double().mean()) < 0.01
        ws.destroy()


def test_norm_of_a_rounded_h_and_in_place():
    g = gen(6)
    T, R, H = 33, 3, 2056
    partials, residual, gamma = [normal((T, H), g) for _ in range(R)], normal((T, H), g), normal((H,), g)
    ws = arf.ar_workspace_create(R, 0, H, T, 1e-5, device=0, flags=arf.AR_WS_NORM_BF16_H | arf.AR_WS_PDL)
    inout = residual.clone()
    q, scales, h = arf.ar_rmsnorm_q8(ws, partials, inout, gamma, 0.0, 1e-5, group=32, residual_out=inout)
    assert h is inout
    check(partials, residual, gamma, 0.0, 1e-5, 32, q, scales, h, None, bf16_h=True)
    # from the h that it stored, the norm is exact to fp32
    x = h.double()
    y = x / torch.sqrt((x * x).mean(1, keepdim=True) + 1e-5) * gamma.double()
    spread = scales.double().repeat_interleave(32, dim=1)[:, :H]
    _attn.check_e4m3(q, y / spread, (y / spread).abs() * 2.0 ** -19, "q")
    ws.destroy()


@pytest.mark.parametrize("group", [0, 32, 128])
def test_rows_of_zeros_and_of_undefined_values(group):
    g = gen(7)
    T, H = 6, 520
    p, residual, gamma = torch.zeros(T, H, dtype=torch.bfloat16, device=DEV), normal((T, H), g), normal((H,), g)
    residual[0] = 0.0
    residual[1, :256] = 0.0                 # whole groups of zeros
    residual[2, 300] = float("nan")
    residual[3, 300] = float("inf")
    residual[4] *= 1e-30                    # below eps: y is tiny
    ws = arf.ar_workspace_create(1, 0, H, T, 1e-6, device=0)
    q, scales, h = arf.ar_rmsnorm_q8(ws, [p], residual, gamma, 0.0, 1e-6, group=group)
    rows = [0, 1, 4, 5]
    check([p[rows]], residual[rows], gamma, 0.0, 1e-6, group, q[rows], scales[rows], h[rows], None)
    assert bool((q[0].float() == 0).all()) and bool((scales[0] == 1).all())
    # a NaN makes the whole row NaN; an infinity makes its own value NaN and the others zeros
    assert bool(torch.isnan(scales[2]).all()) and bool(torch.isnan(q[2].float()).all())
    size = group or H
    assert bool(torch.isnan(scales[3, 300 // size])) and bool(torch.isnan(q[3, 300].float()))
    if group:
        other = torch.arange(scales.shape[1], device=DEV) != 300 // size
        assert bool((scales[3][other] == 1).all())
    ws.destroy()


def test_captured_chain():
    """Calls under each other's ends, each reading the residual that the one before wrote, captured and replayed."""
    g = gen(8)
    T, R, H, steps = 5, 2, 7168, 6
    partials = [[normal((T, H), g) for _ in range(R)] for _ in range(steps)]
    first, gamma = normal((T, H), g), (torch.rand(H, device=DEV, generator=g) + 0.5).bfloat16()
    ws = arf.ar_workspace_create(R, 0, H, T, 1e-6, device=0, flags=arf.AR_WS_PDL)
    hs = [first] + [torch.empty_like(first) for _ in range(steps)]
    outs = [(torch.empty(T, H, dtype=F8, device=DEV), torch.empty(T, H // 128, device=DEV)) for _ in range(steps)]

    def chain():
        for i in range(steps):
            arf.ar_rmsnorm_q8(ws, partials[i], hs[i], gamma, 0.0, 1e-6, q=outs[i][0], scales=outs[i][1], residual_out=hs[i + 1])

    chain()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain()
    for seed in (1, 2):
        first.copy_(normal((T, H), gen(seed)))
        graph.replay()
        torch.cuda.synchronize()
        for i in range(steps):
            check(partials[i], hs[i], gamma, 0.0, 1e-6, 128, *outs[i], hs[i + 1], None)
    ws.destroy()
