"""Refusals of the few-token MoE entry points, on the host: bad arguments are answered before anything could launch."""
import ctypes

import pytest
import torch

import tp_reduce_moe_gb300 as arf

BASE, MB = 1 << 40, 1 << 28
E, S, K, H, I, TMAX = 8, 1, 2, 256, 128, 16


@pytest.fixture(scope="module")
def lib():
    from tp_reduce_moe_gb300 import build
    build.build()
    return arf.load_library()


@pytest.fixture()
def moe(lib):
    m = arf.ar_moe_create(E, K, H, I, TMAX, shared=S, flags=arf.AR_WS_DRY_RUN)
    yield m
    m.destroy()


def addr(i):
    return BASE + i * MB


@pytest.mark.parametrize("args,status", [
    ((8, 0, 2, 256, 128, 0, 0), arf.AR_ERR_INVALID_ARG),      # max_tokens
    ((8, 0, 2, 256, 128, 65, 0), arf.AR_ERR_UNSUPPORTED),
    ((0, 0, 2, 256, 128, 4, 0), arf.AR_ERR_INVALID_ARG),      # experts
    ((8, -1, 2, 256, 128, 4, 0), arf.AR_ERR_INVALID_ARG),     # shared
    ((8, 0, 0, 256, 128, 4, 0), arf.AR_ERR_INVALID_ARG),      # top_k
    ((8, 0, 9, 256, 128, 4, 0), arf.AR_ERR_INVALID_ARG),
    ((32, 0, 17, 256, 128, 4, 0), arf.AR_ERR_UNSUPPORTED),
    ((32, 1, 16, 256, 128, 4, 0), arf.AR_ERR_UNSUPPORTED),    # slots
    ((512, 1, 2, 256, 128, 4, 0), arf.AR_ERR_UNSUPPORTED),    # experts + shared
    ((2147483647, 2147483647, 2, 256, 128, 4, 0), arf.AR_ERR_UNSUPPORTED),
    ((8, 0, 2, 0, 128, 4, 0), arf.AR_ERR_UNSUPPORTED),        # hidden
    ((8, 0, 2, 260, 128, 4, 0), arf.AR_ERR_ALIGNMENT),
    ((8, 0, 2, 16392, 128, 4, 0), arf.AR_ERR_UNSUPPORTED),
    ((8, 0, 2, 256, -8, 4, 0), arf.AR_ERR_INVALID_ARG),       # inter
    ((8, 0, 2, 256, 132, 4, 0), arf.AR_ERR_ALIGNMENT),
    ((8, 0, 2, 256, 16392, 4, 0), arf.AR_ERR_UNSUPPORTED),
    ((8, 0, 2, 256, 128, 4, arf.AR_WS_NORM_BF16_H), arf.AR_ERR_INVALID_ARG),
])
def test_create_rejects(lib, args, status):
    h = ctypes.c_void_p(1)
    e, s, k, hid, inter, t, flags = args
    assert lib.ar_moe_create(0, e, s, k, hid, inter, t, flags | arf.AR_WS_DRY_RUN, ctypes.byref(h)) == status
    assert not h.value


def test_null_handles(lib):
    assert lib.ar_moe_create(0, 8, 0, 2, 256, 128, 4, arf.AR_WS_DRY_RUN, None) == arf.AR_ERR_INVALID_ARG
    assert lib.ar_moe_destroy(None) == arf.AR_OK
    assert lib.ar_moe_device_error(None, None) == arf.AR_ERR_INVALID_ARG
    assert lib.ar_moe_route(None, addr(0), addr(1), None, 0, 1, 1.0, 1, 1, 1, addr(2), addr(3), None) == arf.AR_ERR_INVALID_ARG
    assert lib.ar_moe_experts(None, *[addr(i) for i in range(5)], 1, addr(6), None) == arf.AR_ERR_INVALID_ARG
    assert lib.ar_moe_experts_w4(None, *[addr(i) for i in range(7)], 32, 1, addr(8), None) == arf.AR_ERR_INVALID_ARG


@pytest.mark.skipif(torch.cuda.is_available(), reason="needs a machine without a GPU")
def test_without_gpu_fails_cleanly(lib):
    h = ctypes.c_void_p()
    assert lib.ar_moe_create(0, E, S, K, H, I, 4, 0, ctypes.byref(h)) == arf.AR_ERR_CUDA and not h.value
    assert lib.ar_matvec_w4(addr(0), addr(1), addr(2), 32, 1, 64, 64, addr(3), 0, None) == arf.AR_ERR_CUDA


def route(lib, m, **over):
    a = dict(x=addr(0), gate=addr(1), bias=addr(2), scoring=1, renorm=1, scale=1.0, n_group=1, topk_group=1, T=4,
             ids=addr(3), w=addr(4))
    a.update(over)
    return lib.ar_moe_route(m.handle, a["x"], a["gate"], a["bias"], a["scoring"], a["renorm"], a["scale"], a["n_group"],
                            a["topk_group"], a["T"], a["ids"], a["w"], None)


def test_route_arguments(lib, moe):
    assert route(lib, moe) == arf.AR_VALIDATED
    assert route(lib, moe, bias=None, scoring=0, n_group=4, topk_group=1) == arf.AR_VALIDATED
    assert route(lib, moe, T=0, x=None) == arf.AR_OK
    for over in (dict(x=None), dict(gate=None), dict(ids=None), dict(w=None), dict(scoring=2), dict(renorm=2), dict(T=-1),
                 dict(n_group=3), dict(n_group=8), dict(n_group=0), dict(n_group=2, topk_group=3), dict(topk_group=0),
                 dict(n_group=64), dict(ids=addr(4)), dict(ids=addr(0)), dict(w=addr(1) + 64), dict(w=addr(2))):
        assert route(lib, moe, **over) == arf.AR_ERR_INVALID_ARG, over
    for over in (dict(x=addr(0) + 8), dict(gate=addr(1) + 2), dict(bias=addr(2) + 2), dict(ids=addr(3) + 1), dict(w=addr(4) + 2)):
        assert route(lib, moe, **over) == arf.AR_ERR_ALIGNMENT, over
    assert route(lib, moe, T=TMAX + 1) == arf.AR_ERR_CAPACITY
    with_16 = arf.ar_moe_create(16, 9, H, I, 4, flags=arf.AR_WS_DRY_RUN)
    assert route(lib, with_16, n_group=2, topk_group=1) == arf.AR_ERR_INVALID_ARG  # one group holds 8 < 9 experts
    with_16.destroy()


def experts(lib, m, w4, **over):
    a = dict(x=addr(0), ids=addr(1), w=addr(2), w13=addr(3), s13=addr(4), w2=addr(5), s2=addr(6), group=32, T=4, out=addr(7))
    a.update(over)
    if w4:
        return lib.ar_moe_experts_w4(m.handle, a["x"], a["ids"], a["w"], a["w13"], a["s13"], a["w2"], a["s2"], a["group"],
                                     a["T"], a["out"], None)
    return lib.ar_moe_experts(m.handle, a["x"], a["ids"], a["w"], a["w13"], a["w2"], a["T"], a["out"], None)


@pytest.mark.parametrize("w4", [False, True])
def test_experts_arguments(lib, moe, w4):
    assert experts(lib, moe, w4) == arf.AR_VALIDATED
    assert experts(lib, moe, w4, T=0, x=None) == arf.AR_OK
    names = ["x", "ids", "w", "w13", "w2", "out"] + (["s13", "s2"] if w4 else [])
    for n in names:
        assert experts(lib, moe, w4, **{n: None}) == arf.AR_ERR_INVALID_ARG, n
        base = {"x": 0, "ids": 1, "w": 2, "w13": 3, "s13": 4, "w2": 5, "s2": 6, "out": 7}[n]
        off = 2 if n in ("ids", "w") else 8
        assert experts(lib, moe, w4, **{n: addr(base) + off}) == arf.AR_ERR_ALIGNMENT, n
        if n != "out":
            assert experts(lib, moe, w4, out=addr(base) + 16 if n in ("w13", "w2") else addr(base)) == arf.AR_ERR_INVALID_ARG, n
    assert experts(lib, moe, w4, T=-1) == arf.AR_ERR_INVALID_ARG
    assert experts(lib, moe, w4, T=TMAX + 1) == arf.AR_ERR_CAPACITY
    only_route = arf.ar_moe_create(E, K, H, 0, TMAX, flags=arf.AR_WS_DRY_RUN)
    assert experts(lib, only_route, w4) == arf.AR_ERR_UNSUPPORTED
    assert route(lib, only_route) == arf.AR_VALIDATED
    only_route.destroy()
    if w4:
        for g in (0, 16, 48, 256, -32):
            assert experts(lib, moe, w4, group=g) == arf.AR_ERR_UNSUPPORTED
        odd = arf.ar_moe_create(E, K, H, 96, TMAX, flags=arf.AR_WS_DRY_RUN)
        assert experts(lib, odd, w4, group=32) == arf.AR_VALIDATED
        assert experts(lib, odd, w4, group=64) == arf.AR_ERR_UNSUPPORTED
        odd.destroy()


def test_matvec_arguments(lib):
    def call(**over):
        a = dict(x=addr(0), q=addr(1), s=addr(2), group=32, T=4, N=64, K=256, out=addr(3), f32=0)
        a.update(over)
        return lib.ar_matvec_w4(a["x"], a["q"], a["s"], a["group"], a["T"], a["N"], a["K"], a["out"], a["f32"], None)
    assert call(T=0) == arf.AR_OK
    for over in (dict(x=None), dict(q=None), dict(s=None), dict(out=None), dict(T=-1), dict(N=-1), dict(K=-32), dict(f32=2),
                 dict(out=addr(0)), dict(out=addr(1) + 16), dict(out=addr(2))):
        assert call(**over) == arf.AR_ERR_INVALID_ARG, over
    for over in (dict(group=16), dict(group=0), dict(group=128, K=192), dict(N=0), dict(K=0), dict(N=1048577), dict(K=65568)):
        assert call(**over) == arf.AR_ERR_UNSUPPORTED, over
    for n, i in (("x", 0), ("q", 1), ("s", 2), ("out", 3)):
        assert call(**{n: addr(i) + 8}) == arf.AR_ERR_ALIGNMENT
    assert call(T=65) == arf.AR_ERR_CAPACITY


def test_binding_checks_tensors(moe):
    x, ids, w = torch.zeros(3, H, dtype=torch.bfloat16), torch.zeros(3, K + S, dtype=torch.int32), torch.zeros(3, K + S)
    w13 = torch.zeros(E + S, 2 * I, H, dtype=torch.bfloat16)
    w2 = torch.zeros(E + S, H, I, dtype=torch.bfloat16)
    assert arf.ar_moe_experts(moe, x, ids, w, w13, w2).shape == (3, H)
    gate = torch.zeros(E, H, dtype=torch.bfloat16)
    got = arf.ar_moe_route(moe, x, gate)
    assert got[0].shape == got[1].shape == (3, K + S) and got[0].dtype == torch.int32
    for bad in (dict(x=x.float()), dict(ids=ids.long()), dict(w=w.double()), dict(w13=w13.half())):
        a = dict(x=x, ids=ids, w=w, w13=w13, w2=w2)
        a.update(bad)
        with pytest.raises(TypeError):
            arf.ar_moe_experts(moe, a["x"], a["ids"], a["w"], a["w13"], a["w2"])
    for bad in (dict(ids=ids[:, :2]), dict(w13=w13[:E]), dict(w2=w2.transpose(1, 2)), dict(x=x[:, :128]),
                dict(w2=torch.zeros(E + S, I, H, dtype=torch.bfloat16).transpose(1, 2))):
        a = dict(x=x, ids=ids, w=w, w13=w13, w2=w2)
        a.update(bad)
        with pytest.raises(ValueError):
            arf.ar_moe_experts(moe, a["x"], a["ids"], a["w"], a["w13"], a["w2"])
    with pytest.raises(arf.ArfuseError):
        arf.ar_moe_route(moe, x, gate, n_group=3)
    q13, s13 = torch.zeros(E + S, 2 * I, H // 2, dtype=torch.uint8), torch.zeros(E + S, 2 * I, H // 64, dtype=torch.bfloat16)
    q2, s2 = torch.zeros(E + S, H, I // 2, dtype=torch.uint8), torch.zeros(E + S, H, I // 64, dtype=torch.bfloat16)
    arf.ar_moe_experts_w4(moe, x, ids, w, q13, s13, q2, s2, 64)
    with pytest.raises(ValueError):
        arf.ar_moe_experts_w4(moe, x, ids, w, q13, s13, q2, s2, 32)
    with pytest.raises(arf.ArfuseError):
        arf.ar_moe_experts_w4(moe, x, ids, w, q13, s13, q2, s2, 48)
    moe.destroy()
    with pytest.raises(arf.ArfuseError):
        arf.ar_moe_experts(moe, x, ids, w, w13, w2)
