"""Refusals of the attention entry points and the 8-bit norm, on the host: bad arguments are answered before anything could launch."""
import ctypes

import pytest
import torch

import tp_reduce_moe_gb300 as arf
from tp_reduce_moe_gb300 import binding

BASE, MB = 1 << 40, 1 << 28
HEADS, KV, D, PAGE, SEQS, PAGES = 8, 2, 128, 16, 4, 10


@pytest.fixture(scope="module")
def lib():
    from tp_reduce_moe_gb300 import build
    build.build()
    return arf.load_library()


@pytest.fixture()
def attn(lib):
    m = arf.ar_attn_create(HEADS, KV, D, PAGE, SEQS, flags=arf.AR_WS_DRY_RUN)
    yield m
    m.destroy()


def addr(i):
    return BASE + i * MB


@pytest.mark.parametrize("args,status", [
    ((0, 1, 128, 16, 4, 0), arf.AR_ERR_INVALID_ARG),      # heads
    ((-8, 1, 128, 16, 4, 0), arf.AR_ERR_INVALID_ARG),
    ((1025, 1025, 128, 16, 4, 0), arf.AR_ERR_UNSUPPORTED),
    ((8, 0, 128, 16, 4, 0), arf.AR_ERR_INVALID_ARG),      # kv_heads
    ((8, 3, 128, 16, 4, 0), arf.AR_ERR_INVALID_ARG),
    ((8, 16, 128, 16, 4, 0), arf.AR_ERR_INVALID_ARG),
    ((8, 2, 96, 16, 4, 0), arf.AR_ERR_UNSUPPORTED),       # head_dim
    ((8, 2, 0, 16, 4, 0), arf.AR_ERR_UNSUPPORTED),
    ((8, 2, 512, 16, 4, 0), arf.AR_ERR_UNSUPPORTED),
    ((8, 2, 128, 0, 4, 0), arf.AR_ERR_INVALID_ARG),       # page_size
    ((8, 2, 128, 65537, 4, 0), arf.AR_ERR_UNSUPPORTED),
    ((8, 2, 128, 16, 0, 0), arf.AR_ERR_INVALID_ARG),      # max_seqs
    ((8, 2, 128, 16, 4097, 0), arf.AR_ERR_UNSUPPORTED),
    ((8, 2, 128, 16, 4, arf.AR_WS_NORM_BF16_H), arf.AR_ERR_INVALID_ARG),
])
def test_create_rejects(lib, args, status):
    h = ctypes.c_void_p(1)
    *sizes, flags = args
    assert lib.ar_attn_create(0, *sizes, flags | arf.AR_WS_DRY_RUN, ctypes.byref(h)) == status
    assert not h.value


def test_null_handles(lib):
    assert lib.ar_attn_create(0, 8, 2, 128, 16, 4, arf.AR_WS_DRY_RUN, None) == arf.AR_ERR_INVALID_ARG
    assert lib.ar_attn_destroy(None) == arf.AR_OK
    assert lib.ar_attn_device_error(None, None) == arf.AR_ERR_INVALID_ARG
    assert lib.ar_attn_set_rope(None, 0, 0, 1, None, None) == arf.AR_ERR_INVALID_ARG
    c = cache()
    assert lib.ar_attn_append(None, ctypes.byref(c), addr(2), None, addr(3), 1, addr(4), None) == arf.AR_ERR_INVALID_ARG
    assert lib.ar_attn_decode(None, ctypes.byref(c), addr(2), addr(3), 4, 4, addr(4), 1, 0, 1.0, addr(5), None, None) == arf.AR_ERR_INVALID_ARG


@pytest.mark.skipif(torch.cuda.is_available(), reason="needs a machine without a GPU")
def test_without_gpu_fails_cleanly(lib):
    h = ctypes.c_void_p()
    assert lib.ar_attn_create(0, HEADS, KV, D, PAGE, SEQS, 0, ctypes.byref(h)) == arf.AR_ERR_CUDA and not h.value


def cache(**over):
    """Pages of tokens of heads, k then v."""
    c = dict(k=addr(0), v=addr(1), pages=PAGES, k_page=PAGE * KV * D, k_token=KV * D, k_head=D,
             v_page=PAGE * KV * D, v_token=KV * D, v_head=D, k_scale=None, v_scale=None)
    c.update(over)
    return binding._KvCacheStruct(*[c[n] for n, _ in binding._KvCacheStruct._fields_])


def append(lib, m, c=None, null_cache=False, **over):
    a = dict(qkv=addr(2), pos=addr(3), slots=addr(4), T=3, q=addr(5))
    a.update(over)
    c = c or cache()
    return lib.ar_attn_append(m.handle, None if null_cache else ctypes.byref(c), a["qkv"], a["pos"], a["slots"], a["T"], a["q"], None)


def decode(lib, m, c=None, null_cache=False, **over):
    a = dict(q=addr(2), table=addr(3), width=5, stride=5, lengths=addr(4), B=3, window=0, scale=0.1, out=addr(5), lse=addr(6))
    a.update(over)
    c = c or cache()
    return lib.ar_attn_decode(m.handle, None if null_cache else ctypes.byref(c), a["q"], a["table"], a["width"], a["stride"],
                              a["lengths"], a["B"], a["window"], a["scale"], a["out"], a["lse"], None)


EXTENT = PAGES * PAGE * KV * D * 2

CACHES = [  # what a cache may not be
    (dict(k=None), arf.AR_ERR_INVALID_ARG),
    (dict(v=None), arf.AR_ERR_INVALID_ARG),
    (dict(pages=0), arf.AR_ERR_INVALID_ARG),
    (dict(pages=-1), arf.AR_ERR_INVALID_ARG),
    (dict(pages=1 << 27), arf.AR_ERR_UNSUPPORTED),
    (dict(pages=1 << 62), arf.AR_ERR_UNSUPPORTED),
    (dict(k_scale=addr(7)), arf.AR_ERR_INVALID_ARG),
    (dict(v_scale=addr(7)), arf.AR_ERR_INVALID_ARG),
    (dict(k=addr(0) + 8), arf.AR_ERR_ALIGNMENT),
    (dict(v=addr(1) + 2), arf.AR_ERR_ALIGNMENT),
    (dict(k_token=KV * D + 4, k_page=PAGE * (KV * D + 4)), arf.AR_ERR_ALIGNMENT),
    (dict(k_scale=addr(7), v_scale=addr(8), k_token=KV * D + 8, k_page=PAGE * (KV * D + 8)), arf.AR_ERR_ALIGNMENT),
    (dict(k_scale=addr(7) + 2, v_scale=addr(8)), arf.AR_ERR_ALIGNMENT),
    (dict(k_head=0), arf.AR_ERR_INVALID_ARG),                       # elements at one place
    (dict(v_head=D - 8), arf.AR_ERR_INVALID_ARG),
    (dict(k_token=D), arf.AR_ERR_INVALID_ARG),
    (dict(v_page=0), arf.AR_ERR_INVALID_ARG),
    (dict(v_page=(PAGE - 1) * KV * D), arf.AR_ERR_INVALID_ARG),
    (dict(k_page=-PAGE * KV * D), arf.AR_ERR_INVALID_ARG),
    (dict(k_page=1 << 62), arf.AR_ERR_INVALID_ARG),
    (dict(k_page=1 << 46), arf.AR_ERR_INVALID_ARG),
]


@pytest.mark.parametrize("over,status", CACHES)
def test_caches(lib, attn, over, status):
    assert append(lib, attn, cache(**over)) == status
    assert decode(lib, attn, cache(**over)) == status


@pytest.mark.parametrize("over", [
    {}, dict(k_scale=addr(7), v_scale=addr(8)),
    dict(k_token=D, k_head=PAGE * D, v_token=D, v_head=PAGE * D),                                  # heads of tokens
    dict(v=addr(0) + PAGE * KV * D * 2, k_page=2 * PAGE * KV * D, v_page=2 * PAGE * KV * D),       # both in one tensor
    dict(k_page=D, k_token=PAGES * D, k_head=PAGES * PAGE * D),                                    # heads of tokens of pages
    dict(pages=1, k_page=0, v_page=-3),                                                            # strides that count nothing
    dict(k_page=1 << 41),
])
def test_caches_taken(lib, attn, over):
    if over.get("k_page") == 1 << 41:  # (its end has to be behind every other argument)
        over = dict(over, k=addr(20))
    assert append(lib, attn, cache(**over)) == arf.AR_VALIDATED
    assert decode(lib, attn, cache(**over)) == arf.AR_VALIDATED


def test_single_page_and_head(lib):
    m = arf.ar_attn_create(4, 1, 64, 1, 2, flags=arf.AR_WS_DRY_RUN)
    one = dict(pages=7, k_page=64, v_page=64, k_token=3, k_head=5, v_token=-1, v_head=0)
    assert decode(lib, m, cache(**one), B=2) == arf.AR_VALIDATED
    assert decode(lib, m, cache(**dict(one, k_page=56)), B=2) == arf.AR_ERR_INVALID_ARG
    m.destroy()


def test_append_arguments(lib, attn):
    assert append(lib, attn, pos=None) == arf.AR_VALIDATED  # no rotary positions
    assert append(lib, attn, T=0, qkv=None) == arf.AR_OK
    arf.ar_attn_set_rope(attn, [0.5] * 64, axis=[0] * 32 + [2] * 32)
    assert append(lib, attn) == arf.AR_VALIDATED
    assert append(lib, attn, null_cache=True) == arf.AR_ERR_INVALID_ARG
    assert append(lib, attn, cache(v=addr(0))) == arf.AR_ERR_INVALID_ARG
    for over in (dict(qkv=None), dict(pos=None), dict(slots=None), dict(q=None), dict(T=-1)):
        assert append(lib, attn, **over) == arf.AR_ERR_INVALID_ARG, over
    for over in (dict(qkv=addr(2) + 8), dict(pos=addr(3) + 2), dict(slots=addr(4) + 1), dict(q=addr(5) + 4)):
        assert append(lib, attn, **over) == arf.AR_ERR_ALIGNMENT, over
    assert append(lib, attn, T=arf.AR_MAX_ATTN_TOKENS + 1) == arf.AR_ERR_CAPACITY
    for over in (dict(q=addr(2) + 16), dict(q=addr(3)), dict(q=addr(4)), dict(q=addr(0) + EXTENT - 16), dict(q=addr(1)),
                 dict(qkv=addr(0)), dict(qkv=addr(1) + EXTENT - 16), dict(slots=addr(1)), dict(pos=addr(0) + 64)):
        assert append(lib, attn, **over) == arf.AR_ERR_INVALID_ARG, over
    eight = cache(k_scale=addr(7), v_scale=addr(8))
    assert append(lib, attn, eight) == arf.AR_VALIDATED
    assert append(lib, attn, eight, q=addr(8)) == arf.AR_ERR_INVALID_ARG
    assert append(lib, attn, cache(k_scale=addr(0) + 64, v_scale=addr(8))) == arf.AR_ERR_INVALID_ARG
    # the axes count: three rows of positions before the slots
    assert append(lib, attn, slots=addr(0) - 3 * 4, pos=addr(2) - 3 * 3 * 4) == arf.AR_VALIDATED
    assert append(lib, attn, q=addr(7), pos=addr(7) - 2 * 3 * 4) == arf.AR_ERR_INVALID_ARG


def test_rope_arguments(lib, attn):
    f = (ctypes.c_double * 64)(*[1.0] * 64)
    ax = (ctypes.c_int32 * 64)(*[0] * 64)
    assert lib.ar_attn_set_rope(attn.handle, 128, 0, 1, f, None) == arf.AR_OK
    assert lib.ar_attn_set_rope(attn.handle, 0, 0, 0, None, None) == arf.AR_OK
    assert lib.ar_attn_set_rope(attn.handle, 112, 1, 4, f, ax) == arf.AR_OK
    for args in ((-16, 0, 1, f, ax), (144, 0, 1, f, ax), (64, 2, 1, f, ax), (64, 0, 0, f, ax), (64, 0, 5, f, ax), (64, 0, 1, None, ax)):
        assert lib.ar_attn_set_rope(attn.handle, *args) == arf.AR_ERR_INVALID_ARG, args
    assert lib.ar_attn_set_rope(attn.handle, 24, 0, 1, f, ax) == arf.AR_ERR_UNSUPPORTED
    for bad in (-1, 2):
        ax[3] = bad
        assert lib.ar_attn_set_rope(attn.handle, 128, 0, 2, f, ax) == arf.AR_ERR_INVALID_ARG
    for bad in (float("nan"), float("inf")):
        f[63] = bad
        assert lib.ar_attn_set_rope(attn.handle, 128, 0, 1, f, None) == arf.AR_ERR_INVALID_ARG
    assert append(lib, attn, pos=None) == arf.AR_ERR_INVALID_ARG  # the table before stands


def test_decode_arguments(lib, attn):
    assert decode(lib, attn) == arf.AR_VALIDATED
    assert decode(lib, attn, lse=None, window=7, stride=9, B=4) == arf.AR_VALIDATED
    assert decode(lib, attn, table=None, width=0, stride=0) == arf.AR_VALIDATED
    assert decode(lib, attn, cache(v=addr(0))) == arf.AR_VALIDATED  # values that are the keys
    assert decode(lib, attn, B=1, stride=0) == arf.AR_VALIDATED
    assert decode(lib, attn, B=0, q=None) == arf.AR_OK
    assert decode(lib, attn, window=1 << 40, width=1 << 30, stride=1 << 30, table=addr(20)) == arf.AR_VALIDATED
    for over in (dict(q=None), dict(table=None), dict(lengths=None), dict(out=None), dict(B=-1), dict(width=-1), dict(window=-1),
                 dict(stride=4), dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=3e38), dict(null_cache=True)):
        assert decode(lib, attn, **over) == arf.AR_ERR_INVALID_ARG, over
    for over in (dict(q=addr(2) + 8), dict(table=addr(3) + 2), dict(lengths=addr(4) + 1), dict(out=addr(5) + 2), dict(lse=addr(6) + 2)):
        assert decode(lib, attn, **over) == arf.AR_ERR_ALIGNMENT, over
    assert decode(lib, attn, B=SEQS + 1) == arf.AR_ERR_CAPACITY
    assert decode(lib, attn, stride=1 << 60) == arf.AR_ERR_UNSUPPORTED
    assert decode(lib, attn, width=1 << 31, stride=1 << 31) == arf.AR_ERR_UNSUPPORTED
    eight = cache(k_scale=addr(7), v_scale=addr(8))
    for c, over in ((None, dict(out=addr(2))), (None, dict(out=addr(3))), (None, dict(out=addr(4))), (None, dict(lse=addr(5) + 64)),
                    (None, dict(out=addr(0) + EXTENT - 16)), (None, dict(lse=addr(1))), (eight, dict(out=addr(7))), (eight, dict(lse=addr(8)))):
        assert decode(lib, attn, c, **over) == arf.AR_ERR_INVALID_ARG, over


def test_python_checks(attn):
    bf, f8 = torch.bfloat16, torch.float8_e4m3fn
    new = lambda *s, dtype=bf: torch.zeros(s, dtype=dtype)  # noqa: E731
    k, v = new(PAGES, PAGE, KV, D), new(PAGES, PAGE, KV, D)
    scales = torch.ones(KV)
    c = arf.ar_kv_cache(k, v)
    arf.ar_kv_cache(k.to(f8), v.to(f8), scales, scales)
    for bad in ((k, v, scales, None), (k[0], v[0]), (k, v[:5]), (k.transpose(2, 3), v.transpose(2, 3))):
        with pytest.raises(ValueError):
            arf.ar_kv_cache(*bad)
    for bad in ((k.float(), v), (k, v, scales, scales), (k.to(f8), v.to(f8))):
        with pytest.raises(TypeError):
            arf.ar_kv_cache(*bad)
    with pytest.raises(ValueError):
        arf.ar_kv_cache(k.to(f8), v.to(f8), scales, torch.ones(KV + 1))
    T, cols = 3, (HEADS + 2 * KV) * D
    qkv, slots, pos = new(T, cols), new(T, dtype=torch.int32), new(3, T, dtype=torch.int32)
    assert arf.ar_attn_append(attn, c, qkv, None, slots).shape == (T, HEADS, D)
    arf.ar_attn_set_rope(attn, [0.1] * 8, axis=[0, 1, 2, 0, 1, 2, 0, 1])
    arf.ar_attn_append(attn, c, qkv, pos, slots)
    with pytest.raises(ValueError):
        arf.ar_attn_set_rope(attn, [0.1] * 8, axis=[0])
    other = arf.ar_kv_cache(new(PAGES, PAGE, KV, 64), new(PAGES, PAGE, KV, 64))
    for args in ((other, qkv, pos, slots), (c, qkv[:, :-8], pos, slots), (c, qkv, pos[:2], slots), (c, qkv, None, slots), (c, qkv, pos, slots[:2])):
        with pytest.raises(ValueError):
            arf.ar_attn_append(attn, *args)
    for args in ((c, qkv.float(), pos, slots), (c, qkv, pos.long(), slots), (c, qkv, pos, slots.long())):
        with pytest.raises(TypeError):
            arf.ar_attn_append(attn, *args)
    q, table, lengths = new(T, HEADS, D), new(T, 4, dtype=torch.int32), new(T, dtype=torch.int32)
    out, lse = arf.ar_attn_decode(attn, c, q, table, lengths, lse=new(T, HEADS, dtype=torch.float32))
    assert out.shape == q.shape and lse.shape == (T, HEADS)
    arf.ar_attn_decode(attn, c, q, new(T, 9, dtype=torch.int32)[:, 2:6], lengths)
    for args in ((other, q, table, lengths), (c, q[:, :4], table, lengths), (c, q, table[:2], lengths), (c, q, table[0], lengths),
                 (c, q, table[:1].expand(T, 4), lengths), (c, q, new(4, T, dtype=torch.int32).t(), lengths), (c, q, table, lengths[:2])):
        with pytest.raises(ValueError):
            arf.ar_attn_decode(attn, *args)
    for args in ((c, q.float(), table, lengths), (c, q, table.long(), lengths), (c, q, table, lengths.long())):
        with pytest.raises(TypeError):
            arf.ar_attn_decode(attn, *args)
    with pytest.raises(arf.ArfuseError) as e:
        arf.ar_attn_decode(attn, c, new(SEQS + 1, HEADS, D), new(SEQS + 1, 4, dtype=torch.int32), new(SEQS + 1, dtype=torch.int32))
    assert e.value.status == arf.AR_ERR_CAPACITY
    attn.destroy()
    assert not attn.alive
    with pytest.raises(arf.ArfuseError):
        arf.ar_attn_decode(attn, c, q, table, lengths)


# --------------------------------------------------------------------- the norm with an 8-bit output
R, H, TMAX, EPS = 2, 1000, 8, 1e-6


@pytest.fixture()
def ws(lib):
    w = arf.ar_workspace_create(R, 0, H, TMAX, EPS, flags=arf.AR_WS_DRY_RUN)
    yield w
    w.destroy()


def norm(lib, w, **over):
    a = dict(p=[addr(0), addr(1)], R=R, residual=addr(2), gamma=addr(3), eps=EPS, T=4, H=H, group=128, q=addr(4), scales=addr(5),
             out=addr(6), r_out=addr(7), fp32=0)
    a.update(over)
    p = (ctypes.c_void_p * len(a["p"]))(*a["p"]) if a["p"] is not None else None
    return lib.ar_rmsnorm_q8(w.handle if w else None, p, a["R"], a["residual"], a["gamma"], 0.0, a["eps"], a["T"], a["H"], a["group"],
                             a["q"], a["scales"], a["out"], a["r_out"], a["fp32"], None)


def test_norm_q8_arguments(lib, ws):
    for over in ({}, dict(out=None), dict(group=0), dict(group=32), dict(group=64, fp32=1), dict(r_out=addr(2)), dict(q=addr(4) + 8)):
        assert norm(lib, ws, **over) == arf.AR_VALIDATED, over
    assert norm(lib, ws, T=0, residual=None) == arf.AR_OK
    assert norm(lib, None) == arf.AR_ERR_INVALID_ARG
    for over in (dict(p=None), dict(p=[addr(0), None]), dict(R=1), dict(R=17), dict(R=0), dict(residual=None), dict(gamma=None), dict(q=None),
                 dict(scales=None), dict(r_out=None), dict(eps=1e-5), dict(T=-1), dict(H=992), dict(fp32=2),
                 dict(r_out=addr(2), fp32=1), dict(r_out=addr(2) + 16), dict(q=addr(2)), dict(q=addr(0)), dict(q=addr(7) + 64),
                 dict(scales=addr(4) + 64), dict(scales=addr(3)), dict(out=addr(7)), dict(out=addr(2)), dict(out=addr(1) + 16),
                 dict(r_out=addr(0))):
        assert norm(lib, ws, **over) == arf.AR_ERR_INVALID_ARG, over
    for over in (dict(p=[addr(0), addr(1) + 8]), dict(residual=addr(2) + 8), dict(gamma=addr(3) + 2), dict(q=addr(4) + 4),
                 dict(scales=addr(5) + 2), dict(out=addr(6) + 8), dict(r_out=addr(7) + 8)):
        assert norm(lib, ws, **over) == arf.AR_ERR_ALIGNMENT, over
    for group in (-1, 1, 16, 48, 256, 1000):
        assert norm(lib, ws, group=group) == arf.AR_ERR_UNSUPPORTED
    assert norm(lib, ws, T=TMAX + 1) == arf.AR_ERR_CAPACITY


def test_norm_q8_python_checks(ws):
    new = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype)  # noqa: E731
    T = 3
    parts, res, gamma = [new(T, H), new(T, H)], new(T, H), new(H)
    q, scales, h = arf.ar_rmsnorm_q8(ws, parts, res, gamma, 0.0, EPS, residual_out=res)
    assert q.dtype == torch.float8_e4m3fn and q.shape == (T, H) and scales.shape == (T, 8) and h is res
    assert arf.ar_rmsnorm_q8(ws, parts, res, gamma, 0.0, EPS, group=0, residual_out_fp32=True)[1].shape == (T, 1)
    for args, kw in (((parts[:1], res, gamma), {}), ((parts, res[:, :-8], gamma), {}), ((parts, res, gamma[:-8]), {}),
                     ((parts, res, gamma), dict(scales=new(T, 7, dtype=torch.float32))), ((parts, res, gamma), dict(q=new(T, 8, dtype=torch.float8_e4m3fn)))):
        with pytest.raises(ValueError):
            arf.ar_rmsnorm_q8(ws, *args, 0.0, EPS, **kw)
    for args, kw in ((([p.float() for p in parts], res, gamma), {}), ((parts, res, gamma), dict(q=new(T, H, dtype=torch.uint8))),
                     ((parts, res, gamma), dict(residual_out=new(T, H), residual_out_fp32=True)), ((parts, res, gamma), dict(out=new(T, H, dtype=torch.float32)))):
        with pytest.raises(TypeError):
            arf.ar_rmsnorm_q8(ws, *args, 0.0, EPS, **kw)
    with pytest.raises(arf.ArfuseError) as e:
        arf.ar_rmsnorm_q8(ws, parts, res, gamma, 0.0, EPS, group=256)
    assert e.value.status == arf.AR_ERR_UNSUPPORTED
    with pytest.raises(TypeError, match=r"partials\[1\]"):
        arf.ar_rmsnorm_q8(ws, [parts[0], parts[1].float()], res, gamma, 0.0, EPS)


# --------------------------------------------------------------------- tensors without a place in memory, calls without work
def test_tensors_that_have_no_memory(attn, ws):
    # their addresses cannot be asked for: an error of Python's, with nothing called
    mode = pytest.importorskip("torch._subclasses.fake_tensor").FakeTensorMode()
    T, cols = 3, (HEADS + 2 * KV) * D
    c = arf.ar_kv_cache(torch.zeros(PAGES, PAGE, KV, D).bfloat16(), torch.zeros(PAGES, PAGE, KV, D).bfloat16())
    new = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype)  # noqa: E731
    with mode:
        fake_q, fake_qkv, fake_res = torch.zeros(T, HEADS, D).bfloat16(), torch.zeros(T, cols).bfloat16(), torch.zeros(T, H).bfloat16()
    table, ints = new(T, 4, dtype=torch.int32), new(T, dtype=torch.int32)
    out = new(T, HEADS, D)
    refused = (arf.ArfuseError, TypeError, ValueError, RuntimeError)
    with pytest.raises(refused):
        arf.ar_attn_decode(attn, c, fake_q, table, ints, out=out)
    with pytest.raises(refused):
        arf.ar_attn_append(attn, c, fake_qkv, None, ints, q=out)
    with pytest.raises(refused):
        arf.ar_attn_append(attn, c, new(T, cols).to_sparse(), None, ints, q=out)
    nested = torch.nested.nested_tensor([new(H), new(H), new(H - 8)])
    for parts, res in (([new(T, H), new(T, H)], fake_res), ([new(T, H), nested], new(T, H))):
        with pytest.raises(refused):
            arf.ar_rmsnorm_q8(ws, parts, res, new(H), 0.0, EPS, q=new(T, H, dtype=torch.float8_e4m3fn),
                              scales=new(T, 8, dtype=torch.float32), residual_out=new(T, H))


def test_calls_without_work(attn, ws):
    new = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype)  # noqa: E731
    c = arf.ar_kv_cache(new(PAGES, PAGE, KV, D), new(PAGES, PAGE, KV, D))
    none = new(0, dtype=torch.int32)
    assert arf.ar_attn_append(attn, c, new(0, (HEADS + 2 * KV) * D), None, none).shape == (0, HEADS, D)
    assert arf.ar_attn_decode(attn, c, new(0, HEADS, D), new(0, 4, dtype=torch.int32), none).shape == (0, HEADS, D)
    # no page of any sequence is named: its length can only be 0
    assert arf.ar_attn_decode(attn, c, new(2, HEADS, D), new(2, 0, dtype=torch.int32), new(2, dtype=torch.int32)).shape == (2, HEADS, D)
    q, scales, h = arf.ar_rmsnorm_q8(ws, [new(0, H), new(0, H)], new(0, H), new(H), 0.0, EPS)
    assert q.shape == h.shape == (0, H) and scales.shape == (0, 8)
