"""Rotary positions into the paged cache, and the attention of one new token over it, against their definitions in 64 bits
(needs a GB300)."""
import math

import pytest
import torch

import tp_reduce_moe_gb300 as arf
from tests import _attn

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _built():
    from tp_reduce_moe_gb300 import build
    build.build()
    arf.load_library()
    torch.cuda.set_device(0)


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def normal(shape, g, std=1.0):
    return torch.randn(shape, generator=g, device=DEV).mul_(std).bfloat16()


def guarded(shape, dtype):
    """A tensor with 64 guard values on both sides, and a check that they stand."""
    n = math.prod(shape)
    buf = torch.full((n + 128,), 77, dtype=dtype, device=DEV)
    return buf[64:64 + n].view(shape), lambda: bool((buf[:64] == 77).all()) and bool((buf[64 + n:] == 77).all())


def paged(pages, page, kv, D, eight, layout, g, fill=None):
    """k, v [pages, page, kv, D] of a layout, and their scales (None for bf16)."""
    if layout == "token":      # pages of tokens of heads
        x = torch.empty(2, pages, page, kv, D, device=DEV, dtype=torch.bfloat16)
    elif layout == "head":     # pages of heads of tokens
        x = torch.empty(2, pages, kv, page, D, device=DEV, dtype=torch.bfloat16).transpose(2, 3)
    elif layout == "pair":     # keys and values in one tensor
        x = torch.empty(pages, 2, page, kv, D, device=DEV, dtype=torch.bfloat16).transpose(0, 1)
    else:                      # rows further apart than they are long, heads before pages
        x = torch.empty(2, kv, pages, page + 1, D + 16, device=DEV, dtype=torch.bfloat16)[:, :, :, :page, 16:].permute(0, 2, 3, 1, 4)
    if fill is None:
        x.copy_(normal(x.shape, g))
    else:
        x.fill_(fill)
    if not eight:
        return x[0], x[1], None, None
    y = torch.empty_strided(x.shape, x.stride(), dtype=torch.uint8, device=DEV).view(F8)
    y.view(torch.uint8).copy_(x.to(F8).view(torch.uint8))
    return y[0], y[1], torch.rand(kv, device=DEV, generator=g) + 0.5, torch.rand(kv, device=DEV, generator=g) + 0.5


# -------------------------------------------------------------------- decode
def tables(lengths, page, pages, width, g):
    """Distinct pages in a random order for every sequence, -7 where a sequence has none."""
    table = torch.full((len(lengths), width), -7, dtype=torch.int32, device=DEV)
    order, at = torch.randperm(pages, generator=g, device=DEV).int(), 0
    for b, n in enumerate(lengths):
        need = -(-max(0, n) // page)
        table[b, :need] = order[at:at + need]
        at += need
    assert at <= pages
    return table


def check_decode(m, q, k, v, ks, vs, table, lengths, window=0, scale=None, runs=2, **kw):
    B, heads, D = q.shape
    cache = arf.ar_kv_cache(k, v, ks, vs)
    out, ok1 = guarded((B, heads, D), torch.bfloat16)
    lse, ok2 = guarded((B, heads), torch.float32)
    lens = torch.tensor(lengths, dtype=torch.int32, device=DEV)
    s = D ** -0.5 if scale is None else scale
    want, slack, want_lse, lse_slack = _attn.decode_ref(q, k, v, table, lengths, k.shape[1], window, s, ks, vs, ks is not None)
    first = None
    for _ in range(runs):  # the second call finds the handle as the first left it, and gives the same bits
        out.zero_()
        lse.zero_()
        arf.ar_attn_decode(m, cache, q, table, lens, scale=scale, window=window, out=out, lse=lse, **kw)
        torch.cuda.synchronize()
        off = (out.double() - want).abs()
        assert bool((off <= slack).all()), f"out: {float((off / slack).max())} of the bound"
        empty = torch.isinf(want_lse)
        assert torch.equal(empty, torch.isinf(lse) & (lse < 0))
        off = (lse.double() - want_lse).abs()[~empty]
        assert bool((off <= lse_slack[~empty]).all()), f"lse: {float((off / lse_slack[~empty]).max())} of the bound"
        assert ok1() and ok2()
        if first is not None:
            assert torch.equal(first[0], out) and torch.equal(first[1], lse)
        first = (out.clone(), lse.clone())
    return out


DECODES = [  # heads, kv, D, page, eight, layout, window, lengths
    (8, 1, 128, 16, False, "token", 0, [1]),
    (8, 1, 128, 16, False, "token", 0, [500]),
    (1, 1, 64, 1, False, "token", 0, [1, 2, 17, 33]),
    (32, 8, 128, 16, False, "token", 0, [0, 1, 15, 16, 17, 31, 33, 64, 1000, 129]),
    (16, 2, 128, 64, False, "head", 0, [5000, 3, 0, 0, 700]),
    (16, 16, 64, 20, False, "token", 100, [0, 1, 99, 100, 101, 119, 400, 1234]),
    (16, 2, 256, 32, False, "head", 0, [1, 31, 32, 33, 2001]),
    (64, 8, 128, 64, True, "pair", 0, [1, 63, 65, 3000, 257]),
    (7, 7, 64, 8, True, "token", 0, [9, 700, 8]),
    (12, 4, 256, 16, True, "head", 0, [1000, 77, 16]),
    (20, 1, 128, 7, False, "odd", 0, [300, 6, 7, 8]),
    (48, 2, 64, 128, True, "odd", 33, [300, 6, 129, 32, 33, 34]),
    (40, 2, 128, 16, False, "pair", 1, [300, 1, 0, 16, 17]),
    (256, 1, 128, 16, False, "token", 0, [900, 30]),
    (256, 256, 64, 16, False, "token", 0, [40, 7]),
    (320, 16, 128, 20, False, "head", 0, [400, 1, 90]),
    (1024, 1024, 64, 16, True, "token", 0, [33]),
    (1024, 8, 256, 16, False, "token", 20, [70, 19]),
    (24, 8, 128, 1000, False, "token", 0, [999, 1000, 1001, 2500]),
    (80, 1, 256, 3, True, "token", 0, [100, 50, 1]),
    (4, 2, 64, 16, False, "token", 5000, [40000, 10]),
    (2, 1, 128, 16, False, "token", 0, [60001]),
    (2, 1, 64, 16, True, "head", 0, [70001, 20000]),
    (3, 1, 256, 16, False, "token", 0, [30001]),
]


@pytest.mark.parametrize("heads,kv,D,page,eight,layout,window,lengths", DECODES)
def test_decode(heads, kv, D, page, eight, layout, window, lengths):
    g = gen(heads * 1000 + D + page)
    need = sum(-(-n // page) for n in lengths)
    pages = need + 3
    k, v, ks, vs = paged(pages, page, kv, D, eight, layout, g)
    table = tables(lengths, page, pages, max(1, max(-(-n // page) for n in lengths)) + 2, g)
    q = normal((len(lengths), heads, D), g, 2.0)
    m = arf.ar_attn_create(heads, kv, D, page, len(lengths), device=0)
    check_decode(m, q, k, v, ks, vs, table, lengths, window)
    check_decode(m, q, k, v, ks, vs, table, lengths, window, scale=-0.5 * D ** -0.5, runs=1)
    assert arf.ar_attn_device_error(m) == 0
    m.destroy()


@pytest.mark.parametrize("B", [3, 160, 700, 4096])
def test_decode_many_sequences(B):
    heads, kv, D, page = 8, 4, 64, 16
    g = gen(B)
    lengths = [(b * 37) % 90 for b in range(B)]
    pages = sum(-(-n // page) for n in lengths) + 1
    k, v, ks, vs = paged(pages, page, kv, D, False, "token", g)
    m = arf.ar_attn_create(heads, kv, D, page, B, device=0)
    check_decode(m, normal((B, heads, D), g), k, v, ks, vs, tables(lengths, page, pages, 6, g), lengths)
    m.destroy()


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("B", [1, 18, 19, 20, 38])
def test_decode_equal_lengths(B, eight):
    # items that have a CTA each, up to all SMs, and more of them than SMs
    heads, kv, D, page, n = 16, 8, 64, 16, 700
    g = gen(300 + B)
    pages = B * -(-n // page) + 1
    k, v, ks, vs = paged(pages, page, kv, D, eight, "head", g)
    m = arf.ar_attn_create(heads, kv, D, page, B, device=0)
    check_decode(m, normal((B, heads, D), g), k, v, ks, vs, tables([n] * B, page, pages, 50, g), [n] * B)
    m.destroy()


@pytest.mark.parametrize("eight", [False, True])
def test_decode_much_work(eight):
    # 400 MB of keys and values to stream (from pages that sequences share): more than all SMs take for two bytes
    heads, kv, D, page, B = 12, 4, 64, 16, 256
    g = gen(29)
    k, v, ks, vs = paged(400, page, kv, D, eight, "token", g)
    lengths = [(b * 577) % 3200 for b in range(B)]
    assert sum(lengths) * kv * D * 2 * (1 if eight else 2) > (200 << 20 if eight else 400 << 20)
    table = torch.randint(0, 400, (B, 200), generator=g, device=DEV, dtype=torch.int32)
    m = arf.ar_attn_create(heads, kv, D, page, B, device=0)
    check_decode(m, normal((B, heads, D), g), k, v, ks, vs, table, lengths)
    assert arf.ar_attn_device_error(m) == 0
    m.destroy()


@pytest.mark.parametrize("heads,kv,D,eight", [(32, 2, 128, False), (24, 2, 64, False), (32, 2, 128, True), (32, 2, 256, False), (40, 1, 64, True)])
def test_decode_heads_in_groups_of_sixteen(heads, kv, D, eight):
    # tables so wide that keys and values could be more than 64 MB: groups of up to sixteen heads, otherwise of eight
    page, lengths = 16, [0, 1, 17, 900, 64, 2500, 33]
    g = gen(heads * D)
    pages = sum(-(-n // page) for n in lengths) + 2
    k, v, ks, vs = paged(pages, page, kv, D, eight, "pair", g)
    q = normal((len(lengths), heads, D), g, 2.0)
    m = arf.ar_attn_create(heads, kv, D, page, len(lengths), device=0)
    for width in (170, 8000):
        check_decode(m, q, k, v, ks, vs, tables(lengths, page, pages, width, g), lengths)
    assert arf.ar_attn_device_error(m) == 0
    m.destroy()


def test_decode_without_work():
    heads, kv, D, page = 8, 2, 128, 16
    g = gen(31)
    k, v, _, _ = paged(3, page, kv, D, False, "token", g)
    cache = arf.ar_kv_cache(k, v)
    m = arf.ar_attn_create(heads, kv, D, page, 4096, device=0)
    for B, width in ((0, 4), (3, 0), (1, 0), (4096, 0), (33, 2)):
        lens = torch.zeros(B, dtype=torch.int32, device=DEV)
        out, ok1 = guarded((B, heads, D), torch.bfloat16)
        lse, ok2 = guarded((B, heads), torch.float32)
        out.fill_(5), lse.fill_(5)
        arf.ar_attn_decode(m, cache, normal((B, heads, D), g), torch.full((B, width), -1, dtype=torch.int32, device=DEV), lens, out=out, lse=lse)
        torch.cuda.synchronize()
        assert bool((out == 0).all()) and bool((lse == float("-inf")).all()) and ok1() and ok2()
    assert arf.ar_attn_device_error(m) == 0
    m.destroy()


def test_decode_scores_of_minus_infinity():
    # they count as no token; a row of nothing else as one without tokens
    heads, kv, D, page, n = 4, 2, 64, 16, 100
    g = gen(32)
    k, v, _, _ = paged(21, page, kv, D, False, "token", g)
    q = normal((3, heads, D), g)
    q[..., 0] = 1.0
    table = tables([n, n, 1], page, 21, 7, g)
    gone = torch.zeros(n, dtype=torch.bool, device=DEV)
    gone[::3] = True
    gone[:48] = True
    for t in range(n):
        for b in range(2):
            if gone[t] or b == 1:
                k[int(table[b, t // page]), t % page, :, 0] = float("-inf")
    m = arf.ar_attn_create(heads, kv, D, page, 3, device=0)
    lse = torch.empty(3, heads, device=DEV)
    out, _ = arf.ar_attn_decode(m, arf.ar_kv_cache(k, v), q, table, torch.tensor([n, n, 1], dtype=torch.int32, device=DEV), lse=lse)
    # the first sequence again, with the tokens that count on pages of one token
    at = torch.arange(n, device=DEV)[~gone]
    k1, v1 = (x[table[0, at // page].long(), at % page].unsqueeze(1).contiguous() for x in (k, v))
    table1 = torch.arange(len(at), dtype=torch.int32, device=DEV).view(1, -1)
    want, slack, want_lse, lse_slack = _attn.decode_ref(q[:1], k1, v1, table1, [len(at)], 1, 0, D ** -0.5)
    torch.cuda.synchronize()
    assert bool(((out[:1].double() - want).abs() <= slack).all())
    assert bool(((lse[:1].double() - want_lse).abs() <= lse_slack).all())
    assert bool((out[1] == 0).all()) and bool((lse[1] == float("-inf")).all())
    assert bool(torch.isfinite(out[2]).all()) and bool(torch.isfinite(lse[2]).all())
    m.destroy()


@pytest.mark.parametrize("eight", [False, True])
def test_decode_reads_nothing_outside_the_tokens(eight):
    # every place that no sequence holds, and what lies before a window, is NaN
    heads, kv, D, page, lengths, window = 8, 2, 128, 16, [37, 16, 1, 0, 200], 50
    g = gen(11)
    for w in (0, window):
        k, v, ks, vs = paged(30, page, kv, D, eight, "token", g, fill=float("nan"))
        table = tables(lengths, page, 30, 14, g)
        for b, n in enumerate(lengths):
            for t in range(max(0, n - w) if w else 0, n):
                p = int(table[b, t // page])
                for x in (k, v):
                    x[p, t % page] = normal((kv, D), g).to(x.dtype)
        m = arf.ar_attn_create(heads, kv, D, page, 5, device=0)
        out = check_decode(m, normal((5, heads, D), g), k, v, ks, vs, table, lengths, window=w)
        assert bool(torch.isfinite(out).all())
        assert arf.ar_attn_device_error(m) == 0
        m.destroy()


def test_decode_bad_pages_and_lengths():
    heads, kv, D, page = 8, 2, 128, 16
    g = gen(12)
    k, v, _, _ = paged(40, page, kv, D, False, "token", g)
    lengths = [100, 40, 16, 70]
    table = tables(lengths, page, 40, 8, g)
    m = arf.ar_attn_create(heads, kv, D, page, 4, device=0)
    q = normal((4, heads, D), g)
    table[0, 2], table[0, 5], table[2, 0], table[3, 0] = 40, -1, 2 ** 31 - 1, -(2 ** 31)  # the third row is left with nothing
    check_decode(m, q, k, v, None, None, table, lengths, runs=1)
    assert arf.ar_attn_device_error(m) == arf.AR_DEVERR_PAGE_RANGE
    assert arf.ar_attn_device_error(m) == 0
    table = tables([128] * 4, page, 40, 8, g)
    check_decode(m, q, k, v, None, None, table, [129, -1, 2 ** 31 - 1, -(2 ** 31)], runs=1)
    assert arf.ar_attn_device_error(m) == arf.AR_DEVERR_LENGTH_RANGE
    # pages that a window leaves behind, or that are beyond the length, are not looked at
    table[:, 0], table[:, 7] = 1000, -1
    check_decode(m, q, k, v, None, None, table, [112, 100, 60, 112], window=40, runs=1)
    assert arf.ar_attn_device_error(m) == 0
    # a table without columns
    lens = torch.tensor([0, 0, 0, 0], dtype=torch.int32, device=DEV)
    out = arf.ar_attn_decode(m, arf.ar_kv_cache(k, v), q, table[:, :0], lens)
    assert bool((out == 0).all()) and arf.ar_attn_device_error(m) == 0
    m.destroy()


def test_decode_rows_of_a_wider_table_and_shared_pages():
    heads, kv, D, page = 8, 2, 64, 16
    g = gen(13)
    k, v, _, _ = paged(20, page, kv, D, False, "token", g)
    wide = tables([100, 40, 16], page, 20, 30, g)
    wide[1, :7] = wide[0, :7]  # a forked sequence reads the first one's pages
    m = arf.ar_attn_create(heads, kv, D, page, 3, device=0)
    check_decode(m, normal((3, heads, D), g), k, v, None, None, wide[:, :9], [100, 107, 16])
    m.destroy()


@pytest.mark.parametrize("eight", [False, True])
def test_decode_extreme_scores(eight):
    heads, kv, D, page = 4, 1, 128, 16
    g = gen(14)
    k, v, ks, vs = paged(10, page, kv, D, eight, "token", g)
    table = tables([150], page, 10, 10, g)
    m = arf.ar_attn_create(heads, kv, D, page, 1, device=0)
    # scores of some thousands: one token takes all, and the running maximum moves by far more than a type's range
    check_decode(m, normal((1, heads, D), g, 300.0), k, v, ks, vs, table, [150])
    # tiny queries: the mean of the values
    check_decode(m, normal((1, heads, D), g, 1e-30), k, v, ks, vs, table, [150])
    check_decode(m, torch.zeros(1, heads, D, dtype=torch.bfloat16, device=DEV), k, v, ks, vs, table, [150])
    # falling and rising scores along the sequence
    for sign in (1.0, -1.0):
        for t in range(150):
            p = int(table[0, t // page])
            k[p, t % page] = torch.full((kv, D), sign * (t - 75) / 16, device=DEV).to(k.dtype)
        check_decode(m, torch.full((1, heads, D), 1.0, dtype=torch.bfloat16, device=DEV), k, v, ks, vs, table, [150])
    m.destroy()


@pytest.mark.parametrize("eight", [False, True])
def test_decode_undefined_values_stay_in_their_row(eight):
    heads, kv, D, page = 8, 2, 128, 16
    g = gen(15)
    k, v, ks, vs = paged(30, page, kv, D, eight, "token", g)
    lengths = [150, 90, 100]
    table = tables(lengths, page, 30, 10, g)
    m = arf.ar_attn_create(heads, kv, D, page, 3, device=0)
    cache = arf.ar_kv_cache(k, v, ks, vs)
    q, lens = normal((3, heads, D), g), torch.tensor(lengths, dtype=torch.int32, device=DEV)
    before = arf.ar_attn_decode(m, cache, q, table, lens)
    q[1, 2, 5] = float("nan")                   # one query head
    k[int(table[2, 3]), 7, 1, 9] = float("nan")  # one key of the second half of the heads
    v[int(table[0, 3]), 7, 0, 9] = float("nan")  # one column of the first half
    out = arf.ar_attn_decode(m, cache, q, table, lens)
    want = torch.zeros(3, heads, D, dtype=torch.bool, device=DEV)
    want[1, 2], want[2, 4:], want[0, :4, 9] = True, True, True
    assert torch.equal(torch.isnan(out), want)
    assert torch.equal(out[~want], before[~want])
    m.destroy()


def test_decode_far_places():
    # pages whose places pass 32 bits, of bytes and of values
    heads, kv, D, page, apart = 8, 1, 128, 16, 3 * 2 ** 30
    g = gen(16)
    store = torch.empty(2 * apart + 4096, dtype=torch.bfloat16, device=DEV)
    k = store.as_strided((3, page, kv, D), (apart, D, D, 1), 0)
    v = store.as_strided((3, page, kv, D), (apart, D, D, 1), page * D)
    for x in (k, v):
        x.copy_(normal(x.shape, g))
    table = torch.tensor([[2, 0, 1], [1, 2, 0]], dtype=torch.int32, device=DEV)
    m = arf.ar_attn_create(heads, kv, D, page, 2, device=0)
    check_decode(m, normal((2, heads, D), g), k, v, None, None, table, [40, 17])
    arf.ar_attn_set_rope(m, [])
    rows = normal((2, (heads + 2 * kv) * D), g)
    arf.ar_attn_append(m, arf.ar_kv_cache(k, v), rows, None, torch.tensor([2 * page + 3, page + 5], dtype=torch.int32, device=DEV))
    assert torch.equal(k[2, 3, 0], rows[0, heads * D:(heads + 1) * D]) and torch.equal(v[1, 5, 0], rows[1, (heads + 1) * D:])
    m.destroy()


def test_decode_captured_and_replayed():
    """One captured call serves other lengths, pages and values; two graphs of two handles run side by side."""
    heads, kv, D, page, pages = 16, 2, 128, 16, 400
    g = gen(17)
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    made = []
    for i in range(2):
        k, v, _, _ = paged(pages, page, kv, D, False, "token", g)
        m = arf.ar_attn_create(heads, kv, D, page, 4, device=0, flags=arf.AR_WS_PDL if i else 0)
        q, table = normal((4, heads, D), g), torch.zeros(4, 200, dtype=torch.int32, device=DEV)
        lens = torch.zeros(4, dtype=torch.int32, device=DEV)
        out, cache = torch.empty_like(q), arf.ar_kv_cache(k, v)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side[i]):
            for _ in range(3):
                arf.ar_attn_decode(m, cache, q, table, lens, out=out)
        made.append((m, q, k, v, table, lens, out, graph))
    for lengths in ([0, 0, 0, 0], [1, 2, 3, 4], [3000, 16, 0, 1500], [1000, 1000, 1000, 1000]):
        for m, q, k, v, table, lens, out, graph in made:
            table.copy_(tables(lengths, page, pages, 200, g))
            lens.copy_(torch.tensor(lengths, dtype=torch.int32))
            q.copy_(normal(q.shape, g))
            out.fill_(99)
        torch.cuda.synchronize()
        for i, (*_, graph) in enumerate(made):
            with torch.cuda.stream(side[i]):
                graph.replay()
        torch.cuda.synchronize()
        for m, q, k, v, table, lens, out, _ in made:
            want, slack, _, _ = _attn.decode_ref(q, k, v, table, lengths, page, 0, D ** -0.5)
            assert bool(((out.double() - want).abs() <= slack).all())
    for m, *_ in made:
        m.destroy()


def test_decode_on_another_stream_and_handles_side_by_side():
    heads, kv, D, page = 8, 2, 128, 16
    g = gen(18)
    k, v, _, _ = paged(300, page, kv, D, False, "token", g)
    cache = arf.ar_kv_cache(k, v)
    lengths = [2000, 100, 900]
    table, q = tables(lengths, page, 300, 130, g), normal((3, heads, D), g)
    lens = torch.tensor(lengths, dtype=torch.int32, device=DEV)
    hs = [arf.ar_attn_create(heads, kv, D, page, 3, device=0) for _ in range(2)]
    want = arf.ar_attn_decode(hs[0], cache, q, table, lens)
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream(), torch.cuda.Stream()], [torch.empty_like(q) for _ in range(2)]
    for _ in range(20):
        for h, s, o in zip(hs, streams, outs):
            arf.ar_attn_decode(h, cache, q, table, lens, out=o, stream=s)
    torch.cuda.synchronize()
    for h, o in zip(hs, outs):
        assert torch.equal(o, want)
        h.destroy()


# -------------------------------------------------------------------- append
APPENDS = [  # heads, kv, D, rot, axes, interleaved, page, eight, layout, T, pad, far
    (8, 1, 128, 128, 1, False, 16, False, "token", 1, 0, 2 ** 17),
    (32, 8, 128, 64, 1, True, 64, True, "token", 48, 3, 1000000),
    (64, 8, 128, 128, 3, False, 16, False, "head", 300, 0, 32768),
    (4, 4, 64, 64, 2, True, 1, False, "pair", 7, 1, 50),
    (5, 5, 64, 48, 4, False, 20, True, "odd", 33, 0, 2 ** 31 - 1),
    (7, 1, 256, 256, 1, False, 16, True, "head", 5, 5, 4000),
    (2, 1, 256, 16, 1, True, 7, False, "odd", 100, 2, 10 ** 7),
    (3, 3, 128, 0, 0, False, 16, False, "token", 9, 1, 10),
    (3, 1, 128, 0, 0, False, 16, True, "token", 9, 1, 10),
    (256, 256, 64, 32, 1, False, 16, False, "token", 3, 0, 99),
    (320, 16, 128, 128, 1, False, 16, True, "token", 70, 3, 4000),
    (1024, 1024, 256, 256, 2, True, 16, False, "token", 9, 1, 99),
    (4, 2, 64, 64, 3, False, 128, False, "token", 5000, 100, 5000),
    (1, 1, 64, 64, 1, False, 16, True, "token", 1300, 0, 5000),
]


@pytest.mark.parametrize("heads,kv,D,rot,axes,interleaved,page,eight,layout,T,pad,far", APPENDS)
def test_append(heads, kv, D, rot, axes, interleaved, page, eight, layout, T, pad, far):
    g = gen(T * 7 + D)
    pages = -(-T // page) + 2
    k, v, ks, vs = paged(pages, page, kv, D, eight, layout, g)
    if eight:
        ks, vs = ks * 0.01, vs * 0.01  # (some values pass 448)
    as_codes = lambda x: x.view(torch.uint8 if eight else torch.int16).clone()  # noqa: E731
    before = as_codes(k), as_codes(v)
    qkv = normal((T, (heads + 2 * kv) * D), g)
    pos = torch.randint(0, far, (max(1, axes), T), dtype=torch.int32, device=DEV, generator=g)
    slots = torch.randperm(pages * page, device=DEV, generator=g)[:T].int()
    if pad:
        slots[T - pad:] = -1
    n = rot // 2
    freq, axis = [10000.0 ** (-i / max(1, n)) for i in range(n)], [(i * 7) % max(1, axes) for i in range(n)]
    m = arf.ar_attn_create(heads, kv, D, page, 1, device=0)
    arf.ar_attn_set_rope(m, freq, axis=axis if axes > 1 else None, interleaved=interleaved, axes=max(1, axes))
    q, ok = guarded((T, heads, D), torch.bfloat16)
    cache = arf.ar_kv_cache(k, v, ks, vs)
    arf.ar_attn_append(m, cache, qkv, pos if rot else None, slots, q=q)
    torch.cuda.synchronize()
    assert ok() and arf.ar_attn_device_error(m) == 0
    x = qkv.view(T, heads + 2 * kv, D)
    turned = x[:, :heads + kv]
    want, slack = _attn.rotated(turned, pos, freq, axis if axes > 1 else None, interleaved), _attn.rope_slack(turned, freq, interleaved)
    assert bool(((q.double() - want[:, :heads]).abs() <= want[:, :heads].abs() * _attn.HALF_BF16 + slack[:, :heads] * (1 + 2.0 ** -7)).all())
    assert torch.equal(q[..., rot:], x[:, :heads, rot:])
    rows = (slots >= 0).nonzero().flatten()
    p, o = slots[rows].long() // page, slots[rows].long() % page
    kw, kslack = want[rows, heads:], slack[rows, heads:]
    if eight:
        _attn.check_e4m3(k[p, o], kw / ks.double().view(1, -1, 1), kslack / ks.double().view(1, -1, 1), "k")
        _attn.check_e4m3(v[p, o], x[rows, heads + kv:].double() / vs.double().view(1, -1, 1), 0.0, "v")
    else:
        assert bool(((k[p, o].double() - kw).abs() <= kw.abs() * _attn.HALF_BF16 + kslack * (1 + 2.0 ** -7)).all())
        assert torch.equal(v[p, o], x[rows, heads + kv:])
    # nothing else of the cache moved
    for now, old in zip((k, v), before):
        now = as_codes(now)
        now[p, o] = old[p, o]
        assert torch.equal(now, old)
    # the same call again gives the same
    kept = q.clone(), as_codes(k), as_codes(v)
    arf.ar_attn_append(m, cache, qkv, pos if rot else None, slots, q=q)
    assert torch.equal(kept[0], q) and torch.equal(kept[1], as_codes(k)) and torch.equal(kept[2], as_codes(v))
    m.destroy()


def test_append_one_axis_takes_a_row_of_positions():
    g = gen(30)
    k, v, _, _ = paged(2, 16, 1, 64, False, "token", g)
    m = arf.ar_attn_create(2, 1, 64, 16, 1, device=0)
    arf.ar_attn_set_rope(m, [1.0] * 8)
    qkv, slots = normal((3, 256), g), torch.tensor([0, 1, 2], dtype=torch.int32, device=DEV)
    pos = torch.tensor([5, -6, 7], dtype=torch.int32, device=DEV)
    a = arf.ar_attn_append(m, arf.ar_kv_cache(k, v), qkv, pos, slots)
    b = arf.ar_attn_append(m, arf.ar_kv_cache(k, v), qkv, pos.view(1, 3), slots)
    assert torch.equal(a, b)
    want = _attn.rotated(qkv.view(3, 4, 64)[:, :2], pos.view(1, 3), [1.0] * 8, None, False)
    slack = _attn.rope_slack(qkv.view(3, 4, 64)[:, :2], [1.0] * 8, False)
    assert bool(((a.double() - want).abs() <= want.abs() * _attn.HALF_BF16 + slack * 1.01).all())
    m.destroy()


@pytest.mark.parametrize("T", [2, 40, 3000])
def test_append_the_last_token_of_a_slot_stands(T):
    heads, kv, D, page = 2, 2, 64, 16
    g = gen(31 + T)
    pages = 5
    k, v, _, _ = paged(pages, page, kv, D, False, "token", g)
    qkv = normal((T, (heads + 2 * kv) * D), g)
    slots = torch.randint(-1, pages * page, (T,), device=DEV, generator=g).int()
    if T == 2:
        slots[:] = 33
    want = {int(s): t for t, s in enumerate(slots.tolist()) if s >= 0}
    m = arf.ar_attn_create(heads, kv, D, page, 1, device=0)
    for _ in range(3):
        q = arf.ar_attn_append(m, arf.ar_kv_cache(k, v), qkv, None, slots)
        x = qkv.view(T, heads + 2 * kv, D)
        assert torch.equal(q, x[:, :heads])
        at = torch.tensor(list(want), device=DEV)
        rows = torch.tensor(list(want.values()), device=DEV)
        assert torch.equal(k.reshape(-1, kv, D)[at], x[rows, heads:heads + kv]) and torch.equal(v.reshape(-1, kv, D)[at], x[rows, heads + kv:])
    assert arf.ar_attn_device_error(m) == 0
    m.destroy()


def test_append_angles_at_the_ends_of_their_range():
    # turns a position rounded to 64 bits, as documented; times the position, less the whole turns, exactly
    from fractions import Fraction
    heads, kv, D, page = 1, 1, 64, 16
    freq = [1.0, -1.0, 3.0, -0.5, 1e-6, -1e-9, 1e4, -12345.678, math.pi, -2 * math.pi, 2 ** 40 * 1.1, 1e300, -1e-300, 0.0, 5e-324, -7.25]
    where = [0, 1, -1, 2, 7, 100, -100, 2 ** 31 - 1, -2 ** 31, -2 ** 31 + 1, 10 ** 9, -123456789]
    g = gen(61)
    k, v, _, _ = paged(2, page, kv, D, False, "token", g)
    qkv = normal((len(where), (heads + 2 * kv) * D), g)
    m = arf.ar_attn_create(heads, kv, D, page, 1, device=0)
    arf.ar_attn_set_rope(m, freq)
    q = arf.ar_attn_append(m, arf.ar_kv_cache(k, v), qkv, torch.tensor([where], dtype=torch.int32, device=DEV),
                           torch.arange(len(where), dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    frac = [[Fraction(f / 6.283185307179586476925286766559) * t % 1 for f in freq] for t in where]
    angle = 2 * math.pi * torch.tensor([[float(x) for x in row] for row in frac], dtype=torch.float64, device=DEV)
    n, c, s = len(freq), torch.cos(angle), torch.sin(angle)
    for got, x in ((q[:, 0], qkv[:, :D]), (k.view(-1, D)[:len(where)], qkv[:, D:2 * D])):
        a, b = x[:, :n].double(), x[:, n:2 * n].double()
        want = torch.cat([a * c - b * s, b * c + a * s, x[:, 2 * n:].double()], 1)
        bound = _attn.HALF_BF16 * want.abs() * (1 + 2.0 ** -8) + _attn.rope_slack(x, freq, False) + 2.0 ** -134
        assert bool(((got.double() - want).abs() <= bound).all()), float(((got.double() - want).abs() / bound).max())
    m.destroy()


def test_append_most_tokens():
    # as many as a call takes, every slot named twice, far apart, and every 9th row padded
    heads, kv, D, page, T = 2, 1, 64, 16, arf.AR_MAX_ATTN_TOKENS
    g = gen(51)
    k, v, _, _ = paged(T // 2 // page, page, kv, D, False, "token", g)
    qkv = normal((T, (heads + 2 * kv) * D), g)
    slots = torch.randperm(T // 2, generator=g, device=DEV).int().repeat(2)
    slots[::9] = -1
    k0, v0 = k.clone(), v.clone()
    m = arf.ar_attn_create(heads, kv, D, page, 1, device=0)
    q = arf.ar_attn_append(m, arf.ar_kv_cache(k, v), qkv, None, slots)
    torch.cuda.synchronize()
    x = qkv.view(T, heads + 2 * kv, D)
    assert torch.equal(q, x[:, :heads])
    wk, wv = k0.view(-1, D), v0.view(-1, D)
    for part in (slice(0, T // 2), slice(T // 2, T)):  # (within a half no slot comes twice)
        s = slots[part].long()
        wk[s[s >= 0]], wv[s[s >= 0]] = x[part, heads][s >= 0], x[part, heads + kv][s >= 0]
    assert torch.equal(k.view(-1, D), wk) and torch.equal(v.view(-1, D), wv)
    assert arf.ar_attn_device_error(m) == 0
    with pytest.raises(arf.ArfuseError) as e:
        arf.ar_attn_append(m, arf.ar_kv_cache(k, v), normal((T + 1, qkv.shape[1]), g), None, torch.zeros(T + 1, dtype=torch.int32, device=DEV))
    assert e.value.status == arf.AR_ERR_CAPACITY
    m.destroy()


def test_append_bad_slots():
    heads, kv, D, page, pages = 2, 1, 64, 16, 3
    g = gen(32)
    k, v, _, _ = paged(pages, page, kv, D, False, "token", g)
    before = k.clone(), v.clone()
    m = arf.ar_attn_create(heads, kv, D, page, 1, device=0)
    qkv = normal((5, (heads + 2 * kv) * D), g)
    slots = torch.tensor([pages * page, -2, 2 ** 31 - 1, -(2 ** 31), -1], dtype=torch.int32, device=DEV)
    q = arf.ar_attn_append(m, arf.ar_kv_cache(k, v), qkv, None, slots)
    assert torch.equal(k, before[0]) and torch.equal(v, before[1])
    assert torch.equal(q, qkv.view(5, 4, D)[:, :2])
    assert arf.ar_attn_device_error(m) == arf.AR_DEVERR_SLOT_RANGE
    m.destroy()


def test_append_undefined_and_large_values_in_8_bits():
    m = arf.ar_attn_create(1, 1, 64, 4, 1, device=0)
    k, v, _, _ = paged(1, 4, 1, 64, True, "token", gen(33))
    one = torch.ones(1, device=DEV)
    qkv = torch.zeros(1, 3 * 64, dtype=torch.bfloat16, device=DEV)
    vals = [float("nan"), float("inf"), -float("inf"), 460.0, -1e30, 448.0, 2.0 ** -9, 2.0 ** -10, 2.0 ** -11, 0.0, -0.0, 17.0, 19.0]
    qkv[0, 128:128 + len(vals)] = torch.tensor(vals).bfloat16()
    arf.ar_attn_append(m, arf.ar_kv_cache(k, v, one, one), qkv, None, torch.tensor([2], dtype=torch.int32, device=DEV))
    got = v[0, 2, 0].float()[:len(vals)].tolist()
    # halves between two codes go to the even one
    assert got[0] != got[0] and got[1:] == [448.0, -448.0, 448.0, -448.0, 448.0, 2.0 ** -9, 0.0, 0.0, 0.0, 0.0, 16.0, 20.0]
    m.destroy()


def test_append_scales_at_the_ends_of_their_range():
    # powers of two: every quotient is exact
    m = arf.ar_attn_create(3, 3, 64, 4, 1, device=0)
    for scales in ([2.0 ** -133, 2.0 ** -126, 2.0 ** -127], [2.0 ** 127, 2.0 ** 100, 1.0], [-2.0 ** -140, -4.0, 2.0 ** -149]):
        k, v, _, _ = paged(1, 4, 3, 64, True, "token", gen(34))
        s = torch.tensor(scales, device=DEV)
        codes = torch.tensor([1.0, -8.0, 448.0, 0.0, 2.0 ** -6, 2.0 ** -9, -0.4375, 13.0], device=DEV)
        values = (codes.double() * s.double().unsqueeze(1)).float().bfloat16()  # (small ones may become 0)
        qkv = torch.zeros(1, 9, 64, dtype=torch.bfloat16, device=DEV)
        qkv[0, 3:6, :8], qkv[0, 6:, 56:] = values, values
        arf.ar_attn_append(m, arf.ar_kv_cache(k, v, s, s), qkv.view(1, -1), None, torch.tensor([1], dtype=torch.int32, device=DEV))
        want = (values.double() / s.double().unsqueeze(1)).clamp(-448, 448).float().to(F8).float()
        assert torch.equal(k[0, 1, :, :8].float(), want) and torch.equal(v[0, 1, :, 56:].float(), want), scales
    m.destroy()
