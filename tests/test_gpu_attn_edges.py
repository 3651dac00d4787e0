"""Calls of the attention of a decode layer at the ends of what its description allows (needs a GB300)."""
import pytest
import torch

import tp_reduce_moe_gb300 as arf
from tests import _attn
from tests.test_gpu_attn import DEV, check_decode, gen, normal, paged

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _built():
    from tp_reduce_moe_gb300 import build
    build.build()
    arf.load_library()
    torch.cuda.set_device(0)


# ---------------------------------------------------------------- rotary positions set again behind captured calls
ROPES = [  # frequencies, axes of the pairs, pairing, axes
    ([1.0, 0.5, 0.25, 0.125] * 4, None, False, 1),
    ([0.3, 0.2, 0.1, 0.05] * 8, [0, 1, 2, 3] * 8, True, 4),    # other columns, pairing and axes
    ([0.7, 0.01, 3.0, 0.125] * 4, None, False, 1),             # other frequencies alone
    ([], None, False, 1),                                      # none
]


def test_captured_append_keeps_the_rotary_positions_it_was_made_with():
    heads, kv, D, page, T = 4, 2, 64, 16, 9
    g = gen(70)
    qkv = normal((T, (heads + 2 * kv) * D), g)
    slots = torch.arange(T, dtype=torch.int32, device=DEV)
    x = qkv.view(T, heads + 2 * kv, D)[:, :heads + kv]
    m = arf.ar_attn_create(heads, kv, D, page, 1, device=0)
    made = []

    def check(q, k, pos, rope):
        freq, axis, near, _ = rope
        want, slack = _attn.rotated(x, pos, freq, axis, near), _attn.rope_slack(x, freq, near)
        for got, ref, lost in ((q, want[:, :heads], slack[:, :heads]), (k[0, :T], want[:, heads:], slack[:, heads:])):
            assert bool(((got.double() - ref).abs() <= ref.abs() * _attn.HALF_BF16 + lost * (1 + 2.0 ** -7)).all())

    for rope in ROPES:  # a graph of each, one after the other on one handle
        freq, axis, near, axes = rope
        k, v, _, _ = paged(1, page, kv, D, False, "token", g)
        cache, q = arf.ar_kv_cache(k, v), torch.zeros(T, heads, D, dtype=torch.bfloat16, device=DEV)
        pos = torch.zeros(axes, T, dtype=torch.int32, device=DEV)
        arf.ar_attn_set_rope(m, freq, axis=axis, interleaved=near, axes=axes)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            arf.ar_attn_append(m, cache, qkv, pos, slots, q=q)
        made.append((graph, cache, q, k, pos, rope))
    for now in ROPES:  # whatever is in force, each replays its own
        freq, axis, near, axes = now
        arf.ar_attn_set_rope(m, freq, axis=axis, interleaved=near, axes=axes)
        for graph, _, q, k, pos, rope in made:
            pos.copy_(torch.randint(-1000, 1000, pos.shape, dtype=torch.int32, device=DEV, generator=g))
            q.fill_(99), k.fill_(99)
            graph.replay()
            torch.cuda.synchronize()
            check(q, k, pos, rope)
        # and calls that are made now take what is in force
        pos = torch.randint(-1000, 1000, (axes, T), dtype=torch.int32, device=DEV, generator=g)
        k, v, _, _ = paged(1, page, kv, D, False, "token", g)
        check(arf.ar_attn_append(m, arf.ar_kv_cache(k, v), qkv, pos, slots), k, pos, now)
    assert arf.ar_attn_device_error(m) == 0
    m.destroy()


def test_calls_in_flight_keep_their_rotary_positions():
    # set again right behind each call, with no wait between; more tables than the handle makes room for at once, and some again
    heads, kv, D, page, T = 2, 1, 128, 16, 16
    g = gen(71)
    qkv, slots = normal((T, (heads + 2 * kv) * D), g), torch.arange(T, dtype=torch.int32, device=DEV)
    k, v, _, _ = paged(1, page, kv, D, False, "token", g)
    cache, m = arf.ar_kv_cache(k, v), arf.ar_attn_create(heads, kv, D, page, 1, device=0)
    pos = torch.randint(0, 500, (1, T), dtype=torch.int32, device=DEV, generator=g)
    ropes = [[0.01 * (i % 100) + 0.001 * j for j in range(64)] for i in range(150)]
    outs = []
    torch.cuda.synchronize()
    for freq in ropes:
        arf.ar_attn_set_rope(m, freq)
        outs.append(arf.ar_attn_append(m, cache, qkv, pos, slots))
    torch.cuda.synchronize()
    x = qkv.view(T, heads + 2 * kv, D)[:, :heads]
    for freq, q in zip(ropes, outs):
        want, slack = _attn.rotated(x, pos, freq, None, False), _attn.rope_slack(x, freq, False)
        assert bool(((q.double() - want).abs() <= want.abs() * _attn.HALF_BF16 + slack * (1 + 2.0 ** -7)).all())
    m.destroy()


# ---------------------------------------------------------------- query rows of values far apart, over an 8-bit cache
@pytest.mark.parametrize("D,heads", [(64, 4), (128, 8), (128, 16), (256, 3)])
@pytest.mark.parametrize("far", [2.0 ** 10, 2.0 ** 20, 2.0 ** 27])
def test_decode_small_columns_beside_a_large_one(D, heads, far):
    # the large column meets keys of zero (or tiny ones): the scores are those of the others
    page, lengths = 16, [150, 33]
    g = gen(80 + D)
    k, v, ks, vs = paged(20, page, 1, D, True, "token", g)
    bits = k.view(torch.uint8)
    bits[..., 5] = 0
    bits[..., 40] = torch.tensor([2.0 ** -9], device=DEV).to(F8).view(torch.uint8)
    q = normal((2, heads, D), g, 2.0)
    q[..., 5] = far
    q[0, 0, 40] = -far
    table = torch.randperm(20, generator=g, device=DEV).int()[:20].view(2, 10)
    m = arf.ar_attn_create(heads, 1, D, page, 2, device=0)
    want, slack, want_lse, lse_slack = _attn.decode_ref(q, k, v, table, lengths, page, 0, D ** -0.5, ks, vs, True)
    # Queries come to halves whose largest is 2^15 at least, so they are multiples of 2^-24 there: off by 2^-25 at most, 2^-40 of
    # the largest.  A score is off by that times the sum of its key's magnitudes; weights and their sum by so much each.
    off = 2.0 ** -40 * far * float(k.float().abs().sum(-1).max() * ks) * D ** -0.5
    slack += 2 * off * 1.01 * float(v.float().abs().max() * vs)
    lse_slack += off
    out, lse = arf.ar_attn_decode(m, arf.ar_kv_cache(k, v, ks, vs), q, table, torch.tensor(lengths, dtype=torch.int32, device=DEV),
                                  lse=torch.empty(2, heads, device=DEV))
    assert bool(((out.double() - want).abs() <= slack).all()), f"out: {float(((out.double() - want).abs() / slack).max())} of the bound"
    assert bool(((lse.double() - want_lse).abs() <= lse_slack).all())
    m.destroy()


@pytest.mark.parametrize("size,scale", [(2.0 ** 126, 2.0 ** -127), (2.0 ** 127, 2.0 ** -126), (2.0 ** -126, 2.0 ** 120), (2.0 ** -133, 2.0 ** 126), (2.0 ** -100, 2.0 ** 97)])
def test_decode_queries_at_the_ends_of_their_range(size, scale):
    # (the scale brings the scores back; keys and queries of few bits, so that no product passes the range on its way)
    heads, D, page, n = 4, 64, 16, 90
    g = gen(81)
    k, v, ks, vs = paged(6, page, 1, D, True, "token", g)
    k.view(torch.uint8).copy_((torch.randint(-2, 3, k.shape, generator=g, device=DEV) / 4).to(F8).view(torch.uint8))
    q = (torch.randint(0, 2, (1, heads, D), generator=g, device=DEV) * size).bfloat16()
    table = torch.arange(6, dtype=torch.int32, device=DEV).view(1, 6)
    m = arf.ar_attn_create(heads, 1, D, page, 1, device=0)
    check_decode(m, q, k, v, torch.ones_like(ks), vs, table, [n], scale=scale)
    m.destroy()


# ---------------------------------------------------------------- infinities among the values
@pytest.mark.parametrize("heads,D,n", [(8, 128, 150), (12, 64, 3000), (4, 256, 700)])
def test_decode_infinite_values_stay_in_their_column(heads, D, n):
    kv, page, lengths = 2, 16, [n, 90]
    g = gen(85 + D)
    pages = -(-n // page) + 7
    k, v, _, _ = paged(pages, page, kv, D, False, "token", g)
    order = torch.randperm(pages, generator=g, device=DEV).int()
    table = torch.full((2, pages), -1, dtype=torch.int32, device=DEV)
    table[0, :-(-n // page)], table[1, :6] = order[:-(-n // page)], order[-6:]
    m = arf.ar_attn_create(heads, kv, D, page, 2, device=0)
    cache, lens = arf.ar_kv_cache(k, v), torch.tensor(lengths, dtype=torch.int32, device=DEV)
    for size in (0.0, 1.0):  # equal weights, whose second parts are zero; others
        q = normal((2, heads, D), g, size)
        lse, lse0 = torch.empty(2, heads, device=DEV), torch.empty(2, heads, device=DEV)
        kept = v.clone()
        before, _ = arf.ar_attn_decode(m, cache, q, table, lens, lse=lse0)
        v[int(table[0, 3]), 7, 0, 9] = float("inf")
        v[int(table[0, 0]), 0, 1, 33] = -float("inf")
        v[int(table[1, 5]), 9, 1, 0] = float("inf")   # the last token of its sequence
        v[int(table[1, 5]), 10, 0, 5] = float("inf")  # behind it
        out, _ = arf.ar_attn_decode(m, cache, q, table, lens, lse=lse)
        hit, G = torch.zeros_like(out, dtype=torch.bool), heads // kv
        hit[0, :G, 9], hit[0, G:, 33], hit[1, G:, 0] = True, True, True
        assert torch.equal(~torch.isfinite(out), hit)
        assert torch.equal(out[~hit], before[~hit]) and torch.equal(lse, lse0)
        v.copy_(kept)
    m.destroy()
