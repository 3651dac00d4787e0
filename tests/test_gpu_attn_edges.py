"""Calls of the attention of a decode layer at the ends of what its description allows (needs a GB300)."""
import pytest
import torch

import tp_reduce_moe_gb300 as arf
from tests import _attn
from tests.test_gpu_attn import DEV, gen, normal, paged

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
