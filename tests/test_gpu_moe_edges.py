"""The few-token MoE layer at its edges: memory that copies and ordinary accesses share, waits that run out, choices that
only exact sums decide (needs a GB300)."""
import math

import pytest
import torch

import tp_reduce_moe_gb300 as arf
from tests import _moe
from tests.test_gpu_moe import DEV, Layer, check, choice, gen, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from tp_reduce_moe_gb300 import build
    build.build()
    arf.load_library()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("group", [0, 32, 128])
@pytest.mark.parametrize("T", [2, 5, 12, 64])
def test_first_copies_land_behind_the_masks(T, group):
    """With 512 experts the masks fill the first warp's first slot: every call gives the same bits, and the right ones."""
    E, K, H, I = 512, 4, 512, 128
    g = gen(T + group)
    layer = Layer(E, H, I, group, g)
    m = arf.ar_moe_create(E, K, H, I, T, device=0)
    x = normal((T, H), g)
    ids, w = choice(T, E, K, g)
    outs = [torch.empty(T, H, dtype=torch.bfloat16, device=DEV) for _ in range(40)]
    for out in outs:
        layer.run(m, x, ids, w, out=out)
    torch.cuda.synchronize()
    y, bound = _moe.experts_ref(x, ids, w, layer.w13, layer.w2)
    _moe.close(outs[0], y, bound, "behind the masks")
    assert all(torch.equal(out, outs[0]) for out in outs)
    assert arf.ar_moe_device_error(m) == 0
    m.destroy()


# The ways through the products: whole rows of few tokens staged, rows in pieces, items one after the other, activations of
# the second product staged or loaded, scales by tensor copies and in pieces, jobs of several rounds, one tile in all.
LOST = [  # T, H, E, K, I, group
    (1, 264, 4, 2, 72, 0), (9, 1024, 24, 3, 264, 0), (64, 256, 64, 4, 1024, 0), (1, 7168, 12, 8, 256, 128),
    (8, 16384, 4, 2, 64, 32), (12, 4096, 64, 4, 64, 32), (40, 256, 16, 8, 1024, 64), (7, 768, 6, 3, 256, 64),
    (64, 896, 40, 8, 128, 128), (1, 32, 1, 1, 32, 32),
]


@pytest.mark.parametrize("T,H,E,K,I,group", LOST)
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_clean(T, H, E, K, I, group):
    g = gen(T + H + I)
    layer = Layer(E, H, I, group, g)
    m = arf.ar_moe_create(E, K, H, I, T, device=0)
    x = normal((T, H), g)
    ids, w = choice(T, E, K, g)
    if T > 1:
        ids[T - 1] = -1  # a padded row
    right = layer.run(m, x, ids, w)
    assert arf.ar_moe_device_error(m) == 0
    for limits in ((50_000, 0), (0, 50_000), (50_000, 50_000)):
        for i in (0, 1):
            arf.ar_moe_inject_wait_timeout(m, i + 1, limits[i])
        out = layer.run(m, x, ids, w)
        assert arf.ar_moe_device_error(m) == arf.AR_DEVERR_TIMEOUT  # (synchronises: the kernels have returned)
        used = T - 1 if limits[1] == 0 and T > 1 else T
        assert bool(torch.isnan(out[:used]).all())
        assert bool((out[used:] == 0).all())
        for i in (0, 1):
            arf.ar_moe_inject_wait_timeout(m, i + 1, 0)
        assert torch.equal(layer.run(m, x, ids, w), right)
        assert arf.ar_moe_device_error(m) == 0
    m.destroy()


@pytest.mark.parametrize("T,H,E,K,I,group", [(16, 7168, 32, 8, 256, 64), (16, 7168, 32, 8, 256, 128), (14, 7168, 32, 8, 256, 32), (6, 4096, 16, 5, 1024, 128)])
def test_second_product_with_one_tile_a_round(T, H, E, K, I, group):
    """Staged activations that leave the sums of one tile room, not those of all."""
    g = gen(T + H + I + group)
    layer = Layer(E, H, I, group, g)
    m = arf.ar_moe_create(E, K, H, I, T, device=0)
    check(m, layer, normal((T, H), g), *choice(T, E, K, g), "one tile a round")
    m.destroy()
