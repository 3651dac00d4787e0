"""The few-token MoE layer at its edges: memory that copies and ordinary accesses share, waits that run out, choices that
only exact sums decide (needs a GB300)."""
import math

import pytest
import torch

import tp_reduce_moe_gb300 as arf
from tests import _moe
from tests.test_gpu_moe import DEV, Layer, choice, gen, normal

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
