"""The norm with an 8-bit output where h times its weight passes fp32's range and the normalised value does not (needs a GB300)."""
import pytest
import torch

import tp_reduce_moe_gb300 as arf
from tests.test_gpu_attn import DEV, gen, normal
from tests.test_gpu_norm_q8 import check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from tp_reduce_moe_gb300 import build
    build.build()
    arf.load_library()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("T,H", [(3, 520), (3, 8200), (400, 1024), (400, 4104)])
@pytest.mark.parametrize("group", [0, 32, 128])
def test_large_rows_with_large_weights(T, H, group):
    g = gen(90 + T)
    R = 2
    partials, residual = [normal((T, H), g) for _ in range(R)], normal((T, H), g)
    for x in (*partials, residual):
        x[1::3] *= 1e16   # (sums of squares up to 1e37)
        x[2::3] *= 1e-3
    gamma = normal((H,), g, 1e30)
    ws = arf.ar_workspace_create(R, 0, H, T, 1e-6, device=0)
    out = torch.empty_like(residual)
    q, scales, h = arf.ar_rmsnorm_q8(ws, partials, residual, gamma, 0.0, 1e-6, group=group, out=out)
    check(partials, residual, gamma, 0.0, 1e-6, group, q, scales, h, out)
    want, _ = arf.ar_rmsnorm(ws, partials, residual, gamma, 0.0, 1e-6)
    assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(want).all())
    ws.destroy()


@pytest.mark.parametrize("T", [3, 400])
def test_an_infinity_of_a_row_is_nan_beside_zeros(T):
    g = gen(95)
    H = 1032
    p, residual, gamma = torch.zeros(T, H, dtype=torch.bfloat16, device=DEV), normal((T, H), g), normal((H,), g, 1e30)
    residual[1, 700] = float("inf")
    ws = arf.ar_workspace_create(1, 0, H, T, 1e-6, device=0)
    q, scales, _ = arf.ar_rmsnorm_q8(ws, [p], residual, gamma, 0.0, 1e-6, group=0)
    assert torch.equal(torch.isnan(scales[:, 0]), torch.arange(T, device=DEV) == 1)
    assert bool(torch.isnan(q[1].float()).all()) and not bool(torch.isnan(q[0].float()).any())
    ws.destroy()


def test_a_workspace_sets_up_what_its_calls_launch():
    # creating one does nothing for this norm's kernels; the first call that launches one of those that stay does, once
    from torch.profiler import ProfilerActivity, profile

    def calls(fn):
        with profile(activities=[ProfilerActivity.CPU, ProfilerActivity.CUDA]) as prof:
            fn()
            torch.cuda.synchronize()
        return [e.name for e in prof.events()]

    g = gen(96)
    T, H = 400, 1024
    p, residual, gamma = normal((T, H), g), normal((T, H), g), normal((H,), g)
    x = torch.ones(1024, device=DEV)
    if not any("cudaLaunchKernel" in calls(lambda: x.mul_(1.0)) for _ in range(3)):
        pytest.skip("the profiler records no calls of the runtime on this machine")
    ws = arf.ar_workspace_create(1, 0, H, T, 1e-6, device=0)

    def norm(rows, group):
        arf.ar_rmsnorm_q8(ws, [p[:rows]], residual[:rows], gamma, 0.0, 1e-6, group=group)

    for rows, group, told in ((3, 32, 0), (T, 32, 1), (T, 32, 0), (T, 128, 1), (T, 0, 1), (T, 128, 0), (3, 0, 0)):
        names = calls(lambda: norm(rows, group))
        assert sum(n.startswith("cudaLaunchKernel") for n in names) == 1
        assert names.count("cudaFuncSetAttribute") == told, (rows, group)
    ws.destroy()
