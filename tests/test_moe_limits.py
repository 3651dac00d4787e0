"""Controls of the few-token MoE handle, on the host (no GPU needed)."""
import pytest

import tp_reduce_moe_gb300 as arf


@pytest.fixture(scope="module")
def lib():
    from tp_reduce_moe_gb300 import build
    build.build()
    return arf.load_library()


def test_wait_timeout_injection_setter(lib):
    m = arf.ar_moe_create(8, 2, 256, 128, 16, flags=arf.AR_WS_DRY_RUN)
    for product in (1, 2):
        for limit in (50_000, 1_000_000_000, 0):
            arf.ar_moe_inject_wait_timeout(m, product, limit)
        for bad in (-1, 1_000_000_001):
            with pytest.raises(arf.ArfuseError) as e:
                arf.ar_moe_inject_wait_timeout(m, product, bad)
            assert e.value.status == arf.AR_ERR_INVALID_ARG
    for product in (-1, 0, 3):
        with pytest.raises(arf.ArfuseError):
            arf.ar_moe_inject_wait_timeout(m, product, 50_000)
    m.destroy()
    assert lib.ar_moe_inject_wait_timeout(None, 1, 1) == arf.AR_ERR_INVALID_ARG


def test_scoring_functions_and_the_groups_rule(lib):
    m = arf.ar_moe_create(8, 2, 256, 0, 16, flags=arf.AR_WS_DRY_RUN)
    base = 1 << 40
    call = lambda scoring, groups: lib.ar_moe_route(m.handle, base, base + (1 << 28), None, scoring, 1, 1.0, groups, 1, 4, base + (2 << 28),
                                                    base + (3 << 28), None)
    for function in (arf.AR_MOE_SOFTMAX, arf.AR_MOE_SIGMOID):
        for groups in (1, 4):
            assert call(function, groups) == call(function | arf.AR_MOE_GROUP_MAX, groups) == arf.AR_VALIDATED
    for bad in (2, 0x11 + 1, 0x20, 0x30, -1, 0x10 | 0x100):
        assert call(bad, 4) == arf.AR_ERR_INVALID_ARG
    m.destroy()
