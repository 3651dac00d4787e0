"""What the attention of one new token says of tensors that it does not take (CPU)."""
import pytest
import torch

import tp_reduce_moe_gb300 as arf

HEADS, KV, D, PAGE, B = 4, 2, 64, 16, 2


@pytest.fixture()
def call():
    from tp_reduce_moe_gb300 import build
    build.build()
    m = arf.ar_attn_create(HEADS, KV, D, PAGE, 4, flags=arf.AR_WS_DRY_RUN)
    cache = arf.ar_kv_cache(new(3, PAGE, KV, D), new(3, PAGE, KV, D))
    ints = new(B, dtype=torch.int32)
    yield lambda q, table, **kw: arf.ar_attn_decode(m, cache, q, table, ints, **kw)
    m.destroy()


def new(*s, dtype=torch.bfloat16):
    return torch.zeros(s, dtype=dtype)


def test_tensors_without_a_place_are_not_called_badly_laid_out(call):
    q, table, out = new(B, HEADS, D), new(B, 3, dtype=torch.int32), new(B, HEADS, D)
    with pytest.raises(TypeError, match="plain strided tensors"):
        torch.func.vmap(lambda x: call(x, table, out=out))(new(5, B, HEADS, D))
    with pytest.raises(TypeError, match="plain strided tensors"):
        torch.func.vmap(lambda x: call(q, x, out=out))(new(5, B, 3, dtype=torch.int32))
    with pytest.raises(TypeError, match="plain strided tensors"):
        call(q, table.to_sparse())


def test_page_tables_that_are_badly_laid_out_are_told_so(call):
    q = new(B, HEADS, D)
    for table in (new(B, 6, dtype=torch.int32)[:, ::2], new(3, B, dtype=torch.int32).t(), new(1, 3, dtype=torch.int32).expand(B, 3),
                  new(8, dtype=torch.int32).as_strided((B, 3), (2, 1))):
        with pytest.raises(ValueError, match="entries of a row must be contiguous"):
            call(q, table)
    for table in (new(B, 0, dtype=torch.int32), new(B, 1, dtype=torch.int32), new(B, 9, dtype=torch.int32)[:, 2:5],
                  new(1, 4, dtype=torch.int32).t()[:B].contiguous()):
        assert call(q, table).shape == q.shape
