"""Every token of long, ragged and windowed sequences is looked at once (needs a GB300)."""
import math

import pytest
import torch

import tp_reduce_moe_gb300 as arf
from tests import _attn_count as count
from tests.test_gpu_attn import DEV, gen, paged, tables

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from tp_reduce_moe_gb300 import build
    build.build()
    arf.load_library()
    torch.cuda.set_device(0)


CASES = [  # heads, kv, D, page, eight, window, lengths, columns of the table at least
    (2, 1, 128, 16, False, 0, [60001], 0),
    (2, 1, 64, 16, True, 0, [70001, 20000], 0),
    (3, 1, 256, 16, False, 0, [30001], 0),
    (2, 1, 256, 64, True, 0, [33000, 5], 0),
    (12, 1, 128, 16, False, 0, [40000, 10, 777], 8000),
    (16, 1, 64, 20, True, 0, [40000, 0, 3001], 20000),
    (20, 1, 128, 16, False, 0, [9000, 1234], 0),
    (4, 2, 64, 1, False, 0, [20001, 65, 3], 0),          # pages of one token: an entry of the table each
    (4, 2, 128, 3, False, 0, [30001, 100], 0),
    (4, 1, 128, 3, True, 0, [30001, 100], 0),
    (4, 1, 256, 1, False, 0, [9001], 0),
    (2, 2, 64, 16, False, 5000, [40000, 10, 5001], 0),
    (8, 8, 64, 7, True, 1000, [(b * 613) % 9000 for b in range(40)], 0),
    (8, 2, 128, 16, False, 0, [(b * 377) % 3000 for b in range(64)], 0),
    (32, 2, 128, 16, False, 0, [(b * 377) % 3000 for b in range(64)], 9000),
    (16, 4, 256, 32, False, 0, [(b * 577) % 2000 for b in range(33)], 0),
    (4, 2, 64, 5, False, 0, [(b * 37) % 90 for b in range(700)], 0),
]


@pytest.mark.parametrize("spread", [0, 8])
@pytest.mark.parametrize("heads,kv,D,page,eight,window,lengths,width", CASES)
def test_each_token_counts_once(heads, kv, D, page, eight, window, lengths, width, spread):
    g = gen(len(lengths) + D)
    B, need = len(lengths), [-(-n // page) for n in lengths]
    k, v, ks, vs = paged(sum(need) + 1, page, kv, D, eight, "token", g, fill=0.0)
    if eight:
        ks, vs = torch.ones_like(ks), torch.ones_like(vs)
    table = tables(lengths, page, sum(need) + 1, max(max(need) + 1, width), g)
    # places of all tokens, and which of their sequence they are
    where, which = [], []
    for b, n in enumerate(lengths):
        t = torch.arange(n, device=DEV)
        where.append(table[b, t // page].long() * page + t % page)
        which.append(t)
    where, which = torch.cat(where), torch.cat(which)
    levels = count.level(which, spread)
    kind = torch.uint8 if eight else torch.int16
    as_kind = lambda x: x.to(k.dtype).view(kind)  # noqa: E731
    kk, vv = k.view(kind).view(-1, kv, D), v.view(kind).view(-1, kv, D)
    kk[where, :, 0] = as_kind(levels.float()).unsqueeze(1)
    q = torch.zeros(B, heads, D, dtype=torch.bfloat16, device=DEV)
    q[..., 0] = 1.0
    lens = torch.tensor(lengths, dtype=torch.int32, device=DEV)
    m = arf.ar_attn_create(heads, kv, D, page, B, device=0)
    cache = arf.ar_kv_cache(k, v, ks, vs)
    G = heads // kv
    for at in range(0, max(lengths), count.chunk(D)):
        vv.zero_()
        now = (which >= at) & (which < at + count.chunk(D))
        t, value = which[now], as_kind(torch.pow(2.0, -levels[now].float()))
        for h in range(kv):
            vv[where[now], h, count.column(t, h, D)] = value
        lse = torch.empty(B, heads, device=DEV)
        out, _ = arf.ar_attn_decode(m, cache, q, table, lens, scale=math.log(2.0), window=window, lse=lse)
        out, lse = out.double().cpu(), lse.double().cpu()
        for b, n in enumerate(lengths):
            for h in range(kv):
                want, total = count.counts(n, window, at, h, D, spread)
                rows = slice(h * G, (h + 1) * G)
                if n == 0:
                    assert bool((out[b] == 0).all()) and bool((lse[b] == -math.inf).all())
                    continue
                off = (out[b, rows] - want).abs()
                assert bool((off <= count.bound(want)).all()), (b, n, h, at, float((off / count.bound(want)).max()))
                # without levels the sums are whole numbers (2^7 times them over 8 bits) that are held exactly: what is left are a
                # logarithm's 2^-22 of it and three roundings of 2^-24, less than a token of 70001 would be; with them weights and sums
                # are off by the bound's 2^-12
                ln = math.log(total)
                lost = 2.0 ** -22 * (1.75 * (ln + 5) + 1) if spread == 0 else 2.0 ** -12
                assert bool(((lse[b, rows] - ln).abs() <= lost).all()), (b, n, h)
    assert arf.ar_attn_device_error(m) == 0
    m.destroy()
