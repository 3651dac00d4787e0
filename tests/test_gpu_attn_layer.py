"""The attention half of a decode layer as it is used: norm, 4-bit q/k/v projection, rotary positions into the cache, attention,
4-bit output projection, the boundary norm; step after step, eager and as one captured graph (needs a GB300)."""
import pytest
import torch

import tp_reduce_moe_gb300 as arf
from tests import _attn, _moe
from tests.test_gpu_attn import DEV, gen, normal, paged

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn
B, H, HEADS, KV, D, PAGE, PAGES, WIDTH, GROUP, EPS = 5, 1024, 8, 2, 64, 16, 40, 8, 64, 1e-6


@pytest.fixture(scope="module", autouse=True)
def _built():
    from tp_reduce_moe_gb300 import build
    build.build()
    arf.load_library()
    torch.cuda.set_device(0)


class Layer:
    def __init__(self, eight, g):
        cpu = torch.Generator().manual_seed(1)
        cols = (HEADS + 2 * KV) * D
        self.qkv = _moe.make_w4((cols,), H, GROUP, cpu, DEV)
        self.o = _moe.make_w4((H,), HEADS * D, GROUP, cpu, DEV)
        self.gamma = [(torch.rand(H, device=DEV, generator=g) + 0.5).bfloat16() for _ in range(2)]
        self.k, self.v, self.ks, self.vs = paged(PAGES, PAGE, KV, D, eight, "token", g)
        if eight:
            self.ks, self.vs = self.ks * 0.05, self.vs * 0.05
        self.cache = arf.ar_kv_cache(self.k, self.v, self.ks, self.vs)
        self.ws = arf.ar_workspace_create(1, 0, H, B, EPS, device=0, flags=arf.AR_WS_PDL)
        self.attn = arf.ar_attn_create(HEADS, KV, D, PAGE, B, device=0, flags=arf.AR_WS_PDL)
        self.freq = [10000.0 ** (-i / 16) for i in range(16)]
        arf.ar_attn_set_rope(self.attn, self.freq)
        new = lambda *s, dtype=torch.bfloat16: torch.empty(s, dtype=dtype, device=DEV)  # noqa: E731
        # what a step reads and leaves
        self.partial, self.residual = normal((B, H), g), normal((B, H), g)
        self.pos, self.slots, self.lengths = (torch.zeros(B, dtype=torch.int32, device=DEV) for _ in range(3))
        self.table = torch.full((B, WIDTH), -1, dtype=torch.int32, device=DEV)
        self.x8, self.scales, self.x, self.h = new(B, H, dtype=F8), new(B, H // 128, dtype=torch.float32), new(B, H), new(B, H)
        self.rows, self.q, self.mixed = new(B, cols), new(B, HEADS, D), new(B, HEADS, D)
        self.lse, self.out, self.h2, self.y = new(B, HEADS, dtype=torch.float32), new(B, H), new(B, H), new(B, H)

    def step(self):
        arf.ar_rmsnorm_q8(self.ws, [self.partial], self.residual, self.gamma[0], 0.0, EPS, q=self.x8, scales=self.scales,
                          residual_out=self.h, out=self.x)
        arf.ar_matvec_w4(self.x, *self.qkv, GROUP, out=self.rows)
        arf.ar_attn_append(self.attn, self.cache, self.rows, self.pos.view(1, B), self.slots, q=self.q)
        arf.ar_attn_decode(self.attn, self.cache, self.q, self.table, self.lengths, out=self.mixed, lse=self.lse)
        arf.ar_matvec_w4(self.mixed.view(B, HEADS * D), *self.o, GROUP, out=self.out)
        arf.ar_rmsnorm(self.ws, [self.out], self.h, self.gamma[1], 0.0, EPS, out=self.y, residual_out=self.h2)

    def check(self, before):
        """Each operator's result from what it was given."""
        y, scale, h = _attn.norm_q8_ref([self.partial], self.residual, self.gamma[0], 0.0, EPS, 128)
        assert bool(((self.x.double() - y).abs() <= y.abs() * (_attn.HALF_BF16 + 2.0 ** -18)).all())
        spread = self.scales.double().repeat_interleave(128, dim=1)
        _attn.check_e4m3(self.x8, y / spread, (y / spread).abs() * 2.0 ** -18, "x8")
        W = _moe.w4_values(*self.qkv)
        rows = self.x.double() @ W.t()
        lost = _moe.gamma(H) * (self.x.double().abs() @ W.abs().t())
        assert bool(((self.rows.double() - rows).abs() <= rows.abs() * _attn.HALF_BF16 + lost).all())
        heads = self.rows.view(B, HEADS + 2 * KV, D)
        want = _attn.rotated(heads[:, :HEADS + KV], self.pos.view(1, B), self.freq, None, False)
        slack = _attn.rope_slack(heads[:, :HEADS + KV], self.freq, False)
        assert bool(((self.q.double() - want[:, :HEADS]).abs() <= want[:, :HEADS].abs() * _attn.HALF_BF16 + slack[:, :HEADS] * 1.01).all())
        there = self.slots >= 0
        p, o = self.slots[there].long() // PAGE, self.slots[there].long() % PAGE
        k, v = before[0].clone(), before[1].clone()
        kind = torch.uint8 if self.ks is not None else torch.int16
        k.view(kind)[p, o], v.view(kind)[p, o] = self.k.view(kind)[p, o], self.v.view(kind)[p, o]
        assert torch.equal(k.view(kind), self.k.view(kind)) and torch.equal(v.view(kind), self.v.view(kind))
        if self.ks is None:
            assert torch.equal(self.v[p, o], heads[there, HEADS + KV:])
            kw = want[there, HEADS:]
            assert bool(((self.k[p, o].double() - kw).abs() <= kw.abs() * _attn.HALF_BF16 + slack[there, HEADS:] * 1.01).all())
        else:
            ks, vs = self.ks.double().view(1, KV, 1), self.vs.double().view(1, KV, 1)
            _attn.check_e4m3(self.k[p, o], want[there, HEADS:] / ks, slack[there, HEADS:] / ks, "k")
            _attn.check_e4m3(self.v[p, o], heads[there, HEADS + KV:].double() / vs, 0.0, "v")
        out, bound, lse, lse_bound = _attn.decode_ref(self.q, self.k, self.v, self.table, self.lengths.tolist(), PAGE, 0, D ** -0.5,
                                                      self.ks, self.vs, self.ks is not None)
        assert bool(((self.mixed.double() - out).abs() <= bound).all())
        full = self.lengths > 0
        assert bool(((self.lse.double() - lse).abs()[full] <= lse_bound[full]).all()) and bool((self.lse[~full] == float("-inf")).all())
        W = _moe.w4_values(*self.o)
        a = self.mixed.view(B, HEADS * D).double()
        want = a @ W.t()
        assert bool(((self.out.double() - want).abs() <= want.abs() * _attn.HALF_BF16 + _moe.gamma(HEADS * D) * (a.abs() @ W.abs().t())).all())
        y, _, h2 = _attn.norm_q8_ref([self.out], self.h, self.gamma[1], 0.0, EPS, 128)
        assert bool(((self.h2.double() - h2).abs() <= h2.abs() * (_attn.HALF_BF16 + 2.0 ** -20)).all())
        assert bool(((self.y.double() - y).abs() <= y.abs() * (_attn.HALF_BF16 + 2.0 ** -18)).all())


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("captured", [False, True])
def test_steps(eight, captured):
    g = gen(50)
    layer = Layer(eight, g)
    # sequences of several lengths, one that is a padded row; pages in a mixed order, taken as they are needed
    lengths, free = [0, 15, 16, 40, 0], torch.randperm(PAGES, generator=g, device=DEV).tolist()
    table = [[] for _ in range(B)]
    for b, n in enumerate(lengths):
        table[b] = [free.pop() for _ in range(-(-n // PAGE))]
    if captured:
        layer.lengths.zero_()
        layer.slots.fill_(-1)
        layer.step()  # (every kernel's first use is outside the capture)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            layer.step()
    for step in range(6):
        slots, pos = [], []
        for b in range(B):
            if b == 4:  # no sequence here: nothing written, nothing to look at
                slots.append(-1)
                pos.append(0)
                continue
            if lengths[b] % PAGE == 0:
                table[b].append(free.pop())
            slots.append(table[b][-1] * PAGE + lengths[b] % PAGE)
            pos.append(lengths[b])
            lengths[b] += 1
        layer.slots.copy_(torch.tensor(slots, dtype=torch.int32))
        layer.pos.copy_(torch.tensor(pos, dtype=torch.int32))
        layer.lengths.copy_(torch.tensor(lengths, dtype=torch.int32))
        layer.table.copy_(torch.tensor([t + [-1] * (WIDTH - len(t)) for t in table], dtype=torch.int32))
        layer.partial.copy_(normal((B, H), g))
        layer.residual.copy_(normal((B, H), g))
        before = layer.k.clone(), layer.v.clone()
        torch.cuda.synchronize()
        graph.replay() if captured else layer.step()
        torch.cuda.synchronize()
        layer.check(before)
        assert bool((layer.mixed[4] == 0).all())
    assert arf.ar_attn_device_error(layer.attn) == 0 and arf.ar_workspace_device_error(layer.ws) == 0
    layer.attn.destroy()
    layer.ws.destroy()


def test_one_call_is_one_kernel_launch():
    from tests.test_gpu_one_launch import _device_activities
    layer = Layer(False, gen(51))
    layer.slots.copy_(torch.arange(B, dtype=torch.int32))
    layer.table[:, 0] = 0
    layer.lengths.copy_(torch.tensor([1, 5, 0, 16, 3], dtype=torch.int32))
    layer.step()
    x = torch.ones(1024, device=DEV)
    if not any(_device_activities(lambda: x.mul_(1.0)) for _ in range(3)):
        pytest.skip("the CUDA profiler records no device activity on this machine")
    for kernel, call in (
            ("norm_q8", lambda: arf.ar_rmsnorm_q8(layer.ws, [layer.partial], layer.residual, layer.gamma[0], 0.0, EPS, q=layer.x8,
                                                  scales=layer.scales, residual_out=layer.h, out=layer.x)),
            ("attn_append", lambda: arf.ar_attn_append(layer.attn, layer.cache, layer.rows, layer.pos.view(1, B), layer.slots, q=layer.q)),
            ("attn_decode", lambda: arf.ar_attn_decode(layer.attn, layer.cache, layer.q, layer.table, layer.lengths, out=layer.mixed))):
        names = _device_activities(call)
        assert len(names) == 1 and kernel in names[0], names
    layer.attn.destroy()
    layer.ws.destroy()


def test_readme_example():
    import os
    import re
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")).read()
    blocks = [b for b in re.findall(r"```python\n(.*?)```", text, re.S) if "ar_attn_append" in b]
    assert len(blocks) == 1
    scope = dict(torch=torch, arf=arf)
    exec(compile(blocks[0], "README.md", "exec"), scope)
    q, k, v, table, lengths = (scope[n] for n in ("q", "k", "v", "table", "lengths"))
    for b in range(2):  # the new token's values are where they belong
        at = int(lengths[b]) - 1
        x = scope["qkv"][b].view(-1, scope["D"])
        assert torch.equal(v[int(table[b, at // scope["page"]]), at % scope["page"]], x[scope["heads"] + scope["kv"]:])
    want, slack, _, _ = _attn.decode_ref(q, k, v, table, lengths.tolist(), scope["page"], 0, scope["D"] ** -0.5)
    assert bool(((scope["ctx"].double() - want).abs() <= slack).all())


def test_first_calls_are_captured():
    # a fresh process, nothing launched before: the kernels load during the capture
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = """
import torch, tp_reduce_moe_gb300 as arf
bf = dict(device="cuda", dtype=torch.bfloat16)
i32 = lambda x: torch.tensor(x, device="cuda", dtype=torch.int32)
k, v = torch.zeros(8, 16, 2, 128, **bf), torch.zeros(8, 16, 2, 128, **bf)
cache = arf.ar_kv_cache(k, v)
attn, ws = arf.ar_attn_create(8, 2, 128, 16, 4), arf.ar_workspace_create(2, 0, 1024, 4096, 1e-6)
qkv, slots, table, lengths = torch.ones(2, 12 * 128, **bf), i32([0, 17]), i32([[0], [1]]), i32([1, 2])
parts = {T: [torch.ones(T, 1024, **bf) for _ in range(3)] for T in (2, 4096)}
gamma = torch.ones(1024, **bf)
torch.cuda.synchronize()
s = torch.cuda.Stream()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g, stream=s):
    q = arf.ar_attn_append(attn, cache, qkv, None, slots)
    out = arf.ar_attn_decode(attn, cache, q, table, lengths)
    norms = [arf.ar_rmsnorm_q8(ws, p[:2], p[2], gamma, 0.0, 1e-6) for p in parts.values()]
g.replay()
torch.cuda.synchronize()
assert bool((out == 1).all())  # (of the second two tokens one is zeros and weighs e^-11)
for y, scale, h in norms:
    assert bool((h == 3).all()) and bool(((y.float() * scale.repeat_interleave(128, 1) - 1).abs() < 2.0 ** -4).all())
print("captured")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]
