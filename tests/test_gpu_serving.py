"""The decoder calls as a serving loop uses them: prompts attend and fill the cache, steps reserve, append and attend,
beams fork, finished sequences leave, the cache is compacted under way.  Every output against fp64 over each
sequence's own history, kept apart from the cache."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import remove_padding_prefix_gb300 as rpp
from gpu_util import TDT, dev
from test_gpu_causal import check_rows

pytestmark = pytest.mark.gpu

EPS = {torch.float16: 2.0 ** -10, torch.bfloat16: 2.0 ** -7}


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=dev())


class Loop:
    """A cache of `layers` layers and, per slot and layer, the rows it should hold."""

    def __init__(self, layers, pages, ps, nh, nkv, d, slots, max_pages, dtype):
        self.layers, self.nh, self.nkv, self.d, self.dt = layers, nh, nkv, d, TDT[dtype]
        self.cache = rpp.KvCache(layers, pages, ps, nkv, d, slots, max_pages, dtype, dev())
        self.cache.pool.fill_(float("nan"))
        self.rows = {}            # slot -> [K, V] per layer
        self.g = torch.Generator(device=dev()).manual_seed(layers)

    def qkv(self, n):
        x = torch.randn((n, (self.nh + 2 * self.nkv) * self.d), generator=self.g, device=dev()).to(self.dt)
        w, u = self.nh * self.d, self.nkv * self.d
        return x[:, :w], x[:, w:w + u], x[:, w + u:]

    def prompt(self, slots, lens):
        c = self.cache
        rpp.kv_reserve(c, ints(slots), ints(lens))
        cu = [0] + np.cumsum(lens).tolist()
        for s in slots:
            self.rows[s] = []
        for layer in range(self.layers):
            q, k, v = self.qkv(cu[-1])
            rpp.kv_append(c, layer, k, v, ints(slots), ints(cu))
            o = rpp.attention_causal_varlen(q, k, v, ints(cu), len(lens), max(lens), self.nh, self.nkv, self.d,
                                            err=c.err)
            check_rows(o, q, k, v, cu, self.nh, self.nkv, self.d)
            for i, s in enumerate(slots):
                self.rows[s].append([k[cu[i]:cu[i + 1]].clone(), v[cu[i]:cu[i + 1]].clone()])

    def took(self, slots, layer, k, v):
        for i, s in enumerate(slots):
            r = self.rows[s][layer]
            r[0], r[1] = torch.cat([r[0], k[i:i + 1]]), torch.cat([r[1], v[i:i + 1]])

    def check(self, o, q, slots, layer):
        per, e = self.nh // self.nkv, EPS[self.dt]
        for i, s in enumerate(slots):
            K, V = (x.double().view(-1, self.nkv, self.d) for x in self.rows[s][layer])
            n = K.shape[0]
            qi = q[i].double().view(self.nkv, per, self.d)
            z = torch.einsum("hgd,nhd->hgn", qi, K) * self.d ** -0.5
            ref = torch.einsum("hgn,nhd->hgd", torch.softmax(z, -1), V)
            mag = (torch.einsum("hgd,nhd->hgn", qi.abs(), K.abs()) * self.d ** -0.5).amax()
            # the decode test's bound, with the largest of its terms for all heads
            bound = V.abs().max() * (2 * ((self.d + 2) * 2.0 ** -24 * mag + 2.0 ** -23 * z.abs().max()) +
                                     2 * (2.0 ** -22 + 2.0 ** -17 + n * 2.0 ** -24))
            off = (o[i].double().view(self.nkv, per, self.d) - ref).abs()
            assert (off <= e / 2 * ref.abs() + bound + 2.0 ** -25).all(), (s, layer, n, float(off.max()))

    def step(self, slots):
        c, ss = self.cache, ints(slots)
        rpp.kv_reserve(c, ss, ints([1] * len(slots)))
        for layer in range(self.layers):
            q, k, v = self.qkv(len(slots))
            rpp.kv_append(c, layer, k, v, ss)
            o = rpp.attention_decode(c, layer, q, ss)
            self.took(slots, layer, k, v)
            self.check(o, q, slots, layer)

    def fork(self, src, dst):
        rpp.kv_fork(self.cache, ints(src), ints(dst))
        for a, b in zip(src, dst):
            self.rows[b] = [list(kv) for kv in self.rows[a]]

    def free(self, slots):
        rpp.kv_free(self.cache, ints(slots))
        for s in slots:
            del self.rows[s]

    def compact(self, apart):
        c = self.cache
        if apart:
            c.adopt(*rpp.kv_compact(c, table_out=torch.empty_like(c.table), refs_out=torch.empty_like(c.refs))[:2])
        else:
            rpp.kv_compact(c)

    def done(self):
        assert rpp.get_device_error(self.cache.err) == 0
        assert self.cache.lens.tolist() == [self.rows[s][0][0].shape[0] if s in self.rows else 0
                                            for s in range(self.cache.cfg.slots)]


@pytest.mark.parametrize("dtype,d,nh,nkv,ps", [("bf16", 128, 8, 2, 16), ("fp16", 64, 6, 6, 32), ("bf16", 64, 20, 1, 48)])
def test_a_serving_loop(dtype, d, nh, nkv, ps):
    r = Loop(2, 160, ps, nh, nkv, d, 8, 24, dtype)     # 24 pages a sequence: room for 16 * 24 rows
    r.prompt([2, 0, 5], [37, ps, 190])
    for _ in range(3):
        r.step([5, 2, 0])
    r.fork([5, 5, 0], [1, 7, 6])                 # two beams of one, one of another
    for _ in range(2):
        r.step([7, 0, 5, 6, 1, 2])
    r.free([5, 0])                               # the pages that beams share stay
    r.compact(apart=False)
    for _ in range(ps):                          # over the end of a page
        r.step([1, 6, 7])
    r.prompt([0, 3], [129, 1])                   # a new prompt in a slot that was freed
    r.free([6, 2])
    r.compact(apart=True)
    r.step([0, 1, 3, 7])
    r.fork([3], [5])
    r.step([5, 3])
    r.done()


def test_a_captured_step():
    """reserve, append and attend for every layer captured once; replays advance the sequences."""
    r = Loop(2, 200, 16, 8, 2, 128, 6, 20, "bf16")
    r.prompt([0, 1, 2, 3], [5, 100, 33, 16])
    slots, ones = ints([3, 1, 0, 2]), ints([1] * 4)
    x = [[t.clone() for t in r.qkv(4)] for _ in range(2)]
    outs = [torch.empty(4, 1024, dtype=torch.bfloat16, device=dev()) for _ in range(2)]
    ws = rpp.attention_decode_workspace(r.cache, 4, 8)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            rpp.kv_reserve(r.cache, slots, ones)
            for layer, (q, k, v) in enumerate(x):
                rpp.kv_append(r.cache, layer, k, v, slots)
                rpp.attention_decode(r.cache, layer, q, slots, out=outs[layer], workspace=ws)
    torch.cuda.synchronize()
    r.done()
    for step in range(20):
        order = [int(i) for i in np.random.default_rng(step).permutation(4)]
        slots.copy_(ints(order))
        for t in x:
            for a, b in zip(t, r.qkv(4)):
                a.copy_(b)
        g.replay()
        for layer, (q, k, v) in enumerate(x):
            r.took(order, layer, k, v)
            r.check(outs[layer], q, order, layer)
    r.done()


def test_what_a_call_makes_belongs_to_its_stream(monkeypatch):
    """Workspace, output and count of a call on a given stream: the current stream gets that memory neither
    while the call's stream is busy nor after, and the call gets none that the current stream has just freed."""
    loop = Loop(1, 20, 16, 4, 2, 64, 4, 8, "bf16")
    c = loop.cache
    q, k, v = loop.qkv(3)
    rpp.kv_reserve(c, ints([0, 1, 2]), ints([1, 1, 1]))
    rpp.kv_append(c, 0, k, v, ints([0, 1, 2]))
    cu = ints([0, 3])
    sizes = [rpp.attention_decode_workspace(c, 3, 4).numel(), q.numel() * 2, q.numel() * 2, 4]
    torch.cuda.synchronize()
    made = []
    make = rpp.attention_decode_workspace
    monkeypatch.setattr(rpp, "attention_decode_workspace", lambda *a: made.append(make(*a)) or made[-1])
    freed = [torch.empty(n, dtype=torch.uint8, device=dev()) for n in sizes]
    before = {t.data_ptr() for t in freed}
    del freed                                     # what the current stream would be given next
    side = torch.cuda.Stream()
    outs = [rpp.attention_decode(c, 0, q, stream=side),
            rpp.attention_causal_varlen(q, k, v, cu, 1, 3, 4, 2, 64, err=c.err, stream=side),
            rpp.kv_compact(c, stream=side)[2]]
    assert len(made) == 1
    mine = {t.data_ptr() for t in made + outs}
    assert not mine & before
    del made[:]
    after = [torch.empty(sizes[0], dtype=torch.uint8, device=dev()) for _ in range(4)]
    assert not mine & {t.data_ptr() for t in after}
    side.synchronize()
    assert rpp.get_device_error(c.err) == 0 and int(outs[2]) == 3
    check_rows(outs[1], q, k, v, [0, 3], 4, 2, 64)
    # a new token's attention over its own key alone is its value
    assert torch.equal(outs[0].view(3, 2, 2, 64), v.view(3, 2, 1, 64).expand(3, 2, 2, 64))


FIRST = """
import sys
sys.path.insert(0, {root!r})
import torch
import remove_padding_prefix_gb300 as rpp
ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
c = rpp.KvCache(1, 40, 16, 2, {d}, 4, 8)
qkv = torch.randn(50, 8 * {d}, device="cuda").bfloat16()
w = {d}
q, k, v = qkv[:, :4 * w], qkv[:, 4 * w:6 * w], qkv[:, 6 * w:]
slots, lens, cu, src, dst, one = ints([0, 1]), ints([20, 30]), ints([0, 20, 50]), ints([0]), ints([2]), ints([1])
ws = rpp.attention_decode_workspace(c, 2, 4)
last = q[[19, 49]]
g = torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(g):
    rpp.kv_reserve(c, slots, lens)
    rpp.kv_append(c, 0, k, v, slots, cu)
    a = rpp.attention_causal_varlen(q, k, v, cu, 2, 50, 4, 2, w, err=c.err)
    b = rpp.attention_decode(c, 0, last, slots, workspace=ws)
    rpp.kv_fork(c, src, dst)
    rpp.kv_free(c, one)
    table, refs, live = rpp.kv_compact(c)
g.replay()
assert rpp.get_device_error(c.err) == 0
assert (a[[19, 49]].float() - b.float()).abs().max() <= 2.0 ** -6 * a.float().abs().max()
assert live.tolist() == [3] and c.lens.tolist() == [20, 0, 20, 0]
print("ok")
"""


@pytest.mark.parametrize("d", [64, 128])
def test_the_first_calls_of_a_process_captured(d):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST.format(root=root, d=d)], capture_output=True, text=True, timeout=200)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stdout + r.stderr
