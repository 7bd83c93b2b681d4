"""The decoder calls over the 8-bit cache as a serving loop uses them: prompts attend and fill the cache, steps reserve,
append and attend, beams fork, finished sequences leave, the cache is compacted under way, sequences are read back.
Outputs against fp64 over the rows as the cache holds them; those against the rows that went in."""
import numpy as np
import pytest
import torch

import remove_padding_prefix_gb300 as rpp
from gpu_util import TDT, dev
from test_gpu_causal import check_rows
from test_gpu_serving import EPS, Loop, ints

pytestmark = pytest.mark.gpu


class Loop8(Loop):
    def __init__(self, layers, pages, ps, nh, nkv, d, slots, max_pages, dtype, kind, block):
        super().__init__(layers, pages, ps, nh, nkv, d, slots, max_pages, dtype)
        self.kind, self.block = kind, block
        self.cache = rpp.KvCache8(layers, pages, ps, nkv, d, slots, max_pages, kind, block, dev())
        self.cache.pool.view(torch.uint8).fill_(0x7f)
        self.cache.scales.fill_(255)

    def held(self, slot, layer):
        """K and V as the cache holds them, each within what quantising may lose: a block whose largest magnitude is a has
        steps of less than a / 63.75 (int8) and a / 232 (e4m3); int8 is off by less than one, e4m3 by 2^-4 of the value and
        2^-9 of one."""
        rows = self.rows[slot][layer]
        n = rows[0].shape[0]
        got = rpp.kv_read(self.cache, layer, ints([slot]), ints([0, n]), rows=n)      # bf16 holds every code * 2^e
        for x, y in zip(got, rows):
            x, y = x.double().view(n, self.nkv, self.d), y.double().view(n, self.nkv, self.d)
            pad = torch.nn.functional.pad(y, (0, 0, 0, 0, 0, -n % self.block))
            a = pad.abs().amax(-1).view(-1, self.block, self.nkv).amax(1).repeat_interleave(self.block, 0)[:n, :, None]
            limit = a / 63.75 if self.kind == "int8" else 2.0 ** -4 * y.abs() + 2.0 ** -9 * a / 232
            assert ((x - y).abs() <= limit).all(), (slot, layer)
        return got

    def check(self, o, q, slots, layer):
        per, e = self.nh // self.nkv, EPS[self.dt]
        top = 127.0 if self.kind == "int8" else 448.0
        for i, s in enumerate(slots):
            K, V = (x.double().view(-1, self.nkv, self.d) for x in self.held(s, layer))
            n = K.shape[0]
            qi = q[i].double().view(self.nkv, per, self.d)
            z = torch.einsum("hgd,nhd->hgn", qi, K) * self.d ** -0.5
            ref = torch.einsum("hgn,nhd->hgd", torch.softmax(z, -1), V)
            mag = (torch.einsum("hgd,nhd->hgn", qi.abs(), K.abs()) * self.d ** -0.5).amax()
            # the decode test's bound, with the largest of its terms for all heads (a scale is below 2 max |V| / top)
            vmax = V.abs().max()
            bound = vmax * (2 * ((self.d + 6) * 2.0 ** -24 * mag + 2.0 ** -22 * z.abs().max()) +
                            2 * (2.0 ** -22 + 2.0 ** -21 + n * 2.0 ** -24)) + n * 2.0 ** -32 * top * 2 * vmax * 2 / top
            off = (o[i].double().view(self.nkv, per, self.d) - ref).abs()
            assert (off <= e / 2 * ref.abs() + bound + 2.0 ** -25).all(), (s, layer, n, float(off.max()))


@pytest.mark.parametrize("dtype,d,nh,nkv,ps,kind,block", [
    ("bf16", 128, 8, 2, 16, "e4m3", 16), ("fp16", 64, 6, 6, 32, "int8", 4), ("bf16", 64, 20, 1, 48, "int8", 1),
    ("fp16", 128, 12, 1, 64, "e4m3", 64)])
def test_a_serving_loop(dtype, d, nh, nkv, ps, kind, block):
    r = Loop8(2, 160, ps, nh, nkv, d, 8, 24, dtype, kind, block)
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
    r.prompt([3, 5], [2 * ps, 1])                # chunks: the rest of a prompt after its first part
    r.compact(apart=True)
    r.step([5, 3, 1])
    r.done()


def test_a_sequence_moves_to_another_cache():
    """Read back from one cache as packed rows, taken in by another of the other kind, and attended to as prompts."""
    r = Loop8(1, 40, 16, 4, 2, 64, 4, 20, "bf16", "int8", 16)
    r.prompt([0, 1], [100, 33])
    cu = ints([0, 100, 133])
    k, v = rpp.kv_read(r.cache, 0, ints([0, 1]), cu, rows=133)
    q, _, _ = r.qkv(133)
    check_rows(rpp.attention_causal_varlen(q, k, v, cu, 2, 100, 4, 2, 64), q, k, v, [0, 100, 133], 4, 2, 64)
    wide = rpp.KvCache(1, 20, 16, 2, 64, 2, 10, "bf16", dev())
    rpp.kv_reserve(wide, ints([1, 0]), ints([100, 33]))
    rpp.kv_append(wide, 0, k, v, ints([1, 0]), cu)
    ko, vo = rpp.kv_read(wide, 0, ints([1, 0]), cu, rows=133)
    assert torch.equal(ko, k) and torch.equal(vo, v)
    again = rpp.KvCache8(1, 20, 16, 2, 64, 2, 10, "int8", 16, dev())
    rpp.kv_reserve(again, ints([1, 0]), ints([100, 33]))
    rpp.kv_append(again, 0, ko, vo, ints([1, 0]), cu)
    kk, vv = rpp.kv_read(again, 0, ints([1, 0]), cu, rows=133)
    # codes of a block were up to 127 and are again: written at once, nothing is lost where no code grew past its top
    assert torch.equal(kk, k) and torch.equal(vv, v)
    for c in (r.cache, wide, again):
        assert rpp.get_device_error(c.err) == 0


@pytest.mark.parametrize("kind,block", [("e4m3", 16), ("int8", 1)])
def test_a_captured_step(kind, block):
    """One step of two layers captured once: reserve, append, attend; eight replays, other slots and rows each."""
    layers, nh, nkv, d = 2, 8, 2, 128
    r = Loop8(layers, 80, 16, nh, nkv, d, 6, 12, "bf16", kind, block)
    r.prompt([0, 1, 2, 3], [15, 31, 3, 100])
    c, n = r.cache, 3
    slots, ones = ints([0, 1, 2]), ints([1] * n)
    x = [torch.empty(n, (nh + 2 * nkv) * d, dtype=torch.bfloat16, device=dev()) for _ in range(layers)]
    out = [torch.empty(n, nh * d, dtype=torch.bfloat16, device=dev()) for _ in range(layers)]
    ws = rpp.attention_decode_workspace(c, n, nh)
    w, u = nh * d, nkv * d
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            rpp.kv_reserve(c, slots, ones)
            for i in range(layers):
                rpp.kv_append(c, i, x[i][:, w:w + u], x[i][:, w + u:], slots)
                rpp.attention_decode(c, i, x[i][:, :w], slots, out=out[i], workspace=ws)
    torch.cuda.synchronize()
    rng = np.random.default_rng(5)
    for _ in range(8):
        pick = [int(a) for a in rng.permutation(4)[:n]]
        slots.copy_(ints(pick))
        for i in range(layers):
            q, k, v = r.qkv(n)
            x[i].copy_(torch.cat([q, k, v], 1))
            r.took(pick, i, k, v)
        g.replay()
        torch.cuda.synchronize()
        for i in range(layers):
            r.check(out[i], x[i][:, :w], pick, i)
    r.done()
