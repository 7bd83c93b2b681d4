"""The 8-bit paged cache on the GPU against the oracle kept from the definition: every array of the state, bit for bit,
after each call; rows read back; refused calls change nothing (or only what they say) and record their error."""
import numpy as np
import pytest
import torch

import oracle.decoder as od
import oracle.decoder8 as o8
import remove_padding_prefix_gb300 as rpp
from gpu_util import TDT, dev

pytestmark = pytest.mark.gpu


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=dev())


def raw(t):
    return t.view(torch.uint8).cpu().numpy()


class Pair:
    """A cache on the GPU and the oracle's, driven together."""

    def __init__(self, layers, pages, ps, nkv, d, slots, max_pages, kind="e4m3", block=16, dtype="bf16", seed=0):
        self.rng = np.random.default_rng(seed)
        self.kind, self.dtype, self.nkv, self.d, self.layers = kind, dtype, nkv, d, layers
        self.gpu = rpp.KvCache8(layers, pages, ps, nkv, d, slots, max_pages, kind, block, dev())
        self.ref = o8.PagedCache8(layers, pages, ps, nkv, d, slots, max_pages, kind, block)
        for ours, theirs in ((self.ref.pool, self.gpu.pool), (self.ref.scales, self.gpu.scales)):
            ours[:] = self.rng.integers(0, 256, ours.shape)          # whatever memory held
            theirs.view(torch.uint8).copy_(torch.from_numpy(ours))

    def rows(self, n, pad=0, spread=1.5):
        """n rows of K | V as columns of wider rows, rows and heads of different sizes: (device k, v, fp64 k, v)."""
        w = self.nkv * self.d
        size = np.exp(spread * self.rng.normal(size=(n, 2 * self.nkv, 1)))
        x = self.rng.normal(size=(n, 2 * self.nkv, self.d)) * size
        x[self.rng.random(x.shape) < 0.02] = 0.0
        x[self.rng.random(x.shape[:2]) < 0.02] = 0.0                  # rows of zeros
        wide = np.concatenate([np.zeros((n, pad)), x.reshape(n, 2 * w)], 1)
        g = torch.from_numpy(wide).to(dev()).to(TDT[self.dtype])
        y = g.double().cpu().numpy()
        return (g[:, pad:pad + w], g[:, pad + w:], y[:, pad:pad + w].reshape(n, self.nkv, self.d),
                y[:, pad + w:].reshape(n, self.nkv, self.d))

    def grow(self, slots, counts, pad=0, rows=None):
        rpp.kv_reserve(self.gpu, ints(slots), ints(counts))
        self.ref.reserve(slots, counts)
        cu = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        for layer in range(self.layers):
            k, v, kw, vw = rows or self.rows(int(cu[-1]) + 3, pad)     # three rows behind the last sequence
            rpp.kv_append(self.gpu, layer, k, v, ints(slots), ints(cu.tolist()))
            self.ref.append(layer, kw, vw, slots, counts)

    def fork(self, src, dst):
        rpp.kv_fork(self.gpu, ints(src), ints(dst))
        self.ref.fork(src, dst)

    def free(self, slots):
        rpp.kv_free(self.gpu, ints(slots))
        self.ref.free(slots)

    def compact(self, apart=False):
        remap = torch.full((self.gpu.cfg.pages,), 77, dtype=torch.int32, device=dev())
        outs = dict(table_out=torch.empty_like(self.gpu.table), refs_out=torch.empty_like(self.gpu.refs)) if apart else {}
        table, refs, live = rpp.kv_compact(self.gpu, remap=remap, **outs)
        if apart:
            self.gpu.adopt(table, refs)
        want, n = self.ref.compact()
        assert int(live) == n
        np.testing.assert_array_equal(remap.cpu().numpy(), want)

    def check(self, code=0):
        assert rpp.get_device_error(self.gpu.err) == code
        self.gpu.err.zero_()
        np.testing.assert_array_equal(self.gpu.lens.cpu().numpy(), self.ref.lens)
        np.testing.assert_array_equal(self.gpu.refs.cpu().numpy(), self.ref.refs)
        np.testing.assert_array_equal(self.gpu.table.cpu().numpy(), self.ref.table())
        np.testing.assert_array_equal(raw(self.gpu.scales), self.ref.scales)
        np.testing.assert_array_equal(raw(self.gpu.pool), self.ref.pool)

    def expect(self, layer, slot, a, e, dtype):
        """What reading positions a .. e - 1 gives, as torch rows K, V on the CPU."""
        t = TDT[dtype]
        got = []
        for x in self.ref.values(layer, slot):
            x = o8.read_back(x[a:e], float(torch.finfo(t).max))
            got.append(torch.from_numpy(x).reshape(e - a, self.nkv * self.d).float().to(t))
        return got


def same(a, b):
    return bool(((a == b) | (torch.isnan(a) & torch.isnan(b))).all())


SHAPES = [
    # layers, pages, page rows, kv heads, head size, slots, pages a sequence, block
    (1, 40, 16, 2, 64, 6, 9, 16),
    (2, 61, 16, 8, 128, 12, 20, 16),
    (2, 37, 16, 1, 64, 6, 12, 1),
    (1, 50, 48, 3, 128, 7, 11, 2),
    (1, 30, 32, 5, 64, 7, 6, 4),
    (2, 30, 16, 3, 128, 7, 6, 8),
    (1, 30, 64, 2, 64, 7, 5, 32),
    (1, 20, 64, 1, 128, 7, 4, 64),
    (1, 14, 256, 1, 64, 6, 2, 128),
]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_calls_one_by_one(shape, kind, dtype):
    p = Pair(*shape[:7], kind=kind, block=shape[7], dtype=dtype)
    ps, mp = shape[2], shape[6]
    p.grow([1], [1])
    p.check()
    p.grow([3, 0], [ps, 0])                      # a whole page; a count of zero
    p.check()
    p.grow([0, 1, 2], [ps + 1, ps - 1, 3], pad=8)
    p.check()
    for _ in range(5):                           # token by token, into blocks that have some
        p.grow([2, 0], [1, 1])
        p.check()
    p.grow([2, 1], [7, 2])
    p.check()
    p.fork([0, 3], [4, len(p.ref.lens) - 1])
    p.check()
    p.free([0, 3])
    p.check()
    p.compact()
    p.check()
    p.grow([4], [1])                             # the fork grows on its own page
    p.check()
    p.free([4])
    p.compact(apart=True)
    p.check()
    p.compact()                                  # nothing to move
    p.grow([0], [mp * ps])                       # the longest sequence
    p.check()
    p.free(list(range(len(p.ref.lens))))
    p.compact()                                  # nothing in use
    p.check()


@pytest.mark.parametrize("kind,block,shape,steps", [("e4m3", 16, (2, 60, 16, 2, 64, 9, 9), 50),
                                                    ("int8", 4, (1, 60, 16, 1, 128, 9, 9), 50),
                                                    ("int8", 32, (1, 40, 32, 1, 64, 9, 6), 50)])
def test_random_calls(kind, block, shape, steps):
    p = Pair(*shape, kind=kind, block=block, seed=steps)
    r = np.random.default_rng(7)
    slots, cap = shape[5], shape[2] * shape[6]
    for _ in range(steps):
        what = r.integers(0, 10)
        pick = [int(s) for s in r.permutation(slots)[:r.integers(1, slots + 1)]]
        room = sum(1 for x in p.ref.refs if x == 0)
        if what < 6:
            most = 2 if what < 3 else cap // 3
            counts = [int(min(r.integers(0, most), cap - p.ref.lens[s])) for s in pick]
            need = sum(-(-(p.ref.lens[s] + c) // p.ref.ps) - len(p.ref.rows[s]) for s, c in zip(pick, counts))
            if need <= room:
                p.grow(pick, counts)
        elif what < 7:
            empty = [s for s in pick if p.ref.lens[s] == 0]
            full = [s for s in range(slots) if p.ref.lens[s]]
            if empty and full and len(empty) <= room:
                p.fork([int(x) for x in r.choice(full, len(empty))], empty)
        elif what < 9:
            p.free(pick[:2])
        else:
            p.compact(apart=bool(r.integers(0, 2)))
        p.check()


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("block", [1, 16])
def test_values_at_the_borders(kind, dtype, block):
    """Ties, the largest and smallest values of the type, zeros of both signs, one infinity, one NaN."""
    t = TDT[dtype]
    big, tiny = torch.finfo(t).max, torch.finfo(t).smallest_normal
    small = 2.0 ** -24 if dtype == "fp16" else 2.0 ** -133
    top, past = o8.TOP[kind], o8.PAST[kind]
    eps = torch.finfo(t).eps
    rows = [[0.0, -0.0], [big, -big, big / 3], [small, -small], [tiny, small, -3 * small], [top, 0.5, 1.5, 2.5, -3.5, -0.5],
            [past, 1.0], [past * (1 + eps), 1.0], [1.0, 127.0, 63.5, 62.5, -61.5], [448.0, 17.0, 19.0, 21.0, 2.0 ** -10, 3 * 2.0 ** -10],
            [2.0 ** -9, 1.0, 1.0625, 1.1875], [float("inf"), 1.0], [1.0, float("nan")], [-float("inf")], [1.0] * 64]
    n = len(rows)
    p = Pair(1, n + 2, 16, 1, 64, n, 1, kind=kind, block=block, dtype=dtype)
    x = torch.zeros(n, 64, dtype=torch.float64)
    for i, r in enumerate(rows):
        x[i, :len(r)] = torch.tensor(r, dtype=torch.float64)
    g = x.to(t).to(dev())
    y = g.double().cpu().numpy().reshape(n, 1, 64)
    slots = list(range(n))
    for _ in range(2):                           # as first rows, then beside rows that are there
        p.grow(slots, [1] * n, rows=(g, g, y, y))
        p.check()
        g, y = g.flip(0).contiguous(), y[::-1]
    k, v = rpp.kv_read(p.gpu, 0, ints(slots), dtype=dtype)
    for s in slots:
        want = p.expect(0, s, 1, 2, dtype)
        assert same(k[s].cpu(), want[0][0]) and same(v[s].cpu(), want[1][0])


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_rows_read_back(shape, kind):
    p = Pair(*shape[:7], kind=kind, block=shape[7])
    ps = shape[2]
    lens = [ps, 1, 2 * ps - 3, 0, ps + 5]
    p.grow(list(range(5)), lens)
    layer = p.layers - 1
    w = p.nkv * p.d
    for dtype in ("fp16", "bf16"):
        # whole sequences, ranges, the same slot twice, nothing; rows behind and columns beside stay
        for slots, starts, counts in ([0, 1, 2, 3, 4], [0] * 5, lens), ([4, 2, 4, 0], [3, ps, 0, ps - 1], [5, ps - 3, ps, 1]), \
                ([2, 4, 1], None, [ps, 7, 1]), ([3, 1], [5, 0], [0, 1]):
            cu = np.concatenate([[0], np.cumsum(counts)]).tolist()
            out = torch.full((cu[-1] + 2, 2 * w + 24), 7.0, dtype=TDT[dtype], device=dev())
            k, v = rpp.kv_read(p.gpu, layer, ints(slots), ints(cu), starts=None if starts is None else ints(starts),
                               k=out[:, 8:8 + w], v=out[:, 16 + w:16 + 2 * w])
            assert rpp.get_device_error(p.gpu.err) == 0
            for i, s in enumerate(slots):
                a = lens[s] - counts[i] if starts is None else starts[i]
                want = p.expect(layer, s, a, a + counts[i], dtype)
                assert torch.equal(k[cu[i]:cu[i + 1]].cpu(), want[0]) and torch.equal(v[cu[i]:cu[i + 1]].cpu(), want[1])
            out[:cu[-1], 8:8 + w] = 7.0
            out[:cu[-1], 16 + w:16 + 2 * w] = 7.0
            assert (out == 7).all()
    p.check()


@pytest.mark.parametrize("nkv,block,kind,dtype", [(2, 1, "int8", "fp16"), (2, 16, "e4m3", "bf16"), (4, 4, "e4m3", "fp16"),
                                                  (3, 8, "int8", "bf16"), (2, 32, "int8", "fp16"), (2, 2, "int8", "bf16")])
def test_more_rows_than_ctas(nkv, block, kind, dtype):
    """Several thousand rows, twice, the second time into blocks that have some."""
    p = Pair(1, 220, 32, nkv, 64, 12, 60, kind=kind, block=block, dtype=dtype)
    p.grow([3, 0, 7, 5], [700, 1, 1801, 333])
    p.check()
    p.grow([0, 7, 3, 9], [900, 90, 801, 1000])
    p.check()


def test_one_row_each_without_cu_seqlens():
    p = Pair(2, 20, 16, 2, 64, 6, 5, kind="int8")
    slots = [4, 0, 2]
    p.grow(slots, [3, 16, 15])
    rpp.kv_reserve(p.gpu, ints(slots), ints([1, 1, 1]))
    p.ref.reserve(slots, [1, 1, 1])
    k, v, kw, vw = p.rows(3)
    rpp.kv_append(p.gpu, 1, k, v, ints(slots))
    p.ref.append(1, kw, vw, slots, [1, 1, 1])
    p.check()
    for starts, at in ((None, [3, 16, 15]), ([0, 5, 14], [0, 5, 14])):
        got = rpp.kv_read(p.gpu, 1, ints(slots), starts=None if starts is None else ints(starts))
        for i, s in enumerate(slots):
            want = p.expect(1, s, at[i], at[i] + 1, "bf16")
            assert torch.equal(got[0][i].cpu(), want[0][0]) and torch.equal(got[1][i].cpu(), want[1][0])


def test_an_append_again_changes_nothing():
    """After an error of its own an append is called once more: the rows that it wrote come out the same."""
    p = Pair(1, 20, 16, 2, 64, 6, 5, kind="int8")
    p.grow([0, 1], [5, 40])
    k, v, kw, vw = p.rows(30)
    p.grow([0, 1], [20, 7], rows=(k, v, kw, vw))
    for _ in range(2):
        rpp.kv_append(p.gpu, 0, k, v, ints([0, 1]), ints([0, 20, 27]))
        p.check()


@pytest.mark.parametrize("dtype,kv", [("fp16", "fp16"), ("bf16", "bf16")])
@pytest.mark.parametrize("shape", [(2, 37, 1, 1, 8, 6, 12), (1, 50, 5, 3, 24, 7, 11), (2, 30, 16, 8, 128, 7, 6)])
def test_rows_of_a_cache_of_16_bits_read_back(shape, dtype, kv):
    layers, pages, ps, nkv, d, slots, mp = shape
    c = rpp.KvCache(layers, pages, ps, nkv, d, slots, mp, dtype, dev())
    lens, w = [ps, 0, 2 * ps + 1], nkv * d
    cu = ints([0, ps, ps, 3 * ps + 1])
    rpp.kv_reserve(c, ints([2, 0, 1]), ints(lens))
    x = torch.randn(3 * ps + 1, 2 * w, device=dev()).to(TDT[dtype])
    rpp.kv_append(c, layers - 1, x[:, :w], x[:, w:], ints([2, 0, 1]), cu)
    k, v = rpp.kv_read(c, layers - 1, ints([2, 0, 1]), cu, rows=3 * ps + 1)
    assert torch.equal(k, x[:, :w]) and torch.equal(v, x[:, w:]) and k.dtype is TDT[kv]
    k, v = rpp.kv_read(c, layers - 1, ints([1, 2, 1]), starts=ints([2 * ps, 0, 1 if ps > 1 else 0]))
    assert torch.equal(k, x[[3 * ps, 0, ps + (1 if ps > 1 else 0)], :w])
    assert rpp.get_device_error(c.err) == 0


def _some(seed=0, **kw):
    p = Pair(2, 12, 16, 2, 64, 6, 5, seed=seed, **kw)
    p.grow([0, 1], [20, 32])
    p.check()
    return p


def test_append_refusals():
    p = _some()
    k, v, kw, vw = p.rows(40)
    p.ref.append(0, kw[1:21], vw[1:21], [0], [20])                   # 21 rows for 20 tokens: the first has no place
    rpp.kv_append(p.gpu, 0, k, v, ints([0]), ints([0, 21]))
    p.check(od.LENGTH)
    p = _some()
    for slots, cu, code in (([0, 0], [0, 1, 2], od.SLOT), ([0], [0, 41], od.ROWS), ([0], [-1, 1], od.ROWS), ([6], [0, 1], od.SLOT),
                            ([-1], [0, 1], od.SLOT), ([0, 1], [0, 2, 1], od.LENGTH), ([2], [0, 1], od.LENGTH),
                            ([0], [2, 2], None)):
        rpp.kv_append(p.gpu, 0, k, v, ints(slots), ints(cu))
        if code is None:                                             # two rows that are nobody's
            code = od.LENGTH
        p.check(code)
    p.fork([1], [3])
    rpp.kv_append(p.gpu, 0, k[:1], v[:1], ints([1]))                 # its last page is shared now
    p.check(od.PAGE)


def test_read_refusals():
    p = _some()
    w = 2 * 64
    out = torch.full((40, 2 * w), 3.0, dtype=torch.bfloat16, device=dev())

    def read(slots, cu, starts=None):
        rpp.kv_read(p.gpu, 0, ints(slots), None if cu is None else ints(cu), starts=None if starts is None else ints(starts),
                    k=out[:, :w], v=out[:, w:])
        got = rpp.get_device_error(p.gpu.err)
        p.gpu.err.zero_()
        return got
    for slots, cu, starts, code in (([0, 6], [0, 1, 2], None, od.SLOT), ([-1], [0, 1], None, od.SLOT), ([0], [0, 41], None, od.ROWS),
                                    ([0], [-1, 1], None, od.ROWS), ([0, 1], [0, 2, 1], None, od.LENGTH),
                                    ([2], [0, 1], None, od.LENGTH), ([0], [0, 1], [20], od.LENGTH), ([0], [0, 1], [-1], od.LENGTH),
                                    ([0], [0, 1], [2 ** 31 - 1], od.LENGTH), ([0], [0, 2], [2 ** 31 - 1], od.LENGTH)):
        assert read(slots, cu, starts) == code, (slots, cu, starts)
        assert (out == 3).all()
    assert read([0], [0, 25]) == od.LENGTH                           # 5 rows too many: those have no place
    assert (out[:5] == 3).all()
    p.gpu.table[0, 1] = 12                                           # one past the pool
    out.fill_(3.0)
    assert read([0], [0, 4]) == od.PAGE
    assert (out == 3).all()
    p.gpu.err.fill_(9)
    rpp.kv_read(p.gpu, 0, ints([1]), k=out[:1, :w], v=out[:1, w:])
    assert (out == 3).all()


def test_a_corrupt_page_number_is_skipped():
    p = _some()
    p.gpu.table[0, 1] = 12                                           # one past the pool
    k, v, _, _ = p.rows(1)
    before = p.gpu.pool.clone(), p.gpu.scales.clone()
    for call in (lambda: rpp.kv_append(p.gpu, 0, k, v, ints([0])), lambda: rpp.kv_fork(p.gpu, ints([0]), ints([2])),
                 lambda: rpp.kv_compact(p.gpu)):
        p.gpu.err.zero_()
        call()
        assert rpp.get_device_error(p.gpu.err) == od.PAGE
        assert torch.equal(raw_t(p.gpu.pool), raw_t(before[0])) and torch.equal(p.gpu.scales, before[1])


def raw_t(t):
    return t.view(torch.uint8)


def test_a_set_error_word_stops_every_call():
    p = _some()
    p.gpu.err.fill_(42)
    k, v, _, _ = p.rows(1)
    rpp.kv_reserve(p.gpu, ints([2]), ints([3]))
    rpp.kv_append(p.gpu, 0, k, v, ints([0]))
    rpp.kv_fork(p.gpu, ints([0]), ints([2]))
    rpp.kv_free(p.gpu, ints([0]))
    rpp.kv_compact(p.gpu)
    p.check(42)


def test_arguments_of_the_binding():
    p = _some()
    c = p.gpu
    k, v, _, _ = p.rows(2)
    with pytest.raises(ValueError):
        rpp.kv_append(c, 0, k.float(), v.float(), ints([0, 1]))
    with pytest.raises(ValueError):
        rpp.kv_append(c, 0, k, v.half(), ints([0, 1]))
    with pytest.raises(ValueError):
        rpp.kv_read(c, 0, ints([0]), ints([0, 1]))                    # rows not given
    with pytest.raises(ValueError):
        rpp.kv_read(c, 0, ints([0]), k=k)
    with pytest.raises(ValueError):
        rpp.kv_read(c, 0, ints([0]), dtype="fp32")
    wide = rpp.KvCache(1, 4, 16, 2, 64, 2, 2, "bf16", dev())
    with pytest.raises(ValueError):
        rpp.kv_read(wide, 0, ints([0]), dtype="fp16")                 # it has bf16 rows
    with pytest.raises(ValueError):
        rpp.kv_read(c, 0, ints([0]), starts=ints([0, 1]))
    for bad in (c.scales[..., :0], c.scales.cpu(), c.scales.to(torch.int8), c.scales[:1], c.scales.transpose(0, 1)):
        with pytest.raises(ValueError):
            rpp.KvCache8.from_tensors(c.pool, bad, c.table, c.lens, c.refs)
    with pytest.raises(ValueError):
        rpp.KvCache8.from_tensors(c.pool.view(torch.uint8), c.scales, c.table, c.lens, c.refs)
    with pytest.raises(ValueError):
        rpp.KvCache8(1, 4, 16, 1, 64, 2, 2, dtype="fp16", device=dev())
    with pytest.raises(ValueError):
        rpp.KvCache8(1, 4, 16, 1, 64, 2, 2, block=32, device=dev())
    with pytest.raises(rpp.RppError):
        rpp.KvCache8(1, 4, 16, 1, 96, 2, 2, device=dev())


def test_a_captured_step_replays():
    """free, reserve, append and read captured once; replays with other slots, counts and rows in the same buffers."""
    p = Pair(1, 60, 16, 2, 64, 8, 10, kind="int8", block=8)
    slots, counts, cu = ints([0, 1, 2]), ints([5, 20, 1]), ints([0, 5, 25, 26])
    k = torch.empty(64, 128, dtype=torch.bfloat16, device=dev())
    v, ko, vo = torch.empty_like(k), torch.empty_like(k), torch.empty_like(k)
    gone = ints([7])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            rpp.kv_free(p.gpu, gone)
            rpp.kv_reserve(p.gpu, slots, counts)
            rpp.kv_append(p.gpu, 0, k, v, slots, cu)
            rpp.kv_read(p.gpu, 0, slots, cu, k=ko, v=vo)
    torch.cuda.synchronize()
    p.check()
    r = np.random.default_rng(3)
    for step in range(6):
        sl = [int(x) for x in r.permutation(7)[:3]]
        ct = [int(x) for x in r.integers(0, 20, 3)]
        leave = int(r.integers(0, 8))
        kg, vg, kw, vw = p.rows(64)
        k.copy_(kg)
        v.copy_(vg)
        slots.copy_(ints(sl))
        counts.copy_(ints(ct))
        cu.copy_(ints([0] + np.cumsum(ct).tolist()))
        gone.copy_(ints([leave]))
        g.replay()
        p.ref.free([leave])
        p.ref.reserve(sl, ct)
        p.ref.append(0, kw, vw, sl, ct)
        p.check()
        at = 0
        for a, n in zip(sl, ct):
            want = p.expect(0, a, p.ref.lens[a] - n, p.ref.lens[a], "bf16") if n else [ko[:0].cpu()] * 2
            assert torch.equal(ko[at:at + n].cpu(), want[0]) and torch.equal(vo[at:at + n].cpu(), want[1])
            at += n


def test_the_longest_lists():
    n = 4096
    p = Pair(1, 4200, 16, 1, 64, 2 * n, 1, kind="e4m3", block=16)
    r = np.random.default_rng(1)
    slots = [int(x) for x in r.permutation(2 * n)[:n]]
    p.grow(slots, [int(x) for x in r.integers(0, 3, n)])
    p.grow(slots, [1] * n)
    p.check()
    k, _ = rpp.kv_read(p.gpu, 0, ints(slots))
    for i in (0, 1, 2047, 4095):
        a = p.ref.lens[slots[i]]
        assert torch.equal(k[i:i + 1].cpu(), p.expect(0, slots[i], a - 1, a, "bf16")[0])


def test_a_given_stream():
    """Rows made, written and read on a stream of the call's own, its memory among it."""
    p = Pair(1, 300, 16, 4, 128, 8, 64, kind="e4m3")
    s = torch.cuda.Stream()
    k, v, kw, vw = p.rows(600)
    slots, counts, cu = ints([0, 1]), ints([500, 100]), ints([0, 500, 600])
    torch.cuda.synchronize()
    rpp.kv_reserve(p.gpu, slots, counts, stream=s)
    rpp.kv_append(p.gpu, 0, k, v, slots, cu, stream=s)
    ko, vo = rpp.kv_read(p.gpu, 0, slots, cu, rows=600, dtype=torch.float16, stream=s)
    s.synchronize()
    p.ref.reserve([0, 1], [500, 100])
    p.ref.append(0, kw, vw, [0, 1], [500, 100])
    p.check()
    want = p.expect(0, 0, 0, 500, "fp16")
    assert torch.equal(ko[:500].cpu(), want[0]) and torch.equal(vo[:500].cpu(), want[1])


def test_pages_past_32_bits():
    """Offsets of codes above 2^32 bytes: one layer of 4.6 GB."""
    pages = 140000
    c = rpp.KvCache8(1, pages, 16, 8, 128, 4, 4, "int8", 16, dev())
    c.refs[:pages - 3] = 1
    rpp.kv_reserve(c, ints([1]), ints([40]))
    assert c.table[1, :3].tolist() == [pages - 3, pages - 2, pages - 1]
    x = torch.randn(40, 2048, device=dev(), dtype=torch.float16)
    rpp.kv_append(c, 0, x[:, :1024], x[:, 1024:], ints([1]), ints([0, 40]))
    k, v = rpp.kv_read(c, 0, ints([1]), ints([0, 40]), rows=40, dtype="fp16")
    assert rpp.get_device_error(c.err) == 0
    step = 2.0 ** (torch.floor(torch.log2(x.view(40, 16, 128).float().abs().amax(-1))) - 6)
    for got, part in ((k, step[:, :8]), (v, step[:, 8:])):
        src = x[:, :1024] if got is k else x[:, 1024:]
        # the block's step is at most its largest row's, doubled where that passes 127.5 steps
        limit = torch.cat([part[a:a + 16].amax(0, keepdim=True).expand(min(16, 40 - a), 8) for a in (0, 16, 32)])
        assert ((got.float() - src.float()).abs().view(40, 8, 128) <= limit[..., None]).all()
