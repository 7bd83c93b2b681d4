"""The paged key-value cache on the GPU against the list-kept oracle: every array of the state, bit for bit, after
each call; refused calls change nothing (or only what they say) and record their error."""
import numpy as np
import pytest
import torch

import oracle.decoder as od
import remove_padding_prefix_gb300 as rpp
from gpu_util import TDT, dev

pytestmark = pytest.mark.gpu


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=dev())


def words(t):
    return t.view(torch.int16).cpu().numpy().view(np.uint16)


class Pair:
    """A cache on the GPU and the oracle's, driven together."""

    def __init__(self, layers, pages, ps, nkv, d, slots, max_pages, dtype="bf16", seed=0):
        self.rng = np.random.default_rng(seed)
        self.dtype, self.nkv, self.d, self.layers = dtype, nkv, d, layers
        self.gpu = rpp.KvCache(layers, pages, ps, nkv, d, slots, max_pages, dtype, dev())
        self.ref = od.PagedCache(layers, pages, ps, nkv, d, slots, max_pages)
        start = self.rng.integers(0, 1 << 16, self.ref.pool.shape, dtype=np.uint16)   # whatever memory held
        self.ref.pool[:] = start
        self.gpu.pool.copy_(torch.from_numpy(start.view(np.int16)).to(dev()).view(TDT[dtype]))

    def rows(self, n, pad=0):
        """n rows of K | V as columns of wider rows: (device k, device v, words k, words v)."""
        w = self.nkv * self.d
        x = self.rng.integers(0, 1 << 16, (n, 2 * w + pad), dtype=np.uint16)
        g = torch.from_numpy(x.view(np.int16)).to(dev()).view(TDT[self.dtype])
        k, v = x[:, pad:pad + w], x[:, pad + w:]
        return g[:, pad:pad + w], g[:, pad + w:], k.reshape(n, self.nkv, self.d), v.reshape(n, self.nkv, self.d)

    def grow(self, slots, counts, pad=0):
        rpp.kv_reserve(self.gpu, ints(slots), ints(counts))
        self.ref.reserve(slots, counts)
        cu = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        for layer in range(self.layers):
            k, v, kw, vw = self.rows(int(cu[-1]) + 3, pad)     # three rows behind the last sequence
            rpp.kv_append(self.gpu, layer, k, v, ints(slots), ints(cu.tolist()))
            self.ref.append(layer, kw, vw, slots, counts)

    def fork(self, src, dst):
        rpp.kv_fork(self.gpu, ints(src), ints(dst))
        self.ref.fork(src, dst)

    def free(self, slots):
        rpp.kv_free(self.gpu, ints(slots))
        self.ref.free(slots)

    def compact(self, apart=False):
        old = (self.gpu.table.clone(), self.gpu.refs.clone())
        remap = torch.full((self.gpu.cfg.pages,), 77, dtype=torch.int32, device=dev())
        if apart:
            outs = dict(table_out=torch.empty_like(old[0]), refs_out=torch.empty_like(old[1]))
        else:
            outs = {}
        table, refs, live = rpp.kv_compact(self.gpu, remap=remap, **outs)
        if apart:
            assert torch.equal(self.gpu.table, old[0]) and torch.equal(self.gpu.refs, old[1])
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
        np.testing.assert_array_equal(words(self.gpu.pool), self.ref.pool)


SHAPES = [
    # layers, pages, page rows, kv heads, head size, slots, pages a sequence
    (1, 40, 16, 2, 64, 6, 9),
    (3, 301, 16, 8, 128, 12, 40),
    (2, 37, 1, 1, 8, 6, 12),        # a page of one row, the smallest head
    (2, 50, 5, 3, 24, 7, 11),       # odd sizes
    (1, 130, 48, 4, 64, 40, 7),
]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_calls_one_by_one(shape, dtype):
    p = Pair(*shape, dtype=dtype)
    ps, mp = shape[2], shape[6]
    p.grow([1], [1])
    p.check()
    p.grow([3, 0], [ps, 0])                      # a whole page; a count of zero
    p.check()
    p.grow([0, 1, 2], [2 * ps + 1, ps - 1, 1], pad=8)
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
    p.check()
    p.grow([0], [mp * ps])                       # the longest sequence
    p.check()
    p.free(list(range(len(p.ref.lens))))
    p.compact()                                  # nothing in use
    p.check()


@pytest.mark.parametrize("shape,steps", [((2, 90, 16, 2, 64, 9, 14), 60), ((1, 700, 4, 1, 16, 33, 60), 60),
                                         ((1, 9000, 1, 1, 8, 64, 400), 25)])
def test_random_calls(shape, steps):
    """A seeded walk through the calls; pages of 9000 pass the stretch of a warp several times."""
    p = Pair(*shape, seed=steps)
    r = np.random.default_rng(7)
    slots, cap = shape[5], shape[2] * shape[6]
    for _ in range(steps):
        what = r.integers(0, 10)
        pick = [int(s) for s in r.permutation(slots)[:r.integers(1, slots + 1)]]
        room = sum(1 for x in p.ref.refs if x == 0)
        if what < 5:
            counts = [int(min(r.integers(0, cap // 3), cap - p.ref.lens[s])) for s in pick]
            need = sum(-(-(p.ref.lens[s] + c) // p.ref.ps) - len(p.ref.rows[s]) for s, c in zip(pick, counts))
            if need <= room:
                p.grow(pick, counts)
            else:
                rpp.kv_reserve(p.gpu, ints(pick), ints(counts))
                p.check(od.FULL)
        elif what < 7:
            empty = [s for s in pick if p.ref.lens[s] == 0]
            full = [s for s in range(slots) if p.ref.lens[s]]
            if empty and full and len(empty) <= room:
                p.fork([int(x) for x in r.choice(full, len(empty))], empty)
        elif what < 9:
            p.free(pick)
        else:
            p.compact(apart=bool(r.integers(0, 2)))
        p.check()


def test_one_row_each_without_cu_seqlens():
    p = Pair(2, 20, 16, 2, 64, 6, 5)
    slots = [4, 0, 2]
    rpp.kv_reserve(p.gpu, ints(slots), ints([1, 1, 1]))
    p.ref.reserve(slots, [1, 1, 1])
    k, v, kw, vw = p.rows(3)
    rpp.kv_append(p.gpu, 1, k, v, ints(slots))
    p.ref.append(1, kw, vw, slots, [1, 1, 1])
    p.check()


def _some(seed=0):
    p = Pair(2, 12, 16, 2, 64, 6, 5, seed=seed)
    p.grow([0, 1], [20, 32])
    p.check()
    return p


@pytest.mark.parametrize("slots,counts,code", [
    ([0, 6], [1, 1], od.SLOT), ([-1], [1], od.SLOT), ([2, 3, 2], [1, 1, 1], od.SLOT),
    ([2], [-1], od.LENGTH), ([0], [61], od.LENGTH), ([0], [2**31 - 1], od.LENGTH),
    ([2, 3], [80, 60], od.FULL),
])
def test_reserve_refusals(slots, counts, code):
    p = _some()
    with pytest.raises(od.CacheError) as e:
        p.ref.reserve(slots, counts)
    assert e.value.code == code
    rpp.kv_reserve(p.gpu, ints(slots), ints(counts))
    p.check(code)


@pytest.mark.parametrize("src,dst,code", [
    ([0], [1], od.SLOT), ([0], [0], od.SLOT), ([0, 1], [2, 2], od.SLOT), ([9], [2], od.SLOT), ([0], [-3], od.SLOT),
    ([2, 0], [3, 2], od.SLOT), ([0] * 4, [2, 3, 4, 5], None),
])
def test_fork_refusals(src, dst, code):
    p = _some()
    if code is None:
        p.fork(src, dst)          # one source several times
        p.check()
        return
    with pytest.raises(od.CacheError):
        p.ref.fork(src, dst)
    rpp.kv_fork(p.gpu, ints(src), ints(dst))
    p.check(code)


def test_fork_without_a_free_page():
    p = Pair(1, 4, 16, 1, 64, 4, 4)
    p.grow([0], [3 * 16 + 1])
    rpp.kv_fork(p.gpu, ints([0]), ints([1]))
    p.check(od.FULL)


@pytest.mark.parametrize("slots", [[0, 0], [6], [-1, 0]])
def test_free_refusals(slots):
    p = _some()
    rpp.kv_free(p.gpu, ints(slots))
    p.check(od.SLOT)


def test_append_refusals():
    p = _some()
    k, v, _, _ = p.rows(40)
    rpp.kv_append(p.gpu, 0, k, v, ints([0]), ints([0, 21]))          # 21 rows for 20 tokens: the first has no place
    assert rpp.get_device_error(p.gpu.err) == od.LENGTH
    p = _some()
    rpp.kv_append(p.gpu, 0, k, v, ints([0, 0]), ints([0, 1, 2]))
    p.check(od.SLOT)
    rpp.kv_append(p.gpu, 0, k, v, ints([0]), ints([0, 41]))          # more rows than there are
    p.check(od.ROWS)
    rpp.kv_append(p.gpu, 0, k, v, ints([2]), ints([0, 1]))           # an empty slot
    p.check(od.LENGTH)
    p.fork([1], [3])
    rpp.kv_append(p.gpu, 0, k[:1], v[:1], ints([1]))                 # its last page is shared now
    p.check(od.PAGE)


def test_a_corrupt_page_number_is_skipped():
    p = _some()
    p.gpu.table[0, 1] = 12                                           # one past the pool
    k, v, _, _ = p.rows(1)
    before = p.gpu.pool.clone()
    rpp.kv_append(p.gpu, 0, k, v, ints([0]))
    assert rpp.get_device_error(p.gpu.err) == od.PAGE
    assert torch.equal(words_t(p.gpu.pool), words_t(before))
    for call in (lambda: rpp.kv_fork(p.gpu, ints([0]), ints([2])), lambda: rpp.kv_compact(p.gpu),
                 lambda: rpp.kv_free(p.gpu, ints([0]))):
        p.gpu.err.zero_()
        call()
        assert rpp.get_device_error(p.gpu.err) == od.PAGE


def words_t(t):
    return t.view(torch.int16)


def test_a_set_error_word_stops_every_call():
    p = _some()
    p.gpu.err.fill_(42)
    k, v, _, _ = p.rows(1)
    table = torch.full_like(p.gpu.table, 5)
    rpp.kv_reserve(p.gpu, ints([2]), ints([3]))
    rpp.kv_append(p.gpu, 0, k, v, ints([0]))
    rpp.kv_fork(p.gpu, ints([0]), ints([2]))
    rpp.kv_free(p.gpu, ints([0]))
    rpp.kv_compact(p.gpu, table_out=table, refs_out=torch.zeros_like(p.gpu.refs))
    assert (table == 5).all()
    p.check(42)


def test_a_captured_step_replays():
    """reserve, append and free captured once; replays with other slots, counts and rows in the same buffers."""
    p = Pair(1, 60, 16, 2, 64, 8, 10)
    slots, counts, cu = ints([0, 1, 2]), ints([5, 20, 1]), ints([0, 5, 25, 26])
    k = torch.empty(64, 128, dtype=torch.bfloat16, device=dev())
    v = torch.empty_like(k)
    gone = ints([7])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            rpp.kv_free(p.gpu, gone)
            rpp.kv_reserve(p.gpu, slots, counts)
            rpp.kv_append(p.gpu, 0, k, v, slots, cu)
    torch.cuda.synchronize()
    p.check()
    r = np.random.default_rng(3)
    for step in range(6):
        sl = [int(x) for x in r.permutation(7)[:3]]
        ct = [int(x) for x in r.integers(0, 20, 3)]
        leave = int(r.integers(0, 8))
        _, _, kw, vw = rows = p.rows(64)
        k.copy_(rows[0])
        v.copy_(rows[1])
        slots.copy_(ints(sl))
        counts.copy_(ints(ct))
        cu.copy_(ints([0] + np.cumsum(ct).tolist()))
        gone.copy_(ints([leave]))
        g.replay()
        p.ref.free([leave])
        p.ref.reserve(sl, ct)
        p.ref.append(0, kw, vw, sl, ct)
        p.check()


def test_rows_before_the_first_sequence():
    p = _some()
    k, v, _, _ = p.rows(4)
    before = p.gpu.pool.clone()
    rpp.kv_append(p.gpu, 0, k[:2], v[:2], ints([0]), ints([2, 2]))   # two rows that are nobody's
    assert rpp.get_device_error(p.gpu.err) == od.LENGTH
    assert torch.equal(words_t(p.gpu.pool), words_t(before))


def test_one_page():
    p = Pair(1, 1, 16, 1, 64, 2, 1)
    p.compact()
    p.grow([1], [16])
    p.compact()
    p.check()
    rpp.kv_reserve(p.gpu, ints([0]), ints([1]))
    p.check(od.FULL)
    p.free([1])
    p.compact(apart=True)
    p.check()


def test_the_longest_lists():
    n = 4096
    p = Pair(1, 9000, 4, 1, 8, 2 * n, 3)
    r = np.random.default_rng(1)
    slots = [int(x) for x in r.permutation(2 * n)[:n]]
    p.grow(slots, [int(x) for x in r.integers(0, 7, n)])
    p.check()
    rest = [s for s in range(2 * n) if p.ref.lens[s] == 0][:n]
    held = [s for s in slots if p.ref.lens[s]]
    p.fork([held[int(x)] for x in r.integers(0, len(held), n)], rest)
    p.check()
    p.free(slots)
    p.check()
    p.compact()
    p.check()


def test_offsets_past_32_bits():
    """A pool of over 2^32 elements, the low pages taken: everything happens behind them."""
    pages, nkv, d, ps = 150000, 8, 128, 16
    c = rpp.KvCache(1, pages, ps, nkv, d, 6, 40, "bf16", dev())
    assert c.pool.numel() > 1 << 32
    held = 140000
    c.refs[:held] = 1
    g = torch.Generator(device=dev()).manual_seed(0)
    rpp.kv_reserve(c, ints([1, 4]), ints([600, 9]))
    x = torch.randn(609, 2 * nkv * d, generator=g, device=dev()).bfloat16()
    rpp.kv_append(c, 0, x[:, :nkv * d], x[:, nkv * d:], ints([1, 4]), ints([0, 600, 609]))
    rpp.kv_fork(c, ints([1]), ints([0]))

    def rows(slot, n):
        t = c.table[slot, :-(-n // ps)].long()
        return c.pool[0, t].permute(1, 0, 3, 2, 4).reshape(2, -1, nkv * d)[:, :n]

    def same():
        for slot, at, n in ((1, 0, 600), (4, 600, 9), (0, 0, 600)):
            assert torch.equal(rows(slot, n)[0], x[at:at + n, :nkv * d])
            assert torch.equal(rows(slot, n)[1], x[at:at + n, nkv * d:])

    assert int(c.table[1, 0]) == held and int(c.table[0].max()) >= held
    same()
    q = torch.randn(3, 16 * d, generator=g, device=dev()).bfloat16()
    out = rpp.attention_decode(c, 0, q, ints([1, 4, 0]))
    for i, (at, n) in enumerate(((0, 600), (600, 9), (0, 600))):
        K, V = (y.double().view(n, nkv, d) for y in (x[at:at + n, :nkv * d], x[at:at + n, nkv * d:]))
        z = torch.einsum("hgd,nhd->hgn", q[i].double().view(nkv, 2, d), K) * d ** -0.5
        ref = torch.einsum("hgn,nhd->hgd", torch.softmax(z, -1), V).flatten()
        # a rounding of the output, and 2^-10 of the largest value for the rest (test_gpu_decode.py derives less)
        assert ((out[i].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -10 * V.abs().max()).all()
    rpp.kv_free(c, ints([4]))
    c.refs[100:200] = 0                              # holes far below
    rpp.kv_compact(c)
    assert rpp.get_device_error(c.err) == 0
    assert int(c.table[1].max()) < held and int(c.table[1, :38].min()) >= 0
    for slot in (1, 0):
        assert torch.equal(rows(slot, 600)[0], x[:600, :nkv * d]) and torch.equal(rows(slot, 600)[1], x[:600, nkv * d:])


@pytest.mark.parametrize("name", ["table_out", "refs_out"])
def test_compact_writes_the_caches_own_table_and_counts_or_neither(name):
    p = _some()
    own = p.gpu.table if name == "table_out" else p.gpu.refs
    with pytest.raises(rpp.RppError):
        rpp.kv_compact(p.gpu, **{name: torch.empty_like(own)})
    p.check()


def test_compact_with_one_corrupt_table_entry_moves_the_others():
    """One page number outside the pool: the other sequences' rows are where the new table says,
    whichever CTAs of the move start after the error word is set."""
    p = Pair(2, 600, 16, 2, 64, 40, 32)
    order = np.random.default_rng(4).permutation(40)
    p.grow([int(s) for s in order], [16 * 14 + int(s) % 16 for s in order])
    p.free([int(s) for s in order[:20]])
    p.gpu.table[int(order[20]), 0] = 600
    old = {int(s): p.gpu.table[int(s)].clone() for s in order[21:]}
    pool = p.gpu.pool.clone()
    table, refs, live = rpp.kv_compact(p.gpu)
    assert rpp.get_device_error(p.gpu.err) == od.PAGE
    n = int(live)
    for s, row in old.items():
        used = -(-int(p.gpu.lens[s]) // 16)
        new = table[s, :used].long()
        assert (new < n).all() and (new >= 0).all()
        assert torch.equal(words_t(p.gpu.pool[:, new]), words_t(pool[:, row[:used].long()]))


def test_fork_with_one_corrupt_source_carries_out_the_others():
    """Page numbers outside the pool in two of the sources, and more pairs than CTAs that run at once: every
    other destination is as the oracle has it, and so are all lengths and the counts of all pages."""
    n = 3000
    p = Pair(1, 9000, 4, 1, 8, 2 * n, 4)
    held = list(range(40))
    p.grow(held, [4 * (s % 3) + 1 + s % 4 for s in held])
    p.check()
    src = [int(x) for x in np.random.default_rng(2).integers(0, 40, n)]
    src[:2] = [10, 5]                                     # of 7 rows and 10: a whole page and a part, two and a part
    dst = list(range(n, 2 * n))
    assert (p.ref.lens[10], p.ref.lens[5]) == (7, 10)
    whole = p.ref.rows[5][0]
    p.gpu.table[5, 0] = 9000
    p.gpu.table[10, 1] = -7
    before = p.ref.pool.copy()
    p.fork(src, dst)
    p.ref.refs[whole] = 1                                 # nobody could share it
    for s, t in [(s, s) for s in held] + list(zip(src, dst)):
        if s == 5:
            p.ref.rows[t][0] = 9000                       # the wrong number goes with the copy
        if s == 10 and t != s:                            # a page of its own, with no rows to copy
            own = p.ref.rows[t][1]
            p.ref.pool[:, own] = before[:, own]
    p.ref.rows[10][1] = -7
    p.check(od.PAGE)


def test_a_refused_fork_leaves_forks_of_before_alone():
    """Again the same fork: the destinations are not empty, and what they have written since stays."""
    p = _some()
    p.fork([0], [2])
    k, v, kw, vw = p.rows(1)
    rpp.kv_append(p.gpu, 0, k, v, ints([2]))
    p.ref.append(0, kw, vw, [2], [1])
    p.check()
    rpp.kv_fork(p.gpu, ints([0]), ints([2]))
    p.check(od.SLOT)


@pytest.mark.parametrize("cu,code", [([0, 5, 3, 8], od.LENGTH), ([0, 8, 5, 5], od.LENGTH), ([0, 2, 2, 1], od.LENGTH),
                                     ([-2, 3, 4, 5], od.ROWS)])
def test_append_with_cu_seqlens_that_step_back(cu, code):
    """A negative count, as for reserve, or rows before the first: nothing is written."""
    p = Pair(1, 12, 16, 2, 64, 4, 5)
    p.grow([0, 1, 2], [20, 20, 20])
    k, v, _, _ = p.rows(40)
    rpp.kv_append(p.gpu, 0, k, v, ints([0, 1, 2]), ints(cu))
    p.check(code)


def test_append_with_a_step_back_far_down_the_list():
    n = 1000
    p = Pair(1, 1100, 2, 1, 8, n, 2)
    p.grow(list(range(n)), [2] * n)
    k, v, _, _ = p.rows(n)
    cu = list(range(n + 1))
    cu[700] -= 2
    rpp.kv_append(p.gpu, 0, k, v, ints(list(range(n))), ints(cu))
    p.check(od.LENGTH)


def test_fork_of_an_empty_sequence():
    p = _some()
    p.fork([3, 0, 3], [2, 4, 5])
    p.check()
    p.grow([2, 5], [17, 3])
    p.check()
