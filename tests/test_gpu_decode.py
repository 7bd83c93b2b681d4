"""Attention of one new token over the paged cache, against fp64.

Tolerance, per output element, from the arithmetic (e = eps of the output type; V the
sequence's values of that head, k its keys):
  * the final rounding: e / 2 of the value;
  * a score is an fp32 sum of d exact products, off by at most (d + 2) 2^-24 sum |q_c k_c|,
    and enters as exp(scale s): twice that, times max |V|, on the weighted mean;
  * exp2 (2^-22), the base change of a score of magnitude z (2^-23 z), P kept to two 16-bit parts
    (2^-17), and fp32 sums over n keys (n 2^-24): each times max |V|, twice (numerator and sum).
"""
import numpy as np
import pytest
import torch

import oracle.decoder as od
import remove_padding_prefix_gb300 as rpp
from gpu_util import TDT, dev

pytestmark = pytest.mark.gpu

EPS = {"fp16": 2.0 ** -10, "bf16": 2.0 ** -7}


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=dev())


def make(dtype, lens, nkv, d, ps, seed=0, layers=1, spare=5, extra_pages=1, nan=True):
    """A cache of sequences on shuffled pages; what no sequence has written holds NaN."""
    rng = np.random.default_rng(seed)
    need = [-(-n // ps) for n in lens]
    pages = sum(need) + spare
    mp = max(need + [1]) + extra_pages
    c = rpp.KvCache(layers, pages, ps, nkv, d, len(lens) + 2, mp, dtype, dev())
    order = rng.permutation(pages)
    table = np.full((len(lens) + 2, mp), -1, np.int32)
    refs = np.zeros(pages, np.int32)
    g = torch.Generator(device=dev()).manual_seed(seed)
    pool = torch.randn(c.pool.shape, generator=g, device=dev()).to(TDT[dtype])
    keep = torch.zeros((pages, ps), dtype=torch.bool)
    at = 0
    for s, n in enumerate(lens):
        for j in range(need[s]):
            p = int(order[at])
            at += 1
            table[s, j] = p
            refs[p] = 1
            keep[p, :n - j * ps] = True
    if nan:
        pool = torch.where(keep.to(dev())[None, :, None, None, :, None], pool, torch.full_like(pool, float("nan")))
    c.pool.copy_(pool)
    c.table.copy_(torch.from_numpy(table))
    c.lens[:len(lens)] = ints(lens)
    c.refs.copy_(torch.from_numpy(refs))
    return c


def sequence(c, layer, slot):
    """fp64 K and V [len, kv heads, d] of a slot (on the GPU: the long cases are large)."""
    n, ps = int(c.lens[slot]), c.cfg.page_size
    x = c.pool[layer, c.table[slot, :-(-n // ps)].long()].double()
    x = x.permute(1, 0, 3, 2, 4).reshape(2, -1, c.cfg.kv_heads, c.cfg.head_dim)
    return x[0, :n], x[1, :n]


def check(got, q, c, layer, slots, nh, scale=None):
    d, nkv = c.cfg.head_dim, c.cfg.kv_heads
    per = nh // nkv
    scale = d ** -0.5 if scale is None else scale
    e = EPS["fp16" if q.dtype is torch.float16 else "bf16"]
    assert rpp.get_device_error(c.err) == 0
    assert torch.isfinite(got.float()).all()
    for i, s in enumerate(slots):
        n = int(c.lens[s])
        if n == 0:
            assert (got[i] == 0).all()
            continue
        K, V = sequence(c, layer, s)
        qi = q[i].double().view(nkv, per, d)
        z = torch.einsum("hgd,nhd->hgn", qi, K) * scale
        ref = torch.einsum("hgn,nhd->hgd", torch.softmax(z, -1), V)
        mag = (torch.einsum("hgd,nhd->hgn", qi.abs(), K.abs()) * scale).amax(-1)          # [nkv, per]
        vmax = V.abs().amax(0).amax(-1)[:, None]
        ds = (d + 2) * 2.0 ** -24 * mag + 2.0 ** -23 * z.abs().amax(-1)
        bound = vmax * (2 * ds + 2 * (2.0 ** -22 + 2.0 ** -17 + n * 2.0 ** -24))
        off = (got[i].double().view(nkv, per, d) - ref).abs()
        limit = e / 2 * ref.abs() + bound[..., None] + 2.0 ** -25    # fp16: half a step of its smallest values
        assert (off <= limit).all(), (i, s, n, float((off - limit).max()), float((off / limit).max()))


def queries(n, nh, d, dtype, seed=1, scale=1.0):
    g = torch.Generator(device=dev()).manual_seed(seed)
    wide = (scale * torch.randn((n, nh * d + 64), generator=g, device=dev())).to(TDT[dtype])
    return wide[:, 64:]          # columns of wider rows


LENS = [1, 2, 15, 16, 17, 31, 32, 33, 0, 47, 48, 63, 64, 65, 100, 127, 128, 129, 255, 257, 0, 500, 1023]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nh,nkv,ps", [(8, 8, 16), (32, 8, 16), (12, 12, 32), (5, 1, 48), (16, 2, 64), (40, 2, 16), (33, 1, 16),
                                       (7, 7, 128), (12, 4, 16)])
def test_lengths_and_heads(dtype, d, nh, nkv, ps):
    c = make(dtype, LENS, nkv, d, ps, seed=nh + ps)
    slots = list(np.random.default_rng(2).permutation(len(LENS)))
    q = queries(len(slots), nh, d, dtype, scale=2.0)
    check(rpp.attention_decode(c, 0, q, ints([int(s) for s in slots])), q, c, 0, slots, nh)


@pytest.mark.parametrize("dtype,d,nh,nkv,ps,lens", [
    ("bf16", 128, 32, 8, 16, [40001]), ("fp16", 64, 16, 16, 64, [70000]), ("bf16", 64, 16, 1, 16, [30000, 1, 30000]),
    ("fp16", 128, 8, 8, 16, [9000, 3, 0, 8191]),
])
def test_long(dtype, d, nh, nkv, ps, lens):
    c = make(dtype, lens, nkv, d, ps)
    q = queries(len(lens), nh, d, dtype)
    check(rpp.attention_decode(c, 0, q), q, c, 0, range(len(lens)), nh)


@pytest.mark.parametrize("n,hi,nh,nkv", [(300, 40, 8, 2), (1000, 5, 4, 4), (4096, 20, 2, 1)])
def test_many_short(n, hi, nh, nkv):
    lens = [int(x) for x in np.random.default_rng(n).integers(0, hi, n)]
    c = make("bf16", lens, nkv, 64, 16)
    q = queries(n, nh, 64, "bf16")
    got = rpp.attention_decode(c, 0, q)
    check(got[:400], q[:400], c, 0, range(min(n, 400)), nh)
    check(got[-200:], q[-200:], c, 0, range(n - 200, n), nh)


def test_nothing_to_attend_to():
    c = make("bf16", [0, 0, 0], 4, 128, 16)
    q = queries(3, 8, 128, "bf16")
    out = torch.full((3, 1024), float("nan"), dtype=torch.bfloat16, device=dev())
    rpp.attention_decode(c, 0, q, out=out)
    check(out, q, c, 0, range(3), 8)


def test_layer_scale_and_the_same_slot_twice():
    c = make("fp16", [40, 300, 7], 2, 64, 16, layers=3)
    q = queries(4, 6, 64, "fp16")
    slots = [1, 1, 0, 2]
    check(rpp.attention_decode(c, 2, q, ints(slots), scale=0.31), q, c, 2, slots, 6, 0.31)


def test_uneven_scores():
    """Scores that climb through the sequence by far more than the lazily moved maximum allows, and keys as
    large as -60000 in fp16."""
    c = make("fp16", [3000, 1], 2, 64, 16)
    n = 3000
    pages = c.table[0, :-(-n // 16)].long()
    ramp = torch.linspace(-30, 30, n, device=dev())
    k = c.pool[0, pages, 0]                                        # [pages, heads, 16, d]
    k[:] = 0
    k.permute(0, 2, 1, 3).reshape(-1, 2, 64)[:n, :, 0] = 0
    rows = torch.zeros(pages.numel() * 16, 2, 64, device=dev())
    rows[:n, :, 0] = ramp[:, None]
    rows[5, :, 0] = -60000.0
    c.pool[0, pages, 0] = rows.view(-1, 16, 2, 64).permute(0, 2, 1, 3).half()
    q = torch.zeros(2, 4 * 64, device=dev(), dtype=torch.float16)
    q[:, ::64] = 8.0
    check(rpp.attention_decode(c, 0, q), q, c, 0, [0, 1], 4)


def test_many_weights_far_below_the_maximum():
    """65536 fp16 keys, the first 26 powers of two above the others in weight: together those are
    2^-10 of the sum, and the output is theirs (the first value is 0, theirs 1).  Queries enough that
    a warp has a sequence whole.

    Tolerance: the output's rounding, 2^-11 of it; weights of up to 2^8 are kept 2^7 times as large,
    so what is below fp16's smallest step, 2^-24, is half a step of 2^-7 of it off: n 2^-32; fp32
    sums of n like terms, n 2^-24 of each of numerator and denominator; 2^-16 for the exponent, 26 2^-23 off."""
    n, rows = 65536, 2048
    c = make("fp16", [n], 1, 64, 64, nan=False)
    c.pool[0, :, 0] = 0
    c.pool[0, :, 1] = 1
    first = int(c.table[0, 0])
    c.pool[0, first, 0, 0, 0, 0] = 18.02                            # score 8 * 18.02 / 8, e^-18.02 = 2^-26
    c.pool[0, first, 1, 0, 0] = 0
    q = torch.zeros(rows, 64, device=dev(), dtype=torch.float16)
    q[:, 0] = 8.0
    got = rpp.attention_decode(c, 0, q, torch.zeros(rows, dtype=torch.int32, device=dev())).double()
    assert rpp.get_device_error(c.err) == 0
    w = torch.exp(-c.pool[0, first, 0, 0, 0, 0].double()) * (n - 1)
    ref = w / (1 + w)
    limit = ref * (2.0 ** -11 + 2 * n * 2.0 ** -24 + 2.0 ** -16) + n * 2.0 ** -32
    assert ((got - ref).abs() <= limit).all(), (float(got.min()), float(got.max()), float(ref))


def test_infinite_scores():
    """-inf scores drop their keys; all of them -inf, or a +inf one, give NaN as the formula does."""
    c = make("bf16", [40, 40, 40], 1, 64, 16, nan=False)
    for s, rows in ((0, range(3, 40)), (1, range(40)), (2, [7])):
        for j in rows:
            c.pool[0, int(c.table[s, j // 16]), 0, 0, j % 16, 0] = float("-inf") if s < 2 else float("inf")
    q = queries(3, 1, 64, "bf16").abs()
    out = rpp.attention_decode(c, 0, q)
    assert torch.isnan(out[1:].float()).all()
    K, V = sequence(c, 0, 0)
    ref = torch.softmax(K[:3, 0] @ q[0].double() / 8, 0) @ V[:3, 0]
    assert (out[0].double() - ref).abs().max() <= 2.0 ** -8 * ref.abs().max() + 1e-4


def test_same_result_every_time():
    lens = [int(x) for x in np.random.default_rng(5).integers(1, 4000, 37)]
    c = make("bf16", lens, 4, 128, 16)
    q = queries(37, 16, 128, "bf16")
    first = rpp.attention_decode(c, 0, q)
    for _ in range(5):
        assert torch.equal(first, rpp.attention_decode(c, 0, q))


def test_device_errors_stay_in_bounds():
    c = make("bf16", [40, 300, 7], 2, 64, 16)
    q = queries(3, 4, 64, "bf16")
    for spoil, code in ((lambda: c.lens.__setitem__(1, -5), rpp.RPP_DERR_LENGTH),
                        (lambda: c.lens.__setitem__(1, 1 << 20), rpp.RPP_DERR_LENGTH),
                        (lambda: c.table.__setitem__((1, 3), c.cfg.pages), rpp.RPP_DERR_PAGE),
                        (lambda: c.table.__setitem__((1, 3), -1), rpp.RPP_DERR_PAGE)):
        lens, table = c.lens.clone(), c.table.clone()
        spoil()
        rpp.attention_decode(c, 0, q)
        assert rpp.get_device_error(c.err) == code
        c.err.zero_()
        c.lens.copy_(lens)
        c.table.copy_(table)
    for slots in ([0, 1, 5], [0, -1, 2]):
        rpp.attention_decode(c, 0, q, ints(slots))
        assert rpp.get_device_error(c.err) == rpp.RPP_DERR_SLOT
        c.err.zero_()
    check(rpp.attention_decode(c, 0, q), q, c, 0, range(3), 4)


def test_a_set_error_word_stops_it():
    c = make("bf16", [40], 2, 64, 16)
    c.err.fill_(9)
    out = torch.full((1, 256), 3.0, dtype=torch.bfloat16, device=dev())
    rpp.attention_decode(c, 0, queries(1, 4, 64, "bf16"), out=out)
    assert (out == 3).all()


def test_captured_and_replayed_with_other_lengths():
    c = make("bf16", [400] * 6, 2, 128, 16)
    q = queries(6, 8, 128, "bf16").clone()
    ws = rpp.attention_decode_workspace(c, 6, 8)
    out = torch.empty(6, 1024, dtype=torch.bfloat16, device=dev())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            rpp.attention_decode(c, 0, q, out=out, workspace=ws)
    torch.cuda.synchronize()
    for lens in ([400] * 6, [1, 0, 400, 33, 16, 7], [0] * 6, [13, 399, 1, 2, 3, 400]):
        c.lens[:6] = ints(lens)
        q.copy_(queries(6, 8, 128, "bf16", seed=sum(lens)))
        ws.fill_(255)
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        check(out, q, c, 0, range(6), 8)


def test_two_streams_with_workspaces_of_their_own():
    a, b = (make("bf16", [2000, 50, 900], 4, 128, 16, seed=x) for x in (1, 2))
    q = queries(3, 16, 128, "bf16")
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = []
    for _ in range(4):
        for c, s in zip((a, b), streams):
            with torch.cuda.stream(s):
                outs.append((c, rpp.attention_decode(c, 0, q)))
    torch.cuda.synchronize()
    for c, o in outs:
        check(o, q, c, 0, range(3), 16)


def test_a_workspace_of_fewer_bytes_than_it_counts_is_refused():
    c = make("bf16", [40], 2, 64, 16)
    q = queries(1, 4, 64, "bf16")
    n = rpp.attention_decode_workspace(c, 1, 4).numel()
    with pytest.raises(ValueError):
        rpp.attention_decode(c, 0, q, workspace=torch.empty(1, dtype=torch.uint8, device=dev()).expand(n))
    with pytest.raises(rpp.RppError):
        rpp.attention_decode(c, 0, q, workspace=torch.empty(n - 1, dtype=torch.uint8, device=dev()))


def put(c, kv, slot, j, head, col, x):
    """One element of a sequence's K (kv 0) or V (1) row j in layer 0."""
    ps = c.cfg.page_size
    c.pool[0, int(c.table[slot, j // ps]), kv, head, j % ps, col] = x


def same(a, b):
    return ((a == b) | (torch.isnan(a) & torch.isnan(b))).all()


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("dtype,d,nh,nkv,lens", [
    ("fp16", 64, 4, 4, [1, 2, 16, 17, 31, 40] * 40),          # a warp has them whole
    ("bf16", 128, 20, 1, [1, 2, 16, 17, 31, 40] * 40),        # above 16 query heads
    ("bf16", 128, 8, 2, [3000]),                              # cut, joined by query head
    ("fp16", 64, 5, 1, [2, 5000, 1]),
    ("fp16", 128, 8, 2, [700, 1, 333, 900] * 25),             # cut, joined by the cut
    ("bf16", 64, 3, 3, [1200, 40] * 128),
])
def test_values_that_are_not_finite(dtype, d, nh, nkv, lens, bad):
    """One element of one value row, first, in the middle or last in its sequence: the outputs of that
    column in the heads that read it are it, every other one is as without it."""
    c = make(dtype, lens, nkv, d, 16)
    q = queries(len(lens), nh, d, dtype)
    want = rpp.attention_decode(c, 0, q).clone()
    for s, n in enumerate(lens):
        put(c, 1, s, (0, n // 2, n - 1)[s % 3], nkv - 1, 5, bad)
    want.view(len(lens), nkv, nh // nkv, d)[:, -1, :, 5] = bad
    assert same(rpp.attention_decode(c, 0, q), want)
    assert rpp.get_device_error(c.err) == 0


@pytest.mark.parametrize("rows", [1, 200, 2048])              # cut and joined by head, by cut; whole
@pytest.mark.parametrize("dtype,far", [("fp16", 30.0), ("fp16", 130.0), ("bf16", 60.0), ("bf16", 130.0)])
@pytest.mark.parametrize("first", [False, True])
def test_an_infinite_value_of_a_small_weight(dtype, far, rows, first):
    """The weight e^-far is above 0 whatever the arithmetic makes of it, so the output is the
    infinity; with the infinite value's key before the largest one, too.  -inf as its score makes the
    weight 0, and 0 times infinity is NaN."""
    n, d = 1000, 64
    c = make(dtype, [n], 1, d, 16, nan=False)
    c.pool[0, :, 0] = 0
    at = 3 if first else 997
    for j in range(n):
        if first and j > 900:
            put(c, 0, 0, j, 0, 0, far)
    if not first:
        put(c, 0, 0, at, 0, 0, -far)
    q = torch.zeros(rows, d, device=dev(), dtype=TDT[dtype])
    q[:, 0] = 8.0
    slots = torch.zeros(rows, dtype=torch.int32, device=dev())
    base = rpp.attention_decode(c, 0, q, slots).clone()
    assert torch.isfinite(base.float()).all()
    put(c, 1, 0, at, 0, 7, float("inf"))
    put(c, 1, 0, at, 0, 8, float("-inf"))
    put(c, 1, 0, at, 0, 9, float("inf"))
    put(c, 1, 0, at + 1, 0, 9, float("-inf"))
    base[:, 7], base[:, 8], base[:, 9] = float("inf"), float("-inf"), float("nan")
    assert same(rpp.attention_decode(c, 0, q, slots), base)
    put(c, 0, 0, at, 0, 0, float("-inf"))
    got = rpp.attention_decode(c, 0, q, slots)
    assert torch.isnan(got[:, 7:10]).all() and torch.isfinite(got[:, 10:].float()).all()


def test_rows_whose_scores_are_no_numbers_stay_nan():
    """A query head that holds NaN beside an infinite value: NaN all over, the other heads have the infinity."""
    c = make("fp16", [700, 90], 1, 64, 16)
    q = queries(2, 5, 64, "fp16").clone()
    q[:, 64 * 3 + 7] = float("nan")
    for s in (0, 1):
        put(c, 1, s, 30, 0, 5, float("inf"))
    out = rpp.attention_decode(c, 0, q).float().view(2, 5, 64)
    assert torch.isnan(out[:, 3]).all()
    rest = out[:, [0, 1, 2, 4]]
    assert (rest[..., 5] == float("inf")).all()
    keep = [e for e in range(64) if e != 5]
    assert torch.isfinite(rest[..., keep]).all()
