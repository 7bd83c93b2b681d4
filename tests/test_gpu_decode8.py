"""Attention of one new token over the 8-bit paged cache, against fp64 over the values that the codes stand for.

Tolerance, per output element, from the arithmetic (e = eps of the output type; V the sequence's values of that head,
k its keys, n their number):
  * the final rounding: e / 2 of the value;
  * a score is an fp32 sum of d exact products (a bf16 query's power of two loses at most 2^-32 of its largest element),
    scaled by two factors that are one rounding each: (d + 6) 2^-24 sum |q_c k_c|, and entering as
    exp(scale s) that, twice, times max |V|, on the weighted mean;
  * exp2 (2^-22), the base change of a score of magnitude z (2^-22 z), P kept to two f16 parts (2^-21), fp32 sums
    over n keys (n 2^-24): each times max |V|, twice (numerator and sum);
  * the lesser part of P is no smaller than f16's smallest step, 2^-24, where the largest weight is 2^7 at least:
    half of that for each key's largest code in units of the largest scale, n 2^-32 top 2^(b - 127).
"""
import numpy as np
import pytest
import torch

import remove_padding_prefix_gb300 as rpp
from gpu_util import TDT, dev

pytestmark = pytest.mark.gpu

EPS = {"fp16": 2.0 ** -10, "bf16": 2.0 ** -7}
CODES = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
TOP = {"int8": 127.0, "e4m3": 448.0}


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=dev())


def make(kind, lens, nkv, d, ps, block, seed=0, layers=1, spare=5, spread=2, junk=True):
    """A cache of sequences on shuffled pages, scales of +- spread; what no sequence has written holds NaN (e4m3) or
    anything, and its scales NaN."""
    rng = np.random.default_rng(seed)
    need = [-(-n // ps) for n in lens]
    pages, mp = sum(need) + spare, max(need + [1]) + 1
    c = rpp.KvCache8(layers, pages, ps, nkv, d, len(lens) + 2, mp, kind, block, dev())
    order = rng.permutation(pages)
    table = np.full((len(lens) + 2, mp), -1, np.int32)
    refs = np.zeros(pages, np.int32)
    keep = torch.zeros((pages, ps), dtype=torch.bool)
    at = 0
    for s, n in enumerate(lens):
        for j in range(need[s]):
            table[s, j] = order[at]
            refs[order[at]] = 1
            keep[order[at], :n - j * ps] = True
            at += 1
    g = torch.Generator(device=dev()).manual_seed(seed)
    x = (torch.randn(c.pool.shape, generator=g, device=dev()) * (TOP[kind] / 3.5)).clamp_(-TOP[kind], TOP[kind])
    codes = (x.round() if kind == "int8" else x).to(CODES[kind]).view(torch.uint8)
    base = 128 - (6 if kind == "int8" else 8)
    scales = torch.randint(base - spread, base + spread + 1, c.scales.shape, generator=g, device=dev(), dtype=torch.uint8)
    if junk:
        k = keep.to(dev())[None, :, None, None, :, None]
        codes = torch.where(k, codes, torch.full_like(codes, 0x7f))
        begun = keep.view(pages, ps // block, block).any(-1).to(dev())[None, :, None, None]
        scales = torch.where(begun, scales, torch.full_like(scales, 255))
    c.pool.view(torch.uint8).copy_(codes)
    c.scales.copy_(scales)
    c.table.copy_(torch.from_numpy(table))
    c.lens[:len(lens)] = ints(lens)
    c.refs.copy_(torch.from_numpy(refs))
    return c


def sequence(c, layer, slot):
    """fp64 K and V [len, kv heads, d] of a slot, and the largest scale of each head's V."""
    n, ps = int(c.lens[slot]), c.cfg.page_size
    pages = c.table[slot, :-(-n // ps)].long()
    b = c.scales[layer, pages].double()
    unit = torch.where(b == 255, torch.full_like(b, float("nan")), torch.exp2(b - 127))
    x = c.pool.view(torch.uint8)[layer, pages].view(c.pool.dtype).double() * unit.repeat_interleave(c.block, -1)[..., None]
    x = x.permute(1, 0, 3, 2, 4).reshape(2, -1, c.cfg.kv_heads, c.cfg.head_dim)
    used = unit[:, 1].permute(0, 2, 1).reshape(-1, c.cfg.kv_heads)[:-(-n // c.block)]
    return x[0, :n], x[1, :n], used.amax(0)


def bound(c, q, K, V, unit, z, scale):
    d, n = c.cfg.head_dim, K.shape[0]
    mag = (torch.einsum("hgd,nhd->hgn", q.abs(), K.abs()) * scale).amax(-1)          # [nkv, per]
    vmax = V.abs().amax(0).amax(-1)[:, None]
    ds = (d + 6) * 2.0 ** -24 * mag + 2.0 ** -22 * z.abs().amax(-1)
    top = 127.0 if c.pool.dtype is torch.int8 else 448.0
    return vmax * (2 * ds + 2 * (2.0 ** -22 + 2.0 ** -21 + n * 2.0 ** -24)) + (n * 2.0 ** -32 * top * unit)[:, None]


def check(got, q, c, layer, slots, nh, scale=None, rows=None):
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
        K, V, unit = sequence(c, layer, s)
        qi = q[i].double().view(nkv, per, d)
        z = torch.einsum("hgd,nhd->hgn", qi, K) * scale
        ref = torch.einsum("hgn,nhd->hgd", torch.softmax(z, -1), V)
        off = (got[i].double().view(nkv, per, d) - ref).abs()
        limit = e / 2 * ref.abs() + bound(c, qi, K, V, unit, z, scale)[..., None] + 2.0 ** -25   # (fp16's smallest values)
        assert (off <= limit).all(), (i, s, n, float((off - limit).max()), float((off / limit).max()))


def queries(n, nh, d, dtype, seed=1, scale=1.0):
    g = torch.Generator(device=dev()).manual_seed(seed)
    wide = (scale * torch.randn((n, nh * d + 64), generator=g, device=dev())).to(TDT[dtype])
    return wide[:, 64:]          # columns of wider rows


LENS = [1, 2, 15, 16, 17, 31, 32, 33, 0, 47, 48, 63, 64, 65, 100, 127, 128, 129, 255, 257, 0, 500, 1023]


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nh,nkv,ps,block", [(8, 8, 16, 16), (32, 8, 16, 1), (12, 12, 32, 32), (5, 1, 48, 2), (16, 2, 64, 64),
                                             (40, 2, 16, 16), (33, 1, 16, 4), (7, 7, 128, 128), (12, 4, 16, 8), (9, 1, 32, 16)])
def test_lengths_and_heads(kind, dtype, d, nh, nkv, ps, block):
    c = make(kind, LENS, nkv, d, ps, block, seed=nh + ps)
    slots = list(np.random.default_rng(2).permutation(len(LENS)))
    q = queries(len(slots), nh, d, dtype, scale=2.0)
    check(rpp.attention_decode(c, 0, q, ints([int(s) for s in slots])), q, c, 0, slots, nh)


@pytest.mark.parametrize("kind,dtype,d,nh,nkv,ps,block,lens", [
    ("e4m3", "bf16", 128, 32, 8, 16, 16, [40001]), ("int8", "fp16", 64, 16, 16, 64, 64, [70000]),
    ("e4m3", "fp16", 64, 16, 1, 16, 1, [30000, 1, 30000]), ("int8", "bf16", 128, 8, 8, 16, 4, [9000, 3, 0, 8191]),
])
def test_long(kind, dtype, d, nh, nkv, ps, block, lens):
    c = make(kind, lens, nkv, d, ps, block)
    q = queries(len(lens), nh, d, dtype)
    check(rpp.attention_decode(c, 0, q), q, c, 0, range(len(lens)), nh)


@pytest.mark.parametrize("n,hi,nh,nkv", [(300, 40, 8, 2), (1000, 5, 4, 4), (4096, 20, 2, 1)])
def test_many_short(n, hi, nh, nkv):
    lens = [int(x) for x in np.random.default_rng(n).integers(0, hi, n)]
    c = make("e4m3", lens, nkv, 64, 16, 16)
    q = queries(n, nh, 64, "bf16")
    got = rpp.attention_decode(c, 0, q)
    check(got[:400], q[:400], c, 0, range(min(n, 400)), nh)
    check(got[-200:], q[-200:], c, 0, range(n - 200, n), nh)


@pytest.mark.parametrize("n,nh,nkv,dtype", [(60, 8, 2, "bf16"), (300, 32, 8, "bf16"), (700, 16, 8, "fp16"), (200, 24, 1, "fp16")])
def test_long_sequences_among_short_ones(n, nh, nkv, dtype):
    """Units of many pieces and units of one or two joined by one call, the long ones at either end and in the middle."""
    lens = [int(x) for x in np.random.default_rng(n).integers(0, 90, n)]
    for i, m in ((0, 9000), (n // 2, 5000), (n // 2 + 1, 700), (n - 1, 12001)):
        lens[i] = m
    c = make("e4m3", lens, nkv, 128, 16, 16)
    q = queries(n, nh, 128, dtype)
    got = rpp.attention_decode(c, 0, q)
    check(got, q, c, 0, range(n), nh)
    assert torch.equal(rpp.attention_decode(c, 0, q), got)


def test_nothing_to_attend_to():
    c = make("int8", [0, 0, 0], 4, 128, 16, 16)
    q = queries(3, 8, 128, "bf16")
    out = torch.full((3, 1024), float("nan"), dtype=torch.bfloat16, device=dev())
    rpp.attention_decode(c, 0, q, out=out)
    check(out, q, c, 0, range(3), 8)


def test_layer_scale_and_the_same_slot_twice():
    c = make("e4m3", [40, 300, 7], 2, 64, 16, 16, layers=3)
    q = queries(4, 6, 64, "fp16")
    for layer in (0, 2):
        check(rpp.attention_decode(c, layer, q, ints([1, 2, 1, 0]), scale=0.3), q, c, layer, [1, 2, 1, 0], 6, scale=0.3)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("spread", [0, 20])
def test_scales_far_apart(kind, spread):
    """Blocks whose scales are up to 2^40 apart, ascending, descending and mixed: the largest decide."""
    c = make(kind, [500, 33, 1000], 2, 64, 16, 4, spread=spread)
    q = queries(3, 4, 64, "bf16", scale=2.0 ** -spread)
    c.scales[:, :, 0] = torch.clamp(c.scales[:, :, 0], max=125 if kind == "int8" else 123)
    check_wide(c, q, 4)
    for flip in (False, True):
        for s, n in enumerate([500, 33, 1000]):
            pages = c.table[s, :-(-n // 16)].long()
            ramp = torch.linspace(80, 120, 4 * len(pages), device=dev()).round()
            c.scales[0, pages, 1] = (ramp.flip(0) if flip else ramp).to(torch.uint8).view(-1, 1, 4).expand(-1, 2, 4)
        for s, n in enumerate([500, 33, 1000]):        # (junk past the sequences as before)
            c.scales[0, int(c.table[s, (n - 1) // 16]), :, :, (n - 1) % 16 // 4 + 1:] = 255
        check_wide(c, q, 4)


def check_wide(c, q, nh):
    check(rpp.attention_decode(c, 0, q), q, c, 0, range(q.shape[0]), nh)


@pytest.mark.parametrize("d,nh,nkv", [(64, 4, 4), (128, 20, 1)])
@pytest.mark.parametrize("zero", ["k", "v", "both"])
def test_blocks_of_zeros(d, nh, nkv, zero):
    """Zeros have the smallest scale there is, byte 0: values of 0 give 0, keys of 0 the values' mean."""
    lens = [1, 2, 7, 8, 9, 15, 16, 17, 24, 33, 300]
    c = make("e4m3", lens, nkv, d, 16, 16)
    for kv in (0, 1):
        if zero in ("kv"[kv], "both"):
            c.pool.view(torch.uint8)[0, :, kv] = 0
            c.scales[0, :, kv] = 0
    q = queries(len(lens), nh, d, "fp16")
    got = rpp.attention_decode(c, 0, q)
    check(got, q, c, 0, range(len(lens)), nh)
    if zero != "k":
        assert (got == 0).all()


@pytest.mark.parametrize("dtype,size", [("bf16", 2.0 ** 90), ("bf16", 2.0 ** -90), ("bf16", 2.0 ** -130), ("fp16", 60000.0),
                                        ("fp16", 2.0 ** -20)])
def test_queries_of_any_size(dtype, size):
    """Scores of ordinary size from queries that are very large or small: the scales of the keys are the inverse."""
    c = make("e4m3", [100, 700], 2, 128, 16, 16)
    q = (queries(2, 8, 128, dtype).float() * size).clamp(-60000 if dtype == "fp16" else -3e38, 60000 if dtype == "fp16" else 3e38)
    q = q.to(TDT[dtype])
    shift = -int(np.log2(size))
    c.scales[:, :, 0] = (c.scales[:, :, 0].int() + max(min(shift, 130), -118)).clamp(0, 254).to(torch.uint8)
    for s, n in enumerate([100, 700]):
        c.scales[0, int(c.table[s, (n - 1) // 16]), 0, :, (n - 1) % 16 // 16 + 1:] = 255
    check(rpp.attention_decode(c, 0, q), q, c, 0, range(2), 8)


@pytest.mark.parametrize("lens", [[1, 16, 40] * 300, [3000, 900]])      # units whole in a warp, and cut ones
@pytest.mark.parametrize("size", [87, -60])
def test_values_of_any_size(lens, size):
    """Values of up to 2^88 and tiny ones, bf16 outputs."""
    c = make("int8", lens, 2, 64, 16, 16, spread=0)
    c.scales[:, :, 1] = torch.where(c.scales[:, :, 1] == 255, 255, c.scales[:, :, 1].int() + size).to(torch.uint8)
    q = queries(len(lens), 4, 64, "bf16")
    check(rpp.attention_decode(c, 0, q), q, c, 0, range(len(lens)), 4)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("d,nh,nkv,lens,block", [
    (64, 4, 4, [1, 2, 16, 17, 31, 40] * 40, 16), (128, 20, 1, [1, 2, 16, 17, 31, 40] * 40, 4), (128, 8, 2, [3000], 16),
    (64, 5, 1, [2, 5000, 1], 1), (128, 8, 2, [700, 1, 333, 900] * 25, 16),
])
@pytest.mark.parametrize("kv", [0, 1])
def test_blocks_that_are_no_numbers(kind, d, nh, nkv, lens, block, kv):
    """One block of NaN in K or V of the last kv head, first, in the middle or last in its sequence: that head's
    queries are NaN all over, every other one is as without it."""
    c = make(kind, lens, nkv, d, 16, block)
    q = queries(len(lens), nh, d, "fp16")
    want = rpp.attention_decode(c, 0, q).clone()
    for s, n in enumerate(lens):
        j = (0, n // 2, n - 1)[s % 3]
        c.scales[0, int(c.table[s, j // 16]), kv, nkv - 1, j % 16 // block] = 255
    want.view(len(lens), nkv, -1)[:, -1] = float("nan")
    got = rpp.attention_decode(c, 0, q)
    assert ((got == want) | (torch.isnan(got) & torch.isnan(want))).all()
    assert rpp.get_device_error(c.err) == 0


@pytest.mark.parametrize("far", [30.0, 200.0])
def test_a_block_of_nan_behind_a_weight_that_underflows(far):
    """The weight e^-far is above 0 whatever the arithmetic makes of it."""
    n, d = 1000, 64
    c = make("int8", [n], 1, d, 16, 16, spread=0, junk=False)
    c.pool[0, :, 0] = 0
    c.scales[0, :, 0] = 127
    page = int(c.table[0, 40])
    c.pool[0, page, 0, 0, :, 0] = -100
    q = torch.zeros(3, d, device=dev(), dtype=torch.float16)
    q[:, 0] = far * 8 / 100
    slots = ints([0, 0, 0])
    assert torch.isfinite(rpp.attention_decode(c, 0, q, slots).float()).all()
    c.scales[0, page, 1] = 255
    assert torch.isnan(rpp.attention_decode(c, 0, q, slots)).all()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_a_query_head_that_is_no_number(dtype, bad):
    c = make("e4m3", [700, 90], 1, 64, 16, 16)
    q = queries(2, 5, 64, dtype).clone()
    want = rpp.attention_decode(c, 0, q).clone().view(2, 5, 64)
    q[:, 64 * 3 + 7] = bad
    got = rpp.attention_decode(c, 0, q).view(2, 5, 64)
    assert torch.isnan(got[:, 3]).all()
    assert torch.equal(got[:, [0, 1, 2, 4]], want[:, [0, 1, 2, 4]])


def test_many_weights_far_below_the_maximum():
    """65535 keys at 2^-26 of the first one's weight: 9.8e-4 of the sum together."""
    n, d = 65536, 64
    c = make("int8", [n], 1, d, 64, 64, spread=0, junk=False)
    c.pool[0, :, 0] = 0
    c.scales[0, :, 0] = 127
    c.scales[0, :, 1] = 121
    c.pool[0, int(c.table[0, 0]), 0, 0, 0, 0] = 64
    c.pool[0, :, 1] = 64                                        # values of 1, the first of 0
    c.pool[0, int(c.table[0, 0]), 1, 0, 0] = 0
    q = torch.zeros(1, d, device=dev(), dtype=torch.float16)
    q[0, 0] = 26 * np.log(2) / 64 * 8
    check(rpp.attention_decode(c, 0, q), q, c, 0, [0], 1)


def test_errors_of_the_state():
    c = make("e4m3", [40, 300, 7], 2, 64, 16, 16)
    q = queries(3, 4, 64, "bf16")
    for spoil, code in ((lambda: c.table[1].fill_(c.cfg.pages), rpp.RPP_DERR_PAGE), (lambda: c.table[0].fill_(-1), rpp.RPP_DERR_PAGE),
                        (lambda: c.lens[2].fill_(-1), rpp.RPP_DERR_LENGTH), (lambda: c.lens[0].fill_(10 ** 6), rpp.RPP_DERR_LENGTH)):
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
    c.err.fill_(9)
    out = torch.full((3, 256), 3.0, dtype=torch.bfloat16, device=dev())
    rpp.attention_decode(c, 0, q, out=out)
    assert (out == 3).all()
    c.err.zero_()
    check(rpp.attention_decode(c, 0, q), q, c, 0, range(3), 4)


def test_arguments_of_the_binding():
    c = make("e4m3", [40], 2, 64, 16, 16)
    q = queries(1, 4, 64, "bf16")
    ws = rpp.attention_decode_workspace(c, 1, 4)
    with pytest.raises(ValueError):
        rpp.attention_decode(c, 0, q.float())
    with pytest.raises(ValueError):
        rpp.attention_decode(c, 0, q, out=torch.empty(1, 256, dtype=torch.float16, device=dev()))
    with pytest.raises(rpp.RppError):
        rpp.attention_decode(c, 0, q, workspace=ws[:-1])
    with pytest.raises(rpp.RppError):
        rpp.attention_decode(c, 0, queries(1, 3, 64, "bf16"))
    with pytest.raises(rpp.RppError):
        rpp.attention_decode(c, 1, q)


def test_captured_and_replayed_with_other_lengths():
    c = make("e4m3", [400] * 6, 2, 128, 16, 16, junk=False)
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
    a, b = (make("int8", [2000, 50, 900], 4, 128, 16, 1, seed=x) for x in (1, 2))
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
    first = {id(a): outs[0][1], id(b): outs[1][1]}
    assert all(torch.equal(o, first[id(c)]) for c, o in outs)         # the same bits each time


def test_pages_past_32_bits():
    """A sequence on the last pages of a layer of 4.6 GB."""
    pages, d = 140000, 128
    c = rpp.KvCache8(1, pages, 16, 8, d, 1, 40, "e4m3", 16, dev())
    small = make("e4m3", [600], 8, d, 16, 16, spare=0)
    n = small.pool.shape[1]
    c.pool.view(torch.uint8)[:, pages - n:] = small.pool.view(torch.uint8)
    c.scales[:, pages - n:] = small.scales
    c.table[0, :n] = small.table[0, :n] + (pages - n)
    c.lens[0] = 600
    q = queries(1, 32, d, "bf16")
    check(rpp.attention_decode(c, 0, q), q, small, 0, [0], 32)
    assert rpp.get_device_error(c.err) == 0
