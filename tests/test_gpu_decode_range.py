"""Attention of one new token over either cache where numbers leave the usual range: scores up to fp32's largest, a
large `scale` beside scores of zero.  Against fp64.

Tolerances (e = eps of the output type).  Scores, one key ahead of all others by far more than scores of that size are
rounded: its weight alone is above 0, whatever that rounding was, so the output is its value, off by
  * the final rounding, e / 2 of it;
  * exp2, 2^-22, of the weight and of the factors of a join (at most two), P in two 16-bit parts (2^-21 in f16, 2^-17 in bf16),
    the products, sum, quotient and unit after it (eight roundings of 2^-24) and as many in a join;
  * fp16's smallest values, 2^-25, and half a step of f16's smallest where the weight is 2^6 at least, 2^-31 of the largest
    code's value.
"""
import pytest
import torch

import remove_padding_prefix_gb300 as rpp
import test_gpu_decode as t16
import test_gpu_decode8 as t8
from gpu_util import TDT, dev
from test_gpu_decode8 import EPS, TOP

pytestmark = pytest.mark.gpu

WHOLE, CUT = [1, 16, 40, 17] * 80, [3000, 1, 700]        # units whole in a warp, and cut ones


def places(c, s):
    """Page and row of each token of a slot."""
    t, ps = torch.arange(int(c.lens[s]), device=dev()), c.cfg.page_size
    return c.table[s].long()[t // ps], t % ps


def ahead(lens, nkv, d, sign, seed=0):
    """Keys [len, nkv, d] of each sequence, one of them ahead: all along one direction of signs, at least half as long
    again as the others (or, where scores are below 0, the shortest), the first, a middle or the last; and the directions."""
    g = torch.Generator(device=dev()).manual_seed(seed)
    u = torch.randn((nkv, d), generator=g, device=dev()).sign()
    rows, top = [], []
    for i, n in enumerate(lens):
        j = (0, n // 2, n - 1)[i % 3]
        r = torch.rand((n, nkv, d), generator=g, device=dev())
        k = 30 + 30 * r if sign > 0 else 60 + 60 * r
        k[j] = 90 + 30 * r[j] if sign > 0 else 30 + 10 * r[j]
        rows.append(sign * u * k)
        top.append(j)
    return rows, top, u


def along(n, u, per, dtype, size, seed=1):
    """Queries along the directions, [n, heads * d]."""
    g = torch.Generator(device=dev()).manual_seed(seed)
    q = u[None, :, None, :] * (0.5 + torch.rand((n, u.shape[0], per, u.shape[1]), generator=g, device=dev()))
    return (q.double() * size).to(TDT[dtype]).flatten(1)


def close(got, want, e, rest, least=2.0 ** -25):
    want = want.double()
    off = (got.double() - want).abs()
    assert torch.isfinite(got.float()).all()
    assert (off <= e / 2 * want.abs() + rest + least).all(), float(off.max())


HEADS = [(64, 4, 4), (128, 8, 2), (64, 12, 1), (128, 20, 1)]


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d,nh,nkv", HEADS)
@pytest.mark.parametrize("lens", [WHOLE, CUT], ids=["whole", "cut"])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("by", ["scale", "rows"])
def test_scores_of_any_size_over_codes(kind, dtype, d, nh, nkv, lens, sign, by):
    c = t8.make(kind, lens, nkv, d, 16, 16, spread=0)
    rows, top, u = ahead(lens, nkv, d, sign)
    want = []
    for s, n in enumerate(lens):
        page, row = places(c, s)
        codes = (rows[s].round() if kind == "int8" else rows[s]).to(t8.CODES[kind])
        c.pool.view(torch.uint8)[0, page, 0, :, row] = codes.view(torch.uint8)
        want.append(t8.sequence(c, 0, s)[1][top[s]].repeat_interleave(nh // nkv, 0).flatten())
    want = torch.stack(want)
    used = c.scales[0, :, 0] != 255
    unit = float(torch.exp2(c.scales[0, :, 1][c.scales[0, :, 1] != 255].double() - 127).max())
    rest = want.abs().max() * (2 * 3 * 2.0 ** -22 + 2.0 ** -21 + 16 * 2.0 ** -24) + 2.0 ** -31 * TOP[kind] * unit
    for z in (20, 26, 28, 30, 31, 33, 40, 60, 110):
        # keys of 2^-7 times their codes: scores are some d log2(e) times the sizes
        up = z - 6
        k_up = 0 if by == "scale" else up - 13 if dtype == "fp16" else up // 2
        q_up = 0 if by == "scale" else up - k_up
        scale = 1.37 * 2.0 ** (up if by == "scale" else 0)
        c.scales[0, :, 0] = torch.where(used, 127 - 7 + k_up, 255).to(torch.uint8)
        q = along(len(lens), u, nh // nkv, dtype, 2.0 ** q_up)
        got = rpp.attention_decode(c, 0, q, scale=scale)
        assert rpp.get_device_error(c.err) == 0
        close(got, want, EPS[dtype], rest)


@pytest.mark.parametrize("dtype,by", [("fp16", "scale"), ("bf16", "scale"), ("bf16", "rows")])
@pytest.mark.parametrize("d,nh,nkv", HEADS)
@pytest.mark.parametrize("lens", [WHOLE, CUT], ids=["whole", "cut"])
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_of_any_size_over_16_bits(dtype, by, d, nh, nkv, lens, sign):
    c = t16.make(dtype, lens, nkv, d, 16)
    rows, top, u = ahead(lens, nkv, d, sign)
    want = []
    for s, n in enumerate(lens):
        want.append(t16.sequence(c, 0, s)[1][top[s]].repeat_interleave(nh // nkv, 0).flatten())
    want = torch.stack(want)
    part = 2.0 ** -21 if dtype == "fp16" else 2.0 ** -17
    rest = want.abs().max() * (2 * 3 * 2.0 ** -22 + part + 16 * 2.0 ** -24) + 2.0 ** -31
    for z in (20, 24, 25, 26, 28, 30, 31, 33, 40, 60, 110):
        up = z - 6
        k_up = 0 if by == "scale" else up // 2
        q_up = 0 if by == "scale" else up - k_up
        scale = 1.37 * 2.0 ** (up if by == "scale" else 0)
        for s in range(len(lens)):
            page, row = places(c, s)
            c.pool[0, page, 0, :, row] = (rows[s].double() * 2.0 ** (k_up - 7)).to(TDT[dtype])
        q = along(len(lens), u, nh // nkv, dtype, 2.0 ** q_up)
        got = rpp.attention_decode(c, 0, q, scale=scale)
        assert rpp.get_device_error(c.err) == 0
        close(got, want, EPS[dtype], rest)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("lens", [WHOLE, CUT], ids=["whole", "cut"])
@pytest.mark.parametrize("zero", ["queries", "keys", "product"])
def test_scores_of_zero_beside_a_large_scale(kind, dtype, lens, zero):
    """0 times any scale is 0: the mean of the values."""
    nkv, d, nh = 2, 64, 6
    c = t8.make(kind, lens, nkv, d, 16, 16, spread=0)
    used = c.scales[0, :, 0] != 255
    q = t8.queries(len(lens), nh, d, dtype).clone()
    if zero == "queries":
        q.zero_()
    for s in range(len(lens)):
        page, row = places(c, s)
        if zero == "keys":
            c.pool.view(torch.uint8)[0, page, 0, :, row] = 0
        elif zero == "product":                    # keys in the even columns, queries in the odd ones
            k = c.pool.view(torch.uint8)[0, page, 0, :, row]
            k[..., 1::2] = 0
            c.pool.view(torch.uint8)[0, page, 0, :, row] = k
    if zero == "product":
        q[:, ::2] = 0
    for b in (121, 200, 248):
        c.scales[0, :, 0] = torch.where(used, b, 255).to(torch.uint8)
        for scale in (1.0, 1e30, 2e38):
            got = rpp.attention_decode(c, 0, q, scale=scale)
            assert rpp.get_device_error(c.err) == 0
            for s, n in enumerate(lens[:8]):
                _, V, unit = t8.sequence(c, 0, s)
                want = V.mean(0).repeat_interleave(nh // nkv, 0).flatten()
                rest = V.abs().max() * 2 * (2.0 ** -21 + 3 * 2.0 ** -22 + n * 2.0 ** -24) + n * 2.0 ** -31 * TOP[kind] * unit.max()
                close(got[s], want, EPS[dtype], rest)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("n,gone", [(40, 17), (40, 33), (3000, 1200), (3000, 2990), (33, 1)])
def test_scores_below_every_number(kind, dtype, n, gone):
    """The first keys' scores are beyond fp32's least: weight 0, the others' mean."""
    d = 64
    c = t8.make(kind, [n], 1, d, 16, 1, spread=0)
    page, row = places(c, 0)
    k = torch.zeros((n, 1, d), device=dev())
    k[:gone, :, 0] = -64
    c.pool.view(torch.uint8)[0, page, 0, :, row] = k.to(t8.CODES[kind]).view(torch.uint8)
    used = c.scales[0, :, 0] != 255
    c.scales[0, :, 0] = torch.where(used, 200, 255).to(torch.uint8)
    q = torch.zeros((1, 3 * d), device=dev())
    q[:, ::d] = 50000.0
    got = rpp.attention_decode(c, 0, q.to(TDT[dtype]), scale=1e38)
    assert rpp.get_device_error(c.err) == 0
    _, V, unit = t8.sequence(c, 0, 0)
    want = V[gone:].mean(0).flatten().repeat(3)
    rest = V.abs().max() * 2 * (2.0 ** -21 + 3 * 2.0 ** -22 + n * 2.0 ** -24) + n * 2.0 ** -31 * TOP[kind] * unit.max()
    close(got[0], want, EPS[dtype], rest)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("lens", [WHOLE, CUT], ids=["whole", "cut"])
def test_a_large_scale_and_large_queries_beside_tiny_keys(kind, lens):
    """scale * q is beyond fp32's largest, scale * (q . k) is not."""
    nkv, d, nh = 2, 64, 6
    c = t8.make(kind, lens, nkv, d, 16, 16, spread=0)
    rows, top, u = ahead(lens, nkv, d, 1)
    want = []
    for s, n in enumerate(lens):
        page, row = places(c, s)
        codes = (rows[s].round() if kind == "int8" else rows[s]).to(t8.CODES[kind])
        c.pool.view(torch.uint8)[0, page, 0, :, row] = codes.view(torch.uint8)
        want.append(t8.sequence(c, 0, s)[1][top[s]].repeat_interleave(nh // nkv, 0).flatten())
    want = torch.stack(want)
    c.scales[0, :, 0] = torch.where(c.scales[0, :, 0] != 255, 3, 255).to(torch.uint8)
    unit = 2.0 ** (1 if kind == "int8" else -1) / 64
    rest = want.abs().max() * (2 * 3 * 2.0 ** -22 + 2.0 ** -21 + 16 * 2.0 ** -24) + 2.0 ** -31 * TOP[kind] * unit
    for q_up in (20, 60, 100):
        q = along(len(lens), u, nh // nkv, "bf16", 2.0 ** q_up)
        got = rpp.attention_decode(c, 0, q, scale=1e38)
        assert rpp.get_device_error(c.err) == 0
        close(got, want, EPS["bf16"], rest)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("lens", [WHOLE, CUT], ids=["whole", "cut"])
@pytest.mark.parametrize("q_up", [-20, -41, -60, -90])
def test_a_tiny_scale_and_tiny_queries_beside_large_keys(kind, lens, q_up):
    """scale times the power of two that queries are held in is below fp32's smallest normal number (at 2^-144 a step is 2^-5
    of it), the scores are about 2^-9."""
    nkv, d, nh = 2, 64, 6
    c = t8.make(kind, lens, nkv, d, 16, 16, spread=0)
    c.scales[:, :, 0] = torch.where(c.scales[:, :, 0] != 255, 246, 255).to(torch.uint8)
    q = t8.queries(len(lens), nh, d, "bf16", scale=2.0 ** q_up)
    scale = 2.0 ** (-137 - q_up) * 1.37
    t8.check(rpp.attention_decode(c, 0, q, scale=scale), q, c, 0, range(len(lens)), nh, scale=scale)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d,nh,nkv", [(64, 4, 2), (128, 8, 2), (128, 20, 1)])
@pytest.mark.parametrize("lens", [[2, 16, 40, 17, 33] * 60, [3000, 2, 700]], ids=["whole", "cut"])
@pytest.mark.parametrize("order", ["near first", "far first", "in turn"])
def test_values_far_apart(kind, dtype, d, nh, nkv, lens, order):
    """Half of a sequence's blocks hold values up to 2^120 larger than the other half's, which the queries hardly look at, or
    some heads at the ones and some at the others.  Error, beside the output's rounding (P_j: weights that add up to 1):
    scores, exp2, P's parts and sums as in the other tests, of sum P_j |V_j|; half a step of f16's smallest for each key's
    code, where the largest P_j 2^(b_j - 127) is held as 2^7 at least."""
    if order == "in turn":
        half = lambda n: (torch.arange(n, device=dev()) // 4) % 2 == 1
    else:
        half = lambda n: (torch.arange(n, device=dev()) >= (n + 1) // 2) ^ (order == "far first")
    per = nh // nkv
    for gap, away, mixed in ((20, 40.0, True), (20, 300.0, True), (45, 40.0, False), (45, 300.0, False), (45, 300.0, True),
                             (100, 40.0, True), (100, 300.0, True), (120, 300.0, False)):
        if dtype == "fp16" and (gap == 100 or gap == 45 and mixed):
            continue                               # (beyond fp16's values)
        c = t8.make(kind, lens, nkv, d, 16, 1, seed=gap, spread=1)
        low = 127 - (12 if kind == "int8" else 14) if dtype == "fp16" else 60
        for s, n in enumerate(lens):
            page, row = places(c, s)
            far = half(n)
            k = torch.zeros((n, nkv, d), device=dev())
            k[:, :, 0] = torch.where(far, -64.0, 64.0)[:, None]
            k[:, :, 1] = torch.arange(n, device=dev())[:, None] % 64 - 32.0
            c.pool.view(torch.uint8)[0, page, 0, :, row] = k.to(t8.CODES[kind]).view(torch.uint8)
            c.scales[0, page, 0, :, row] = 121
            c.scales[0, page, 1, :, row] = (low + gap * far.int())[:, None].to(torch.uint8)
        q = torch.zeros((len(lens), nkv, per, d), device=dev())
        q[..., 0] = away / 2 * d ** 0.5
        if mixed:
            q[:, :, 1::2, 0] *= -1
        q[..., 1] = 1.5
        q = q.to(TDT[dtype]).flatten(1)
        got = rpp.attention_decode(c, 0, q)
        assert rpp.get_device_error(c.err) == 0 and torch.isfinite(got.float()).all()
        e = EPS[dtype]
        for s in list(range(min(len(lens), 10))) + [len(lens) - 1]:
            n = lens[s]
            K, V, _ = t8.sequence(c, 0, s)
            qi = q[s].double().view(nkv, per, d)
            z = torch.einsum("hgd,nhd->hgn", qi, K) * d ** -0.5
            P = torch.softmax(z, -1)
            ref = torch.einsum("hgn,nhd->hgd", P, V)
            page, row = places(c, s)
            unit = torch.exp2(c.scales[0, page, 1, :, row].double() - 127).T[:, None]                # [nkv, 1, n]
            codes = (V / unit[:, 0].T[..., None]).abs().sum(0)[:, None]                                # [nkv, 1, d]
            mag = (torch.einsum("hgd,nhd->hgn", qi.abs(), K.abs()) * d ** -0.5).amax(-1)
            ds = (d + 6) * 2.0 ** -24 * mag + 2.0 ** -22 * z.abs().amax(-1)
            part = torch.einsum("hgn,nhd->hgd", P, V.abs())
            limit = e / 2 * ref.abs() + (2 * ds + 2 * (2.0 ** -22 + 2.0 ** -21 + n * 2.0 ** -24))[..., None] * part + \
                2.0 ** -32 * (P * unit).amax(-1, keepdim=True) * codes + (2.0 ** -25 if dtype == "fp16" else 2.0 ** -134)
            off = (got[s].double().view(nkv, per, d) - ref).abs()
            assert (off <= limit).all(), (gap, away, mixed, s, n, float((off / limit).max()))


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("d,nh,nkv", HEADS)
@pytest.mark.parametrize("size", [110, 87, -60])
def test_values_of_any_size_in_pieces(kind, d, nh, nkv, size):
    """Units that several warps share: what they leave for the join is held in units of its own sum."""
    lens = [3000, 1, 900, 20]
    c = t8.make(kind, lens, nkv, d, 16, 16, spread=0)
    c.scales[:, :, 1] = torch.where(c.scales[:, :, 1] == 255, 255, c.scales[:, :, 1].int() + size).to(torch.uint8)
    q = t8.queries(len(lens), nh, d, "bf16", scale=3.0)
    t8.check(rpp.attention_decode(c, 0, q), q, c, 0, range(len(lens)), nh)
