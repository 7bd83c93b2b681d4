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


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d,nh,nkv", HEADS)
@pytest.mark.parametrize("lens", [WHOLE, CUT], ids=["whole", "cut"])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("by", ["scale", "rows"])
def test_scores_of_any_size_over_16_bits(dtype, d, nh, nkv, lens, sign, by):
    if by == "rows" and dtype == "fp16":
        pytest.skip("fp16 rows reach scores of 2^38, with the scale of the other case")
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
