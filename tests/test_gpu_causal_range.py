"""Causal attention over packed prompts at scores up to fp32's largest, against the values that fp64 picks.

In every row one key is ahead of all others that the row sees by far more than scores of that size are rounded: its weight alone
is above 0, whatever that rounding was, so the output is its value, off by the final rounding (e / 2 of it, e = eps of the
type), the rounding of the weight to the type (e / 2, which the sum does not share), exp2 (2^-22) and the products and
quotient after it (eight roundings of 2^-24), and fp16's smallest values, 2^-25."""
import pytest
import torch

import remove_padding_prefix_gb300 as rpp
from gpu_util import TDT, dev
from test_gpu_decode8 import EPS, ints
from test_gpu_decode_range import along

pytestmark = pytest.mark.gpu

LENS = [1, 2, 64, 129, 16, 300, 700, 33]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d,nh,nkv", [(64, 4, 4), (128, 8, 2), (64, 6, 1), (128, 3, 3)])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("by", ["scale", "rows"])
def test_scores_of_any_size(dtype, d, nh, nkv, sign, by):
    g = torch.Generator(device=dev()).manual_seed(d + nh)
    total, cu = sum(LENS), [0]
    u = torch.randn((nkv, d), generator=g, device=dev()).sign()
    r = torch.rand((total, nkv, d), generator=g, device=dev())
    size = 30 + 15 * r if sign > 0 else 70 + 30 * r
    want = torch.zeros(total, dtype=torch.long, device=dev())
    for n in LENS:                       # the first key ahead of all behind it, and one in the middle ahead of that
        a, p = cu[-1], cu[-1] + n // 2
        size[a] = 60 + 20 * r[a] if sign > 0 else 45 + 15 * r[a]
        size[p] = 100 + 20 * r[p] if sign > 0 else 25 + 10 * r[p]
        want[a:p], want[p:a + n] = a, p
        cu.append(a + n)
    v = torch.randn((total, nkv * d), generator=g, device=dev()).to(TDT[dtype])
    ref = v[want].double().view(total, nkv, 1, d).expand(total, nkv, nh // nkv, d).reshape(total, nh * d)
    e = EPS[dtype]
    for z in (20, 24, 25, 26, 28, 30, 31, 33, 36) + ((60, 110) if dtype == "bf16" or by == "scale" else ()):
        up = z - 6
        k_up = 0 if by == "scale" else 15 if dtype == "fp16" else up // 2
        q_up = 0 if by == "scale" else up - k_up
        k = (sign * u * size * 2.0 ** (min(k_up, 8) - 7)).double()
        k = (k * 2.0 ** (k_up - min(k_up, 8))) if dtype == "bf16" else k
        q = along(total, u, nh // nkv, dtype, 2.0 ** (q_up if dtype == "bf16" else min(q_up, 14)))
        if z == 33 and by == "scale":             # the largest scale there is, and rows as much smaller
            up, q = 127.5, (q.double() * 2.0 ** -14).to(TDT[dtype])
            k = k * 2.0 ** -12 if dtype == "bf16" else k
        # what fp16's range leaves over goes to the scale
        left = up - (min(k_up, 8) + min(q_up, 14)) if by == "rows" and dtype == "fp16" else up if by == "scale" else 0
        out = rpp.attention_causal_varlen(q, k.to(TDT[dtype]).flatten(1), v, ints(cu), len(LENS), max(LENS), nh, nkv, d,
                                          scale=min(1.37 * 2.0 ** left, 2e38))
        assert torch.isfinite(out.float()).all(), z
        off = (out.double() - ref).abs()
        assert (off <= (e / 2 + e / 2 + 2.0 ** -22 + 8 * 2.0 ** -24) * ref.abs() * (1 + e) + 2.0 ** -25).all(), (z, float(off.max()))
