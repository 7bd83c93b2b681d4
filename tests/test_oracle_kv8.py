"""Pins of the 8-bit cache's oracle: code tables, rounding, the scale rule, and what repeated raises cost."""
import numpy as np
import pytest
import torch

import oracle.decoder8 as o8

KINDS = ["int8", "e4m3"]


def test_tables_are_the_types():
    for kind, t in (("int8", torch.int8), ("e4m3", torch.float8_e4m3fn)):
        want = torch.arange(256, dtype=torch.uint8).view(t).double().numpy()
        np.testing.assert_array_equal(o8.VALUES[kind], want)


@pytest.mark.parametrize("kind", KINDS)
def test_rounding_is_the_types(kind):
    r = np.random.default_rng(1)
    top = o8.TOP[kind]
    x = np.concatenate([r.uniform(-top, top, 4000), np.ldexp(r.uniform(-1, 1, 2000), r.integers(-12, 8, 2000)),
                        np.arange(-256, 257) / 2.0, np.arange(-64, 65) * 2.0 ** -10, [top, -top, 0.0, -0.0]])
    x = np.clip(x, -top, top).astype(np.float32)
    t = torch.from_numpy(x)
    want = t.round().to(torch.int8) if kind == "int8" else t.to(torch.float8_e4m3fn)
    np.testing.assert_array_equal(o8.encode(x, kind), want.view(torch.uint8).numpy())


@pytest.mark.parametrize("kind", KINDS)
def test_the_scale_is_the_smallest_that_is_half_a_step_off_at_most(kind):
    r = np.random.default_rng(2)
    for a in np.concatenate([np.exp(r.uniform(-60, 80, 300)), [o8.PAST[kind], np.nextafter(o8.PAST[kind], 1e9), 1.0, 0.0]]):
        b = o8.scale_byte(a, kind)
        assert a <= o8.PAST[kind] * 2.0 ** (b - 127) and (b == 0 or a > o8.PAST[kind] * 2.0 ** (b - 128))
    assert o8.scale_byte(np.inf, kind) == 255


@pytest.mark.parametrize("block", [1, 4, 16])
@pytest.mark.parametrize("kind", KINDS)
def test_what_a_value_loses(kind, block):
    """int8: half a step written at once, below one step token by token; e4m3: 2^-4 of the value and the subnormal step."""
    r = np.random.default_rng(3)
    n = 48
    x = (r.normal(size=(n, 2, 64)) * np.exp(0.1 * np.arange(n))[:, None, None]).astype(np.float16).astype(np.float64)
    for counts in ([n], [1] * n, [5, 3, 1, 20, 1, 18]):
        c = o8.PagedCache8(1, 4, 16, 2, 64, 2, 4, kind, block)
        at = 0
        for m in counts:
            c.reserve([1], [m])
            c.append(0, x[at:at + m], -x[at:at + m], [1], [m])
            at += m
        k, v = c.values(0, 1)
        step = np.concatenate([np.repeat(o8.scale(c.scales[0, p, 0]), block, -1) for p in c.rows[1]], -1).T[..., None]
        if kind == "int8":
            limit = step / 2 if counts == [n] else step
        else:
            limit = 2.0 ** -4 * np.abs(x) + step * 2.0 ** (-10 if counts == [n] else -9)
        assert (np.abs(k - x) <= limit).all()
        np.testing.assert_array_equal(v, -k)


def test_one_row_that_is_not_finite_spoils_its_block_only():
    c = o8.PagedCache8(1, 4, 16, 1, 64, 2, 4, "e4m3", 4)
    x = np.ones((12, 1, 64))
    x[5, 0, 3] = np.inf
    c.reserve([0], [12])
    c.append(0, x, x, [0], [12])
    k, _ = c.values(0, 0)
    bad = np.isnan(k).all((1, 2))
    assert bad.tolist() == [4 <= i < 8 for i in range(12)] and not np.isnan(k[~bad]).any()
