"""Pins of the decoder oracle: causal attention against torch, the list-kept cache against plain sequences."""
import numpy as np
import pytest
import torch

import oracle.decoder as od


def test_causal_attention_against_torch():
    rng = np.random.default_rng(0)
    lens, nh, nkv, d = [5, 0, 1, 9], 6, 2, 8
    cu = np.concatenate([[0], np.cumsum(lens)])
    q, k, v = (rng.standard_normal((cu[-1], n * d)) for n in (nh, nkv, nkv))
    got = od.causal_attention(q, k, v, cu, nh, nkv, d)
    for b, n in enumerate(lens):
        if not n:
            continue
        def heads(x, h):
            return torch.tensor(x[cu[b]:cu[b + 1]]).view(n, h, d).transpose(0, 1)
        kk, vv = (heads(x, nkv).repeat_interleave(nh // nkv, 0) for x in (k, v))
        want = torch.nn.functional.scaled_dot_product_attention(heads(q, nh), kk, vv, is_causal=True)
        np.testing.assert_allclose(got[cu[b]:cu[b + 1]], want.transpose(0, 1).reshape(n, -1).numpy(), atol=1e-12)


def test_the_last_row_is_the_decode_of_its_sequence():
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((3, 7, 8))
    rows = od.causal_attention(q, k, v, [0, 7], 1, 1, 8)
    np.testing.assert_allclose(rows[6], od.attend(q[6], k, v, 8 ** -0.5), atol=1e-14)
    np.testing.assert_allclose(rows[0], v[0], atol=1e-14)
    assert (od.attend(q[0], k[:0], v[:0], 1.0) == 0).all()


def test_cache_keeps_what_plain_lists_keep():
    """A walk through the calls; every slot reads back the rows that a list of its own holds."""
    rng = np.random.default_rng(2)
    c = od.PagedCache(2, 40, 4, 2, 8, 6, 8)
    plain = [[] for _ in range(6)]
    for _ in range(300):
        what = rng.integers(0, 5)
        s = int(rng.integers(0, 6))
        try:
            if what < 2:
                n = int(rng.integers(0, 6))
                c.reserve([s], [n])
                rows = rng.integers(0, 1 << 16, (2, 2, n, 2, 8), dtype=np.uint16)     # K / V, layer
                for layer in range(2):
                    c.append(layer, rows[0, layer], rows[1, layer], [s], [n])
                plain[s] += [rows[:, :, j] for j in range(n)]
            elif what == 2:
                t = int(rng.integers(0, 6))
                c.fork([t], [s])
                plain[s] = list(plain[t])
            elif what == 3:
                c.free([s])
                plain[s] = []
            else:
                _, live = c.compact()
                assert all(r == 0 for r in c.refs[live:]) and all(r > 0 for r in c.refs[:live])
        except od.CacheError:
            pass
        for s in range(6):
            for layer in range(2):
                k, v = c.sequence(layer, s)
                assert len(k) == len(plain[s])
                for j, row in enumerate(plain[s]):
                    assert (k[j] == row[0, layer]).all() and (v[j] == row[1, layer]).all()
        used = [p for row in c.rows for p in row]
        assert [used.count(p) for p in range(40)] == c.refs


@pytest.mark.parametrize("call,code", [
    (lambda c: c.reserve([0, 0], [1, 1]), od.SLOT), (lambda c: c.reserve([4], [1]), od.SLOT),
    (lambda c: c.reserve([0], [13]), od.LENGTH), (lambda c: c.reserve([0, 1, 2], [12, 12, 5]), od.FULL),
    (lambda c: c.fork([3], [3]), od.SLOT), (lambda c: c.fork([0], [3]), od.SLOT), (lambda c: c.free([1, 1]), od.SLOT),
])
def test_refusals_leave_the_state(call, code):
    c = od.PagedCache(1, 7, 4, 1, 8, 4, 3)
    c.reserve([3], [2])
    before = (c.table().copy(), list(c.lens), list(c.refs))
    with pytest.raises(od.CacheError) as e:
        call(c)
    assert e.value.code == code
    assert (c.table() == before[0]).all() and c.lens == before[1] and c.refs == before[2]
