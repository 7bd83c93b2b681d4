"""Rows read back: what the binding refuses, and reads of more rows than one pass of the grid has."""
import pytest
import torch

import remove_padding_prefix_gb300 as rpp
from gpu_util import TDT, dev
from test_gpu_kv8 import ints

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("make", [lambda: rpp.KvCache8(1, 8, 16, 2, 64, 4, 4, "e4m3", 16, dev()),
                                  lambda: rpp.KvCache(1, 8, 16, 2, 64, 4, 4, "bf16", dev())])
def test_rows_and_dtype_beside_tensors_that_have_their_own(make):
    c = make()
    rpp.kv_reserve(c, ints([1]), ints([5]))
    x = torch.randn(5, 256, device=dev()).to(torch.bfloat16)
    cu = ints([0, 5])
    rpp.kv_append(c, 0, x[:, :128], x[:, 128:], ints([1]), cu)
    out = torch.full((5, 256), 3.0, dtype=torch.bfloat16, device=dev())
    k, v = out[:, :128], out[:, 128:]
    for kw in (dict(dtype="fp16"), dict(dtype=torch.float16), dict(dtype=torch.float32), dict(rows=4), dict(rows=6)):
        with pytest.raises(ValueError):
            rpp.kv_read(c, 0, ints([1]), cu, k=k, v=v, **kw)
    assert (out == 3).all()
    rpp.kv_read(c, 0, ints([1]), cu, k=k, v=v, rows=5, dtype="bf16")
    want = rpp.kv_read(c, 0, ints([1]), cu, rows=5, dtype=torch.bfloat16)
    assert rpp.get_device_error(c.err) == 0
    assert torch.equal(k, want[0]) and torch.equal(v, want[1])
