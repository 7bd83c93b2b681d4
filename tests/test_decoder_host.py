"""Decoder-serving calls, host side: argument checks return before any launch (no GPU needed)."""
import ctypes as C

import pytest

from remove_padding_prefix_gb300 import _abi

EINVAL, EUNSUPPORTED, EWORKSPACE = -1, -2, -4


@pytest.fixture(scope="module")
def lib():
    import os
    from remove_padding_prefix_gb300 import build
    if not os.path.exists(_abi.LIB_PATH):
        build.build()
    return _abi.load()


def cfg(**kw):
    d = dict(layers=2, pages=10, page_size=16, kv_heads=2, head_dim=64, slots=4, max_pages=5, dtype=_abi.RPP_BF16)
    d.update(kw)
    return _abi.KvCfg(**d)


def cache(**kw):
    d = dict(pool=256, table=256, lens=256, refs=256)
    d.update(kw)
    return _abi.KvArrays(**d)


BAD_CFG = [
    (dict(layers=0), EINVAL), (dict(pages=0), EINVAL), (dict(page_size=0), EINVAL), (dict(kv_heads=-1), EINVAL),
    (dict(head_dim=0), EINVAL), (dict(slots=0), EINVAL), (dict(max_pages=0), EINVAL),
    (dict(slots=65536, max_pages=65536), EINVAL), (dict(max_pages=1 << 28), EINVAL),
    (dict(dtype=_abi.RPP_F32), EUNSUPPORTED), (dict(dtype=_abi.RPP_I8), EUNSUPPORTED),
    (dict(slots=1, page_size=3, max_pages=715827882), EINVAL),        # 2^31 - 2 tokens: a page more is past an int
    (dict(pages=(1 << 30) + 1), EUNSUPPORTED),
    (dict(pages=1 << 30, layers=1 << 16, page_size=1 << 16, kv_heads=512, head_dim=128), EUNSUPPORTED),   # 2^80 bytes
    (dict(pages=1 << 30, layers=1 << 16, page_size=16, kv_heads=32, head_dim=128), EUNSUPPORTED),         # 2^64 bytes
    (dict(head_dim=60), EUNSUPPORTED), (dict(slots=65537), EUNSUPPORTED), (dict(kv_heads=1025), EUNSUPPORTED),
]


def calls(lib, c, a, **kw):
    """The status of each call on a cache, with arguments that are fine unless given."""
    g = dict(list=256, n=2, err=256, k=256, v=256, ld=128, rows=2, layer=0, cu=256, ws=256, ws_bytes=1 << 40, out=256,
             q=256, ldq=256, nh=4, scale=0.125, counts=256, to=256)
    g.update(kw)
    p, r = C.byref(c), C.byref(a)
    return {
        "reserve": lambda: lib.rpp_kv_reserve(p, r, g["list"], g["counts"], g["n"], g["err"], None),
        "append": lambda: lib.rpp_kv_append(p, r, g["layer"], g["k"], g["v"], g["ld"], g["list"], g["cu"], g["n"],
                                            g["rows"], g["err"], None),
        "fork": lambda: lib.rpp_kv_fork(p, r, g["list"], g["to"], g["n"], g["err"], None),
        "free": lambda: lib.rpp_kv_free(p, r, g["list"], g["n"], g["err"], None),
        "compact": lambda: lib.rpp_kv_compact(p, r, g["out"], 256, 256, 256, g["ws"], g["ws_bytes"], g["err"], None),
        "decode": lambda: lib.rpp_attention_decode(p, r, g["layer"], g["q"], g["ldq"], g["list"], g["n"], g["nh"],
                                                   g["scale"], g["out"], g["ws"], g["ws_bytes"], g["err"], None),
    }


ALL = ("reserve", "append", "fork", "free", "compact", "decode")


@pytest.mark.parametrize("kw,status", BAD_CFG)
def test_configurations(lib, kw, status):
    c = cfg(**kw)
    for name, call in calls(lib, c, cache()).items():
        assert call() == status, name
    assert lib.rpp_kv_pool_bytes(C.byref(c)) == 0
    assert lib.rpp_kv_compact_workspace_bytes(C.byref(c)) == 0
    assert lib.rpp_attention_decode_workspace_bytes(C.byref(c), 1, 4) == 0


@pytest.mark.parametrize("kw", [dict(pool=None), dict(table=None), dict(lens=None), dict(refs=None), dict(pool=264),
                                dict(refs=260)])
def test_arrays(lib, kw):
    for name, call in calls(lib, cfg(), cache(**kw)).items():
        assert call() == EINVAL, name


@pytest.mark.parametrize("kw,status,names", [
    (dict(n=0), EINVAL, ("reserve", "append", "fork", "free", "decode")),
    (dict(n=4097, rows=5000), EUNSUPPORTED, ("reserve", "append", "fork", "free", "decode")),
    (dict(list=None), EINVAL, ("reserve", "append", "fork", "free")),
    (dict(list=None, n=5), EINVAL, ("decode",)),                       # more rows than slots
    (dict(err=None), EINVAL, ("reserve", "append", "fork", "free", "compact")),
    (dict(counts=None), EINVAL, ("reserve",)),
    (dict(to=None), EINVAL, ("fork",)),
    (dict(layer=2), EINVAL, ("append", "decode")), (dict(layer=-1), EINVAL, ("append", "decode")),
    (dict(k=None), EINVAL, ("append",)), (dict(v=258), EINVAL, ("append",)),
    (dict(ld=127), EINVAL, ("append",)), (dict(ld=120), EINVAL, ("append",)),
    (dict(rows=0x7fffffff), EUNSUPPORTED, ("append",)),
    (dict(rows=0), EINVAL, ("append",)), (dict(cu=None, rows=1), EINVAL, ("append",)),
    (dict(out=None), EINVAL, ("compact", "decode")),
    (dict(ws=None), EINVAL, ("compact", "decode")), (dict(ws=260), EINVAL, ("compact", "decode")),
    (dict(out=512), EINVAL, ("compact",)),                             # a new table, but the cache's own counts
    (dict(ws_bytes=8), EWORKSPACE, ("compact", "decode")),
    (dict(q=None), EINVAL, ("decode",)), (dict(q=264), EINVAL, ("decode",)), (dict(ldq=255), EINVAL, ("decode",)),
    (dict(ldq=248), EINVAL, ("decode",)), (dict(nh=3), EINVAL, ("decode",)), (dict(nh=0), EINVAL, ("decode",)),
    (dict(scale=0.0), EINVAL, ("decode",)), (dict(scale=float("nan")), EINVAL, ("decode",)),
    (dict(scale=float("inf")), EINVAL, ("decode",)), (dict(scale=-1.0), EINVAL, ("decode",)),
])
def test_arguments(lib, kw, status, names):
    every = calls(lib, cfg(), cache(), **kw)
    for name in names:
        assert every[name]() == status, name


def test_decode_takes_64_and_128_on_pages_of_whole_sixteens(lib):
    for kw in (dict(head_dim=96), dict(head_dim=32), dict(page_size=8), dict(page_size=24)):
        assert calls(lib, cfg(**kw), cache(), ldq=1024)["decode"]() == EUNSUPPORTED


def test_sizes(lib):
    c = cfg()
    assert lib.rpp_kv_pool_bytes(C.byref(c)) == 2 * 10 * 2 * 2 * 16 * 64 * 2
    assert lib.rpp_kv_compact_workspace_bytes(C.byref(c)) == (2 + 10) * 4
    big = cfg(pages=1 << 20, layers=80, kv_heads=8, head_dim=128)
    assert lib.rpp_kv_pool_bytes(C.byref(big)) == (1 << 20) * 80 * 2 * 8 * 16 * 128 * 2
    small = lib.rpp_attention_decode_workspace_bytes(C.byref(c), 1, 2)
    assert 0 < small < lib.rpp_attention_decode_workspace_bytes(C.byref(c), 1, 32)
    assert lib.rpp_attention_decode_workspace_bytes(C.byref(c), 1, 3) == 0      # not a multiple of the kv heads
    assert lib.rpp_attention_decode_workspace_bytes(C.byref(c), 4097, 2) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), EINVAL), (dict(k=None), EINVAL), (dict(v=None), EINVAL), (dict(cu=None), EINVAL),
    (dict(out=None), EINVAL), (dict(B=0), EINVAL), (dict(T=0), EINVAL), (dict(max_len=0), EINVAL), (dict(nh=0), EINVAL),
    (dict(nkv=0), EINVAL), (dict(nh=5), EINVAL), (dict(d=0), EINVAL), (dict(q=264), EINVAL), (dict(v=258), EINVAL),
    (dict(out=8), EINVAL), (dict(ldq=260), EINVAL), (dict(ldq=248), EINVAL), (dict(ld=127), EINVAL), (dict(ld=120), EINVAL),
    (dict(scale=0.0), EINVAL), (dict(scale=float("nan")), EINVAL),
    (dict(dtype=_abi.RPP_F32), EUNSUPPORTED), (dict(dtype=_abi.RPP_I8), EUNSUPPORTED),
    (dict(d=96, ldq=1024, ld=1024), EUNSUPPORTED), (dict(B=4097), EUNSUPPORTED), (dict(max_len=262145), EUNSUPPORTED),
    (dict(nh=1 << 24, T=1 << 20, ldq=1 << 30), EUNSUPPORTED),
    (dict(T=0x7fffffff), EUNSUPPORTED),
])
def test_causal_arguments(lib, kw, status):
    g = dict(q=256, k=256, v=256, ldq=256, ld=128, cu=256, B=3, T=100, max_len=60, nh=4, nkv=2, d=64,
             dtype=_abi.RPP_BF16, scale=0.125, out=256)
    g.update(kw)
    assert lib.rpp_attention_causal_varlen(g["q"], g["k"], g["v"], g["ldq"], g["ld"], g["cu"], g["B"], g["T"],
                                           g["max_len"], g["nh"], g["nkv"], g["d"], g["dtype"], g["scale"], g["out"],
                                           None, None) == status


@pytest.mark.parametrize("scale", [3.0e38, 2.4e38])
def test_scales_whose_base_2_form_overflows(lib, scale):
    """The kernels work with scale * log2(e): past the largest float it would make 0 scores NaN."""
    assert calls(lib, cfg(), cache(), scale=scale)["decode"]() == EINVAL
    assert lib.rpp_attention_causal_varlen(256, 256, 256, 256, 128, 256, 3, 100, 60, 4, 2, 64, _abi.RPP_BF16, scale, 256,
                                           None, None) == EINVAL
