"""The 8-bit cache's calls, host side: argument checks return before any launch (no GPU needed)."""
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


def cfg(block=16, **kw):
    d = dict(layers=2, pages=10, page_size=32, kv_heads=2, head_dim=64, slots=4, max_pages=5, dtype=_abi.RPP_E4M3)
    d.update(kw)
    return _abi.Kv8Cfg(_abi.KvCfg(**d), block)


def cache(scales=256, **kw):
    d = dict(pool=256, table=256, lens=256, refs=256)
    d.update(kw)
    return _abi.Kv8Arrays(_abi.KvArrays(**d), scales)


def calls(lib, c, a, **kw):
    """The status of each call on a cache, with arguments that are fine unless given."""
    g = dict(list=256, n=2, err=256, k=256, v=256, ld=128, rows=2, layer=0, cu=256, starts=None, ws=256, ws_bytes=1 << 40,
             out=256, q=256, ldq=256, nh=4, scale=0.125, counts=256, to=256, dtype=_abi.RPP_BF16)
    g.update(kw)
    p, r = C.byref(c) if c is not None else None, C.byref(a) if a is not None else None
    return {
        "reserve": lambda: lib.rpp_kv8_reserve(p, r, g["list"], g["counts"], g["n"], g["err"], None),
        "append": lambda: lib.rpp_kv8_append(p, r, g["layer"], g["k"], g["v"], g["dtype"], g["ld"], g["list"], g["cu"],
                                             g["n"], g["rows"], g["err"], None),
        "read": lambda: lib.rpp_kv8_read(p, r, g["layer"], g["list"], g["starts"], g["cu"], g["n"], g["rows"], g["k"],
                                         g["v"], g["dtype"], g["ld"], g["err"], None),
        "fork": lambda: lib.rpp_kv8_fork(p, r, g["list"], g["to"], g["n"], g["err"], None),
        "free": lambda: lib.rpp_kv8_free(p, r, g["list"], g["n"], g["err"], None),
        "compact": lambda: lib.rpp_kv8_compact(p, r, g["out"], 256, 256, 256, g["ws"], g["ws_bytes"], g["err"], None),
        "decode": lambda: lib.rpp_attention_decode8(p, r, g["layer"], g["q"], g["dtype"], g["ldq"], g["list"], g["n"],
                                                    g["nh"], g["scale"], g["out"], g["ws"], g["ws_bytes"], g["err"], None),
    }


def refused(lib, c, status):
    for name, call in calls(lib, c, cache()).items():
        assert call() == status, name
    p = C.byref(c)
    assert lib.rpp_kv8_pool_bytes(p) == lib.rpp_kv8_scales_bytes(p) == lib.rpp_kv8_compact_workspace_bytes(p) == 0
    assert lib.rpp_attention_decode8_workspace_bytes(p, 1, 4) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(layers=0), EINVAL), (dict(pages=0), EINVAL), (dict(page_size=0), EINVAL), (dict(kv_heads=-1), EINVAL),
    (dict(head_dim=0), EINVAL), (dict(slots=0), EINVAL), (dict(max_pages=0), EINVAL), (dict(block=0), EINVAL),
    (dict(block=-16), EINVAL), (dict(slots=65536, max_pages=65536), EINVAL),
    (dict(dtype=_abi.RPP_F32), EUNSUPPORTED), (dict(dtype=_abi.RPP_F16), EUNSUPPORTED),
    (dict(dtype=_abi.RPP_BF16), EUNSUPPORTED), (dict(dtype=5), EUNSUPPORTED), (dict(dtype=-1), EUNSUPPORTED),
    (dict(block=64), EUNSUPPORTED), (dict(block=3), EUNSUPPORTED), (dict(block=12, page_size=48), EUNSUPPORTED),
    (dict(block=256, page_size=256), EUNSUPPORTED), (dict(block=32, page_size=48), EUNSUPPORTED),
    (dict(head_dim=32), EUNSUPPORTED), (dict(head_dim=96), EUNSUPPORTED), (dict(head_dim=256), EUNSUPPORTED),
    (dict(page_size=8, block=8), EUNSUPPORTED), (dict(page_size=24, block=8), EUNSUPPORTED),
    (dict(pages=(1 << 30) + 1), EUNSUPPORTED), (dict(slots=65537), EUNSUPPORTED), (dict(kv_heads=1025), EUNSUPPORTED),
    (dict(pages=1 << 30, layers=1 << 16, page_size=32, kv_heads=32, head_dim=128), EUNSUPPORTED),      # 2^64 bytes
])
def test_configurations(lib, kw, status):
    refused(lib, cfg(**kw), status)


def test_no_configuration_or_cache(lib):
    for name, call in calls(lib, None, cache()).items():
        assert call() == EINVAL, name
    for name, call in calls(lib, cfg(), None).items():
        assert call() == EINVAL, name


@pytest.mark.parametrize("kw", [dict(pool=None), dict(table=None), dict(lens=None), dict(refs=None), dict(pool=264),
                                dict(refs=260), dict(scales=None), dict(scales=264)])
def test_arrays(lib, kw):
    for name, call in calls(lib, cfg(), cache(**kw)).items():
        assert call() == EINVAL, name


@pytest.mark.parametrize("kw,status,names", [
    (dict(n=0), EINVAL, ("reserve", "append", "read", "fork", "free", "decode")),
    (dict(n=4097, rows=5000), EUNSUPPORTED, ("reserve", "append", "read", "fork", "free", "decode")),
    (dict(list=None), EINVAL, ("reserve", "append", "read", "fork", "free")),
    (dict(list=None, n=5), EINVAL, ("decode",)),
    (dict(err=None), EINVAL, ("reserve", "append", "read", "fork", "free", "compact")),
    (dict(counts=None), EINVAL, ("reserve",)), (dict(to=None), EINVAL, ("fork",)),
    (dict(layer=2), EINVAL, ("append", "read", "decode")), (dict(layer=-1), EINVAL, ("append", "read", "decode")),
    (dict(k=None), EINVAL, ("append", "read")), (dict(v=258), EINVAL, ("append", "read")),
    (dict(ld=127), EINVAL, ("append", "read")), (dict(ld=120), EINVAL, ("append", "read")),
    (dict(rows=0x7fffffff), EUNSUPPORTED, ("append", "read")), (dict(rows=0), EINVAL, ("append", "read")),
    (dict(cu=None, rows=1), EINVAL, ("append", "read")),
    (dict(dtype=_abi.RPP_F32), EUNSUPPORTED, ("append", "read", "decode")),
    (dict(dtype=_abi.RPP_E4M3), EUNSUPPORTED, ("append", "read", "decode")),
    (dict(out=None), EINVAL, ("compact", "decode")),
    (dict(ws=None), EINVAL, ("compact", "decode")), (dict(ws=260), EINVAL, ("compact", "decode")),
    (dict(out=512), EINVAL, ("compact",)), (dict(ws_bytes=8), EWORKSPACE, ("compact", "decode")),
    (dict(q=None), EINVAL, ("decode",)), (dict(q=264), EINVAL, ("decode",)), (dict(ldq=255), EINVAL, ("decode",)),
    (dict(ldq=248), EINVAL, ("decode",)), (dict(nh=3), EINVAL, ("decode",)), (dict(nh=0), EINVAL, ("decode",)),
    (dict(scale=0.0), EINVAL, ("decode",)), (dict(scale=float("nan")), EINVAL, ("decode",)),
    (dict(scale=3.0e38), EINVAL, ("decode",)),
])
def test_arguments(lib, kw, status, names):
    every = calls(lib, cfg(), cache(), **kw)
    for name in names:
        assert every[name]() == status, name


def test_reading_a_cache_of_16_bits(lib):
    """rpp_kv_read's own checks; a cache of codes is not one of its."""
    def status(dtype=_abi.RPP_F16, **kw):
        g = dict(k=256, v=256, ld=128, rows=2, n=2, layer=0, err=256, list=256, cu=None, starts=None)
        g.update(kw)
        c = cfg(dtype=dtype).kv
        return lib.rpp_kv_read(C.byref(c), C.byref(cache().kv), g["layer"], g["list"], g["starts"], g["cu"], g["n"],
                               g["rows"], g["k"], g["v"], g["ld"], g["err"], None)
    for kw in (dict(k=None), dict(v=8), dict(ld=124), dict(rows=1), dict(n=0), dict(layer=2), dict(err=None), dict(list=None)):
        assert status(**kw) == EINVAL, kw
    assert status(dtype=_abi.RPP_I8) == status(dtype=_abi.RPP_E4M3) == status(n=4097, rows=5000) == EUNSUPPORTED


def test_sizes(lib):
    c = cfg(block=4)
    assert lib.rpp_kv8_pool_bytes(C.byref(c)) == 2 * 10 * 2 * 2 * 32 * 64
    assert lib.rpp_kv8_scales_bytes(C.byref(c)) == 2 * 10 * 2 * 2 * 8
    assert lib.rpp_kv8_compact_workspace_bytes(C.byref(c)) == (2 + 10) * 4
    small = lib.rpp_attention_decode8_workspace_bytes(C.byref(c), 1, 2)
    assert 0 < small < lib.rpp_attention_decode8_workspace_bytes(C.byref(c), 1, 8)
    assert lib.rpp_attention_decode8_workspace_bytes(C.byref(c), 1, 3) == 0
    assert lib.rpp_attention_decode8_workspace_bytes(C.byref(c), 4097, 2) == 0
