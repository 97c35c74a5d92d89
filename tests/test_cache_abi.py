"""The paged-cache entry points refuse bad arguments before they touch a device, and the
workspace size follows from the arguments."""
import ctypes

import numpy as np
import pytest
import torch

import cache_ref
import online_softmax_flashattention_attention_gb300 as pkg
from online_softmax_flashattention_attention_gb300 import build as pkgbuild


@pytest.fixture(scope="module")
def lib():
    pkgbuild.build_library()
    return pkg.load_library()


def _cache(**kw):
    a = dict(size=ctypes.sizeof(pkg.AttnCache), k=0x10000, v=0x20000, k_scale=0x30000, v_scale=0x40000,
             type=pkg.CACHE_E4M3, num_pages=4, page_size=64, num_heads=8, d=128)
    a.update(kw)
    return pkg.AttnCache(*[a[name] for name, _ in pkg.AttnCache._fields_])


def _strides(a, b):
    return (ctypes.c_int64 * 2)(a, b)


def _write(lib, cache, **kw):
    a = dict(K=0x50000, V=0x60000, ks=_strides(1024, 128), vs=_strides(1024, 128), table=0x70000, max_pages=4,
             cu=0x80000, start=0x90000, B=2, total=7)
    a.update(kw)
    return lib.attn_cache_write(None if cache is None else ctypes.byref(cache), a["K"], a["V"], a["ks"], a["vs"],
                                a["table"], a["max_pages"], a["cu"], a["start"], a["B"], a["total"], None)


def _read(lib, cache, **kw):
    a = dict(K=0x50000, V=0x60000, table=0x70000, max_pages=4, cu=0x80000, start=0x90000, B=2, total=7)
    a.update(kw)
    return lib.attn_cache_read(None if cache is None else ctypes.byref(cache), a["K"], a["V"], a["table"],
                               a["max_pages"], a["cu"], a["start"], a["B"], a["total"], None)


def _tree(lib, cache, **kw):
    a = dict(Q=0x50000, O=0x60000, LSE=0xa0000, table=0x70000, max_pages=4, cu=0x80000, ctx=0x90000, mask=0xb0000, B=2,
             Hq=32, max_q=8, total=7, scale=0.1, ws=0xc0000, ws_bytes=1 << 30)
    a.update(kw)
    return lib.attn_fwd_tree(a["Q"], None if cache is None else ctypes.byref(cache), a["O"], a["LSE"], a["table"],
                             a["max_pages"], a["cu"], a["ctx"], a["mask"], a["B"], a["Hq"], a["max_q"], a["total"],
                             a["scale"], a["ws"], a["ws_bytes"], None)


CACHE_FAULTS = [(dict(size=8), -8), (dict(d=96), -3), (dict(type=2), -8), (dict(type=-1), -8), (dict(page_size=0), -2),
                (dict(page_size=24), -2), (dict(page_size=-16), -2), (dict(num_pages=-1), -2), (dict(num_heads=0), -2),
                (dict(k=0), -1), (dict(v=0), -1), (dict(k_scale=0), -1), (dict(v_scale=0), -1), (dict(k=0x10008), -4),
                (dict(v_scale=0x40004), -4)]


@pytest.mark.parametrize("call", [_write, _read, _tree])
@pytest.mark.parametrize("fault,status", CACHE_FAULTS)
def test_cache_faults(lib, call, fault, status):
    assert call(lib, _cache(**fault)) == status
    assert lib.attn_last_error().decode() != ""


@pytest.mark.parametrize("call", [_write, _read, _tree])
def test_common_faults(lib, call):
    assert call(lib, None) == -1
    assert call(lib, _cache(), max_pages=-1) == -2
    assert call(lib, _cache(), max_pages=2 ** 31 // 64) == -2   # 2^31 positions
    assert call(lib, _cache(), B=-1) == -2
    assert call(lib, _cache(), total=-1) == -2
    assert call(lib, _cache(), cu=0) == -1
    assert call(lib, _cache(), table=0) == -1
    assert call(lib, _cache(), table=0x70002) == -4
    assert call(lib, _cache(), cu=0x80001) == -4
    # nothing to do: no pointer is needed, no device either
    assert call(lib, _cache(), B=0, cu=0, table=0) == 0
    assert call(lib, _cache(), total=0, cu=0, table=0) == 0


@pytest.mark.parametrize("call", [_write, _read, _tree])
def test_positions_that_round_past_32_bits(lib, call):
    for page in (16, 32, 64, 128):  # 2^31 - page positions
        assert call(lib, _cache(page_size=page), max_pages=2 ** 31 // page - 1) == -2


@pytest.mark.parametrize("call", [_write, _read])
def test_row_pointers(lib, call):
    assert call(lib, _cache(), K=0) == -1
    assert call(lib, _cache(), V=0x60002) == -4


@pytest.mark.parametrize("strides", [(-8, 128), (1024, 12), (1 << 38, 128)])
def test_write_strides(lib, strides):
    assert _write(lib, _cache(), ks=_strides(*strides)) == -8
    assert _write(lib, _cache(), vs=_strides(*strides)) == -8


@pytest.mark.parametrize("args,status", [
    (dict(max_q=65), -2), (dict(max_q=-1), -2), (dict(Hq=-8), -2), (dict(Hq=12), -2), (dict(scale=0.0), -8),
    (dict(scale=float("nan")), -8), (dict(Q=0), -1), (dict(O=0), -1), (dict(LSE=0), -1), (dict(Q=0x50008), -4),
    (dict(LSE=0xa0002), -4), (dict(mask=0xb0004), -4), (dict(ctx=0x90002), -4), (dict(ws=0), -1), (dict(ws=0xc0008), -4),
    (dict(ws_bytes=1000), -8),
])
def test_tree_faults(lib, args, status):
    assert _tree(lib, _cache(), **args) == status


def test_tree_no_rows(lib):
    assert _tree(lib, _cache(), max_q=0, Q=0, ws=0) == 0
    assert _tree(lib, _cache(), Hq=0, Q=0, ws=0) == 0


def test_workspace_bytes(lib):
    f = pkg.tree_workspace_bytes
    assert f(32, 8, 1, 128) > 0 and f(32, 8, 1, 64) > 0
    assert f(32, 8, 1, 96) == 0 and f(32, 0, 1, 128) == 0 and f(30, 8, 1, 128) == 0 and f(32, 8, 65, 128) == 0
    assert f(32, 8, 0, 128) == 0


def test_python_refusals():
    """The binding's own checks (shapes, types, placement) raise before any call."""
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt)  # noqa: E731
    with pytest.raises(ValueError):
        pkg.attn_cache_write(z(3, 2, 64), z(3, 2, 64), z(4, 2, 16, 64), z(4, 2, 16, 64), z(1, 2, dt=torch.int32),
                             z(2, dt=torch.int32))  # on the CPU
    with pytest.raises(ValueError):
        pkg.attn_cache_read(z(4, 2, 16, 64), z(4, 2, 16, 32), z(1, 2, dt=torch.int32), z(2, dt=torch.int32), 3)
    with pytest.raises(ValueError):
        pkg.attn_fwd_tree(z(1, 2, 64), z(2, 16, 64), z(2, 16, 64), z(1, 2, dt=torch.int32), None, z(2, dt=torch.int32), 1)


def test_reference_quantiser():
    """The tests' own rounding: every e4m3 value is its own nearest, and ties go to even."""
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    fine = codes[~np.isnan(codes)]
    assert np.array_equal(cache_ref.e4m3_round(fine), fine)
    grid = np.unique(np.abs(fine))
    mid = (grid[1:] + grid[:-1]) / 2
    even = torch.from_numpy(mid.astype(np.float32)).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(cache_ref.e4m3_round(mid), even)
    assert cache_ref.quantise_row(np.array([448.0, 1.0]))[1] == 127
    assert cache_ref.quantise_row(np.array([449.0, 1.0]))[1] == 128
    assert cache_ref.quantise_row(np.zeros(4))[1] == 1
