"""Limits of sizes that include/attn.h states for the paged cache and its attention: refused beyond, and the
message says which."""
import ctypes

import pytest

import online_softmax_flashattention_attention_gb300 as pkg
from online_softmax_flashattention_attention_gb300 import build as pkgbuild


@pytest.fixture(scope="module")
def lib():
    pkgbuild.build_library()
    return pkg.load_library()


def _cache(page=64, heads=8):
    return pkg.AttnCache(ctypes.sizeof(pkg.AttnCache), 0x10000, 0x20000, 0x30000, 0x40000, pkg.CACHE_E4M3, 4, page,
                         heads, 128)


def _tree(lib, cache, Hq):
    return lib.attn_fwd_tree(0x50000, ctypes.byref(cache), 0x60000, 0xa0000, 0x70000, 4, 0x80000, 0x90000, None, 2, Hq,
                             8, 7, 0.1, 0xc0000, 1 << 30, None)


def _read(lib, cache):
    return lib.attn_cache_read(ctypes.byref(cache), 0x50000, 0x60000, 0x70000, 4, 0x80000, 0x90000, 2, 7, None)


def _error(lib):
    return lib.attn_last_error().decode()


def test_pages(lib):
    assert _read(lib, _cache(page=65536 + 16)) == -2 and "65536" in _error(lib)
    assert _tree(lib, _cache(page=65536 + 16), 32) == -2 and "65536" in _error(lib)


def test_heads(lib):
    assert _read(lib, _cache(heads=65537)) == -2 and "65536" in _error(lib)
    assert _tree(lib, _cache(), 65536 + 8) == -2
    assert "65536" in _error(lib) and "multiple" not in _error(lib)
    assert _tree(lib, _cache(), 12) == -2 and "multiple" in _error(lib)
