"""attn_cache_evict refuses new lengths that lie on the old ones: a sequence's CTAs read its old length while
another's write the new ones."""
import ctypes

import pytest

import online_softmax_flashattention_attention_gb300 as pkg
from online_softmax_flashattention_attention_gb300 import build as pkgbuild

LENS, B = 0x70000, 5


@pytest.mark.parametrize("out,overlaps", [(LENS, True), (LENS + 4, True), (LENS - 4, True), (LENS + 4 * (B - 1), True),
                                          (LENS - 4 * (B - 1), True), (LENS + 4 * B, False), (LENS - 4 * B, False)])
def test_overlapping_lengths(out, overlaps):
    pkgbuild.build_library()
    lib = pkg.load_library()
    c = pkg.AttnCache(ctypes.sizeof(pkg.AttnCache), 0x10000, 0x20000, 0x30000, 0x40000, pkg.CACHE_E4M3, 4, 64, 8, 128)
    # (kept is out of line, which is looked at after the overlap: no call goes further than the checks)
    rc = lib.attn_cache_evict(ctypes.byref(c), 0x50000, 0x60000, 4, None, 0, LENS, 0x80001, out, B, 100, 4, 16, None)
    assert rc == (-8 if overlaps else -4)
    assert ("overlap" in lib.attn_last_error().decode()) == overlaps
