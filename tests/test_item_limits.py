"""Launches are refused whose items a CTA could not count past in 32 bits: a CTA goes through its items by an
index that ends up to two rounds of CTAs after the last one, and one that wrapped would name items that are
not there."""
import ctypes

import pytest

import online_softmax_flashattention_attention_gb300 as pkg
from online_softmax_flashattention_attention_gb300 import build as pkgbuild

MOST = 2 ** 31 - 1 - 2 * 4096
BAD_SHAPE, NULLPTR = -2, -1


@pytest.fixture(scope="module")
def lib():
    pkgbuild.build_library()
    return pkg.load_library()


def _varlen(lib, B, H, max_q, total=7, total_k=9):
    return lib.attn_fwd_varlen(None, None, None, None, None, None, None, B, H, max_q, total, total_k, 64, 0.125, 1, None)


def _prompt(lib, B, H, max_q, total=7):
    st = (ctypes.c_int64 * 2)(64, 64)
    return lib.attn_fwd_prompt(None, None, None, None, None, st, st, st, st, None, None, B, H, 1, max_q, total, 9, 64, 0.125, 1,
                               None, 0, None)


@pytest.mark.parametrize("call", [_varlen, _prompt])
@pytest.mark.parametrize("B,H,max_q,status", [
    (151 * 331, 42966, 1, BAD_SHAPE),             # 2147483646 items, a prime's neighbour
    (1, 42966, 128 * 151 * 331, BAD_SHAPE),       # the same, as tiles of one sequence
    (2 ** 15, 2 ** 16 - 1, 1, NULLPTR),           # 2^31 - 2^15: enough room, so the pointers are looked at
    (2 ** 15, 2 ** 16 - 1, 129, BAD_SHAPE),
    (2 ** 15, 2 ** 16 - 2, 1, NULLPTR),
    (1, 1, 2 ** 31 - 255, BAD_SHAPE),             # rows are rounded up to a block of 128 in 32 bits
    (1, 1, 2 ** 31 - 1, BAD_SHAPE),
    (1, 1, 2 ** 31 - 256, NULLPTR),
])
def test_items(lib, call, B, H, max_q, status):
    assert H <= 65536 and (status == NULLPTR) == (max_q <= 2 ** 31 - 256 and B * H * -(-max_q // 128) <= MOST)
    assert call(lib, B, H, max_q) == status


def test_packed_rows(lib):
    for kw in (dict(total=2 ** 31 - 255), dict(total_k=2 ** 31 - 1)):
        assert _varlen(lib, 1, 1, 8, **kw) == BAD_SHAPE
    assert _varlen(lib, 1, 2 ** 30, 1, total=2 ** 31 - 256) == BAD_SHAPE  # 2^68 values: more than 64 bits hold


def test_dense_and_splits(lib):
    def fwd(BH, Nq):
        return pkg.attn_fwd_raw(None, None, None, None, None, 1, BH, Nq, 16, 64, 0.125, 0, None, None)
    assert fwd(2 ** 31 - 2, 1) == BAD_SHAPE and fwd(MOST + 1, 1) == BAD_SHAPE and fwd(MOST, 1) == NULLPTR
    def states(BH, S):  # noqa: E306
        return lib.attn_fwd_states(0x10000, 0x20000, 0x30000, 0x40000, 0x50000, 0x60008, 1, BH, 1, 16, 64, 0.125, 0, None, S, None)
    assert states(4, 3) == -4  # (the last pointer is out of line: no call goes further than the checks)
    def states_ok(BH, S):  # noqa: E306
        return lib.attn_fwd_states(0x10000, 0x20000, 0x30000, 0x40000, 0x50000, 0x60000, 1, BH, 1, 16, 64, 0.125, 0, None, S, None)
    assert states_ok(2 ** 29, 4) == BAD_SHAPE and states_ok((MOST + 1) // 3 + 1, 3) == BAD_SHAPE


@pytest.mark.parametrize("ctas", [1, 132, 152, 4096])
def test_the_index_after_the_last_stays_in_32_bits(ctas):
    """item_of: round r takes items r G .. r G + G - 1, forward and backward in turn."""
    for cta in (0, ctas // 2, ctas - 1):
        for r in range(max(0, MOST // ctas - 2), MOST // ctas + 3):
            item = r * ctas + (ctas - 1 - cta if r & 1 else cta)
            assert r * ctas + ctas - 1 < 2 ** 31
            if item >= MOST:
                break
        else:
            raise AssertionError("the walk ends")
