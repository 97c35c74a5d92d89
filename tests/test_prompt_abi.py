"""attn_qk_rotate, attn_fwd_prompt, attn_cache_weigh and attn_cache_evict refuse bad arguments before they
touch a device."""
import ctypes

import pytest
import torch

import online_softmax_flashattention_attention_gb300 as pkg
from online_softmax_flashattention_attention_gb300 import build as pkgbuild


@pytest.fixture(scope="module")
def lib():
    pkgbuild.build_library()
    return pkg.load_library()


def _st(a, b):
    return (ctypes.c_int64 * 2)(a, b)


def _cache(**kw):
    a = dict(size=ctypes.sizeof(pkg.AttnCache), k=0x10000, v=0x20000, k_scale=0x30000, v_scale=0x40000,
             type=pkg.CACHE_E4M3, num_pages=4, page_size=64, num_heads=8, d=128)
    a.update(kw)
    return pkg.AttnCache(*[a[name] for name, _ in pkg.AttnCache._fields_])


def _rotate(lib, **kw):
    a = dict(Q=0x10000, K=0x20000, Qo=0x30000, Ko=0x40000, qs=_st(4096, 128), ks=_st(1024, 128), qos=_st(4096, 128),
             kos=_st(1024, 128), cu=0x50000, start=0x60000, pos=0x70000, freq=0x80000, r=64, inter=0, qw=0x90000, kw=0xa0000,
             wt=0, eps=1e-6, B=2, Hq=32, Hkv=8, d=128, total=7)
    a.update(kw)
    return lib.attn_qk_rotate(*[a[n] for n in ("Q", "K", "Qo", "Ko", "qs", "ks", "qos", "kos", "cu", "start", "pos", "freq", "r",
                                               "inter", "qw", "kw", "wt", "eps", "B", "Hq", "Hkv", "d", "total")], None)


def _prompt(lib, **kw):
    a = dict(Q=0x10000, K=0x20000, V=0x30000, O=0x40000, LSE=0x50000, qs=_st(4096, 128), ks=_st(1024, 128), vs=_st(1024, 128),
             os=_st(4096, 128), cuq=0x60000, cuk=0x70000, B=2, Hq=32, Hkv=8, maxq=7, tq=7, tk=9, d=128, scale=0.1, causal=1, ws=None, wsb=0)
    a.update(kw)
    return lib.attn_fwd_prompt(*[a[n] for n in ("Q", "K", "V", "O", "LSE", "qs", "ks", "vs", "os", "cuq", "cuk", "B", "Hq", "Hkv",
                                                "maxq", "tq", "tk", "d", "scale", "causal", "ws", "wsb")], None)


def _weigh(lib, cache=None, **kw):
    a = dict(Q=0x50000, LSE=0x60000, w=0x70000, out=0x80000, table=0x90000, max_pages=4, cu=0xa0000, ctx=0xb0000, B=2, Hq=32,
             total=7, scale=0.1, decay=0.5)
    a.update(kw)
    c = _cache() if cache is None else cache
    return lib.attn_cache_weigh(a["Q"], a["LSE"], ctypes.byref(c), *[a[n] for n in (
        "w", "out", "table", "max_pages", "cu", "ctx", "B", "Hq", "total", "scale", "decay")], None)


def _evict(lib, cache=None, **kw):
    a = dict(w=0x50000, table=0x60000, max_pages=4, to=0, to_pages=0, lens=0x70000, kept=0x80000, out_lens=0x90000, B=2, keep=100,
             sink=4, recent=16)
    a.update(kw)
    c = _cache() if cache is None else cache
    return lib.attn_cache_evict(ctypes.byref(c), *[a[n] for n in ("w", "table", "max_pages", "to", "to_pages", "lens", "kept",
                                                                  "out_lens", "B", "keep", "sink", "recent")], None)


@pytest.mark.parametrize("args,status", [
    (dict(d=96), -3), (dict(B=-1), -2), (dict(total=-1), -2), (dict(Hq=-1), -2), (dict(Hkv=65537), -2), (dict(r=12), -2),
    (dict(r=72), -2), (dict(r=-8), -2), (dict(wt=2), -8), (dict(eps=-1.0), -8), (dict(eps=float("nan")), -8), (dict(cu=0), -2),
    (dict(Q=0), -1), (dict(Ko=0), -1), (dict(K=0x20008), -4), (dict(Qo=0x30002), -4), (dict(qs=None), -1), (dict(kos=None), -1),
    (dict(qs=_st(4096, 12)), -8), (dict(ks=_st(-8, 128)), -8), (dict(qos=_st(4096, 0)), -8), (dict(kos=_st(1 << 38, 128)), -8),
    (dict(freq=0), -1), (dict(freq=0x80002), -4), (dict(pos=0x70001), -4), (dict(cu=0x50002), -4), (dict(start=0x60002), -4),
    (dict(qw=0x90001), -4), (dict(kw=0xa0002, wt=1), -4),
])
def test_rotate_faults(lib, args, status):
    assert _rotate(lib, **args) == status
    assert lib.attn_last_error().decode() != ""


def test_rotate_nothing_to_do(lib):
    assert _rotate(lib, total=0, Q=0, qs=None, freq=0) == 0
    assert _rotate(lib, B=0, Q=0) == 0
    assert _rotate(lib, Hq=0, Hkv=0, Q=0, K=0) == 0


@pytest.mark.parametrize("args,status", [
    (dict(d=32), -3), (dict(B=-1), -2), (dict(Hq=30), -2), (dict(Hkv=0), -2), (dict(Hkv=-8), -2), (dict(Hq=65544), -2),
    (dict(maxq=-1), -2), (dict(tq=-1), -2), (dict(tk=-1), -2), (dict(maxq=2 ** 31 - 255), -2), (dict(tk=2 ** 31 - 1), -2),
    (dict(B=65536, Hq=65536, maxq=128), -2), (dict(scale=0.0), -8), (dict(scale=float("inf")), -8), (dict(Q=0), -1), (dict(V=0), -1),
    (dict(LSE=0), -1), (dict(cuk=0), -1), (dict(O=0x40008), -4), (dict(K=0x20004), -4), (dict(LSE=0x50002), -4),
    (dict(cuq=0x60001), -4), (dict(qs=_st(4095, 128)), -8), (dict(os=_st(0, 128)), -8), (dict(ks=_st(1024, 0)), -8),
    (dict(vs=_st(1 << 38, 128)), -8), (dict(vs=None), -1),
])
def test_prompt_faults(lib, args, status):
    assert _prompt(lib, **args) == status
    assert lib.attn_last_error().decode() != ""


def test_prompt_nothing_to_do(lib):
    for kw in (dict(B=0), dict(Hq=0), dict(maxq=0), dict(tq=0)):
        assert _prompt(lib, Q=0, O=0, LSE=0, cuq=0, qs=None, **kw) == 0


@pytest.mark.parametrize("args,status", [
    (dict(B=-1), -2), (dict(Hq=-8), -2), (dict(total=-1), -2), (dict(Hq=12), -2), (dict(Hq=65544), -2), (dict(max_pages=-1), -2),
    (dict(max_pages=2 ** 25), -2), (dict(scale=-1.0), -8), (dict(decay=float("nan")), -8), (dict(decay=float("inf")), -8),
    (dict(Q=0), -1), (dict(LSE=0), -1), (dict(out=0), -1), (dict(w=0), -1), (dict(table=0), -1), (dict(cu=0), -1),
    (dict(Q=0x50004), -4), (dict(LSE=0x60001), -4), (dict(w=0x70002), -4), (dict(out=0x80002), -4), (dict(ctx=0xb0002), -4),
])
def test_weigh_faults(lib, args, status):
    assert _weigh(lib, **args) == status
    assert lib.attn_last_error().decode() != ""


CACHE_FAULTS = [(dict(size=8), -8), (dict(d=96), -3), (dict(type=7), -8), (dict(page_size=24), -2), (dict(num_heads=0), -2),
                (dict(num_pages=-1), -2), (dict(k=0), -1), (dict(k_scale=0), -1), (dict(k=0x10008), -4), (dict(k_scale=0x30004), -4)]


@pytest.mark.parametrize("fault,status", CACHE_FAULTS)
def test_cache_faults(lib, fault, status):
    assert _weigh(lib, _cache(**fault)) == status
    assert _evict(lib, _cache(**fault)) == status


def test_weigh_needs_no_values(lib):
    """A cache without values gets as far as the other checks; packing needs them."""
    assert _weigh(lib, _cache(v=0, v_scale=0), Q=0) == -1
    assert "LSE" in lib.attn_last_error().decode()
    assert _evict(lib, _cache(v=0)) == -1 and _evict(lib, _cache(v_scale=0)) == -1


def test_weigh_nothing_to_do(lib):
    for kw in (dict(B=0), dict(Hq=0), dict(total=0)):
        assert _weigh(lib, Q=0, out=0, cu=0, table=0, **kw) == 0


@pytest.mark.parametrize("args,status", [
    (dict(B=-1), -2), (dict(keep=-1, sink=0, recent=0), -2), (dict(sink=-1), -2), (dict(recent=-1), -2), (dict(sink=90, recent=11), -2),
    (dict(sink=2 ** 31 - 1, recent=2 ** 31 - 1), -2), (dict(to=0xa0000, to_pages=1), -2), (dict(to=0xa0000, to_pages=-1), -2),
    (dict(to=0xa0000, to_pages=2 ** 25), -2), (dict(to=0x60000, to_pages=3), -2), (dict(max_pages=2 ** 25), -2), (dict(lens=0), -1),
    (dict(out_lens=0), -1), (dict(kept=0), -1), (dict(w=0), -1), (dict(table=0), -1), (dict(out_lens=0x70000), -8),
    (dict(w=0x50002), -4), (dict(kept=0x80001), -4), (dict(to=0xa0002, to_pages=4), -4), (dict(lens=0x70002), -4),
])
def test_evict_faults(lib, args, status):
    assert _evict(lib, **args) == status
    assert lib.attn_last_error().decode() != ""


def test_evict_nothing_to_do(lib):
    assert _evict(lib, B=0, w=0, table=0, lens=0, kept=0, out_lens=0) == 0


def test_python_refusals():
    """The binding's own checks (shapes, types, placement) raise before any call."""
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt)  # noqa: E731
    i = lambda *s: z(*s, dt=torch.int32)  # noqa: E731
    f = lambda *s: z(*s, dt=torch.float32)  # noqa: E731
    with pytest.raises(ValueError):
        pkg.attn_qk_rotate(z(3, 4, 64), z(3, 2, 64))  # on the CPU
    with pytest.raises(ValueError):
        pkg.attn_fwd_prompt(z(3, 4, 64), z(3, 2, 64), z(3, 2, 64), i(2), i(2), 3)
    with pytest.raises(ValueError):
        pkg.attn_cache_weigh(z(1, 4, 64), f(4, 1), z(2, 2, 16, 64), f(2, 2, 16), i(1, 2), None, i(2))
    with pytest.raises(ValueError):
        pkg.attn_cache_evict(z(2, 2, 16, 64), z(2, 2, 16, 64), f(2, 2, 16), i(1, 2), i(1), 4)


def test_most_positions(lib):
    """Steps of a kernel must not pass 2^31: a sequence of more than 2^31 - 2^17 positions is refused."""
    most = (2 ** 31 - 2 ** 17) // 16
    page = _cache(page_size=16)
    for n, status in ((most + 1, -2), (2 ** 27 - 16, -2), (most, -1)):  # (then the missing pointer is found)
        assert _weigh(lib, page, max_pages=n, Q=0) == status
        assert _evict(lib, page, max_pages=n, lens=0) == status
    for keep, status in ((2 ** 31 - 1, -2), (2 ** 31 - 2 ** 17 + 1, -2), (2 ** 31 - 2 ** 17, -1)):
        assert _evict(lib, keep=keep, lens=0) == status
