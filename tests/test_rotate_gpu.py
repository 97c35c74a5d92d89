"""attn_qk_rotate on the GPU against the definition in 64 bits."""
import numpy as np
import pytest
import torch

from prompt_ref import bf16, f64, ref_rotate

pytestmark = pytest.mark.gpu

CASES = [
    # Hq, Hkv, d, lengths, starts, num_freq, norm, interleaved, gap, behind
    (32, 8, 128, [1], [100000], 64, "bf16", False, 0, 0),
    (4, 1, 64, [1, 1, 1], [0, 7, 2 ** 31 - 1], 32, None, False, 0, 0),
    (3, 3, 128, [5, 0, 130], [0, 3, 1000], 64, "fp32", True, 2, 3),
    (7, 1, 64, [33], [5], 8, "bf16", True, 0, 1),
    (5, 5, 128, [9, 1], [12345678, 0], 48, "bf16", False, 1, 0),
    (2, 1, 128, [700], [0], 0, "fp32", False, 0, 0),
    (1, 0, 64, [17], [0], 16, None, False, 0, 0),
    (0, 9, 128, [3, 2], [1, 2], 32, "bf16", True, 0, 0),
    (40, 8, 64, [1300], [9], 32, "bf16", False, 0, 0),
    (65, 2, 128, [31] * 70, list(range(70)), 64, None, True, 0, 0),
]


def _pkg():
    import online_softmax_flashattention_attention_gb300 as pkg
    return pkg


def _i32(a):
    return torch.as_tensor(np.asarray(a, np.int32)).cuda()


def _freq(r, base=10000.0):
    return (base ** (-np.arange(r) / max(r, 1))).astype(np.float32)


def _positions(total, cu, start):
    pos = np.full(total, -1, np.int64)
    for b in range(len(cu) - 1):
        pos[cu[b]:cu[b + 1]] = start[b] + np.arange(cu[b + 1] - cu[b])
    return pos


def _hold(got, x, w, freq, pos, eps, interleaved, rows):
    want, tol = ref_rotate(f64(x), w, freq, pos, eps, interleaved)
    got = f64(got)
    assert np.all(np.abs(got[rows] - want[rows]) <= tol[rows])
    assert np.isnan(got[~rows]).all()  # left as they were


@pytest.mark.parametrize("joint", [False, True])
@pytest.mark.parametrize("case", CASES)
def test_against_definition(case, joint):
    Hq, Hkv, d, lens, start, r, norm, inter, gap, behind = case
    pkg, rng = _pkg(), np.random.default_rng(3)
    cu = (np.concatenate([[0], np.cumsum(lens)]) + gap).tolist()
    total = cu[-1] + behind
    if joint:
        x = bf16(rng, (total, Hq + 2 * Hkv + 1, d), 2.0).cuda()
        Q, K = x[:, 1:1 + Hq], x[:, 1 + Hq:1 + Hq + Hkv]
    else:
        Q, K = (bf16(rng, (total, n, d)).cuda() for n in (Hq, Hkv))
    dt = {"bf16": torch.bfloat16, "fp32": torch.float32, None: None}[norm]
    w = [None if dt is None else torch.from_numpy(1 + 0.3 * rng.standard_normal(d).astype(np.float32)).to(dt).cuda() for _ in range(2)]
    freq = _freq(r) if r else None
    Qo, Ko = (torch.full((total, n, d), float("nan"), dtype=torch.bfloat16, device="cuda") for n in (Hq, Hkv))
    out = pkg.attn_qk_rotate(Q, K, _i32(cu), None if freq is None else torch.from_numpy(freq).cuda(), Qo, Ko,
                             start_lens=_i32(start), q_weight=w[0], k_weight=w[1], eps=1e-5, interleaved=inter)
    assert out[0] is Qo and out[1] is Ko
    pos = _positions(total, cu, start)
    rows = pos >= 0
    for got, src, wt in ((Qo, Q, w[0]), (Ko, K, w[1])):
        _hold(got, src, None if wt is None else f64(wt), freq, pos, 1e-5, inter, rows)


def test_explicit_positions_and_no_sequences():
    pkg, rng = _pkg(), np.random.default_rng(4)
    Q, K = bf16(rng, (37, 4, 64)).cuda(), bf16(rng, (37, 2, 64)).cuda()
    freq = _freq(32)
    f = torch.from_numpy(freq).cuda()
    pos = rng.integers(-2 ** 31, 2 ** 31, 37)
    Qo, Ko = pkg.attn_qk_rotate(Q, K, None, f, positions=_i32(pos))
    for got, src in ((Qo, Q), (Ko, K)):
        _hold(got, src, None, freq, pos, 0.0, False, np.ones(37, bool))
    Qo, Ko = pkg.attn_qk_rotate(Q, K, None, f, start_lens=_i32([11]))
    _hold(Qo, Q, None, freq, 11 + np.arange(37), 0.0, False, np.ones(37, bool))


@pytest.mark.parametrize("inter", [False, True])
def test_in_place(inter):
    pkg, rng = _pkg(), np.random.default_rng(5)
    joint = bf16(rng, (333, 12, 128)).cuda()
    before = joint.clone()
    w = torch.ones(128, device="cuda")
    f = torch.from_numpy(_freq(64)).cuda()
    want = pkg.attn_qk_rotate(joint[:, :8], joint[:, 8:10], None, f, q_weight=w, interleaved=inter)
    pkg.attn_qk_rotate(joint[:, :8], joint[:, 8:10], None, f, joint[:, :8], joint[:, 8:10], q_weight=w, interleaved=inter)
    assert torch.equal(joint[:, :8], want[0]) and torch.equal(joint[:, 8:10], want[1])
    assert torch.equal(joint[:, 10:], before[:, 10:])


def test_repeated_heads_as_input():
    """An input may show one head several times (stride 0)."""
    pkg, rng = _pkg(), np.random.default_rng(6)
    one = bf16(rng, (9, 1, 64)).cuda()
    f = torch.from_numpy(_freq(16)).cuda()
    Qo, Ko = pkg.attn_qk_rotate(one.expand(9, 6, 64), one, None, f)
    for h in range(6):
        assert torch.equal(Qo[:, h], Ko[:, 0])


def test_special_values():
    """Rows of zeros, infinities and NaN stay among themselves; a frequency that is none makes NaN."""
    pkg = _pkg()
    x = torch.ones((6, 2, 64), dtype=torch.bfloat16, device="cuda")
    x[1], x[2, 0, 3], x[3, 1, 63], x[4] = 0.0, float("inf"), float("nan"), 2.0 ** -100
    freq = torch.from_numpy(_freq(16)).cuda()
    w = torch.full((64,), 0.5, device="cuda")
    Qo, Ko = pkg.attn_qk_rotate(x, x, None, freq, q_weight=w)
    Qo, Ko = Qo.float(), Ko.float()
    assert torch.isfinite(Qo[[0, 1, 4, 5]]).all() and (Qo[1] == 0).all()
    assert torch.isnan(Qo[3, 1]).all() and torch.isfinite(Qo[3, 0]).all()       # one NaN: its whole normed row
    assert torch.isfinite(Ko[2, 0, 32:]).all() and not torch.isfinite(Ko[2, 0, [3, 19]]).any() and torch.isfinite(Ko[2, 1]).all()
    assert torch.isnan(Ko[3, 1, 63]) and torch.isfinite(Ko[3, 1, :63]).all()
    freq[2] = float("inf")
    Ko = pkg.attn_qk_rotate(x, x, None, freq)[1].float()
    assert torch.isnan(Ko[0][:, [2, 18]]).all() and torch.isfinite(Ko[0][:, [0, 1, 3, 17, 19, 32]]).all()


def test_captured_call_follows_the_lengths():
    pkg, rng = _pkg(), np.random.default_rng(8)
    Q, K = bf16(rng, (50, 4, 128)).cuda(), bf16(rng, (50, 2, 128)).cuda()
    f = torch.from_numpy(_freq(64)).cuda()
    cu, start = _i32([0, 20, 50]), _i32([0, 0])
    Qo, Ko = (torch.empty_like(t) for t in (Q, K))
    pkg.attn_qk_rotate(Q, K, cu, f, Qo, Ko, start_lens=start)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkg.attn_qk_rotate(Q, K, cu, f, Qo, Ko, start_lens=start)
    for c, s in (([0, 20, 50], [5, 6]), ([0, 1, 50], [1000, 3]), ([0, 0, 50], [0, 70000])):
        cu.copy_(_i32(c))
        start.copy_(_i32(s))
        g.replay()
        torch.cuda.synchronize()
        pos = _positions(50, c, s)
        _hold(Qo, Q, None, _freq(64), pos, 0.0, False, np.ones(50, bool))


def test_offsets_past_32_bits():
    """Strides that lead past 2^31 elements."""
    pkg, rng = _pkg(), np.random.default_rng(9)
    step = 2 ** 30 + 64
    big = torch.empty(2 * step + 2 * 64, dtype=torch.bfloat16, device="cuda")
    Q = torch.as_strided(big, (3, 2, 64), (step, 64, 1))
    src = bf16(rng, (3, 2, 64)).cuda()
    Q.copy_(src)
    f = torch.from_numpy(_freq(32)).cuda()
    want = pkg.attn_qk_rotate(src, src, None, f)
    got = pkg.attn_qk_rotate(src, Q, None, f)  # read there
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    pkg.attn_qk_rotate(Q, src, None, f, Q, None)  # and written
    assert torch.equal(Q, want[0])


def test_streams():
    """Outputs made on another stream than the current one, in stream order."""
    pkg, rng = _pkg(), np.random.default_rng(10)
    Q, K = bf16(rng, (4000, 8, 128)).cuda(), bf16(rng, (4000, 2, 128)).cuda()
    f = torch.from_numpy(_freq(64)).cuda()
    want = pkg.attn_qk_rotate(Q, K, None, f)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = pkg.attn_qk_rotate(Q, K, None, f, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
