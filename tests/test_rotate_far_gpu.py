"""attn_qk_rotate's angles at far positions, either sense of turning."""
import numpy as np
import pytest
import torch

from cache_ref import HALF_BF16

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("sign", [1, -1])
def test_small_frequencies_far_away(sign, interleaved):
    """Pairs (1, 0) turn into (cos, sin), with no other product or sum in the result.  The angle is off by
    2^-23 rad and 2^-52 of itself, the functions by 2^-21 of their value (two units), the result rounds to
    bf16 once; among these many angles some have a sine or a cosine small enough for that to show."""
    import online_softmax_flashattention_attention_gb300 as pkg
    rng = np.random.default_rng(21)
    total, r = 20000, 64
    freq = (sign * np.float32(10.0) ** -rng.uniform(6, 9.5, r)).astype(np.float32)
    pos = rng.integers(2 ** 30, 2 ** 31, total)
    pos[::2] *= -1
    first = slice(0, None, 2) if interleaved else slice(0, r)
    second = slice(1, None, 2) if interleaved else slice(r, None)
    x = torch.zeros((total, 1, 2 * r), dtype=torch.bfloat16, device="cuda")
    x[..., first] = 1.0
    got, _ = pkg.attn_qk_rotate(x, x[:, :0], None, torch.from_numpy(freq).cuda(),
                                positions=torch.from_numpy(pos.astype(np.int32)).cuda(), interleaved=interleaved)
    got = got[:, 0].double().cpu().numpy()
    t = pos[:, None] * freq[None].astype(np.float64)
    for cols, want in ((first, np.cos(t)), (second, np.sin(t))):
        tol = 2.0 ** -23 + 2.0 ** -52 * np.abs(t) + np.abs(want) * (HALF_BF16 + 2.0 ** -21)
        tol += 2.0 ** -53 * np.abs(t)  # the reference's own product
        assert np.all(np.abs(got[:, cols] - want) <= tol)


def test_turning_back():
    """A frequency and its negative turn by the same angle either way, to the last bit."""
    import online_softmax_flashattention_attention_gb300 as pkg
    rng = np.random.default_rng(22)
    freq = torch.from_numpy((np.float32(10.0) ** -rng.uniform(0, 9.5, 32)).astype(np.float32)).cuda()
    pos = torch.from_numpy(rng.integers(-2 ** 31, 2 ** 31, 999).astype(np.int32)).cuda()
    x = torch.zeros((999, 1, 64), dtype=torch.bfloat16, device="cuda")
    x[..., :32] = 1.0
    a, _ = pkg.attn_qk_rotate(x, x[:, :0], None, freq, positions=pos)
    b, _ = pkg.attn_qk_rotate(x, x[:, :0], None, -freq, positions=pos)
    assert torch.equal(a[..., :32], b[..., :32]) and torch.equal(a[..., 32:], -b[..., 32:])
