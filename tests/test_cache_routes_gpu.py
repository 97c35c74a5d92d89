"""Routes through the paged cache that a program takes and the other files leave out."""
import numpy as np
import pytest
import torch

from cache_ref import HALF_BF16, Batch

pytestmark = pytest.mark.gpu


def _pkg():
    import online_softmax_flashattention_attention_gb300 as pkg
    return pkg


def _i32(a):
    return torch.as_tensor(np.asarray(a, np.int32)).cuda()


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("hkv,G,d", [(2, 4, 128), (1, 8, 64), (3, 1, 64)])
def test_a_prompt_over_a_prefix_read_back_with_grouped_heads(hkv, G, d, f8):
    """What attn_cache_read returns, each K/V head repeated for its group, through the packed forward:
    a chain's tokens as attn_fwd_tree has them.  As they are, with fewer heads, they are refused."""
    pkg = _pkg()
    b = Batch(61, hkv, G, d, 32, f8, [150, 7], [9, 4], masks="chain")
    args, kw = b.dev()
    O, LSE = pkg.attn_fwd_tree(*args, **kw)
    cu_k = _i32([0, 159, 170])
    sc = {n: kw[n] for n in ("k_scale", "v_scale") if n in kw}
    K, V = pkg.attn_cache_read(args[1], args[2], args[3], cu_k, 170, **sc)
    cu_q = args[5]
    if G > 1:
        with pytest.raises(ValueError, match="repeat"):
            pkg.attn_fwd_varlen(args[0], K, V, cu_q, cu_k, 9, causal=True)
    K, V = (x.repeat_interleave(G, 1) for x in (K, V))
    O2, LSE2 = pkg.attn_fwd_varlen(args[0], K, V, cu_q, cu_k, 9, causal=True)
    pkg.cache_check()
    # each is off by half a bf16 step of O, and by one of every probability: 2^-8 (|O| + A), both at most max |v|
    assert bool(((O - O2).float().abs() <= 4 * HALF_BF16 * V.float().abs().max()).all())
    # scores: d 2^-24 |q| |k| / sqrt(d) each, |q| |k| under 250 here, and 2^-17 of the query row's largest where
    # a value is 2^-9 of it and less
    assert bool(((LSE - LSE2).abs() <= 4e-4).all())


def test_workspaces_go_with_their_threads():
    """The workspaces kept for threads that have ended, and all of them after release_workspace(), no
    longer take device memory."""
    import gc
    import threading
    pkg = _pkg()
    b = Batch(62, 2, 4, 128, 16, False, [300], [9])  # tiles: 21 MB a workspace
    args, kw = b.dev()
    O, LSE = torch.empty_like(args[0]), torch.empty((8, 9), device="cuda")
    pkg.release_workspace()
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    one = pkg.tree_workspace_bytes(8, 2, 9, 128)
    ready, go = threading.Barrier(5), threading.Event()

    def work():
        pkg.attn_fwd_tree(*args, O, LSE, **kw)
        ready.wait()
        go.wait()

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    ready.wait()
    torch.cuda.synchronize()
    assert torch.cuda.memory_allocated() - before >= 4 * one
    go.set()
    for t in threads:
        t.join()
    gc.collect()
    assert torch.cuda.memory_allocated() - before < one
    pkg.attn_fwd_tree(*args, O, LSE, **kw)
    ready, go = threading.Barrier(2), threading.Event()
    t = threading.Thread(target=work)
    t.start()
    ready.wait()
    assert torch.cuda.memory_allocated() - before >= 2 * one
    pkg.release_workspace()
    assert torch.cuda.memory_allocated() - before < one
    go.set()
    t.join()
    pkg.cache_check()


def test_packed_forward_refuses_outputs_that_do_not_fit():
    pkg = _pkg()
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731
    Q, cu = z(5, 8, 64), _i32([0, 5])
    for O, LSE in ((z(5, 2, 64), None), (z(5, 8, 64, dt=torch.float32), None), (z(5, 8, 128)[:, :, ::2], None),
                   (None, z(5, 8, dt=torch.float32)), (None, z(8, 5)), (z(5, 8, 64).cpu(), None)):
        with pytest.raises(ValueError):
            pkg.attn_fwd_varlen(Q, Q, Q, cu, cu, 5, O, LSE)
    with pytest.raises(ValueError, match="K must be"):
        pkg.attn_fwd_varlen(Q, z(5, 8, 128)[:, :, ::2], Q, cu, cu, 5)
    assert bool((pkg.attn_fwd_varlen(Q, Q, Q, cu, cu, 5)[0] == 0).all())
