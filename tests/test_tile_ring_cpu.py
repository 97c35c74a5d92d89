"""The ring of V blocks of the 128-row bf16 kernel, as a model of its barriers run under schedules
that starve one role: nobody may meet another block than the one it waits for, and all must end.

The model has an mbarrier's semantics (a wait by parity is over while the last completed phase has
it), the kernel's roles and its counts; how many arrivals free a stage of V, and whether the warp
that repairs ragged blocks is one of them, is read from the source."""
import os
import random
import re

import pytest

SOURCE = os.path.join(os.path.dirname(__file__), "..", "online_softmax_flashattention_attention_gb300", "csrc",
                      "attn_tree_tile_kernel.cuh")


class Bar:
    def __init__(self, count):
        self.count, self.left, self.done = count, count, 0

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.left, self.done = self.count, self.done + 1

    def over(self, parity):
        return (self.done & 1) != parity


def roles(n, rk, rv, nb, ragged, v_free_count):
    """Generators that yield what they wait for, as functions."""
    k_full, k_free = [Bar(1) for _ in range(rk)], [Bar(1) for _ in range(rk)]
    v_full, v_fixed = ([Bar(1) for _ in range(rv)] for _ in range(2))
    v_free = [Bar(v_free_count) for _ in range(rv)]
    s_full, p_full, pv_done = ([Bar(1) for _ in range(nb)] for _ in range(3))
    in_k, in_v = [None] * rk, [None] * rv

    def producer():
        for g in range(n):
            yield lambda: k_free[g % rk].over((g // rk & 1) ^ 1)
            in_k[g % rk] = g
            k_full[g % rk].arrive()
            yield lambda: v_free[g % rv].over((g // rv & 1) ^ 1)
            in_v[g % rv] = g
            v_full[g % rv].arrive()

    def scores():
        for g in range(n):
            if g >= nb:
                yield lambda: pv_done[g % nb].over((g - nb) // nb & 1)
            yield lambda: k_full[g % rk].over(g // rk & 1)
            assert in_k[g % rk] == g
            s_full[g % nb].arrive()
            k_free[g % rk].arrive()

    def softmax():
        for g in range(n):
            yield lambda: s_full[g % nb].over(g // nb & 1)
            p_full[g % nb].arrive()

    def values():
        par = [0] * rv
        for g in range(n):
            st = g % rv
            yield lambda: v_full[st].over(g // rv & 1)
            if g in ragged:
                yield lambda: v_fixed[st].over(par[st])
                par[st] ^= 1
            yield lambda: p_full[g % nb].over(g // nb & 1)
            assert in_v[st] == g
            pv_done[g % nb].arrive()
            v_free[st].arrive()

    def repair():
        for g in range(n):
            st = g % rv
            yield lambda: v_full[st].over(g // rv & 1)
            assert in_v[st] == g, f"the repair looks for block {g} and finds {in_v[st]}"
            if g in ragged:
                v_fixed[st].arrive()
            if v_free_count == 2:
                v_free[st].arrive()

    return {"producer": producer(), "scores": scores(), "softmax": softmax(), "values": values(), "repair": repair()}


def run(parts, starved, patience, seed):
    """Steps a random role that can go on; the starved one only every `patience` steps, or alone."""
    r = random.Random(seed)
    waits = {}
    for name, gen in list(parts.items()):
        waits[name] = next(gen)
    step = 0
    while waits:
        step += 1
        ready = [n for n, w in waits.items() if w()]
        assert ready, f"nobody can go on: {sorted(waits)}"
        others = [n for n in ready if n != starved]
        name = r.choice(others) if others and (starved not in ready or step % patience) else starved
        try:
            waits[name] = next(parts[name])
        except StopIteration:
            del waits[name]


def counted():
    with open(SOURCE) as f:
        return int(re.search(r"mbar_init\(bar_v_free\(s\), kF8 \? 4 : (\d)\)", f.read()).group(1))


@pytest.mark.parametrize("starved", ["producer", "scores", "softmax", "values", "repair"])
@pytest.mark.parametrize("rk,rv,nb", [(3, 3, 3), (4, 4, 3)])  # d = 128 and d = 64
@pytest.mark.parametrize("ragged", [{199}, {0, 57, 58, 120, 198, 199}])
def test_no_role_is_passed_by_the_ring(starved, rk, rv, nb, ragged):
    for seed in range(20):
        for patience in (7, 61, 10 ** 9):
            run(roles(200, rk, rv, nb, ragged, counted()), starved, patience, seed)


def test_the_model_finds_a_repair_that_is_not_counted():
    with pytest.raises(AssertionError):
        run(roles(200, 3, 3, 3, {199}, 1), "repair", 10 ** 9, 1)
