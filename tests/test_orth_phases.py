"""The phases of the orthogonalisation's grid form (no device needed): which CTA pairs have a tile in which phase, by
the planner restated, and the waits that keep a pair without one from running ahead, as a model of the barriers.

An mbarrier wait tells a phase from the one before by its parity, so it is right only for a thread that is at most one
completion behind.  A pair with a Poly tile but no Gram tile is two behind unless it waits in the Gram phase too."""
import os
import random
import re

import pytest

import structured_sparse_transformer_b200 as sp

CSRC = os.path.join(os.path.dirname(os.path.abspath(sp.__file__)), "csrc")
GRAM, POLY, APPLY = 0, 1, 2


# ------------------------------------------------------------------ the planner, restated (sp24_lib.cu)

def _sym_tiles(m, bn):
    rb, r, cb = -(-m // 256), 256 // bn, -(-m // bn)
    return r * rb * (rb - 1) // 2 + min(cb, r * rb)


def _stage_us(bn, apply, use):
    share = use / 74.0
    return 0.25 + 0.10 * share if bn == 128 else 0.31 + (0.14 if apply else 0.07) * share


def _shape(tiles, kt, P, bn, apply, most=4):
    split, use = 1, min(tiles, P)
    us = _stage_us(bn, apply, P) * (tiles // P * kt) + (2.4 if bn == 256 else 1.4)
    tail = tiles % P
    if tail:
        least = _stage_us(bn, apply, tail) * kt
        s = 2
        while s <= most and s <= kt and tail * s <= P:
            t = _stage_us(bn, apply, tail * s) * ((kt + s - 1) // s) + (3.5 if bn == 256 else 2.8) + 0.4 * (s - 2)
            if t < least:
                least, split = t, s
            s += 1
        us += least
        if tiles < P:
            use = tail * split
    return dict(bn=bn, split=split, use=use, us=us)


def _plan(m, n, batch, P):
    """(pairs of the grid, [(tiles, split) of Gram, Poly, Apply])."""
    mb, grid, kinds = -(-m // 256), 0, []
    for k in (GRAM, POLY, APPLY):
        kt = -(-(n if k == GRAM else m) // 64)
        best = None
        for bn in (128, 256):
            per = mb * -(-n // bn) if k == APPLY else _sym_tiles(m, bn)
            o = _shape(batch * per, kt, P, bn, k == APPLY)
            if best is None or o["us"] <= best["us"]:
                best = dict(o, per=per)
        kinds.append((best, kt))
        grid = max(grid, best["use"])
    return grid, [(batch * b["per"], _shape(batch * b["per"], kt, grid, b["bn"], k == APPLY)["split"])
                  for k, (b, kt) in enumerate(kinds)]


def _has_tile(pair, grid, tiles, split):
    full = tiles // grid * grid if split > 1 else tiles
    return pair < full or (split > 1 and pair < (tiles - full) * split)


def _idle_in_gram(m, n, batch, P):
    """Pairs with a Poly tile and no Gram tile."""
    grid, kinds = _plan(m, n, batch, P)
    return [p for p in range(grid) if _has_tile(p, grid, *kinds[POLY]) and not _has_tile(p, grid, *kinds[GRAM])]


def test_plans_with_such_pairs_exist():
    """On parts of 142 and 152 SMs; on 148 this time model gives none, but nothing but its constants keeps it so."""
    assert _idle_in_gram(1793, 60000, 1, 71) and _idle_in_gram(786, 27070, 4, 76)


# ------------------------------------------------------------------ the barriers

def _run(has, phases, waits_each_phase, seed):
    """Random interleaving of every pair's producer and epilogue; the loads of G that came before the phase that
    writes it was over."""
    rng = random.Random(seed)
    pairs = len(has)
    counted = [0] * phases                       # pairs that have left the phase
    ready = [0] * pairs                          # completions of the pair's `ready`
    stale = []

    def passed(pair, ph):                        # a wait on `ready` with phase ph's parity
        return ready[pair] & 1 != ph & 1

    def producer(pair):
        for ph in range(phases):
            while ph > 0 and counted[ph - 1] < pairs:
                yield
            ready[pair] += 1
            yield

    def epilogue(pair):
        for ph in range(phases):
            kind = ph % 3
            if has[pair][kind]:
                while kind == POLY and not passed(pair, ph):
                    yield
                if kind == POLY and counted[ph - 1] < pairs:
                    stale.append((pair, ph))
                while ready[pair] < ph + 1:      # the accumulator: its operands are loaded behind the producer's wait
                    yield
                yield
            while waits_each_phase and not passed(pair, ph):
                yield
            counted[ph] += 1
            yield

    agents = [f(p) for p in range(pairs) for f in (producer, epilogue)]
    for _ in range(400 * pairs * phases):
        if not agents:
            return stale
        a = rng.choice(agents)
        try:
            next(a)
        except StopIteration:
            agents.remove(a)
    raise AssertionError("the phases do not end")


def _waits_each_phase():
    """Whether the kernel's epilogue waits on `ready` at the end of every phase in the grid form."""
    text = open(os.path.join(CSRC, "ortho_gemm.cuh")).read()
    kernel = text[text.index("orth_products_kernel(const __grid_constant__"):text.index("orth_small_kernel(const __grid_constant__")]
    end = kernel[kernel.index("this warp's stores of the phase are complete"):]
    at_count = end.index("flag_add_release(p.counters + ph")
    grid_branch = end[:at_count].rindex("if (!CLUSTER)")
    return re.search(r"mbar_wait_bounded\(ready, \(uint32_t\)ph & 1u", end[:grid_branch]) is not None


CASES = [[(1, 1, 1), (1, 1, 1), (0, 1, 1)], [(1, 0, 1), (0, 1, 0), (1, 1, 1), (0, 1, 1)], [(1, 1, 1), (0, 0, 1), (1, 1, 0)],
         [(1, 1, 1)] * 3]


@pytest.mark.parametrize("has", CASES)
def test_g_is_read_after_it_is_written(has):
    for seed in range(300):
        assert not _run(has, 14, _waits_each_phase(), seed)


def test_g_is_read_after_it_is_written_on_a_planned_grid():
    grid, kinds = _plan(1793, 60000, 1, 71)
    has = [tuple(_has_tile(p, grid, *k) for k in kinds) for p in range(grid)]
    for seed in range(3):
        assert not _run(has, 8, _waits_each_phase(), seed)


def test_the_model_finds_the_fault_without_the_wait():
    assert any(_run(CASES[0], 14, False, seed) for seed in range(300))


def test_set_up_comes_before_the_first_launch():
    """What can fail without a launch (tensor maps, a kernel's set-up on its device) does so before the first kernel
    advances the momentum: a refused step leaves every buffer as it was."""
    text = open(os.path.join(CSRC, "sp24_lib.cu")).read()
    run = text[text.index("sp24_status run_orth("):]
    run = run[:run.index("\n}\n")]
    behind = run[run.index("launch_pdl("):]
    for what in ("make_map_", "pairs_of<", "orth_clusters", "plan_orth_products(", "last(false)"):
        assert what not in behind, what
    assert run.index("plan_orth_products(") < run.index("last(false)") < run.index("launch_pdl(")
    launch = text[text.index("sp24_status launch_orth_products("):]
    launch = launch[:launch.index("\n}\n")]
    assert "pairs_of" not in launch and "orth_clusters" not in launch
