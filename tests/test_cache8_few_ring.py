"""The stages of the 8-bit cache's kernel for few rows as a model on the CPU: four loading warps in
turn, the warps that take the halves of each stage, and the warp that joins what they leave of a
piece, run in random orders.  A wait by parity tells a phase only from the ones next to it, so a warp
may wait for the phase behind the last that it has seen, and for no other."""
import random

import pytest

from test_cache_weights_ring import Barrier, Wrong


def run(warps, loaders, stages, pieces, seed, slow):
    """One random order.  pieces: stages of each; both halves of a stage are chunks (the upper one may
    hold no key: its warp gives the stage back all the same)."""
    rng = random.Random(seed)
    full, empty = [Barrier(1) for _ in range(stages)], [Barrier(2) for _ in range(stages)]
    done, taken = Barrier(warps), Barrier(1)
    data, left = [None] * stages, [None] * warps

    def load(w):
        i = 0
        for n in pieces:
            for _ in range(n):
                if i % loaders == w:
                    st = i % stages
                    if i >= stages:
                        yield lambda b=empty[st], x=(i // stages - 1) & 1: b.passes(x)
                    data[st] = None
                    yield True  # (the copies land)
                    data[st] = i
                    full[st].arrive()
                i += 1
        return

    def take(w):
        before = first = 0
        for at, n in enumerate(pieces):
            q = (w - first) % warps
            while q < 2 * n:
                i = before + q // 2
                st = i % stages
                yield lambda b=full[st], x=i // stages & 1: b.passes(x)
                was = data[st]
                yield True  # (reads them for a while)
                if was != i or data[st] != i:
                    raise Wrong(f"stage {i} read as {was}, {data[st]}")
                empty[st].arrive()
                q += warps
            before, first = before + n, (first + 2 * n) % warps
            if at > 0:
                yield lambda x=(at - 1) & 1: taken.passes(x)
            left[w] = at
            yield True
            done.arrive()

    def join():
        for at in range(len(pieces)):
            yield lambda x=at & 1: done.passes(x)
            if any(x != at for x in left):
                raise Wrong(f"piece {at} joined from {left}")
            yield True
            taken.arrive()

    actors = {f"load{w}": load(w) for w in range(loaders)}
    actors.update({f"take{w}": take(w) for w in range(warps)}, join=join())
    ready = {name: True for name in actors}
    weight = {name: 0.03 if slow in name else 1.0 for name in actors}
    while actors:
        able = [x for x in actors if ready[x] is True or ready[x]()]
        if not able:
            raise Wrong("every warp waits: " + ", ".join(actors))
        x = rng.choices(able, [weight[a] for a in able])[0]
        try:
            ready[x] = next(actors[x])
        except StopIteration:
            del actors[x]


SLOW = ["none", "load", "load0", "load2", "take", "take0", "take3", "take7", "join"]
PIECES = [[60], [1] * 40, [9, 1, 17, 2, 30, 3, 1, 12], [5, 4, 3] * 8, [13] * 6]


def failures(warps, loaders, stages):
    bad = 0
    for i in range(180):
        try:
            run(warps, loaders, stages, PIECES[i % len(PIECES)], i, SLOW[i % len(SLOW)])
        except (Wrong, AssertionError):
            bad += 1
    return bad


@pytest.mark.parametrize("stages", [8, 16])
def test_stages_and_pieces_stay_together(stages):
    assert failures(8, 4, stages) == 0


def test_the_model_sees_stages_that_go_from_warp_to_warp():
    """Eight stages under twelve warps (a launch failure, before they had to belong to one warp each),
    and under loading warps that do not divide them."""
    assert failures(12, 4, 8) > 0
    assert failures(12, 4, 12) == 0


def test_numbers_of_the_kernel():
    import os
    import re

    from ragged_gqa_attention_varlen_gb300 import _build

    src = open(os.path.join(_build.CSRC, "cache8_few.cuh")).read()
    assert re.search(r"kFewLoads = 4;", src) and re.search(r"kFewWarps = 8,", src)
    assert re.search(r"kStages = HD == 64 \? 16 : 8;", src)
    assert "static_assert(2 * kStages % kFewWarps == 0 && kStages % kFewLoads == 0" in src
    assert "mbar_init(&bars->empty[b], 2);" in src and "mbar_init(&bars->done, kFewWarps);" in src and "mbar_init(&bars->taken, 1);" in src
