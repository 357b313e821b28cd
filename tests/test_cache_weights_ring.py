"""The key weights' ring of Q tiles as a model on the CPU: four loading warps, the warp
that issues the products, the tensor core and the two groups of summing warps, run in
random orders.  A parity wait tells a phase only from the ones next to it, so a warp that
passes over tiles can mistake an older phase for its own; the rules by which the warps
share the ring have to hold whoever is slow."""
import random

import pytest

WARPS, INFOS, BUFFERS = 4, 8, 4


class Barrier:
    def __init__(self, count):
        self.count, self.pending, self.phase = count, count, 0

    def arrive(self, n=1):
        self.pending -= n
        assert self.pending >= 0, "more arrivals than a phase takes"
        if self.pending == 0:
            self.phase, self.pending = self.phase + 1, self.count

    def passes(self, parity):
        return (self.phase & 1) != parity


class Wrong(Exception):
    pass


def run(stages, rule, pieces, seed, slow):
    """One random order.  pieces: (Q tiles, key tiles): several Q tiles of one key tile stream
    by, each fetched by one warp; a single one stays for all key tiles and is fetched by all.
    rule: "own" (a warp waits for its own tiles' places only), "watch" (for every tile's place)
    or "all" (it arrives for every tile besides)."""
    rng = random.Random(seed)
    everyone = rule == "all"
    q_full = [Barrier(WARPS) for _ in range(stages)]
    q_empty = [Barrier(1) for _ in range(stages)]
    info_full, info_read = ([Barrier(WARPS) for _ in range(INFOS)], [Barrier(2) for _ in range(INFOS)])
    s_full, s_read = [Barrier(1) for _ in range(BUFFERS)], [Barrier(1) for _ in range(BUFFERS)]
    q, info, queue, buffers = [None] * stages, [None] * INFOS, [], [None] * BUFFERS

    def loader(w):
        n = 0
        for tiles, _ in pieces:
            many = tiles > 1
            for _ in range(tiles):
                at, own = n % stages, not many or n % WARPS == w
                if n >= stages and (own or rule != "own"):
                    yield lambda b=q_empty[at], x=(n // stages & 1) ^ 1: b.passes(x)
                if own:
                    i = n % INFOS
                    if n >= INFOS:
                        yield lambda b=info_read[i], x=(n // INFOS & 1) ^ 1: b.passes(x)
                    info[i] = n
                    info_full[i].arrive(WARPS if many else 1)
                    yield True
                    q[at] = n
                    yield True
                    q_full[at].arrive(1 if everyone or not many else WARPS)
                elif everyone:
                    q_full[at].arrive()
                n += 1

    def products():
        n = step = 0
        for tiles, keys in pieces:
            many = tiles > 1
            for k in range(keys):
                for t in range(tiles):
                    at = n % stages
                    if many or k == 0:
                        yield lambda b=q_full[at], x=n // stages & 1: b.passes(x)
                    if step >= BUFFERS:
                        yield lambda b=s_read[step % BUFFERS], x=(step // BUFFERS - 1) & 1: b.passes(x)
                    last = many or k == keys - 1
                    queue.append((at, n, step, last))
                    yield True
                    step += 1
                    n += last
        return

    def tensor_core(total):
        for _ in range(total):
            yield lambda: queue
            at, n, step, last = queue[0]
            first = q[at]
            yield True  # (the product reads its tile for a while)
            if q[at] != n or first != n:
                raise Wrong(f"product of tile {n} read tile {q[at]}")
            queue.pop(0)
            buffers[step % BUFFERS] = n
            s_full[step % BUFFERS].arrive()
            if last:
                q_empty[at].arrive()

    def sums(half):
        used = step = 0
        for tiles, keys in pieces:
            many = tiles > 1
            for k in range(keys):
                for _ in range(tiles):
                    last, i = many or k == keys - 1, used % INFOS
                    if step & 1 == half:
                        yield lambda b=info_full[i], x=used // INFOS & 1: b.passes(x)
                        yield lambda b=s_full[step % BUFFERS], x=step // BUFFERS & 1: b.passes(x)
                        if info[i] != used or buffers[step % BUFFERS] != used:
                            raise Wrong(f"tile {used} summed with the scalars of {info[i]}")
                        yield True
                        s_read[step % BUFFERS].arrive()
                    elif last:
                        yield lambda b=info_full[i], x=used // INFOS & 1: b.passes(x)
                    if last:
                        info_read[i].arrive()
                        used += 1
                    step += 1

    total = sum(a * b for a, b in pieces)
    actors = {f"load{w}": loader(w) for w in range(WARPS)}
    actors.update(issue=products(), core=tensor_core(total), sums0=sums(0), sums1=sums(1))
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


SLOW = ["none", "load", "load0", "load1", "load2", "load3", "issue", "core", "sums", "sums0"]
STREAM = [(40, 1)]
MIXED = [(9, 1), (1, 5), (1, 1), (13, 1), (2, 1), (1, 3), (3, 1), (30, 1), (1, 1), (17, 1)]


def failures(stages, rule):
    bad = 0
    for i in range(200):
        try:
            run(stages, rule, (STREAM, MIXED)[i & 1], i, SLOW[i % len(SLOW)])
        except (Wrong, AssertionError):
            bad += 1
    return bad


@pytest.mark.parametrize("stages", [2, 3, 4])
def test_tiles_and_scalars_stay_together(stages):
    assert failures(stages, "all") == 0


@pytest.mark.parametrize("stages", [2, 3, 4])
def test_the_model_sees_warps_that_pass_over_tiles(stages):
    """Waiting for one's own tiles only takes a place that is still read (unless every place has
    one warp), and watching the others' without arriving for them can fall a phase behind."""
    assert (failures(stages, "own") > 0) == (stages < WARPS)
    assert failures(stages, "watch") > 0


def test_ring_sizes_of_the_kernel():
    """The kernel's numbers are those of the model, and every warp arrives for every tile."""
    import os
    import re

    from ragged_gqa_attention_varlen_gb300 import _build

    src = open(os.path.join(_build.CSRC, "cache_weights.cuh")).read()
    assert re.search(r"kQS = HD == 160 \? 2 : \(HD == 128 \? 3 : 4\);", src)
    assert re.search(r"kIS = %d;" % INFOS, src)
    assert "mbar_init(&bars->q_full[b], %d);" % WARPS in src
    assert src.count("arrive(&bars->q_full[qs])") == 1 and "arrive_n(&bars->q_full" not in src
