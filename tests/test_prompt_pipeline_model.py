"""A model of the barriers of the kernel for prompts (host only): raw tiles, tiles in fp16, scores, products and marks.
MMAs complete in the order they are issued, warps run at any pace, and a wait by parity cannot tell a phase from the one
two before it."""
import os
import random

import pytest

KERNEL = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "nvfp4_block_scaled_gemv_gb300",
                      "csrc_layer", "attention_prompt.cu")


class Barrier:
    def __init__(self, count):
        self.count, self.arrived, self.phases = count, 0, 0

    def arrive(self):
        self.arrived += 1
        if self.arrived == self.count:
            self.arrived, self.phases = 0, self.phases + 1

    def passed(self, parity):
        return self.phases & 1 != parity


def run(rng, halves, tiles, warps, own_p, slots, raws, o_of, marks=4, converters=4):
    """One row tile.  o_of(u, j): (barrier, parity) of the product of tile j in half u.  Returns what went wrong, or None."""
    def bars(n, count):
        return [Barrier(count) for _ in range(n)]

    s_full, p_ready, s_free, o_done = bars(2, 1), bars(2, warps), bars(2, warps), bars(2, 1)
    raw_full, raw_empty, marks_full = bars(raws, 1), bars(raws, converters), bars(marks, converters)
    slot_full, slot_empty = bars(slots, converters), bars(slots, 1)
    steps, queue, copies, done = tiles * halves, [], [], set()
    raw, slot, mark = [None] * raws, [{} for _ in range(slots)], [{} for _ in range(marks)]

    def expect(what, got, want):
        if got != want:
            raise AssertionError(f"{what}: {got}, expected {want}")

    def loader():
        for j in range(tiles):
            yield lambda: raw_empty[j % raws].passed((j // raws & 1) ^ 1)
            copies.append(j)

    def copier():
        while True:
            yield lambda: copies
            j = copies.pop(0)
            raw[j % raws] = j
            raw_full[j % raws].arrive()

    def converter(w):
        for j in range(tiles):
            yield lambda: raw_full[j % raws].passed(j // raws & 1)
            mark[j % marks][w] = j
            marks_full[j % marks].arrive()
            for fill in (2 * j, 2 * j + 1):
                i = fill % slots
                yield lambda: slot_empty[i].passed((fill // slots & 1) ^ 1)
                expect("raw tile", raw[j % raws], j)
                slot[i][w] = fill
                slot_full[i].arrive()
            raw_empty[j % raws].arrive()

    def filled(fill):
        i = fill % slots
        yield lambda: slot_full[i].passed(fill // slots & 1)
        expect("fill", slot[i], {w: fill for w in range(converters)})

    def scores(x):
        j, u = x // halves, x % halves
        yield from filled(2 * j)
        queue.append(([s_full[x & 1]] + [slot_empty[2 * j % slots]] * (u == halves - 1), 2 * j, None))

    def issuer():
        for x in range(min(2, steps)):
            yield from scores(x)
        for x in range(steps):
            if own_p and x + 2 < steps:
                yield lambda: s_free[x & 1].passed(x >> 1 & 1)
                yield from scores(x + 2)
            j, u = x // halves, x % halves
            yield from filled(2 * j + 1)
            yield lambda: p_ready[x & 1].passed(x >> 1 & 1)
            queue.append(([o_done[o_of(u, j)[0]]] + [slot_empty[(2 * j + 1) % slots]] * (u == halves - 1), 2 * j + 1, (u, j)))
            if not own_p and x + 2 < steps:
                yield from scores(x + 2)

    def pipe():
        while True:
            yield lambda: queue
            signals, fill, what = queue.pop(0)
            expect("tile of a product", set(slot[fill % slots].values()), {fill})
            done.add(what)
            for barrier in signals:
                barrier.arrive()

    def softmax(u, raises, masked):
        def product(j):
            at, parity = o_of(u, j)
            yield lambda: o_done[at].passed(parity)
            expect(f"product of tile {j} of {tiles} in half {u}", (u, j) in done, True)

        for j in range(tiles):
            x = halves * j + u
            yield lambda: s_full[x & 1].passed(x >> 1 & 1)
            if own_p:
                s_free[x & 1].arrive()
                if j:
                    yield from product(j - 1)
            elif j and raises[j]:
                yield from product(j - 1)
            if masked[j]:
                yield lambda: marks_full[j % marks].passed(j // marks & 1)
                expect("marks", mark[j % marks], {w: j for w in range(converters)})
            p_ready[x & 1].arrive()
        yield from product(tiles - 1)

    def some(share):
        return [rng.random() < share for _ in range(tiles)]

    actors = [issuer(), pipe(), loader(), copier()] + [converter(w) for w in range(converters)]
    last = len(actors)
    actors += [softmax(u, some(0.3), some(0.4)) for u in range(halves) for _ in range(warps)]
    pace = [rng.choice([0.05, 0.3, 1.0]) for _ in actors]
    waits = [next(a, None) for a in actors]
    try:
        while any(w is not None for w in waits[last:]):
            ready = [i for i, w in enumerate(waits) if w is not None and w()]
            if not ready:
                return "nobody can go on"
            i = rng.choices(ready, [pace[k] for k in ready])[0]
            waits[i] = next(actors[i], None)
    except AssertionError as e:
        return str(e)
    return None


def in_turn(u, j):
    return j & 1, j >> 1 & 1


def by_half(u, j):
    return u, j & 1


# halves, warps that announce P, P beside S, slots, raw tiles: heads of 256 on one SM and on a pair, of 128, of 64
KERNELS = [(1, 4, False, 3, 2, in_turn), (1, 8, False, 3, 2, in_turn), (2, 4, False, 3, 2, by_half), (2, 4, True, 6, 4, by_half)]


@pytest.mark.parametrize("halves,warps,own_p,slots,raws,o_of", KERNELS)
def test_what_is_waited_for_is_there(halves, warps, own_p, slots, raws, o_of):
    rng = random.Random(warps + halves)
    for _ in range(500):
        assert run(rng, halves, rng.randint(1, 9), warps, own_p, slots, raws, o_of) is None


def test_one_barrier_for_one_half_would_let_warps_by():
    rng = random.Random(5)
    assert any("product of tile" in (run(rng, 1, rng.randint(2, 7), 4, False, 3, 2, by_half) or "") for _ in range(500))


def test_the_kernel_has_these_barriers():
    with open(KERNEL) as f:
        code = f.read()
    assert "(NQ == 2 ? (uint32_t)u : (uint32_t)j & 1u)" in code and "(uint32_t)(NQ == 2 ? j : j >> 1) & 1u" in code
    assert code.count("wait_phase(o_done(u, j - 1), o_phase(j - 1), ok)") == 2
    assert code.count("wait_phase(o_done(u, tiles - 1), o_phase(tiles - 1), ok)") == 1
    assert code.count("o_done(") == 4
