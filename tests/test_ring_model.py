"""A model of the tiles' rings: a producer of codes and one of tokens, sets of unpacking warps, the tensor core, and barriers
that are waited on by parity. Copies land and commits signal in any order, some much later than others. It shows what the number of
barriers decides: with one per place sets read other blocks than theirs, with as many as ring.h says they never do."""
import random

import pytest

KB = 128                                                     # columns of a block of codes


def barriers_for(places, step):
    return -(-places // step) * step


class Barrier:
    def __init__(self, count):
        self.count = self.pending = count
        self.phase = self.copies = 0

    def arrive(self):
        self.pending -= 1
        assert self.pending >= 0, "arrived on twice"
        self.check()

    def landed(self):
        self.copies -= 1
        self.check()

    def check(self):
        if not self.pending and not self.copies:
            self.phase, self.pending = self.phase + 1, self.count

    def passes(self, use):                                   # a parity: the barrier is not in this use's phase
        return self.phase % 2 != use % 2


class Wrong(Exception):
    pass


def run(agents, later, rng):
    """Steps of agents (generators of (barrier, use) to wait for, or None) and of what is on its way, in any order."""
    slow = rng.choice([0.0, 0.5, 0.9])
    waits = {a: next(a) for a in agents}
    while waits:
        ready = [a for a, w in waits.items() if w is None or w[0].passes(w[1])]
        if not ready and not later:
            raise Wrong("nobody goes on")
        if ready and (not later or rng.random() < slow or rng.random() < 0.5):
            a = rng.choice(ready)
            try:
                waits[a] = next(a)
            except StopIteration:
                del waits[a]
        else:
            later.pop(rng.randrange(len(later)))()


def tiles(seed, d, n_tiles, sets, slabs, blocks, kc, enough):
    """Tiles of one CTA, a warp for each set. `slabs`, `blocks`: places; `kc`: columns of a slab; `enough`: barriers by the rule."""
    rng, later = random.Random(seed), []
    step, d_pad = max(1, sets * kc // KB), -(-d // KB) * KB
    n_empty, n_landed = (barriers_for(slabs, sets), barriers_for(blocks, step)) if enough else (slabs, blocks)
    full, empty = [Barrier(2) for _ in range(slabs)], [Barrier(1) for _ in range(n_empty)]
    landed, free = [Barrier(1) for _ in range(n_landed)], [Barrier(KB // kc) for _ in range(blocks)]
    code, operand = [None] * blocks, [None] * slabs

    def after(f):
        left = [rng.choice([0, 0, 0, 40])]

        def go():
            if left[0]:
                left[0] -= 1
                later.append(go)
            else:
                f()
        later.append(go)

    def slab_free(n):
        u = n + n_empty - slabs
        return empty[u % n_empty], u // n_empty - 1

    def tokens():
        n = 0
        for _ in range(n_tiles):
            for k in range(0, d_pad, kc):
                yield slab_free(n)
                b = full[n % slabs]
                if k < d:
                    b.copies += 1
                    after(b.landed)
                b.arrive()
                n += 1

    def codes():
        for n in range(n_tiles * d_pad // KB):
            yield free[n % blocks], n // blocks - 1

            def land(n=n):
                code[n % blocks] = n
                landed[n % n_landed].landed()
            landed[n % n_landed].copies += 1
            landed[n % n_landed].arrive()
            after(land)

    def products():
        n = 0
        for _ in range(n_tiles):
            for k in range(0, d_pad, kc):
                yield full[n % slabs], n // slabs
                if k < d and operand[n % slabs] != n:
                    raise Wrong(f"a product of slab {operand[n % slabs]} for {n}")
                after(empty[n % n_empty].arrive)
                n += 1

    def unpack(s):
        for n in range(s, n_tiles * d_pad // kc, sets):
            cb, k = n * kc // KB, n * kc % d_pad
            yield landed[cb % n_landed], cb // n_landed
            yield slab_free(n)
            if k < d:
                for _ in range(2):
                    yield None
                    if code[cb % blocks] != cb:
                        raise Wrong(f"codes {code[cb % blocks]} read for {cb}")
                operand[n % slabs] = n
            full[n % slabs].arrive()
            free[cb % blocks].arrive()

    run([tokens(), codes(), products()] + [unpack(s) for s in range(sets)], later, rng)


FORMS = {"bf16, 4 bits": (4, 4, 3, 64), "e4m3, 4 bits": (2, 4, 3, 128), "bf16, 2 and 3 bits": (4, 4, 4, 64), "e4m3, 2 and 3 bits": (4, 4, 4, 128),
         "bf16, 8 bits": (2, 3, 2, 64)}


@pytest.mark.parametrize("d", [64, 128, 320, 448, 1024])
@pytest.mark.parametrize("form", FORMS)
def test_no_set_reads_another_block(form, d):
    for seed in range(120):
        tiles(seed, d, 4, *FORMS[form], enough=True)


@pytest.mark.parametrize("form", ["bf16, 4 bits", "e4m3, 4 bits", "bf16, 8 bits"])
def test_a_barrier_for_each_place_is_too_few(form):
    wrong = 0
    for seed in range(200):
        try:
            tiles(seed, 1024, 3, *FORMS[form], enough=False)
        except (Wrong, AssertionError):
            wrong += 1
    assert wrong > 0
