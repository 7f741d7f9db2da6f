"""The split that decode calls run (a fixed cost per unit, whole short units), and the windowed block-causal one:
properties that the kernels and the combine rely on, by the code that they share with the host."""
import random

import pytest

from two_tower_block_b200 import ops


def cases():
    rng = random.Random(5)
    for U, C in ((1, 148), (16, 144), (40, 148), (73, 148), (147, 148), (148, 148), (149, 148), (300, 148), (7, 3), (3, 1)):
        for kind in ("equal", "ragged", "short", "one long"):
            for cost in (0, 1, 5, 8):
                Hkv = rng.choice([h for h in (1, 2, 3, 7) if U % h == 0])
                B = U // Hkv
                top = {"equal": 1, "ragged": 300, "short": 3, "one long": 4}[kind]
                tiles = [rng.randint(1, top) for _ in range(B)] if kind != "equal" else [rng.randint(1, 90)] * B
                if kind == "one long":
                    tiles[rng.randrange(B)] = 5000
                yield tiles, Hkv, C, cost, rng.choice([0, 6])
    for U in (10, 100):           # T just below, at and above the number of ranges
        for T in (U, 147, 148, 149, 150, 160):
            if T >= U:
                yield [1 + (T - U) // U + (1 if n < (T - U) % U else 0) for n in range(U)], 1, 148, 5, 0


@pytest.mark.parametrize("i", range(20))
def test_decode_split(i):
    for tiles, Hkv, C, want, whole in list(cases())[i::20]:
        what = (tiles[:8], len(tiles), Hkv, C, want, whole)
        starts, cost, segments, records = ops.decode_split(tiles, Hkv, C, want, whole)
        unit_tiles = [t for t in tiles for _ in range(Hkv)]
        U = len(unit_tiles)
        assert 0 <= cost <= want, what
        # every tile once, in order; every used range holds at least one
        at = [(u, t) for u in range(U) for t in range(unit_tiles[u])]
        got = [(u, t) for _, u, lo, hi, _ in segments for t in range(lo, hi)]
        assert got == at, what
        used = sorted({s[0] for s in segments})
        T = sum(unit_tiles) + U * cost
        assert used == list(range(len(used))), what
        stays_whole = U <= C and max(tiles) <= whole
        assert len(used) == (U if stays_whole else min(C, T)), what
        assert all(a < b for a, b in zip(starts[:len(used)], starts[1:])), what
        # a whole unit needs no slot; the pieces of a cut one have slots of their own
        slots = [s[4] for s in segments if s[4] >= 0]
        assert len(slots) == len(set(slots)) and all(0 <= s < 2 * C for s in slots), what
        pieces = {}
        for c, u, lo, hi, slot in segments:
            assert (slot < 0) == (hi - lo == unit_tiles[u]), what
            assert slot < 0 or slot // 2 == c, what
            if slot >= 0:
                pieces.setdefault(u, []).append((c, slot))
        # and its record, in the range that it begins in, leads to every one of them in order
        assert {r[0]: c for c, r in enumerate(records) if r[0] >= 0} == {u: p[0][0] for u, p in pieces.items()}, what
        for u, p in pieces.items():
            first = p[0][0]
            _, last, which = records[first]
            assert p == [(first, 2 * first + which)] + [(c, 2 * c) for c in range(first + 1, last + 1)], what
        if stays_whole:
            assert not pieces, what


def test_decode_split_evens_out_the_fixed_cost():
    """Ragged units: a range's tiles and the costs of the unit edges in it differ from the mean by one cost."""
    rng = random.Random(6)
    tiles = [rng.randint(1, 257) for _ in range(64)]
    starts, cost, segments, _ = ops.decode_split(tiles, 2, 148, 5)
    assert cost == 5
    work = [0.0] * 148
    unit_tiles = [t for t in tiles for _ in range(2)]
    for c, u, lo, hi, _ in segments:
        work[c] += hi - lo + (cost / 2 if lo == 0 else 0) + (cost / 2 if hi == unit_tiles[u] else 0)
    mean = sum(work) / len(work)
    assert max(work) <= mean + cost + 1


def test_decode_split_refuses_bad_arguments():
    for args in (([0], 1, 4), ([1], 0, 4), ([1], 1, 4, -1), ([1], 1, 4, 0, -1)):
        with pytest.raises(ops.TTError) as e:
            ops.decode_split(*args)
        assert e.value.status == ops.TT_ERR_INVALID_ARG


@pytest.mark.parametrize("cost", [-1, 0, 3])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (64, 4), (1000, 100), (10 ** 6, 7)])
@pytest.mark.parametrize("B,Hkv,N,S,C", [(1, 1, 8, 8, 148), (2, 1, 1000, 8, 148), (4, 2, 8192, 16, 148), (1, 3, 2100, 21, 37)])
def test_windowed_causal_split(B, Hkv, N, S, C, window, sinks, cost):
    def tiles(b):
        L = S * b
        runs = [L] if not window or L - window <= sinks else [sinks, window]
        return -(-S // 64) + sum(-(-r // 64) for r in runs)
    T = B * Hkv * sum(tiles(b) for b in range(N // S))
    starts = ops.causal_split(B, Hkv, N, S, 64, C, cost, window, sinks)
    used = min(C, T)
    assert starts[0] == 0 and starts[used:] == [T] * (C + 1 - used)
    assert all(a < b for a, b in zip(starts[:used], starts[1:]))
    if cost == 0:
        assert starts[:used] == [c * T // used for c in range(used)]
    if window == 0:
        assert starts == ops.causal_split(B, Hkv, N, S, 64, C, cost)


def test_windowed_causal_split_refuses_bad_windows():
    for window, sinks in ((-1, 0), (4, -1), (0, 3)):
        with pytest.raises(ops.TTError):
            ops.causal_split(1, 1, 64, 8, 64, 4, -1, window, sinks)


def test_a_causal_split_of_the_longest_sequence_is_refused_before_its_table_is_made():
    """2^31 - 1 blocks: too many tiles, found long before 8 GB of prefix sums are."""
    import resource
    before = resource.getrusage(resource.RUSAGE_SELF).ru_maxrss
    with pytest.raises(ops.TTError) as e:
        ops.causal_split(1, 1, 2 ** 31 - 1, 1, 64, 4)
    assert e.value.status == ops.TT_ERR_UNSUPPORTED
    assert resource.getrusage(resource.RUSAGE_SELF).ru_maxrss - before < 1 << 20   # KB
