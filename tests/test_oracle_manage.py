"""The page-management oracle keeps what it must keep (CPU)."""
import random

import pytest

from oracle import manage


def invariants(s):
    held = [e for row in s.table for e in row if e >= 0]
    assert [held.count(p) for p in range(len(s.ref))] == s.ref


def contents(s, b):
    return [None if s.table[b][p] < 0 else s.data[s.table[b][p]] for p in range(-(-s.lens[b] // s.ps))]


@pytest.mark.parametrize("seed", range(20))
def test_random_traffic_keeps_counts_and_contents(seed):
    rng = random.Random(seed)
    s = manage.State(40, 6, 8, 4)
    stamp = 0
    for _ in range(60):
        what = rng.choice(["reserve", "fork", "free", "trim", "compact"])
        before = [contents(s, b) for b in range(6)]
        if what == "reserve":
            want = [rng.choice([0, L + rng.randrange(6)]) for L in s.lens]
            if not manage.reserve(s, want):
                for b in range(6):
                    for p in range(-(-s.lens[b] // 4), -(-want[b] // 4)):
                        s.data[s.table[b][p]] = stamp = stamp + 1
                    s.lens[b] = max(s.lens[b], want[b])
            for b in range(6):
                assert contents(s, b)[:len(before[b])] == before[b]
        elif what == "fork":
            rows = rng.sample(range(6), rng.randrange(2, 6))
            n = rng.randrange(1, len(rows))
            src = [rng.choice(rows[n:]) for _ in range(n)]
            if not manage.fork(s, src, rows[:n]):
                for a, b in zip(src, rows[:n]):
                    assert contents(s, b) == before[a] and s.lens[a] == s.lens[b]
                    if s.lens[a] % 4 and s.table[a][s.lens[a] // 4] >= 0:
                        assert s.table[a][s.lens[a] // 4] != s.table[b][s.lens[a] // 4]
        elif what == "free":
            b = rng.randrange(6)
            assert not manage.free(s, [b, b])
            assert s.lens[b] == 0 and max(s.table[b]) == -1
        elif what == "trim":
            assert not manage.free(s, None, window=rng.randrange(12), sinks=rng.randrange(6))
        else:
            live, errors = manage.compact(s)
            assert not errors and all(s.ref[:live]) and not any(s.ref[live:])
            assert [contents(s, b) for b in range(6)] == before
        invariants(s)


def test_copy_refuses_what_would_race():
    s = manage.State(6, 1, 1, 4)
    s.data = list("abcdef")
    assert manage.copy(s, [0, 0, 3], [1, 2, 3]) == set() and s.data == list("aaadef")
    assert manage.copy(s, [3, 4], [5, 5]) == {"bounds"} and s.data == list("aaadef")
    assert manage.copy(s, [3, 4, 5], [4, 0, 9]) == {"bounds"} and s.data == list("eaadef")
