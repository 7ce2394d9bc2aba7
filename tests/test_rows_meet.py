"""Whether the rows of two activations share memory, against counting every element, on the CPU."""

import random

import pytest
import torch


def views(rng):
    """Two [T, H, .] views of one buffer."""
    T, H, D, V = rng.randint(1, 5), rng.randint(1, 4), rng.randint(1, 6), rng.randint(1, 6)
    kind = rng.randrange(4)
    if kind == 0:  # tokens of queries, then results
        a, b = (H * D + H * V + rng.randint(0, 2), D), None
        b = (a[0], V)
        off = rng.choice([H * D, H * D - 1, H * D + 1, -H * V, rng.randint(-40, 40)])
    elif kind == 1:  # heads of queries, then results
        s = D + V + rng.randint(0, 2)
        a = b = (H * s, s) if rng.random() < 0.5 else (s, T * s)
        off = rng.choice([D, D - 1, s - V, s - V + 1, rng.randint(-40, 40)])
    elif kind == 2:
        a, b = (H * D, D), (H * V, V)
        off = rng.choice([T * H * D, T * H * D - 1, -T * H * V, 1 - T * H * V, rng.randint(-40, 40)])
    else:
        a, b = [(rng.randint(0, 20), rng.randint(0, 20)) for _ in range(2)]
        off = rng.randint(-60, 60)
    buf = torch.zeros(2000, dtype=torch.int16)
    return buf.as_strided((T, H, D), (*a, 1), 800), buf.as_strided((T, H, V), (*b, 1), 800 + off)


@pytest.mark.parametrize("seed", range(40))
def test_against_counting(seed):
    from speculative_decoding_verification_29_gb300.api import _rows_meet

    rng, seen = random.Random(seed), set()
    for _ in range(100):
        x, y = views(rng)
        at = [set((t.storage_offset() + i * t.stride(0) + j * t.stride(1) + k for i in range(t.shape[0])
                   for j in range(t.shape[1]) for k in range(t.shape[2]))) for t in (x, y)]
        meet = bool(at[0] & at[1])
        assert _rows_meet(x, y) == meet, (x.shape, x.stride(), y.shape, y.stride(), y.storage_offset() - 800)
        seen.add(meet)
    assert seen == {False, True}


def test_more_rows_than_are_looked_at():
    """2^25 rows: told apart by their strides, or taken to meet."""
    from speculative_decoding_verification_29_gb300.api import _meet

    T, H = 1 << 15, 1 << 10
    side = (T, H, 8, H * 16, 16, 8, H * 16, 16)
    assert not _meet(*side, 8) and _meet(*side, 16)
    assert not _meet(T, H, H * 8, H * 24, 8, 8, H * 24, 16, 16)
    assert _meet(T, H, 8, H * 24, 16, 8, H * 24, 24, 8)
