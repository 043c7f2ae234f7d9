"""The plain oracle of the 4-bit cache against its definition in exact arithmetic, at the top of f16."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import int4_oracle as io


@pytest.mark.parametrize("top", [65504.0, 65472.0, 65408.0, 65376.0])
def test_f16_steps_at_the_top_of_the_type(top):
    """Every step is the type's next one up or, where 15 of it would pass 65504, the next one down; no code stands for
    more than the type holds, and none is further from its value than half a step."""
    torch = pytest.importorskip("torch")
    lows = np.concatenate([-np.geomspace(65504, 2.0 ** -24, 60), [0.0], np.geomspace(2.0 ** -24, top, 60)]).astype(np.float16)
    u = np.random.default_rng(0).random((len(lows), 32))
    u[:, 3], u[:, 9] = 0, 1
    x = torch.from_numpy((lows[:, None].astype(float) + (top - lows[:, None].astype(float)) * u).astype(np.float16))
    codes, step, low = io.quantise(x, 32)
    down = 0
    for row, code, st, lo in zip(x, codes, step[:, 0], low[:, 0]):
        row, st, lo = [Fraction(float(v)) for v in row], Fraction(float(st)), Fraction(float(lo))
        most = max(row)
        want = max((most - lo) / 15, Fraction(1, 2 ** 24))
        at = np.float16(float(st))
        assert lo == min(row) and Fraction(float(at)) == st
        up = st if st >= want else Fraction(float(np.nextafter(at, np.float16(np.inf))))
        before = Fraction(float(np.nextafter(np.float16(float(up)), np.float16(0))))
        assert before < want <= up
        assert st == (before if lo + 15 * up > 65504 and most > lo else up)
        down += st < want
        for v, c in zip(row, code):
            assert 0 <= c <= 15 and abs(lo + int(c) * st - v) <= st / 2 and abs(lo + int(c) * st) <= 65504
    assert down > 10 or top < 65440   # (few lows of the smaller tops need it)
