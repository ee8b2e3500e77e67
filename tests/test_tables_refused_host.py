"""The tables' model: what a step that was refused as a whole says (no GPU)."""

import numpy as np
import pytest

from oracle import tables as OT


@pytest.mark.parametrize("new,count,most,lacking,good", [
    (3, 10, 8, 0, True), (3, 10, 2, -1, False), (3, -1, 8, -1, False), (3, 11, 8, -1, False), (20, 0, 30, 1, True),
    (20, -1, 30, 1, False), (20, 0, 19, 1, False), (20, 10, 19, -1, False), (0, 10, 0, 0, True), (100, 10, 30, 0, False),
])
def test_what_a_step_says(new, count, most, lacking, good):
    # one request of 5 tokens, a table of 48, a stack of 10
    t, ctx, qs, slots, pos, bs, n, lack, ok = OT.extend(np.zeros((1, 3), dtype=np.int32), [5], [new],
                                                        np.arange(10, dtype=np.int32), count, 16, most, 50)
    assert (lack, ok) == (lacking, good)
    if lacking:                                       # nothing was done
        assert ctx[0] == 5 and not qs.any() and not bs.any() and n == count and (slots == -1).all() and (pos == -1).all()
