"""The append's row order in the plain replay: of the rows next to a stream's first
one those count whose position fits their distance from it, up to the first break in
their page."""
import numpy as np
import pytest

from oracle.kv8 import Kv8Replay

# positions of one stream's rows (slots of its segment, pages of 16) and those dropped
BREAKS = [
    ([*range(7), 99, *range(8, 16)], list(range(7, 16))),      # one far off
    ([*range(7), -1, *range(8, 16)], list(range(7, 16))),
    ([21, 30, 23], [1, 2]),
    ([4, 5, 9, 7, 8], [2, 3, 4]),
    ([3, 4, 4, 6, 7], [2, 3, 4]),                              # one twice
    ([3, 4, 6, 6, 7], [2, 3, 4]),                              # one left out
    ([13, 15, 15, 16, 17], [1, 2]),                            # fits again at a page's start
    ([*range(5, 16), 0, *range(17, 40)], list(range(11, 27))),
    ([*range(10, 20), *range(10, 20)], list(range(10, 20))),   # the run once more
    ([5, 4, 3, 8, 9], [1, 2, 3, 4]),
]


def dropped_of(slots, page):
    """The rule by its words: a row counts when it and all rows of the run that lie
    before it in its page are at their places."""
    fits = [x - slots[0] == j for j, x in enumerate(slots)]
    return [j for j, x in enumerate(slots) if not all(fits[max(0, j - x % page):j + 1])]


@pytest.mark.parametrize("slots,drop", BREAKS)
def test_rows_behind_a_break_in_their_page_are_dropped(slots, drop):
    assert dropped_of(slots, 16) == drop
    tab = [[3, 5, 6, 7], [1, 4, 2, 0]]
    g = np.random.default_rng(1)
    k = g.standard_normal((len(slots) + 2, 1, 2)).astype(np.float32)
    sid = [1] + [2] * len(slots) + [1]
    pos = [7] + [7 + x if x >= 0 else x for x in slots] + [8]
    r, kept = Kv8Replay(1, 2, 16, 8, 7, [], tab), Kv8Replay(1, 2, 16, 8, 7, [], tab)
    assert r.append(k, k, sid, pos) == [i + 1 for i in drop] + [len(slots) + 1]
    # the same as the kept rows by themselves, a page a call
    keep = [0] + [i + 1 for i in range(len(slots)) if i not in drop]
    for s, pg in sorted({(sid[i], (pos[i] - 7) // 16) for i in keep}):
        part = [i for i in keep if (sid[i], (pos[i] - 7) // 16) == (s, pg)]
        assert kept.append(k[part], k[part], [s] * len(part), [pos[i] for i in part]) == []
    for t in ("k", "v", "k_scale", "v_scale"):
        assert np.array_equal(getattr(r, t), getattr(kept, t)), t
