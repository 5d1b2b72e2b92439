"""The copying thread of the drafted trees' tensor-core kernel, gone through on
counters: host logic, checked on a machine without a GPU.  Whichever wait runs
out, and where none does, the thread stays until the last copy to each barrier
has landed, so that no copy reaches shared memory that is another block's."""
import os

import pytest

from polar_attention_b200 import native


@pytest.fixture(scope="module")
def copies():
    if not os.path.exists(native.LIB_PATH):
        pytest.skip("library not built")
    return native.tree_copies


@pytest.mark.parametrize("steps", [[], [1], [2], [3], [7], [1, 1], [1, 1, 1], [4, 1], [1, 4, 2],
                                   [5, 1, 1, 6], [3] * 9, [2] * 8])
def test_every_copy_lands(copies, steps):
    missed, waits = copies(steps)
    # A wait for each tile's queries but the first, and for each step past two stages.
    assert missed == 0 and waits == max(len(steps) - 1, 0) + max(sum(steps) - 2, 0)
    for n in range(waits):
        assert copies(steps, n) == (0, n + 1), (steps, n)


def test_bad_arguments(copies):
    with pytest.raises(ValueError):
        copies([3, 0])
