"""The oracle's reading of draft probabilities that are none: what is not above 0 counts as 0, as the target's do."""

import numpy as np
import pytest

import oracle

NAN = float("nan")


@pytest.mark.parametrize("none", [0.0, -0.0, -0.5, NAN, -np.inf])
def test_what_is_no_draft_probability_counts_as_zero(none):
    p = np.array([[0.25, 0.25, 0.5], [0.5, 0.25, 0.25]])
    q = np.array([[0.5, none, 0.25], [NAN, NAN, NAN]])
    # word 1 has no draft probability: it stays at any random number, as u * 1 * 0 < 0.25
    assert oracle.tree.verify([0, 1], [-1, 0], p, [0.0, 0.99], q) == ([0, 1], 0)
    # word 0 is refused (0.6 * 0.5 > 0.25): r = max(p - q, 0) = [0, 0.25, 0.25]
    assert oracle.tree.verify([0, 0], [-1, 0], p, [0.49, 0.6], q) == ([0], 1)
    assert oracle.tree.verify([0, 0], [-1, 0], p, [0.51, 0.6], q) == ([0], 2)
    # and then word 1 stays, and a random number of 0 gives the first word of the row behind it
    assert oracle.tree.verify([0, 0, 1], [-1, 0, 0], p[[0, 0, 0]], [0.0, 0.6, 0.99], q[[0, 0, 0]]) == ([0, 2], 0)
    # after a second refusal c is 1 + 0.5: word 2 has r = 0.5 - 1.5 * 0.25 left, word 1 all of its 0.25
    assert oracle.tree.verify([0, 0, 0], [-1, 0, 0], p[[0, 0, 0]], [0.66, 0.6, 0.9], q[[0, 0, 0]]) == ([0], 1)
    assert oracle.tree.verify([0, 0, 0], [-1, 0, 0], p[[0, 0, 0]], [0.67, 0.6, 0.9], q[[0, 0, 0]]) == ([0], 2)


@pytest.mark.parametrize("none", [0.0, -0.5, NAN, -np.inf])
def test_what_is_no_target_probability_counts_as_zero(none):
    p = np.array([[0.5, none, 0.5]])
    assert oracle.tree.verify([0], [-1], p, [0.49]) == ([0], 0)
    assert oracle.tree.verify([0], [-1], p, [0.51]) == ([0], 2)
    assert oracle.tree.verify([0, 1], [-1, 0], p[[0, 0]], [0.51, 0.0]) == ([0], 2)
