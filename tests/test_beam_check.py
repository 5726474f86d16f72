"""The check of selected candidates itself, on fabricated results: it takes the oracle's and refuses wrong ones."""
import numpy as np
import pytest

from oracle import beam as obeam
from test_gpu_beam_order import check_exactly

torch = pytest.importorskip("torch")


def fabricate(x, scores, n, finished=None, end=-1):
    s, p, t = obeam.select(x, scores, n, finished, end)
    return s.astype(np.float32), p.copy(), t.copy()


def refuses(x, scores, n, change, finished=None, end=-1):
    got = fabricate(x, scores, n, finished, end)
    check_exactly(torch.from_numpy(x), scores, n, finished, end, got)
    change(*got)
    with pytest.raises(AssertionError):
        check_exactly(torch.from_numpy(x), scores, n, finished, end, got)


def test_a_wrong_last_place_is_refused():
    x = np.random.default_rng(1).standard_normal((2, 5000)).astype(np.float32)
    zero = np.zeros((2, 1), np.float32)

    def other_token(s, p, t):
        t[1, -1] = (t[1, -1] + 123) % 5000

    refuses(x, zero, 1, other_token)
    refuses(x, zero, 4, other_token)


def test_equal_logits_out_of_order_are_refused():
    x = np.zeros((1, 700), np.float32)
    zero = np.zeros((1, 1), np.float32)

    def later_tokens(s, p, t):
        t += 500

    def swapped(s, p, t):
        t[0, :2] = t[0, 1::-1]

    refuses(x, zero, 4, later_tokens)
    refuses(x, zero, 4, swapped)


def test_a_score_of_another_candidate_is_refused():
    x = np.random.default_rng(2).standard_normal((3, 400)).astype(np.float32)
    scores = np.array([[0, -0.5, -1]], np.float32)

    def off(s, p, t):
        s[0, 3] += 1e-5

    def twice(s, p, t):
        p[0, 3], t[0, 3], s[0, 3] = p[0, 2], t[0, 2], s[0, 2]

    refuses(x, scores, 6, off)
    refuses(x, scores, 6, twice)


def test_an_end_token_before_its_turn_is_refused():
    x = np.zeros((1, 10), np.float32)

    def first(s, p, t):
        t[0] = [7, 0, 1]

    refuses(x, np.full((1, 1), -np.inf, np.float32), 3, first, np.array([[True]]), 7)
