"""Beam selection, candidate by candidate: which one stands at each place, and how far its score is from 64 bits."""
import numpy as np
import pytest

from kvq_helpers import dev, host
from test_gpu_beam import TYPES, logits, run_select

pytestmark = pytest.mark.gpu

# What the logarithm of a row's sum may be off by, relative errors of the sum's terms added up. A term at distance d from
# the maximum: its exponent's rounding, d 2^-24, and d 1.4e-8 of log2(e)'s; the exponential's two steps, 2^-22. With n terms
# there d counts with at most n exp(-d) / (1 + n exp(-d)) of the sum: 1.1e-6 for n = 2^22. Additions in float32: 16 terms one
# after the other (8.5 2^-24 on average of what they have added), 64 steps (32.5 2^-24), 4 2^-24 for the thread's and the
# part's factors and the logarithm. 3.8e-6 in all, which is 2^-18.
LOG = 2.0**-18
FP32_MAX = float(np.finfo(np.float32).max)


def row_totals(x, scores, finished, end):
    """Scores of all candidates in 64 bits [R, W, V], and the logits as they count."""
    r, w = scores.shape
    x = host(x.float()).astype(np.float64).reshape(r, w, -1)
    x = np.minimum(np.where(np.isnan(x), -np.inf, x), FP32_MAX)
    total = np.full(x.shape, -np.inf)
    for g, i in np.ndindex(r, w):
        s = float(scores[g, i])
        if not np.isfinite(s):
            continue
        if finished is not None and finished[g, i]:
            total[g, i, end] = s
        elif x[g, i].max() > -np.inf:
            d = x[g, i] - x[g, i].max()
            total[g, i] = s + (d - np.log(np.exp(d).sum()))
    return total, x


def check_exactly(x, scores, n, finished=None, end=-1, got=None):
    """Every place's candidate: those of one beam are its best ones in the order of their logits, equal ones by the token;
    candidates at -inf come last, by their index; beams are interleaved by scores that 64 bits give, but where two are
    closer than what the logarithms and the outputs' rounding (2^-24 of their size) leave."""
    s, p, t = run_select(x, scores, n, finished, end) if got is None else got
    total, x = row_totals(x, scores, finished, end)
    r, w, v = total.shape
    for g in range(r):
        own = total[g, p[g], t[g]]
        fin = np.isfinite(own)
        k = int(min(n, np.isfinite(total[g]).sum()))
        assert fin[:k].all() and not fin[k:].any()
        off = LOG + 2.0**-24 * np.abs(own[:k])
        assert (np.abs(s[g, :k] - own[:k]) <= off).all() and (s[g, k:] == -np.inf).all()
        assert (np.diff(s[g, :k]) <= 0).all()
        for i in range(w):
            mine = t[g, :k][p[g, :k] == i]
            order = np.lexsort((np.arange(v), -x[g, i], -total[g, i]))[: len(mine)]
            assert np.array_equal(mine, order), (g, i, mine, order)
        # what stands at a place is no worse than the best of what comes behind it, the candidates left out among them
        best = np.sort(total[g].ravel())[::-1][:k]
        assert (np.abs(own[:k] - best) <= 2 * LOG).all()
        flat = np.flatnonzero(np.isneginf(total[g].ravel()))[: n - k]
        assert np.array_equal(p[g, k:] * v + t[g, k:], flat)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("w,n", [(1, 3), (2, 9), (3, 16), (40, 20)])
@pytest.mark.parametrize("score", [-np.inf, np.inf, np.nan])
def test_select_ended_beams_without_a_finite_score(kind, w, n, score):
    """They are dead beams: their tokens go by their index, the end token among them."""
    import torch
    rng = np.random.default_rng(w)
    v, end = 300, 7
    x = torch.full((2 * w, v), -float("inf"), dtype=getattr(torch, kind), device="cuda")
    x[:, 5], x[:, 200] = 1.0, 3.0
    scores = rng.uniform(-9, 0, (2, w)).astype(np.float32)
    finished = rng.random((2, w)) < 0.3
    scores[:, 0], finished[:, 0] = score, True
    scores[1], finished[1] = score, True
    check_exactly(x, scores, n, finished, end)


@pytest.mark.parametrize("kind", ["float32", "bfloat16"])
@pytest.mark.parametrize("w,n", [(1, 2), (1, 3), (1, 128), (3, 5), (2, 100)])
def test_select_orders_a_beam_by_its_logits(kind, w, n):
    """Logits so near to one another that their scores are equal in 64 bits, the larger ones further back in the row."""
    import torch
    v = 64000
    x = torch.full((w, v), -1.0, dtype=getattr(torch, kind), device="cuda")
    x[:, 31] = 30.0
    at = torch.arange(100, device="cuda") * 601 + 7
    x[:, at] = (torch.arange(100, device="cuda") + 1).to(x.dtype) * 2.0**-80
    check_exactly(x, np.zeros((1, w), np.float32), n)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("below", [3.6875, 4.125, 6.1875])
def test_select_sums_of_long_rows(kind, below):
    """Four million tokens, one in four of them the largest: additions to a long sum whose roundings all point one way. The
    beam's score takes the logarithm off, so that the output's rounding hides nothing."""
    import torch
    v, w = 1 << 22, 64
    x = torch.empty((w, v), dtype=getattr(torch, kind), device="cuda")
    x[0] = -below
    x[0, ::4] = 0.0
    log = np.log(v / 4 * (1 + 3 * np.exp(-below)))
    scores = np.full((1, w), -np.inf, np.float32)
    scores[0, 0] = log
    s, p, t = run_select(x, scores, 3)
    assert p.tolist() == [[0, 0, 0]] and t.tolist() == [[0, 4, 8]]
    assert np.abs(s - (float(scores[0, 0]) - log)).max() <= LOG


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("w", [1, 16])
def test_select_sums_of_constant_tails(kind, w):
    """One large logit and 128000 equal ones: every term carries the same rounding."""
    import torch
    rng = np.random.default_rng(w)
    v = 128000
    for below in (2.5, 5.625, 8.25, 11.125, 12.0):
        x = torch.full((w, v), 20.0 - below, dtype=getattr(torch, kind), device="cuda")
        x[torch.arange(w, device="cuda"), dev(rng.integers(0, v, w))] = 20.0
        log = np.log1p((v - 1) * np.exp(float(x[0].min()) - 20.0))
        scores = np.full((1, w), log, np.float32)
        check_exactly(x, scores, 2 * w)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("r,w,v,n", [
    (1, 1, 1, 1), (2, 3, 17, 5), (1, 4, 32000, 4), (3, 5, 999, 10), (7, 1, 50021, 1), (2, 8, 4097, 16), (1, 64, 300, 128),
    (40, 4, 2048, 8), (1, 3, 131072, 128), (5, 16, 16385, 32), (9, 2, 50021, 1)])
def test_select_every_place(r, w, v, n, kind):
    rng = np.random.default_rng(r * 1000 + w * 100 + v)
    x = logits(rng, r * w, v, kind)
    check_exactly(x, rng.uniform(-20, 0, (r, w)).astype(np.float32), n)
    finished = rng.random((r, w)) < 0.3
    check_exactly(x, rng.uniform(-20, 0, (r, w)).astype(np.float32), n, finished, v // 2)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("n", [1, 4, 16, 128])
def test_select_equal_logits_go_by_the_token(kind, n):
    import torch
    v = 70000
    i = torch.arange(v, device="cuda", dtype=torch.float32)
    for row in (0 * i, i // 9000, -(i // 9000), (i * 7919) % 5, (i * 7919) % 4000 // 1000):
        x = row.to(getattr(torch, kind)).repeat(4, 1)
        check_exactly(x, np.array([[0, -1.5], [-2.25, -2.25]], np.float32), n)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("left", [0, 1, 3, 40])
def test_select_what_bans_leave_goes_by_the_index(kind, left):
    rng = np.random.default_rng(left)
    x = logits(rng, 6, 40000, kind)
    for row in range(6):
        banned = np.ones(40000, bool)
        banned[rng.permutation(40000)[:left]] = False
        x[row, dev(banned)] = float("nan") if row % 2 else -float("inf")
    check_exactly(x, rng.uniform(-9, -3, (2, 3)).astype(np.float32), 12)


@pytest.mark.parametrize("at", [-65536.0, -1e6, 30000.0, 65536.0, 1e6, 1e30])
def test_select_every_place_of_large_logits(at):
    rng = np.random.default_rng(11)
    x = rng.integers(-8, 8, (6, 30000)).astype(np.float32)
    x[:3] += np.float32(at)
    x[3:, 15000:] += np.float32(at)
    check_exactly(dev(x), rng.uniform(-9, 0, (2, 3)).astype(np.float32), 5)


@pytest.mark.parametrize("kind,v", [("float32", 300003), ("float16", 600001), ("bfloat16", 600001)])
@pytest.mark.parametrize("shift", [0, 3])
def test_select_every_place_of_long_rows(kind, v, shift):
    """Rows whose sums are folded on the way: banned, rising, with NaN and infinities, on any boundary."""
    import torch
    rng = np.random.default_rng(shift)
    w = 16
    whole = torch.full((w, v + 5), float("nan"), dtype=getattr(torch, kind), device="cuda")
    x = whole[:, shift:shift + v]
    x.copy_(logits(rng, w, v, kind))
    ramp = torch.arange(v, device="cuda") / v
    x[1] = (3 * ramp).to(x.dtype)
    x[2] = (0.01 * ramp - 70000 * (kind != "float16")).to(x.dtype)
    x[3] = -float("inf")
    x[4, : v - 4] = float("nan")
    x[5, : v // 2] = -float("inf")
    x[6, v // 3] = float("inf")
    scores = rng.uniform(-14, -10, (1, w)).astype(np.float32)
    scores[0, 7] = -np.inf
    check_exactly(x, scores, 40)
    finished = rng.random((1, w)) < 0.3
    check_exactly(x, scores, 128, finished, v - 1)


def test_select_of_many_small_requests():
    import torch
    rng = np.random.default_rng(3)
    x = logits(rng, 70000 * 2, 21, "float16")
    scores = rng.uniform(-9, 0, (70000, 2)).astype(np.float32)
    s, p, t = run_select(x, scores, 5)
    y = x.double().view(70000, 2, 21)
    y = torch.log_softmax(y, 2) + dev(scores).double()[..., None]
    best = y.view(70000, 42).sort(dim=1, descending=True).values
    assert np.abs(s - host(best[:, :5])).max() <= LOG + 2.0**-24 * float(best.abs().max())
    own = host(y.view(70000, 42).gather(1, dev((p * 21 + t).astype(np.int64))))
    assert np.abs(own - host(best[:, :5])).max() <= 2 * LOG
