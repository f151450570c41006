"""Beam selection on logits of every finite size, against the 64-bit reference
(ref_requests.py): masks of large finite values, large maxima, rows masked throughout."""
import numpy as np
import pytest
import torch

import ref_requests as ref
import weight_only_quantized_wql_gb300 as wql
from ref64 import f64

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
T = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ORDERS = [wql.BEAM_RANKED, wql.BEAM_ANCHORED]

# The error of a score before its rounding.  Of the logarithm of the sum: a term is
# an exponential (2^-22) and passes at most 16 rescalings in its lane and three in the
# joins (2^-22 each); the arguments' roundings, two of each part of d = top - l and
# log2 e's own, add up to 2^-23 d + 2^-26 d, d's mean under the softmax being at most
# log n < 14; at most 65 additions on a term's way, 2^-24 each; the logarithm's
# mantissa 2^-23.  In rows far from zero the exponents hold a rounding R of the
# maximum's product besides, 2^-24 R (R <= 10 where logits are less than 14 apart), and
# products in two parts 2^-24.  In two fp32 parts a score of size s is off by 2^-45 s more.
SCORE = 20 * 2.0 ** -22 + 14 * (2.0 ** -23 + 2.0 ** -26) + 76 * 2.0 ** -24 + 2.0 ** -23
PARTS = 2.0 ** -45

LOWEST = {k: torch.finfo(v).min for k, v in T.items()}
LARGE = [-1e4, -1e9, -1e10, -1e11, -1e12, -1e20, -1e30, -1e38, -2.2e38]
MASKS = [(dt, m) for dt in ("f32", "bf16") for m in LARGE + [LOWEST[dt] / 2, LOWEST[dt]]]
MASKS += [("f16", -1e4), ("f16", LOWEST["f16"])]


def compare(logits, scores, eos, order):
    """A call against the reference; False where the inputs decide something by less
    than the errors."""
    tokens, parents, best, ended, gap = ref.beam_select(f64(logits), f64(scores), -1 if eos is None else eos,
                                                        order == wql.BEAM_ANCHORED)
    sizes = [np.abs(v[np.isfinite(v)]).max(initial=0.0) for v in (best, ended)]
    if gap <= 2 * (SCORE + PARTS * max(sizes)):
        return False
    t, p, s, e = wql.wql_beam_select(logits.to(DEV), scores.to(DEV), eos, order)

    def near(x, want):
        x, fine = f64(x), np.isfinite(want)
        np.testing.assert_array_equal(np.isfinite(x), fine)
        assert np.all(x[~fine] == -np.inf)
        err = np.abs(x[fine] - want[fine])
        tol = SCORE + (PARTS + 2.0 ** -24) * np.abs(want[fine])
        assert np.all(err <= tol), (err - tol).max()

    near(s, best)
    if eos is not None:
        near(e, ended)
    np.testing.assert_array_equal(t.cpu().numpy(), tokens)
    np.testing.assert_array_equal(p.cpu().numpy(), parents)
    return True


def first_clear(make, eos, order):
    for seed in range(20):
        if compare(*make(seed), eos, order):
            return
    raise AssertionError("no clear inputs")


def inputs(batch, beams, n, dt, seed):
    g = torch.Generator().manual_seed(seed)
    logits = (3 * torch.randn(batch, beams, n, generator=g)).to(T[dt])
    scores = -torch.rand(batch, beams, generator=g).cumsum(-1) * 2
    return g, logits, scores


# ---------------------------------------------------------------------------
# Rows far from zero
# ---------------------------------------------------------------------------
CENTERS = [("f16", 300.0), ("f16", 1000.0), ("f16", 3e4), ("bf16", 300.0), ("bf16", 1000.0)]
CENTERS += [("f32", c) for c in (300.0, 1000.0, 3e4, 7e5, 3e6, 3e7)]


@pytest.mark.parametrize("dt,center", CENTERS)
@pytest.mark.parametrize("sign", [1, -1])
def test_differences_of_large_logits(dt, center, sign):
    """Rows far from zero whose logits differ by ordinary amounts."""
    def make(seed):
        _, logits, scores = inputs(80, 4, 20000, dt, seed)
        return (logits.float() + sign * center).to(T[dt]), scores

    first_clear(make, 19, wql.BEAM_RANKED)


# ---------------------------------------------------------------------------
# Rows that are masked throughout
# ---------------------------------------------------------------------------
def check_whole_rows(dt, mask, order, n):
    """Every token of a masked row has the probability 1 / n."""
    def make(seed):
        _, logits, scores = inputs(4, 4, n, dt, seed)
        logits[0, 1] = mask
        logits[1, :3] = mask
        logits[2] = mask
        return logits, scores

    first_clear(make, 3, order)


@pytest.mark.parametrize("order", ORDERS)
@pytest.mark.parametrize("dt", T)
@pytest.mark.parametrize("n", [5, 20000])
def test_whole_rows_of_the_lowest_value(dt, order, n):
    check_whole_rows(dt, LOWEST[dt], order, n)


@pytest.mark.parametrize("order", ORDERS)
@pytest.mark.parametrize("dt,mask", MASKS)
@pytest.mark.parametrize("n", [5, 20000])
def test_whole_rows_masked(dt, mask, order, n):
    check_whole_rows(dt, mask, order, n)


# ---------------------------------------------------------------------------
# Rows that are masked in part, and large maxima
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("order", ORDERS)
@pytest.mark.parametrize("dt,mask", MASKS)
def test_few_tokens_allowed(dt, mask, order):
    """Six tokens of 20000 (the first, the last and the end token among them): whole
    lanes, warps and parts see nothing but the mask."""
    def make(seed):
        g, logits, scores = inputs(4, 4, 20000, dt, seed)
        allowed = torch.zeros(4, 4, 20000, dtype=torch.bool)
        allowed.scatter_(-1, torch.randint(1, 19999, (4, 4, 3), generator=g), True)
        allowed[..., [0, 77, -1]] = True
        return logits.masked_fill(~allowed, mask), scores

    first_clear(make, 77, order)


@pytest.mark.parametrize("dt,mask", MASKS)
def test_lanes_masked_before_and_after(dt, mask):
    """Rows of several steps, the first, the last or every other stretch of them masked."""
    def make(seed):
        _, logits, scores = inputs(80, 4, 20000, dt, seed)
        logits[0::4, :, :10000] = mask
        logits[1::4, :, 10000:] = mask
        for at in range(0, 20000, 1024):
            logits[2::4, :, at:at + 512] = mask
        return logits, scores

    first_clear(make, 19, wql.BEAM_RANKED)


@pytest.mark.parametrize("order", ORDERS)
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("top", [2e6, 1e10, 1e30, 1e38, 2.2e38, 3e38])
def test_large_maxima(dt, top, order):
    """Six equal maxima in half of the rows: they share the probability."""
    def make(seed):
        g, logits, scores = inputs(3, 4, 20000, dt, seed)
        logits[:, ::2].scatter_(-1, torch.randint(0, 20000, (3, 2, 6), generator=g), top)
        logits[2, :, 5000:] = -top
        return logits, scores

    first_clear(make, None, order)


@pytest.mark.parametrize("order", ORDERS)
@pytest.mark.parametrize("sign", [1, -1])
def test_maxima_on_both_sides_of_the_border(sign, order):
    """Lanes' maxima next to 2^31 / log2 e, where the sums change their form; one step
    of fp32 is 128 there."""
    def make(seed):
        g, logits, scores = inputs(3, 4, 20000, "f32", seed)
        steps = torch.randint(0, 3, (3, 4, 20000), generator=g) - 4
        steps.scatter_(-1, torch.randint(0, 20000, (3, 4, 6), generator=g), 2)
        steps[0, 0] = torch.randint(-2, 3, (20000,), generator=g)
        return (sign * 1488522240.0 + 128 * steps.double()).float(), scores

    first_clear(make, None, order)


# ---------------------------------------------------------------------------
# Scores far below the best
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("order", ORDERS)
def test_beams_meet_far_below_the_best(order):
    """A beam 5000 below another continues before that one's token 5000 below its best,
    by 3e-5."""
    logits = torch.full((1, 2, 40), -torch.inf)
    logits[0, :, 0] = 0.0
    logits[0, 1, 1] = -5000.0
    scores = torch.tensor([[-5000.0, -3e-5]])
    assert compare(logits, scores, None, order)


@pytest.mark.parametrize("order", ORDERS)
@pytest.mark.parametrize("dt,mask", MASKS)
def test_masked_tokens_are_selected(dt, mask, order):
    """Fewer allowed tokens than beams, and one beam: masked ones follow, the lowest first."""
    _, logits, scores = inputs(2, 4, 3000, dt, 0)
    allowed = torch.zeros(3000, dtype=torch.bool)
    allowed[[1, 2999]] = True
    logits.masked_fill_(~allowed, mask)
    scores[:, 0], scores[:, 1:] = -1.25, -torch.inf
    assert compare(logits, scores, 2, order)


# ---------------------------------------------------------------------------
# Scores below fp32's range
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("order", ORDERS)
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("mask", [-9e37, -1.7e38, -3e38])
def test_scores_below_the_range(dt, mask, order):
    """The lowest finite score and masked tokens: their sum rounds to -inf, which is no
    continuation; nor does a beam end with it."""
    logits = torch.full((1, 3, 50), mask).to(T[dt])
    logits[0, :2, 5] = 2.0                      # the end token: all that is left of beam 1
    logits[0, 0, 7] = 1.0
    logits[0, 2, 9] = 0.0
    low = torch.finfo(torch.float32).min
    t, p, s, e = wql.wql_beam_select(logits.to(DEV), torch.tensor([[0.0, low, low]], device=DEV), 5, order)
    # beam 0's two, its masked ones with a finite score; beam 2's token 9
    assert t.tolist() == [[7, 0, 1]] and p.tolist() == [[0, 0, 0]]
    assert torch.isfinite(s).all()
    lse = np.log(np.exp(2.0) + np.exp(1.0))
    assert abs(s[0, 0].item() - (1.0 - lse)) <= 1e-5 and abs(e[0, 0].item() - (2.0 - lse)) <= 1e-5
    assert torch.all(s[0, 1:] == logits[0, 0, 0].float().item())
    # beam 1 alone: what it has is its end; beam 2: one token
    t, p, s, e = wql.wql_beam_select(logits[:, 1:].to(DEV), torch.tensor([[low, low]], device=DEV), 5, order)
    at = 1 if order == wql.BEAM_ANCHORED else 0
    want = [[-1, -1]]
    want[0][at] = 9
    assert t.tolist() == want and p.tolist() == [[1 if v == 9 else -1 for v in want[0]]]
    assert s[0, at].item() == low and s[0, 1 - at].item() == -np.inf
    assert e[0, 0].item() == low and e[0, 1].item() == -np.inf
