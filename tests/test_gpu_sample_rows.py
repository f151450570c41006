"""wql_sample on rows that do not fit shared memory, one and two blocks to a
row: the modes that a large batch runs in, every filter, lists that run over."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import ref64
import test_gpu_operators as small
import weight_only_quantized_wql_gb300 as wql

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
LOG2E = float(np.float32(1.44269504088896340736))       # as a temperature: c = 1
T = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def sample_exact(l, top_k, top_p, min_p, u):
    """ref64.sample_exact for whole logits at c = 1, in integer arrays."""
    l = np.asarray(l, dtype=np.int64)
    n = l.size
    d = l.max() - l
    w = np.where(d <= 31, np.int64(1) << (31 - np.minimum(d, 31)), 0)
    order = np.argsort(d, kind="stable")                # by logit descending, then by index
    if 0 < top_k < n:
        order = order[:top_k]
    if top_p < 1:
        reach = Fraction(float(np.float32(top_p))) * int(w[order].sum())
        before = np.cumsum(w[order]) - w[order]
        order = order[:max(1, int(np.searchsorted(before, -(-reach.numerator // reach.denominator))))]
    if min_p > 0:
        least = Fraction(min(float(np.float32(min_p)), 1.0)) * (1 << 31)
        order = order[w[order] >= -(-least.numerator // least.denominator)]
    at = np.sort(order)
    run = np.cumsum(w[at])
    total = int(run[-1])
    r = min(int(Fraction(float(np.float32(u))) * total), total - 1)
    i = int(at[np.searchsorted(run, r, side="right")])
    return i, int(w[i]), total


FILTERS = [  # top_k, top_p, min_p, spread of the logits
    (0, 1.0, 0.0, 20), (0, 1.0, 0.25, 12), (50, 1.0, 0.0, 30), (20, 0.8, 0.1, 12),
    (500, 1.0, 0.0, 8),        # a list with many ties: more than a block's own
    (512, 0.9, 0.0, 3),        # and more than it can hold
    (800, 1.0, 0.0, 6), (9000, 0.99, 0.0, 3), (0, 0.9, 0.0, 30), (0, 0.5, 0.05, 12),
    (0, 0.9, 0.0, 3), (0, 0.6, 0.0, 1),       # more open tokens than the list holds
    (0, 1e-9, 0.0, 8)]
ROWS = [  # rows, logits, type, elements past a 16-byte boundary
    (160, 40008, "bf16", 0), (160, 40001, "f16", 0), (160, 40008, "bf16", 3),
    (160, 20000, "f32", 0), (160, 20003, "f32", 1), (100, 151936, "bf16", 0),
    (100, 100003, "f16", 5), (100, 60000, "f32", 0), (30, 200001, "f32", 0)]


def test_the_reference_is_the_other_one():
    g = torch.Generator().manual_seed(3)
    for n, spread in ((1, 3), (50, 5), (700, 2)):
        for top_k, top_p, min_p, _ in FILTERS:
            l = torch.randint(-spread, spread + 1, (n,), generator=g).tolist()
            u = float(torch.rand(1, generator=g))
            assert sample_exact(l, top_k, top_p, min_p, u) == \
                ref64.sample_exact([float(v) for v in l], LOG2E, top_k, top_p, min_p, u)


def full(v, m, dtype=torch.float32):
    return torch.full((m,), v, dtype=dtype, device=DEV)


def shifted(l, shift):
    if shift == 0:
        return l
    off = torch.empty(l.numel() + shift, dtype=l.dtype, device=DEV)[shift:].view(l.shape)
    off.copy_(l)
    return off


@pytest.mark.parametrize("top_k,top_p,min_p,spread", FILTERS)
@pytest.mark.parametrize("m,n,dt,shift", ROWS)
def test_long_rows_exact(m, n, dt, shift, top_k, top_p, min_p, spread):
    g = torch.Generator().manual_seed(n + top_k + spread)
    l = torch.randint(-spread, spread + 1, (m, n), generator=g, dtype=torch.int8)
    # one row's largest logits lie in its last quarter
    l[1, :n - n // 4].clamp_(max=spread - 2)
    u = torch.rand(m, generator=g)
    u[0], u[1] = 0.0, 1.0 - 2.0 ** -24
    ids, logp = wql.wql_sample(
        shifted(l.to(DEV).to(T[dt]), shift), u.to(DEV), full(LOG2E, m), full(top_k, m, torch.int32),
        full(top_p, m), full(min_p, m))
    for i in (0, 1, 2, m // 2, m - 1):
        want, w, total = sample_exact(l[i].numpy(), top_k, top_p, min_p, float(u[i]))
        assert int(ids[i]) == want, i
        # two roundings to fp32, a division and logf (2 ulp of the result)
        lp = np.log(w / total)
        assert abs(float(logp[i]) - lp) <= 4 * 2.0 ** -24 + 2.0 ** -22 * abs(lp)


@pytest.mark.parametrize("mode", ["plain", "top_k", "top_p", "min_p", "all", "wide", "flat"])
@pytest.mark.parametrize("m,n,dt", [(160, 40001, "bf16"), (160, 40008, "f16"), (160, 20003, "f32"),
                                    (100, 60000, "bf16")])
def test_long_rows_of_real_logits(mode, m, n, dt):
    small.test_sample_real_logits(mode, m, n, dt)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m,shift", [(160, 0), (160, 1), (2, 0), (2, 3)])
@pytest.mark.parametrize("top_k,top_p,min_p", [(0, 1.0, 0.0), (0, 0.7, 0.0), (300, 0.9, 0.0),
                                               (1 << 19, 0.5, 0.1)])
def test_longest_rows_all_equal(m, shift, dt, top_k, top_p, min_p):
    """The largest sums that the histograms and the stretches hold, ties all over."""
    n = wql.SAMPLE_MAX_N
    l = shifted(torch.zeros(m, n, dtype=T[dt], device=DEV), shift)
    u = (torch.arange(m, device=DEV).float() + 0.5) / m
    ids, logp = wql.wql_sample(l, u, full(1.0, m), full(top_k, m, torch.int32), full(top_p, m),
                               full(min_p, m))
    keep = top_k or n
    if top_p < 1:
        reach = Fraction(float(np.float32(top_p))) * keep
        keep = -(-reach.numerator // reach.denominator)
    want = [min(int(Fraction(float(v)) * keep), keep - 1) for v in u.cpu()]
    assert ids.cpu().tolist() == want
    assert torch.all((logp.double() + np.log(keep)).abs() <= 2.0 ** -21 * np.log(keep))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("m", [160, 3])
def test_longest_rows_exact(m, dt):
    n = wql.SAMPLE_MAX_N - 5
    g = torch.Generator().manual_seed(m)
    l = torch.randint(-6, 7, (m, n), generator=g, dtype=torch.int8)
    u = torch.rand(m, generator=g)
    for top_k, top_p, min_p in ((0, 1.0, 0.0), (0, 0.97, 0.01), (40, 0.9, 0.0), (100000, 0.9, 0.0)):
        ids, _ = wql.wql_sample(l.to(DEV).to(T[dt]), u.to(DEV), full(LOG2E, m),
                                full(top_k, m, torch.int32), full(top_p, m), full(min_p, m))
        for i in (0, m - 1):
            assert int(ids[i]) == sample_exact(l[i].numpy(), top_k, top_p, min_p, float(u[i]))[0]
