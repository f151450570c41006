"""wql_sample where its definition is decided by the last bit: products of a
32-bit float and an exact sum, and temperatures next to zero."""
import numpy as np
import pytest
import torch

import ref64
import weight_only_quantized_wql_gb300 as wql

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
LOG2E = float(np.float32(1.44269504088896340736))       # as a temperature: c = 1
T = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def powers(total, top):
    """Exponents of powers of two, at most 2^top, that sum to total, descending."""
    out = [top] * (total >> top)
    return out + [b for b in range(top - 1, -1, -1) if total >> b & 1]


def logits_of(exponents):
    """Logits whose weights at c = 1 are those powers of two (the largest is 2^31)."""
    assert max(exponents) == 31
    return [float(b - 31) for b in exponents]


def draw(l, dt, u, top_k=None, top_p=None):
    one = lambda v, d=torch.float32: None if v is None else torch.tensor([v], dtype=d, device=DEV)  # noqa: E731
    ids, _ = wql.wql_sample(torch.tensor([l], device=DEV).to(T[dt]), one(u), one(LOG2E),
                            one(top_k, torch.int32), one(top_p))
    return int(ids[0])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("total", [2 ** 33 + 3, 2 ** 33 + 25, 2 ** 35 + 7])
@pytest.mark.parametrize("top_k", [None, 400])
def test_draw_just_below_a_running_sum(dt, total, top_k):
    """u * total lies 2^-24 below the running sum of the first tokens: in 53
    bits it would round up to it, and the next token be drawn."""
    k = -pow(total, -1, 1 << 24) % (1 << 24)
    first = (k * total + 1) >> 24
    u = k / 2.0 ** 24
    assert float(np.float32(u)) == u and float(u) * float(total) == first
    a, b = powers(first, 31), powers(total - first, 31)
    pad = [float("-inf")] * 500
    l = logits_of(a + b) + pad
    want, _, s = ref64.sample_exact(l, LOG2E, top_k or 0, 1.0, 0.0, u)
    assert want == len(a) - 1 and s == total
    assert draw(l, dt, u, top_k) == want


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("top_k", [None, 400, 600])
@pytest.mark.parametrize("step", [129, 141])
def test_nucleus_just_above_a_running_sum(dt, top_k, step):
    """top_p * total lies 2^-24 above the sum of the first ranks: the next rank
    is kept, which 53 bits would lose."""
    total = (step << 24) - 1
    p = 1.0 - 2.0 ** -24
    rest = step                                       # total = before + rest
    before = total - rest
    assert (((1 << 24) - 1) * total - 1) >> 24 == before and p * float(total) == before
    assert before % 2 == 0                            # the rest: weights of 1, below the head's
    tail = powers(rest, 0)
    head = powers(before, 31)
    # the first rank of the rest at index 0, drawn by u = 0 if it is kept
    l = logits_of([tail[0]] + head + tail[1:]) + [float("-inf")] * 700
    want, _, _ = ref64.sample_exact(l, LOG2E, top_k or 0, p, 0.0, 0.0)
    assert want == 0
    assert draw(l, dt, 0.0, top_k, p) == want


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n,top_k,top_p,spread", [
    (1000, 50, 1.0, 12), (1000, 0, 0.5, 12), (1000, 20, 0.8, 12), (5003, 2500, 0.6, 3),
    (40001, 40, 0.95, 30), (40001, 0, 0.9, 3), (100003, 0, 0.6, 1), (100003, 30000, 0.5, 1)])
def test_temperature_next_to_zero(n, top_k, top_p, spread, dt):
    """c = 2^126 and logits that far below 1: four times c is no float."""
    m, tiny = 4, 2.0 ** -126
    t = LOG2E * tiny
    assert float(np.float32(t)) == t
    g = torch.Generator().manual_seed(n + top_k)
    l = torch.randint(-spread, spread + 1, (m, n), generator=g).float() * tiny
    u = torch.tensor([0.0, 0.3, 0.77, 1.0 - 2.0 ** -24])
    full = lambda v, d=torch.float32: torch.full((m,), v, dtype=d, device=DEV)  # noqa: E731
    ids, logp = wql.wql_sample(l.to(T[dt]).to(DEV), u.to(DEV), full(t), full(top_k, torch.int32),
                               full(top_p))
    for i in range(m):
        want, w, total = ref64.sample_exact(l[i].tolist(), t, top_k, top_p, 0.0, float(u[i]))
        assert int(ids[i]) == want
        lp = np.log(w / total)
        assert abs(float(logp[i]) - lp) <= 4 * 2.0 ** -24 + 2.0 ** -22 * abs(lp)
