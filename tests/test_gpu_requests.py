"""Adapters beside a projection, beam selection and reordering on the GPU,
against 64-bit references (ref_requests.py)."""
import numpy as np
import pytest
import torch

import ref_requests as ref
import weight_only_quantized_wql_gb300 as wql
from ref64 import f64

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
T = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ULP = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}            # half an ulp, relative
TINY = {"f16": 2.0 ** -25, "bf16": 1e-38}               # half the smallest subnormal


def gen(seed):
    return torch.Generator().manual_seed(seed)


def placed(t, shift):
    """t on the GPU, `shift` elements behind a 16-byte boundary."""
    buf = torch.empty(t.numel() + shift, dtype=t.dtype, device=DEV)
    v = buf[shift:].view(t.shape)
    v.copy_(t)
    return v


# ---------------------------------------------------------------------------
# lora_add
# ---------------------------------------------------------------------------
def lora_inputs(m, n, k, r, count, dt, seed, size=1.0):
    g = gen(seed)
    y = (2 * torch.randn(m, n, generator=g)).to(T[dt])
    x = (size * torch.randn(m, k, generator=g)).to(T[dt])
    a = (torch.randn(count, r, k, generator=g) / k ** 0.5).to(T[dt])
    b = (0.3 * torch.randn(count, n, r, generator=g)).to(T[dt])
    scale = 0.5 + torch.rand(count, generator=g)
    # every adapter, none (three ways), in no order
    ids = torch.randint(-1, count + 1, (m,), generator=g, dtype=torch.int32)
    if m > 4:
        ids[1], ids[3] = -2 ** 31, 2 ** 31 - 1
    else:
        ids[:] = count - 1
    return y, x, a, b, scale, ids


def check_lora(got, y, x, a, b, scale, ids, dt):
    want, size, split = ref.lora(f64(y), f64(x), f64(a), f64(b),
                                 None if scale is None else f64(scale), ids.tolist())
    k, r = x.shape[-1], a.shape[1]
    # an fp32 sum of products on the tensor cores loses at most 2^-22 of the
    # summands' size a step of 16 (their truncation included), over the k / 16
    # steps of u, its 32 partial sums and the 2 * r / 16 steps of the product;
    # u in two parts of 16 bits leaves 2^-17 of it, or in fp16 2^-22 of the row's
    # largest; scale, factor and addition are 4 fp32 roundings
    tol = (k / 16 + 32 + r / 8 + 16) * 2.0 ** -22 * size + 2.0 ** -17 * size + 2.0 ** -22 * split
    tol += 4 * 2.0 ** -24 * (np.abs(want) + size)
    err = np.abs(f64(got) - want)
    bad = err > tol + ULP[dt] * (np.abs(want) + tol) + TINY[dt]
    assert not bad.any(), (int(bad.sum()), float((err - tol)[bad].max()))
    none = (ids < 0) | (ids >= a.shape[0])
    assert torch.equal(got.cpu()[none], y[none])


LORA = [(1, 1, 8, 8, 1), (1, 1000, 64, 16, 3), (1, 999, 5120, 16, 2), (5, 777, 72, 24, 2),
        (16, 128, 512, 32, 1), (17, 64, 40, 32, 1), (33, 1003, 136, 8, 5), (40, 264, 1032, 56, 40),
        (300, 520, 256, 64, 7), (257, 97, 1024, 128, 3), (9, 2056, 5120, 40, 9),
        (520, 72, 96, 104, 2), (530, 72, 200, 24, 3), (513, 40, 136, 64, 9), (700, 80, 5120, 16, 20)]


@pytest.mark.parametrize("m,n,k,r,count", LORA)
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_lora(m, n, k, r, count, dt):
    y, x, a, b, scale, ids = lora_inputs(m, n, k, r, count, dt, m + n)
    ad = wql.LoraAdapters(a.to(DEV), b.to(DEV), scale.to(DEV))
    yd = y.to(DEV)
    got = wql.wql_lora_add(yd, x.to(DEV), ad, ids.to(DEV))
    check_lora(got, y, x, a, b, scale, ids, dt)
    assert torch.equal(yd.cpu(), y)                       # y stays
    again = wql.wql_lora_add(yd, x.to(DEV), ad, ids.to(DEV), out=yd)
    assert again is yd and torch.equal(yd, got)           # in place: the same


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_lora_runs_and_leading_shape(dt):
    """Prompts: long runs of one adapter; no scale."""
    m, n, k, r, count = 600, 136, 64, 16, 3
    y, x, a, b, _, _ = lora_inputs(m, n, k, r, count, dt, 3)
    ids = (torch.arange(m) * count // m).to(torch.int32)
    ad = wql.LoraAdapters(a.to(DEV), b.to(DEV))
    got = wql.wql_lora_add(y.view(3, 200, n).to(DEV), x.view(3, 200, k).to(DEV), ad,
                           ids.view(3, 200).to(DEV))
    assert got.shape == (3, 200, n)
    check_lora(got.view(m, n), y, x, a, b, None, ids, dt)


@pytest.mark.parametrize("shift,out_shift", [(1, 1), (4, 4), (7, 7), (0, 3), (5, 2), (2, 1)])
@pytest.mark.parametrize("n", [72, 301, 1, 33, 290])
def test_lora_on_any_boundary(shift, out_shift, n):
    """Rows and tensors that start anywhere, y and out apart: what the same
    columns give in a tensor of whole groups."""
    wide = (n + 7) // 8 * 8
    y, x, a, b, scale, ids = lora_inputs(21, wide, 64, 16, 2, "bf16", shift)
    ad = wql.LoraAdapters(a.to(DEV), b.to(DEV), scale.to(DEV))
    want = wql.wql_lora_add(y.to(DEV), x.to(DEV), ad, ids.to(DEV))[:, :n]
    ad = wql.LoraAdapters(a.to(DEV), b[:, :n].contiguous().to(DEV), scale.to(DEV))
    store = torch.full((21 * n + out_shift + 9,), 7.0, dtype=y.dtype, device=DEV)
    out = store[out_shift:out_shift + 21 * n].view(21, n)
    wql.wql_lora_add(placed(y[:, :n].contiguous(), shift), x.to(DEV), ad, ids.to(DEV), out=out)
    assert torch.equal(out, want)
    assert (store[:out_shift] == 7).all() and (store[out_shift + 21 * n:] == 7).all()


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("size", [2.0 ** -12, 2.0 ** 9])
def test_lora_sizes_of_u(dt, size):
    """u far above what fp16 holds (x 2^9, a of 2^6), and far below."""
    y, x, a, b, scale, ids = lora_inputs(20, 80, 256, 16, 2, dt, 5, size)
    a = (a * (64 if size > 1 else 2.0 ** -4)).to(T[dt])
    b = (b * 2.0 ** -14 if size > 1 else b).to(T[dt])
    ad = wql.LoraAdapters(a.to(DEV), b.to(DEV), scale.to(DEV))
    check_lora(wql.wql_lora_add(y.to(DEV), x.to(DEV), ad, ids.to(DEV)), y, x, a, b, scale, ids, dt)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_lora_bad_rows_stay_alone(bad, dt):
    y, x, a, b, scale, _ = lora_inputs(20, 64, 64, 16, 3, dt, 6)
    ids = (torch.arange(20) % 4 - 1).to(torch.int32)      # 3 adapters and none
    ad = wql.LoraAdapters(a.to(DEV), b.to(DEV), scale.to(DEV))
    clean = wql.wql_lora_add(y.to(DEV), x.to(DEV), ad, ids.to(DEV))
    x[5, 7] = bad                                          # adapter 0
    x[4, 7] = bad                                          # none
    got = wql.wql_lora_add(y.to(DEV), x.to(DEV), ad, ids.to(DEV))
    rows = [i for i in range(20) if i != 5]
    assert torch.equal(got[rows], clean[rows])
    assert not torch.isfinite(got[5]).any()
    # adapters that are not finite concern their own tokens only
    b[1, 3, 2] = bad
    a[2] = bad
    ad = wql.LoraAdapters(a.to(DEV), b.to(DEV), scale.to(DEV))
    got = wql.wql_lora_add(y.to(DEV), x.to(DEV), ad, ids.to(DEV))
    keep = [i for i in range(20) if int(ids[i]) in (-1, 0) and i != 5]
    assert torch.equal(got[keep], clean[keep])
    cols = [c for c in range(64) if c != 3]
    one = [i for i in range(20) if int(ids[i]) == 1]
    assert torch.equal(got[one][:, cols], clean[one][:, cols])
    assert not torch.isfinite(got[one][:, 3]).any()


def test_lora_none_at_all_and_empty():
    y, x, a, b, scale, ids = lora_inputs(6, 40, 64, 8, 2, "bf16", 8)
    ad = wql.LoraAdapters(a.to(DEV), b.to(DEV), scale.to(DEV))
    none = torch.full((6,), -1, dtype=torch.int32, device=DEV)
    assert torch.equal(wql.wql_lora_add(y.to(DEV), x.to(DEV), ad, none).cpu(), y)
    got = wql.wql_lora_add(y[:0].to(DEV), x[:0].to(DEV), ad, none[:0])
    assert got.shape == (0, 40)
    no = wql.LoraAdapters(a[:0].to(DEV), b[:0].to(DEV))
    assert torch.equal(wql.wql_lora_add(y.to(DEV), x.to(DEV), no, ids.to(DEV)).cpu(), y)


def test_lora_offsets_past_32_bits():
    count, n, r = 33, 1 << 20, 128                         # 4.4e9 values of b, 8.9 GB
    g = gen(2)
    b = torch.zeros(count, n, r, dtype=torch.bfloat16, device=DEV)
    last = (0.3 * torch.randn(1000, r, generator=g)).bfloat16()
    b[-1, -1000:] = last.to(DEV)
    a = torch.randn(count, r, 64, generator=g).bfloat16()
    x = torch.randn(2, 64, generator=g).bfloat16()
    y = torch.randn(2, n, generator=g).bfloat16()
    ids = torch.tensor([count - 1, -1], dtype=torch.int32)
    got = wql.wql_lora_add(y.to(DEV), x.to(DEV), wql.LoraAdapters(a.to(DEV), b), ids.to(DEV)).cpu()
    del b
    assert torch.equal(got[:, :-1000], y[:, :-1000]) and torch.equal(got[1], y[1])
    check_lora(got[:, -1000:], y[:, -1000:], x, a[-1:], last[None], None,
               torch.tensor([0, -1], dtype=torch.int32), "bf16")


def test_lora_refusals_of_the_binding():
    y, x, a, b, scale, ids = (t.to(DEV) for t in lora_inputs(6, 40, 64, 8, 2, "bf16", 8))
    ad = wql.LoraAdapters(a, b, scale)
    ok = lambda **kw: wql.wql_lora_add(**{"y": y, "x": x, "adapters": ad, "ids": ids, **kw})  # noqa: E731
    ok()
    bad = [dict(ids=ids.long()), dict(ids=ids[:5]), dict(x=x.half()), dict(x=x[:, :56]), dict(y=y[:5]),
           dict(y=y.float()), dict(y=y.t()), dict(y=y.view(-1)), dict(out=y[:, :39]),
           dict(adapters=wql.LoraAdapters(a, b[:1], scale)),
           dict(adapters=wql.LoraAdapters(a[:, :4], b, scale)),
           dict(adapters=wql.LoraAdapters(a.half(), b.half(), scale)),
           dict(adapters=wql.LoraAdapters(a, b, scale[:1])),
           dict(adapters=wql.LoraAdapters(a, b, scale.half())),
           dict(adapters=wql.LoraAdapters(a, b.transpose(1, 2), scale)),
           dict(workspace=torch.empty(64, device=DEV))]
    for kw in bad:
        with pytest.raises(ValueError):
            ok(**kw)
    with pytest.raises(wql.WQLError, match="EWORKSPACE"):
        ok(workspace=torch.empty(64, dtype=torch.uint8, device=DEV))
    with pytest.raises(wql.WQLError, match="EUNSUPPORTED"):
        ok(adapters=wql.LoraAdapters(a[:, :4].contiguous(), b[:, :, :4].contiguous()))


# ---------------------------------------------------------------------------
# beam_select
# ---------------------------------------------------------------------------
# The error of a score before its rounding.  Of the logarithm of the sum: each
# exponential 2^-22 and its argument (two roundings of d = top - l, and log2 e's
# own, 2^-26) 2^-23 d + 2^-26 d, d's mean under the softmax being at most log n
# < 14; 32 additions in a row and 13 joining them, 2^-24 each; the logarithm's
# mantissa 2^-23.
SCORE = 2.0 ** -22 + 14 * (2.0 ** -23 + 2.0 ** -26) + 45 * 2.0 ** -24 + 2.0 ** -23


def check_select(logits, scores, eos, order, got=None, ties=False):
    """Compares a call with the reference; where two beams' scores are nearer
    than their errors (ties: equal ones aside) the inputs say nothing."""
    batch, beams = scores.shape
    l = f64(logits.view(batch, beams, -1))
    tokens, parents, best, ended, gap = ref.beam_select(l, f64(scores), -1 if eos is None else eos,
                                                        order == wql.BEAM_ANCHORED)
    if gap <= 2 * SCORE:
        return False
    if got is None:
        got = wql.wql_beam_select(logits.to(DEV), scores.to(DEV), eos, order)
    t, p, s, e = got
    assert t.dtype == torch.int32 and p.dtype == torch.int32 and t.shape == (batch, beams)
    np.testing.assert_array_equal(t.cpu().numpy(), tokens)
    np.testing.assert_array_equal(p.cpu().numpy(), parents)

    def near(x, want):
        x, fine = f64(x), np.isfinite(want)
        np.testing.assert_array_equal(np.isfinite(x), fine)
        assert np.all(x[~fine] == -np.inf)
        err = np.abs(x[fine] - want[fine])
        assert np.all(err <= SCORE + 2.0 ** -24 * np.abs(want[fine])), err.max()

    near(s, best)
    assert (e is None) == (eos is None)
    if eos is not None:
        near(e, ended)
    return True


def select_inputs(batch, beams, n, dt, seed, spread=3.0):
    g = gen(seed)
    logits = (spread * torch.randn(batch, beams, n, generator=g)).to(T[dt])
    scores = -torch.rand(batch, beams, generator=g).cumsum(-1) * 2
    return logits, scores


def first_clear(make, eos, order, shift=0):
    """The first seed whose inputs say something (one in a hundred may not)."""
    for seed in range(20):
        logits, scores = make(seed)
        if check_select(logits, scores, eos, order,
                        got=wql.wql_beam_select(placed(logits, shift), scores.to(DEV), eos, order)):
            return
    raise AssertionError("no clear inputs")


SELECT = [(1, 1, 1), (1, 4, 2), (2, 3, 5), (1, 4, 151), (3, 2, 2047), (2, 5, 2049), (2, 4, 8192),
          (1, 16, 8193), (2, 32, 700), (1, 32, 20011), (9, 7, 50303), (1, 4, 151936),
          (80, 4, 9001), (40, 8, 16384)]


@pytest.mark.parametrize("batch,beams,n", SELECT)
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("order", [wql.BEAM_RANKED, wql.BEAM_ANCHORED])
def test_select(batch, beams, n, dt, order):
    for eos in (None, n // 2):
        first_clear(lambda s: select_inputs(batch, beams, n, dt, s), eos, order)


@pytest.mark.parametrize("dt,shifts", [("f32", (1, 2, 3)), ("bf16", (1, 2, 3, 4, 5, 6, 7))])
@pytest.mark.parametrize("n", [4099, 4096, 3])
def test_select_on_any_boundary(dt, shifts, n):
    logits, scores = select_inputs(2, 3, n, dt, 1)
    want = wql.wql_beam_select(logits.to(DEV), scores.to(DEV), 1)
    for shift in shifts:
        got = wql.wql_beam_select(placed(logits, shift), scores.to(DEV), 1)
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_select_largest_vocabulary():
    n = wql.BEAM_MAX_N
    first_clear(lambda s: select_inputs(1, 3, n, "bf16", s), n - 1, wql.BEAM_RANKED)
    first_clear(lambda s: select_inputs(3, 32, n, "f16", s), 0, wql.BEAM_ANCHORED)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("beams", [1, 4, 32])
def test_select_equal_logits(dt, beams):
    """Whole rows equal (the lowest tokens win), and rows of few values."""
    n = 10007
    scores = -torch.arange(beams, dtype=torch.float32)[None] * 3
    logits = torch.full((1, beams, n), 0.5, dtype=T[dt])
    assert check_select(logits, scores, 2, wql.BEAM_RANKED)
    logits = torch.randint(0, 2, (1, beams, n), generator=gen(1)).to(T[dt])
    logits[0, 0] = -0.0
    logits[0, 0, 5000:] = 0.0                     # -0 is 0
    assert check_select(logits, scores, None, wql.BEAM_RANKED)
    # all beams the same: the lower beam first, on rows of every alignment
    logits = (3 * torch.randn(n, generator=gen(2))).to(T[dt]).expand(1, beams, n).contiguous()
    assert check_select(logits, torch.full((1, beams), -1.5), 7, wql.BEAM_RANKED)
    assert check_select(logits, torch.full((1, beams), -1.5), 7, wql.BEAM_ANCHORED)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("order", [wql.BEAM_RANKED, wql.BEAM_ANCHORED])
def test_select_masks(dt, order):
    """Masked by -inf, by the type's lowest value, by NaN; few tokens allowed."""
    batch, beams, n = 4, 4, 20000
    logits, scores = select_inputs(batch, beams, n, dt, 3)
    low = torch.finfo(T[dt]).min
    keep = torch.rand(batch, beams, n, generator=gen(4)) < 0.0002
    logits[0][~keep[0]] = float("-inf")
    logits[1][~keep[1]] = low
    logits[2][~keep[2]] = float("nan")
    logits[3, 1:] = float("-inf")                 # one beam left, with two tokens
    logits[3, 0, 2:] = float("-inf")
    assert check_select(logits, scores, 1, order)
    logits[0] = float("-inf")                     # nothing left at all
    logits[1] = float("nan")
    logits[2, :, :2] = 1.0
    logits[2, :, 2:] = low
    assert check_select(logits, scores, 1, order)


@pytest.mark.parametrize("order", [wql.BEAM_RANKED, wql.BEAM_ANCHORED])
def test_select_infinities_and_scores(order):
    batch, beams, n = 3, 4, 9000
    logits, scores = select_inputs(batch, beams, n, "f32", 5)
    logits[0, 1, [17, 8999]] = float("inf")
    logits[0, 2, 100] = float("nan")
    scores[1] = torch.tensor([0.0, float("-inf"), float("nan"), float("inf")])   # a first step
    logits[2, 3, 4] = float("inf")
    assert check_select(logits, scores, 4, order)
    scores[:] = float("-inf")
    t, p, s, e = wql.wql_beam_select(logits.to(DEV), scores.to(DEV), 4, order)
    assert (t == -1).all() and (p == -1).all() and (s == -float("inf")).all() and torch.equal(s, e)


def test_select_the_end():
    """The end of a beam counts while it is among the best, not by its rank
    among those that go on."""
    n = 3000
    logits = torch.zeros(1, 3, n)
    logits[0, :, 9] = torch.tensor([9.0, 4.0, 8.0])         # eos
    logits[0, 0, :3] = torch.tensor([8.5, 8.25, 1.0])
    logits[0, 1, 3] = 9.5
    scores = torch.tensor([[0.0, -0.3, -0.7]])
    for order in (wql.BEAM_RANKED, wql.BEAM_ANCHORED):
        assert check_select(logits, scores, 9, order)
        t, p, s, e = wql.wql_beam_select(logits.to(DEV), scores.to(DEV), 9, order)
        assert 9 not in t.tolist()[0] and torch.isfinite(e).any()


def test_select_offsets_past_32_bits():
    batch, beams, n = 1030, 4, 1 << 20                      # 4.3e9 logits, 8.6 GB
    logits = torch.zeros(batch, beams, n, dtype=torch.bfloat16, device=DEV)
    tail, scores = select_inputs(1, beams, n, "bf16", 0)
    logits[-1] = tail[0].to(DEV)
    all_scores = scores.expand(batch, beams).contiguous().to(DEV)
    got = wql.wql_beam_select(logits, all_scores, 3)
    one = wql.wql_beam_select(tail.to(DEV), scores.to(DEV), 3)
    for a, b in zip(got, one):
        torch.testing.assert_close(a[-1:], b, rtol=0, atol=2 * SCORE)


def test_select_in_place_scores_and_refusals():
    logits, scores = select_inputs(2, 3, 500, "bf16", 7)
    l, s = logits.to(DEV), scores.to(DEV)
    want = wql.wql_beam_select(l.view(6, 500), s, 3)
    lib, ws = wql.load(), torch.empty(wql.wql_beam_workspace_size(2, 3, 500), dtype=torch.uint8, device=DEV)
    t, p, e = torch.empty_like(want[0]), torch.empty_like(want[0]), torch.empty_like(s)
    assert lib.wql_beam_select(l.data_ptr(), wql.BF16, 2, 3, 500, s.data_ptr(), 3, 0, t.data_ptr(),
                               p.data_ptr(), s.data_ptr(), e.data_ptr(), ws.data_ptr(), ws.numel(),
                               torch.cuda.current_stream().cuda_stream) == 0
    for a, b in zip((t, p, s, e), want):
        assert torch.equal(a, b)
    s = scores.to(DEV)
    for args in ((l, s[:, :2]), (l, s.double()), (l, s.view(-1)), (l, s, 500), (l, s, -1),
                 (l, s, None, 2), (l.transpose(1, 2), s)):
        with pytest.raises(ValueError):
            wql.wql_beam_select(*args)
    with pytest.raises(wql.WQLError, match="EUNSUPPORTED"):
        wql.wql_beam_select(torch.zeros(33, 10, device=DEV), torch.zeros(1, 33, device=DEV))
    empty = wql.wql_beam_select(l[:0], s[:0], 3)
    assert all(v.shape == (0, 3) for v in empty)


# ---------------------------------------------------------------------------
# beam_reorder
# ---------------------------------------------------------------------------
def some_parents(batch, beams, seed):
    p = torch.randint(-1, beams + 1, (batch, beams), generator=gen(seed), dtype=torch.int32)
    p[0] = torch.arange(beams)                            # nothing moves
    if batch > 1:
        p[1] = torch.arange(beams - 1, -1, -1)            # all swap
    return p


def numbers(shape, dtype, seed):
    return torch.randint(0, 200, shape, generator=gen(seed)).to(dtype)


def check_reorder(tensors, parents, lengths, dim):
    """tensors: (storage, view of it that is reordered)."""
    want = []
    for store, view in tensors:
        w = store.cpu().clone()
        v = w.as_strided(view.size(), view.stride(), view.storage_offset())
        v.copy_(torch.from_numpy(ref.reorder(v.double().numpy(), parents.numpy(),
                                             None if lengths is None else lengths.numpy(), dim)))
        want.append(w)
    got = wql.wql_beam_reorder([v for _, v in tensors], parents.to(DEV),
                               None if lengths is None else lengths.to(DEV), dim)
    assert all(a is b for a, (_, b) in zip(got, tensors))
    for (store, _), w in zip(tensors, want):
        assert torch.equal(store.cpu(), w)


@pytest.mark.parametrize("beams", [1, 2, 3, 4, 5, 8, 13, 16, 17, 32])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32, torch.uint8, torch.int64])
def test_reorder(beams, dtype):
    batch, rows = 3, 3 * beams + 2                        # rows behind the last sequence
    st = [numbers(s, dtype, i).to(DEV) for i, s in
          enumerate([(rows, 2, 37, 16), (rows, 1, 1, 3), (rows, 5), (rows,), (rows, 3, 64, 128)])]
    check_reorder([(t, t) for t in st], some_parents(batch, beams, beams), None, None)


LAYOUTS = {                                               # [rows] and where the positions are
    "heads, positions, dim": ((3, 40, 24), 2),
    "positions, heads, dim": ((40, 3, 24), 1),
    "positions": ((40,), 1),
    "positions, odd dim": ((40, 7), 1),
}


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", [torch.float16, torch.int32, torch.uint8])
@pytest.mark.parametrize("beams", [4, 11])
def test_reorder_lengths(layout, dtype, beams):
    shape, dim = LAYOUTS[layout]
    lengths = torch.tensor([40, 0, 1, 17, 39, -5, 1000], dtype=torch.int32)
    batch = len(lengths)
    parents = torch.stack([torch.randperm(beams, generator=gen(i)) for i in range(batch)]).int()
    parents[3, 1:] = 0
    st = [numbers((batch * beams, *shape), dtype, i).to(DEV) for i in range(3)]
    check_reorder([(t, t) for t in st], parents, lengths, dim)


def test_reorder_views():
    """Slices, keys and values in one tensor, rows inside positions, odd starts."""
    batch, beams, h, l, d = 2, 4, 3, 20, 24
    rows = batch * beams
    parents = torch.tensor([[1, 1, 3, 0], [2, 0, 2, 2]], dtype=torch.int32)
    lengths = torch.tensor([13, 20], dtype=torch.int32)
    n = lambda *s, dt=torch.bfloat16: numbers(s, dt, len(s)).to(DEV)  # noqa: E731
    a = n(rows, h, 64, d)
    kv = n(rows, 2, h, l, d)
    inner = n(rows, h, l, 2 * d)
    heads = n(rows, l, h, d)
    turned = n(l, rows, h * d)
    extra = n(rows + 3, h, l, d)
    odd = n(rows * l * 5 + 1, dt=torch.uint8)
    check_reorder([(a, a[:, :, :l])], parents, lengths, 2)
    w = kv.cpu().clone()
    wql.wql_beam_reorder([kv[:, 0], kv[:, 1]], parents.to(DEV), lengths.to(DEV), 2)
    for i in (0, 1):
        w[:, i] = torch.from_numpy(ref.reorder(w[:, i].double().numpy(), parents.numpy(), lengths.numpy(), 2))
    assert torch.equal(kv.cpu(), w)
    check_reorder([(inner, inner[..., d:])], parents, lengths, 2)
    check_reorder([(heads, heads[:, :, 1])], parents, lengths, 1)
    check_reorder([(heads, heads[:, 3:, 1:])], parents, lengths, 1)
    check_reorder([(turned, turned.transpose(0, 1))], parents, lengths, 1)
    check_reorder([(extra, extra[3:])], parents, lengths, 2)
    v = odd[1:].view(rows, l, 5)
    check_reorder([(odd, v)], parents, lengths, 1)
    check_reorder([(inner, inner[:, :, ::2, :d])], parents, None, None)


def test_reorder_many_states_of_every_kind():
    batch, beams = 2, 3
    parents = torch.tensor([[2, 2, 0], [1, 2, 0]], dtype=torch.int32)
    st = []
    for i in range(150):
        dt = (torch.bfloat16, torch.int32, torch.uint8)[i % 3]
        st.append(numbers((batch * beams, 1 + i % 7, 3), dt, i).to(DEV))
    check_reorder([(t, t) for t in st], parents, None, None)


@pytest.mark.parametrize("beams", [2, 4, 7, 16])
@pytest.mark.parametrize("some", [False, True])
def test_reorder_many_columns(beams, some):
    """Enough to move for a thread to take many pieces of a row: whole ones, ends of
    rows and of positions, lengths."""
    batch, l = 64, 40
    rows = batch * beams
    g = gen(beams)
    parents = torch.randint(-1, beams + 1, (batch, beams), generator=g, dtype=torch.int32)
    parents[0] = torch.arange(beams)
    lengths = torch.randint(-1, l + 2, (batch,), generator=g, dtype=torch.int32) if some else None
    big = numbers((rows, 2, l, 264), torch.bfloat16, 1).to(DEV)
    st = [(big, big)]
    for i in range(13):
        gaps = numbers((rows, 3, l, 24), torch.bfloat16, i).to(DEV)
        thin = numbers((rows, 1, l, 6), torch.uint8, i).to(DEV)
        ends = numbers((rows, 2, l + 8, 5), torch.float16, i).to(DEV)
        st += [(gaps, gaps[..., :12]), (thin, thin), (ends, ends[:, :, :l])]
    check_reorder(st, parents, lengths, 2)


def test_reorder_offsets_past_32_bits():
    rows, row = 4, (1 << 31) + 64                         # 8.6 GB
    s = torch.zeros(rows, row, dtype=torch.uint8, device=DEV)
    s[:, -32:] = torch.arange(rows, dtype=torch.uint8, device=DEV)[:, None]
    s[:, :32] = s[:, -32:] + 10
    wql.wql_beam_reorder([s], torch.tensor([[3, 1, 0, 1]], dtype=torch.int32, device=DEV))
    assert s[:, -1].tolist() == [3, 1, 0, 1] and s[:, 31].tolist() == [13, 11, 10, 11]
    assert s[:, row // 2].tolist() == [0] * 4


def test_reorder_refusals():
    p = torch.zeros(2, 3, dtype=torch.int32, device=DEV)
    s = torch.zeros(6, 4, 10, 8, device=DEV)
    for args in (([s], p.long()), ([s], p.view(-1)), ([s[:5]], p), ([s.cpu()], p), ([s], p.cpu()),
                 ([s], p, torch.zeros(2, dtype=torch.int32, device=DEV)),       # no position_dim
                 ([s], p, torch.zeros(3, dtype=torch.int32, device=DEV), 2),
                 ([s], p, None, 0), ([s], p, None, 4), ([s], p, None, -1),
                 ([s[..., ::2]], p, None, 2), ([s[:, ::3, :, :4].transpose(1, 3)], p, None, 3)):
        with pytest.raises(ValueError):
            wql.wql_beam_reorder(*args)
    for st in ([s, s], [s, s[:, 1:]], [s[:1].expand(6, 4, 10, 8)]):
        with pytest.raises(wql.WQLError, match="EINVAL"):
            wql.wql_beam_reorder(st, p)
    assert not s.any()
    wql.wql_beam_reorder([s[:, :0]], p)
    wql.wql_beam_reorder([s], p[:0])


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
def search(batch, beams, n, k, steps, graph, order, seed=0):
    """Beam search with an adapter per sequence over a random recurrent state."""
    g = gen(seed)
    rows = batch * beams
    w = 0.3 * torch.randn(n, k, generator=g)
    qw = wql.wql_quantize(w.to(DEV), 4, 64)
    mix = (torch.randn(k, k, generator=g) / k ** 0.5).half().to(DEV)
    ad = wql.LoraAdapters((torch.randn(2, 8, k, generator=g) / k ** 0.5).half().to(DEV),
                          (0.5 * torch.randn(2, n, 8, generator=g)).half().to(DEV))
    ids = (torch.arange(rows) // beams % 3 - 1).int().to(DEV)
    hidden = torch.zeros(rows, k, dtype=torch.float16, device=DEV)
    history = torch.zeros(rows, steps, dtype=torch.int32, device=DEV)
    cache = torch.zeros(rows, 2, steps, 16, dtype=torch.float16, device=DEV)
    scores = torch.full((batch, beams), float("-inf"), device=DEV)
    tokens = torch.zeros(batch, beams, dtype=torch.int32, device=DEV)
    length = torch.zeros(batch, dtype=torch.int32, device=DEV)
    at = torch.arange(steps, device=DEV)
    workspace = wql.Workspace(DEV)

    def reset():
        hidden.zero_(), history.zero_(), cache.zero_(), tokens.zero_(), length.zero_()
        scores.fill_(float("-inf"))
        scores[:, 0] = 0

    def step():
        x = wql.wql_embed_gather(tokens.view(-1), qw, torch.float16)
        hidden.copy_(torch.tanh((hidden + x) @ mix))
        here = (at == length[0])
        cache.copy_(torch.where(here[:, None], hidden.view(rows, 1, 1, k)[..., :16], cache))
        logits, _, _ = wql.wql_logits(hidden, qw, workspace=workspace)
        wql.wql_lora_add(logits, hidden, ad, ids, out=logits)
        t, parents, s, ended = wql.wql_beam_select(logits, scores, 3, order)
        wql.wql_beam_reorder([hidden, history], parents)
        wql.wql_beam_reorder([cache], parents, length + 1, 2)
        history.copy_(torch.where(here, t.view(rows, 1), history))
        tokens.copy_(t), scores.copy_(s), length.add_(1)
        return logits, parents, ended

    reset()
    if graph:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            out = step()
        reset()
    log = []
    for _ in range(steps):
        before = scores.clone()
        if graph:
            captured.replay()
        else:
            out = step()
        log.append([t.clone().cpu() for t in (before, *out, tokens, scores, history, hidden, cache)])
    return log


@pytest.mark.parametrize("order", [wql.BEAM_RANKED, wql.BEAM_ANCHORED])
def test_beam_search_steps(order):
    """Every step's selection against the reference on the logits it had, the
    histories against what was selected, and a graph against eager calls."""
    batch, beams, n, k, steps = 3, 4, 1000, 128, 6
    log = search(batch, beams, n, k, steps, False, order)
    hist = torch.zeros(batch * beams, steps, dtype=torch.int32)
    for i, (before, logits, parents, ended, tokens, scores, history, hidden, cache) in enumerate(log):
        check_select(logits.view(batch, beams, n), before, 3, order, (tokens, parents, scores, ended))
        hist = torch.from_numpy(ref.reorder(hist.numpy(), parents.numpy(), None, 1))
        hist[:, i] = tokens.view(-1)
        assert torch.equal(history, hist)
        assert torch.equal(cache[:, 0, i], hidden[:, :16])         # moved along
    assert torch.isfinite(log[-1][5]).all()
    for a, b in zip(log, search(batch, beams, n, k, steps, True, order)):
        for x, y in zip(a, b):
            assert torch.equal(x, y)


def test_streams_do_not_disturb_one_another():
    """The same calls on two streams at once give what they give alone."""
    l = [select_inputs(4, 4, 30000, "bf16", i) for i in (1, 2)]
    lo = [lora_inputs(64, 2048, 256, 16, 4, "bf16", i) for i in (3, 4)]
    dev = [[t.to(DEV) for t in v] for v in (*l, *lo)]
    ad = [wql.LoraAdapters(*dev[i][2:5]) for i in (2, 3)]

    def call(i):
        y, x, ids = dev[2 + i][0], dev[2 + i][1], dev[2 + i][5]
        return [*wql.wql_beam_select(dev[i][0], dev[i][1], 5), wql.wql_lora_add(y, x, ad[i], ids)]

    want = [call(0), call(1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(call(i))
    torch.cuda.synchronize()
    for i in (0, 1):
        for g in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(g, want[i]))


def test_graphs_follow_their_inputs():
    """Two captured graphs, replayed on two streams at once, with other ids, logits and
    parents than those of the capture."""
    def inputs(seed):
        y, x, a, b, scale, ids = lora_inputs(70, 1003, 256, 24, 5, "f16", seed)
        logits, scores = select_inputs(5, 4, 30001, "f16", seed)
        cache = numbers((20, 3, 50, 16), torch.float16, seed)
        return [t.to(DEV) for t in (y, x, ids, logits, scores, cache)], [t.to(DEV) for t in (a, b, scale)]

    def call(ad, y, x, ids, logits, scores, cache):
        lo = wql.wql_lora_add(y, x, ad, ids)
        t, parents, s, ended = wql.wql_beam_select(logits, scores, 7, wql.BEAM_ANCHORED)
        wql.wql_beam_reorder([cache], parents)
        return lo, t, parents, s, ended, cache

    made = []
    for i in (0, 1):
        now, ad = inputs(i)
        made.append([now, wql.LoraAdapters(*ad)])
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            call(made[i][1], *now)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = call(made[i][1], *now)
        made[i] += [graph, out, side]
    for seed in (2, 4, 6):
        want, new = [], []
        for i, (now, ad, graph, out, side) in enumerate(made):
            new.append(inputs(seed + i)[0])
            want.append([t.clone() for t in call(ad, *[t.clone() for t in new[i]])])
        torch.cuda.synchronize()
        for i, (now, ad, graph, out, side) in enumerate(made):
            with torch.cuda.stream(side):
                for a, b in zip(now, new[i]):
                    a.copy_(b)
                graph.replay()
        torch.cuda.synchronize()
        for i in (0, 1):
            assert all(torch.equal(a, b) for a, b in zip(made[i][3], want[i])), (seed, i)


def test_lora_out_apart():
    """An output that overlaps y without being y is refused."""
    y, x, a, b, scale, ids = (t.to(DEV) for t in lora_inputs(6, 40, 64, 8, 2, "bf16", 8))
    ad = wql.LoraAdapters(a, b, scale)
    store = torch.zeros(7, 40, dtype=y.dtype, device=DEV)
    with pytest.raises(wql.WQLError, match="EINVAL"):
        wql.wql_lora_add(store[:6], x, ad, ids, out=store[1:])
    assert not store.any()


def test_example_runs():
    """examples/beam_step.py, eagerly and as a graph."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "beam_step.py")
    spec = importlib.util.spec_from_file_location("beam_step", path)
    mod = importlib.util.module_from_spec(spec)
    import sys
    sys.modules["beam_step"] = mod                 # dataclasses look it up
    spec.loader.exec_module(mod)
    eager = mod.search(3, 4, 2000, 128, 5, graph=False)
    graph = mod.search(3, 4, 2000, 128, 5, graph=True)
    assert all(torch.equal(x, y) for x, y in zip(eager, graph))
    assert torch.isfinite(eager[1]).all() and eager[0].shape == (3, 4, 5)
    assert (eager[0] != mod.EOS).all()
