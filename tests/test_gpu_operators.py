"""The operators around the head on the GPU against 64-bit references
(ref64.py): add_rmsnorm, microscaled codes, their product, sampling."""
import numpy as np
import pytest
import torch

import ref64
import weight_only_quantized_wql_gb300 as wql
from ref64 import f64

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
T = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ULP = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}            # half an ulp, relative (11 and 8 bits)
TINY = {"f16": 2.0 ** -25, "bf16": 1e-38}               # half the smallest subnormal
LOG2E = float(np.float32(1.44269504088896340736))       # as a temperature: c = 1


def gen(seed):
    return torch.Generator().manual_seed(seed)


# ---------------------------------------------------------------------------
# add_rmsnorm
# ---------------------------------------------------------------------------
def norm_inputs(m, k, dt, seed):
    g = gen(seed)
    x = torch.randn(m, k, generator=g).to(T[dt])
    r = (4 * torch.randn(m, k, generator=g)).to(T[dt])
    w = (1 + 0.3 * torch.randn(k, generator=g)).to(T[dt])
    return x, r, w


# fp32 steps of y: the sum of k squares (pairwise over threads, at most 64 in a
# row), mean, rsqrt (2 ulp), two products
def rel32(k):
    return 96 * 2.0 ** -24


@pytest.mark.parametrize("m,k", [(1, 1), (3, 7), (2, 33), (5, 1024), (130, 1000), (1, 5120),
                                 (2, 4099), (1, 8193), (2, 65535), (1, 65536)])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("residual", [True, False])
def test_norm_same(m, k, dt, residual):
    x, r, w = norm_inputs(m, k, dt, m * 7 + k)
    eps = 1e-5
    y, ro, sc = wql.wql_add_rmsnorm(x.to(DEV), w.to(DEV), r.to(DEV) if residual else None, eps)
    h, want = ref64.rmsnorm(f64(x), f64(r) if residual else None, f64(w), eps)
    assert sc is None and (ro is None) == (not residual)
    err = np.abs(f64(y) - want)
    assert np.all(err <= (ULP[dt] * 1.001 + rel32(k)) * np.abs(want) + TINY[dt])
    if residual:
        # fp32 holds x + r of 16-bit inputs to 2^-24, then one rounding
        assert np.all(np.abs(f64(ro) - h) <= (ULP[dt] + 2.0 ** -23) * np.abs(h) + TINY[dt])


@pytest.mark.parametrize("m,k", [(1, 5), (3, 64), (131, 1000), (7, 4099), (2, 5120)])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_norm_e4m3(m, k, dt):
    x, r, w = norm_inputs(m, k, dt, k)
    x[0] = 0                                         # with r: a row like any other
    r[0] = 0                                         # a row of zeros
    y, ro, sc = wql.wql_add_rmsnorm(x.to(DEV), w.to(DEV), r.to(DEV), 1e-6, wql.NORM_E4M3)
    assert y.dtype == torch.float8_e4m3fn and y.shape == x.shape and sc.shape == (m,)
    _, want = ref64.rmsnorm(f64(x), f64(r), f64(w), 1e-6)
    s = np.maximum(np.abs(want).max(-1) / 448, 1e-8)
    assert np.all(np.abs(f64(sc) - s) <= (rel32(k) + 2.0 ** -22) * s)
    v = want / s[:, None]
    # half a step of e4m3 (3 bits of fraction, subnormals of 2^-9), and the fp32 steps
    tol = np.maximum(2.0 ** -4 * np.abs(v), 2.0 ** -10) + (rel32(k) + 2.0 ** -21) * np.abs(v) * 2
    assert np.all(np.abs(f64(y.float()) - v) <= tol)


@pytest.mark.parametrize("fmt", [wql.NORM_MX_FP8, wql.NORM_MX_FP4])
@pytest.mark.parametrize("m,k", [(1, 32), (3, 96), (128, 160), (129, 1024), (2, 5120),
                                 (1, 16416), (1, 65536)])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_norm_mx(fmt, m, k, dt):
    x, r, w = norm_inputs(m, k, dt, k + 1)
    y, ro, sc = wql.wql_add_rmsnorm(x.to(DEV), w.to(DEV), r.to(DEV), 1e-6, fmt)
    f = y.fmt
    assert sc is None and f == (wql.MX_FP8 if fmt == wql.NORM_MX_FP8 else wql.MX_FP4)
    tiles = y.scales.cpu().numpy()
    byte = ref64.untile(tiles, m, k // 32)
    np.testing.assert_array_equal(tiles, ref64.tile(byte))          # zeros elsewhere
    _, want = ref64.rmsnorm(f64(x), f64(r), f64(w), 1e-6)
    b = np.abs(want).reshape(m, k // 32, 32).max(-1)
    lo = np.frexp(b * (1 - rel32(k)))[1] - 1 - ref64.EMAX[f] + 127
    hi = np.frexp(b * (1 + rel32(k)))[1] - 1 - ref64.EMAX[f] + 127
    assert np.all((byte == lo) | (byte == hi))
    s = np.repeat(2.0 ** (byte.astype(float) - 127), 32, axis=1)
    v = np.abs(want) / s
    got = ref64.mx_values(y.codes.cpu().numpy(), byte, f) / s
    top = ref64.grid(f)[-1]
    step = 2.0 ** (np.floor(np.log2(np.maximum(v, 2.0 ** (0 if f == 0 else -6)))) -
                   (1 if f == 0 else 3))
    clipped = np.minimum(v, top)
    assert np.all(np.abs(np.abs(got) - clipped) <= step / 2 + rel32(k) * v)
    assert np.all((got == 0) | (np.sign(got) == np.sign(want)))


@pytest.mark.parametrize("fmt", [wql.NORM_SAME, wql.NORM_E4M3])
@pytest.mark.parametrize("shift", [1, 3, 8])
def test_norm_any_alignment(fmt, shift):
    """Tensors that start anywhere give what aligned ones give, and rows that
    share 16 bytes leave each other alone."""
    m, k = 5, 1003
    x, r, w = norm_inputs(m, k, "bf16", 9)
    want = wql.wql_add_rmsnorm(x.to(DEV), w.to(DEV), r.to(DEV), fmt=fmt)
    off = [torch.empty(t.numel() + shift, dtype=t.dtype, device=DEV)[shift:].view(t.shape)
           for t in (x, r, w)]
    for o, t in zip(off, (x, r, w)):
        o.copy_(t)
    got = wql.wql_add_rmsnorm(off[0], off[2], off[1], fmt=fmt)
    for a, b in zip(want, got):
        if a is not None and fmt == wql.NORM_SAME:
            # the order of the sum differs: one ulp of the output at most
            assert np.all(np.abs(f64(a) - f64(b)) <= 2.0 ** -7 * np.abs(f64(a)))
        elif a is not None:
            assert np.all(np.abs(f64(a.float()) - f64(b.float())) <= 2.0 ** -3 * np.abs(f64(a.float())) + 2.0 ** -9)


def test_norm_in_place_and_leading_shape():
    x, r, w = norm_inputs(6, 512, "bf16", 1)
    xd, rd, wd = x.view(2, 3, 512).to(DEV), r.view(2, 3, 512).to(DEV), w.to(DEV)
    y0, r0, _ = wql.wql_add_rmsnorm(xd, wd, rd)
    y1, r1, _ = wql.wql_add_rmsnorm(xd, wd, rd, residual_out=rd)
    assert r1 is rd and y0.shape == xd.shape
    assert torch.equal(y0, y1) and torch.equal(r0, rd)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_norm_bad_rows_stay_alone(bad):
    x, r, w = norm_inputs(4, 256, "f16", 2)
    clean, _, cs = wql.wql_add_rmsnorm(x.to(DEV), w.to(DEV), r.to(DEV), fmt=wql.NORM_E4M3)
    x[1, 77] = bad
    y, _, sc = wql.wql_add_rmsnorm(x.to(DEV), w.to(DEV), r.to(DEV), fmt=wql.NORM_E4M3)
    assert torch.isnan(sc[1]) and torch.isfinite(sc[[0, 2, 3]]).all()
    for i in (0, 2, 3):
        assert torch.equal(y[i].view(torch.uint8), clean[i].view(torch.uint8)) and sc[i] == cs[i]
    m, _, _ = wql.wql_add_rmsnorm(x.to(DEV), w.to(DEV), r.to(DEV), fmt=wql.NORM_MX_FP4)
    v = wql.wql_mx_dequantize(m)
    assert torch.isnan(v[1, 64:96]).all() and torch.isfinite(v[[0, 2, 3]]).all()


# ---------------------------------------------------------------------------
# microscaled codes
# ---------------------------------------------------------------------------
def mx_input(rows, k, dt, seed):
    g = gen(seed)
    x = torch.randn(rows, k, generator=g) * torch.exp2(torch.randint(-20, 15, (rows, 1),
                                                                     generator=g).float())
    # ties and exact powers of two: a coarse grid
    x = torch.where(torch.rand(rows, k, generator=g) < 0.3, torch.round(x * 4) / 4, x)
    return x.to(T[dt])


def plain_nans(codes, byte, fmt):
    """NaN codes (of a block with a NaN scale, e4m3) may have any sign."""
    if fmt == wql.MX_FP8:
        return np.where(np.repeat(byte == 255, 32, axis=1), codes & 127, codes)
    return codes


@pytest.mark.parametrize("fmt", [wql.MX_FP4, wql.MX_FP8])
@pytest.mark.parametrize("rows,k", [(1, 32), (3, 64), (2, 160), (128, 128), (129, 96), (300, 1056)])
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_mx_bit_exact(fmt, rows, k, dt):
    x = mx_input(rows, k, dt, rows + k)
    a = wql.wql_mx_quantize(x.to(DEV), fmt)
    codes, byte = ref64.mx_quantize(f64(x), fmt)
    np.testing.assert_array_equal(a.scales.cpu().numpy(), ref64.tile(byte))
    np.testing.assert_array_equal(plain_nans(a.codes.cpu().numpy(), byte, fmt), codes)
    want = ref64.mx_values(codes, byte, fmt)
    np.testing.assert_array_equal(f64(wql.wql_mx_dequantize(a, torch.float32)), want)
    for out in ("f16", "bf16"):
        got = wql.wql_mx_dequantize(a, T[out]).cpu()
        np.testing.assert_array_equal(f64(got), f64(torch.from_numpy(want).float().to(T[out])))


@pytest.mark.parametrize("fmt", [wql.MX_FP4, wql.MX_FP8])
def test_mx_edge_blocks(fmt):
    top = float(torch.finfo(torch.float32).max)
    x = torch.zeros(8, 32)
    x[1, 3] = 2.0 ** -149                            # subnormals: scale 2^-127
    x[2, 0], x[2, 1] = 2.0 ** -126, -(2.0 ** -127)
    x[3, 5], x[3, 6] = top, -top
    x[4, 0] = -0.0
    x[5, 31] = float("nan")
    x[6, 8], x[6, 9] = float("-inf"), 1.0
    x[7] = torch.linspace(-7.99, 7.99, 32)           # past the largest element: saturates
    a = wql.wql_mx_quantize(x.to(DEV), fmt)
    codes, byte = ref64.mx_quantize(f64(x), fmt)
    assert list(byte[:, 0])[5:7] == [255, 255]
    np.testing.assert_array_equal(a.scales.cpu().numpy(), ref64.tile(byte))
    np.testing.assert_array_equal(plain_nans(a.codes.cpu().numpy(), byte, fmt), codes)
    assert torch.isnan(wql.wql_mx_dequantize(a)[5:7]).all()


def test_mx_empty():
    a = wql.wql_mx_quantize(torch.empty(0, 64, dtype=torch.float16, device=DEV))
    assert a.rows == 0 and wql.wql_mx_dequantize(a).shape == (0, 64)
    w = wql.wql_mx_quantize(torch.ones(5, 64, dtype=torch.float16, device=DEV))
    assert wql.wql_mx_logits(a, w).shape == (0, 5)


# ---------------------------------------------------------------------------
# the product
# ---------------------------------------------------------------------------
def mx_operands(m, n, k, fmt, seed):
    g = gen(seed)
    x = torch.randn(m, k, generator=g) * (1 + 15 * (torch.rand(k, generator=g) < 0.02))
    w = 0.02 * torch.randn(n, k, generator=g)
    xa = wql.wql_mx_quantize(x.to(DEV), fmt)
    wa = wql.wql_mx_quantize(w.to(DEV), wql.MX_FP4)
    xv = ref64.mx_values(*ref64.mx_quantize(f64(x), fmt), fmt)
    wv = ref64.mx_values(*ref64.mx_quantize(f64(w), 0), 0)
    return xa, wa, xv, wv


def check_logits(got, xv, wv, dt, bias=0.0):
    want = xv @ wv.T + bias
    absacc = np.abs(xv) @ np.abs(wv).T
    k = xv.shape[1]
    # exact products, fp32 sums (the bound the tensor-core tests use), one rounding
    tol = k * 2.0 ** -22 * (absacc + np.abs(bias)) + ULP[dt] * 1.001 * np.abs(want) + TINY[dt]
    err = np.abs(f64(got) - want)
    assert np.all(err <= tol), f"worst {np.max(err / tol):.2f} of the tolerance"


@pytest.mark.parametrize("fmt", [wql.MX_FP8, wql.MX_FP4])
@pytest.mark.parametrize("m,n,k", [
    (1, 1, 32), (1, 127, 64), (2, 128, 96), (3, 129, 128), (1, 4099, 160), (8, 1000, 1024),
    (16, 300, 224), (17, 513, 256), (33, 1000, 512), (64, 777, 2080), (100, 260, 1056),
    (128, 999, 512), (129, 1000, 512), (200, 300, 288), (256, 640, 1024), (257, 500, 320),
    (300, 131, 5120), (700, 400, 64), (5, 20001, 5120)])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_mx_logits(fmt, m, n, k, dt):
    xa, wa, xv, wv = mx_operands(m, n, k, fmt, m + n + k)
    ws = wql.Workspace(DEV)
    got = wql.wql_mx_logits(xa, wa, T[dt], workspace=ws)
    torch.cuda.synchronize()
    assert ws.error_word() == 0
    check_logits(got, xv, wv, dt)
    assert torch.equal(got, wql.wql_mx_logits(xa, wa, T[dt]))      # no order changes the sums


def test_mx_logits_bias_and_out():
    xa, wa, xv, wv = mx_operands(5, 1001, 256, wql.MX_FP8, 3)
    b = torch.randn(1001, generator=gen(4)).to(torch.bfloat16)
    out = torch.full((5, 1001), float("nan"), dtype=torch.bfloat16, device=DEV)
    r = wql.wql_mx_logits(xa, wa, torch.bfloat16, bias=b.to(DEV), out=out)
    assert r is out
    check_logits(out, xv, wv, "bf16", f64(b))
    with pytest.raises(ValueError):
        wql.wql_mx_logits(xa, wa, torch.bfloat16, bias=b.half().to(DEV))
    with pytest.raises(ValueError):
        wql.wql_mx_logits(xa, wa, torch.bfloat16, out=out[:4])


@pytest.mark.parametrize("fmt", [wql.MX_FP8, wql.MX_FP4])
def test_mx_logits_nan_scales(fmt):
    """A NaN block makes its token's or its vocab row's logits NaN, no others."""
    x = torch.randn(4, 128, generator=gen(5))
    w = torch.randn(200, 128, generator=gen(6))
    x[2, 40] = float("inf")
    w[150, 3] = float("nan")
    got = wql.wql_mx_logits(wql.wql_mx_quantize(x.to(DEV), fmt),
                            wql.wql_mx_quantize(w.to(DEV)), torch.float16)
    want = torch.zeros(4, 200, dtype=torch.bool)
    want[2] = True
    want[:, 150] = True
    assert torch.equal(torch.isnan(got).cpu(), want)


def test_mx_logits_extreme_scales():
    """Scales far from 1 on both sides, products within fp32."""
    g = gen(8)
    x = torch.randn(3, 64, generator=g) * 2.0 ** 60
    w = torch.randn(130, 64, generator=g) * 2.0 ** -60
    xa, wa = wql.wql_mx_quantize(x.to(DEV), wql.MX_FP8), wql.wql_mx_quantize(w.to(DEV))
    xv = ref64.mx_values(*ref64.mx_quantize(f64(x), 1), 1)
    wv = ref64.mx_values(*ref64.mx_quantize(f64(w), 0), 0)
    check_logits(wql.wql_mx_logits(xa, wa, torch.bfloat16), xv, wv, "bf16")


@pytest.mark.parametrize("fmt,k", [(wql.MX_FP8, 512), (wql.MX_FP8, 544), (wql.MX_FP4, 512)])
def test_mx_logits_wait_timeout_is_reported_and_recovers(fmt, k):
    """A stalled issuing warp: every role's bounded wait runs out, the call
    returns, the error word says so, and the next call is right."""
    xa, wa, xv, wv = mx_operands(20, 3000, k, fmt, 1)
    ws = wql.Workspace(DEV)
    try:
        wql.wql_debug_set_waits(2_000_000, True)          # SM cycles, about 1 ms
        wql.wql_mx_logits(xa, wa, torch.float16, workspace=ws)
        torch.cuda.synchronize()
    finally:
        wql.wql_debug_set_waits(0, False)
    assert ws.error_word() == 8
    ws.clear_error()
    got = wql.wql_mx_logits(xa, wa, torch.float16, workspace=ws)
    assert ws.error_word() == 0
    check_logits(got, xv, wv, "f16")


# ---------------------------------------------------------------------------
# sampling
# ---------------------------------------------------------------------------
def par(v, m, dtype=torch.float32):
    if v is None:
        return None
    t = torch.as_tensor(v, dtype=dtype)
    return (t.expand(m) if t.dim() == 0 else t).contiguous().to(DEV)


def run_sample(l, u, t=1.0, k=None, p=None, mp=None):
    m = l.shape[0]
    return wql.wql_sample(l.to(DEV), par(u, m), par(t, m), par(k, m, torch.int32), par(p, m),
                          par(mp, m))


# whole logits and c = 1: every weight is a power of two, every sum exact
EXACT = [  # n, top_k, top_p, min_p, spread of the logits
    (1, 0, 1.0, 0.0, 3), (2, 1, 1.0, 0.0, 3), (7, 3, 0.7, 0.0, 4), (64, 0, 0.9, 0.0, 10),
    (1000, 50, 1.0, 0.0, 12), (1000, 0, 0.5, 0.0, 12), (1000, 0, 1.0, 0.25, 12),
    (1000, 20, 0.8, 0.1, 12), (1001, 0, 1.0, 0.0, 20), (3000, 900, 1.0, 0.0, 6),
    (5003, 0, 0.9, 0.0, 2), (5003, 2500, 0.6, 0.0, 3), (20011, 40, 0.95, 0.0, 30),
    (20011, 0, 0.9, 0.0, 3), (40001, 3000, 0.999, 0.0, 5), (40001, 10, 1.0, 0.0, 1),
    (40001, 0, 1e-9, 0.0, 8), (40001, 39999, 1.0, 0.0, 4), (40001, 0, 0.97, 2.0, 30),
    # more equal logits than the lists hold: the descent over the rank key
    (40001, 0, 0.6, 0.0, 1), (100003, 0, 0.97, 0.0, 2), (100003, 30000, 0.5, 0.0, 1),
]


@pytest.mark.parametrize("n,top_k,top_p,min_p,spread", EXACT)
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_sample_exact(n, top_k, top_p, min_p, spread, dt):
    """Many equal logits, cuts inside ties, one to eight blocks per row."""
    m = 5
    l = torch.randint(-spread, spread + 1, (m, n), generator=gen(n + top_k)).float()
    u = torch.tensor([0.0, 0.25, 0.5, 0.731, 1.0 - 2.0 ** -24])
    ids, logp = run_sample(l.to(T[dt]), u, LOG2E, top_k, top_p, min_p)
    for i in range(m):
        want, w, total = ref64.sample_exact(l[i].tolist(), LOG2E, top_k, top_p, min_p,
                                            float(u[i]))
        assert int(ids[i]) == want
        # two roundings to fp32, a division and logf (2 ulp of the result)
        lp = np.log(w / total)
        assert abs(float(logp[i]) - lp) <= 4 * 2.0 ** -24 + 2.0 ** -22 * abs(lp)


def test_sample_exact_many_rows():
    """One block per row: as many rows as fill the GPU."""
    m, n = 400, 3001
    l = torch.randint(-6, 7, (m, n), generator=gen(1)).float()
    u = torch.rand(m, generator=gen(2))
    k = torch.randint(0, 3100, (m,), generator=gen(3))
    p = torch.where(torch.rand(m, generator=gen(4)) < 0.5, torch.rand(m, generator=gen(5)), 1.0)
    ids, _ = run_sample(l.to(torch.bfloat16), u, LOG2E, k, p)
    for i in range(m):
        want = ref64.sample_exact(l[i].tolist(), LOG2E, int(k[i]), float(p[i]), 0.0, float(u[i]))
        assert int(ids[i]) == want[0], i


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n", [5, 9000, 70001])
def test_sample_masked_rows(dt, n):
    """Rows with nothing left, with one token left, with NaN, with the type's
    lowest value as a mask."""
    ninf, nan = float("-inf"), float("nan")
    low = float(torch.finfo(T[dt]).min)
    l = torch.full((8, n), ninf)
    l[1, n - 2] = -3.0                              # one token
    l[2] = nan                                      # all NaN: nothing left
    l[3], l[3, 3] = low, 1.0                        # masked by the lowest value
    l[4] = low                                      # everything at the lowest value
    l[5], l[5, 1], l[5, 4] = nan, 2.0, 2.0          # NaN counts as -inf
    l[6, 2], l[6, 4] = float("inf"), float("inf")   # the infinite ones share it all
    l[7], l[7, 0] = 0.0, ninf
    u = torch.tensor([0.5, 0.9, 0.5, 0.9, 0.5, 0.9, 0.9, 0.0])
    for k, p, mp in ((None, None, None), (3, None, None), (None, 0.9, None), (None, None, 0.1),
                     (2, 0.999, 0.01)):
        ids, logp = run_sample(l.to(T[dt]), u, 1.0, k, p, mp)
        ids, logp = ids.cpu().tolist(), logp.cpu()
        assert ids[0] == -1 and ids[2] == -1 and torch.isnan(logp[[0, 2]]).all()
        assert ids[1] == n - 2 and logp[1] == 0
        assert ids[3] == 3 and logp[3] == 0
        kept4 = min(n, k or n) if p is None else None
        if p is None:
            assert ids[4] == int(0.5 * kept4)
        assert ids[5] == 4 and ids[6] == 4 and ids[7] == 1
        assert abs(float(logp[5]) - np.log(0.5)) < 1e-6
    ids, logp = run_sample(l.to(T[dt]), u, 0.0)     # greedy
    assert ids.cpu().tolist() == [-1, n - 2, -1, 3, 0, 1, 2, 1]
    assert torch.isnan(logp[[0, 2]]).all() and (logp[[1, 3, 4, 5, 6, 7]] == 0).all()


def test_sample_odd_parameters():
    l = torch.tensor([[1.0, 3.0, 2.0, 3.0]]).expand(9, 4).contiguous()
    nan, inf = float("nan"), float("inf")
    t = torch.tensor([nan, -1.0, 1e-38, 1e30, inf, 1.0, 1.0, 1.0, 1.0])
    u = torch.tensor([0.9, 0.9, 0.9, 0.9, 0.99, 1.0, -1.0, nan, 0.9])
    p = torch.tensor([1.0, 1.0, 1.0, 1.0, 1.0, 1.0, 1.0, 1.0, -0.5])
    k = torch.tensor([0, 0, 0, 0, 0, -3, 99, 4, 0])
    ids, logp = run_sample(l, u, t, k, p)
    # NaN, <= 0: greedy; near 0: the maxima share; near inf: uniform; u >= 1:
    # the last; u <= 0 or NaN: the first; top_p <= 0: the first by rank
    assert ids.cpu().tolist() == [1, 1, 3, 3, 3, 3, 0, 0, 1]
    assert abs(float(logp[3]) - np.log(0.25)) < 1e-6 and logp[8] == 0


@pytest.mark.parametrize("mode", ["plain", "top_k", "top_p", "min_p", "all", "wide", "flat"])
@pytest.mark.parametrize("m,n,dt", [(1, 50304, "bf16"), (3, 30011, "f16"), (40, 8192, "f32"),
                                    (320, 2500, "bf16")])
def test_sample_real_logits(mode, m, n, dt):
    """Logits as they come, against 64 bits: the draw lies where u says."""
    g = gen(m + n)
    spread = 0.5 if mode == "flat" else 3.0
    l = (spread * torch.randn(m, n, generator=g)).to(T[dt])
    u, t = torch.rand(m, generator=g), 0.5 + torch.rand(m, generator=g)
    k = {"top_k": 40, "all": 200, "wide": n // 2}.get(mode)
    p = {"top_p": 0.8, "all": 0.9, "wide": 0.99, "flat": 0.9}.get(mode)
    mp = {"min_p": 0.02, "all": 0.005}.get(mode)
    ids, logp = run_sample(l, u, t, k, p, mp)
    again = run_sample(l, u, t, k, p, mp)
    assert torch.equal(ids, again[0]) and torch.equal(logp, again[1])
    # a weight is off by its exponent's error (|x| <= 31, four roundings), exp2f
    # (2 ulp), and the truncation to 2^-31 of the largest
    rel = 0.7 * 31 * 2.0 ** -22 + 2.0 ** -22
    slack = 2 * (rel + n * 2.0 ** -31)
    lv = f64(l)
    for i in range(0, m, max(1, m // 25)):
        args = (lv[i], float(t[i]), k or 0, float(np.float32(p)) if p else 1.0,
                float(np.float32(mp)) if mp else 0.0)
        e, order, lo = ref64.kept(*args, slack=-slack)
        hi = ref64.kept(*args, slack=slack)[2]
        ok = False
        for keep in {lo, hi, *range(lo, min(hi, lo + 50))}:
            inside = np.zeros(n, bool)
            inside[order[:keep]] = True
            w = np.where(inside, e, 0.0)
            cum = np.cumsum(w) / w.sum()
            j = int(ids[i])
            near = cum[j] - w[j] / w.sum() - slack <= float(u[i]) <= cum[j] + slack
            lp = np.log(w[j] / w.sum()) if inside[j] else -np.inf
            near = near and abs(lp - float(logp[i])) <= 2 * slack + 2.0 ** -30 / e[j] + 1e-6
            ok = ok or bool(near)
        assert ok, f"row {i}: token {int(ids[i])}, kept {lo}..{hi}"


@pytest.mark.parametrize("n", [9, 4096, 40001, 200000])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_sample_any_alignment(n, dt):
    """Logits that start on any element draw what aligned ones do."""
    m = 3
    l = (3 * torch.randn(m, n, generator=gen(n))).to(T[dt]).to(DEV)
    u = torch.rand(m, generator=gen(1))
    for k, p, mp in ((None, None, None), (20, 0.9, None), (None, 0.95, 0.001), (n // 2, 0.99, None)):
        want = run_sample(l, u, 0.9, k, p, mp)
        for shift in (1, 3, 7):
            off = torch.empty(l.numel() + shift, dtype=l.dtype, device=DEV)[shift:].view(m, n)
            off.copy_(l)
            got = run_sample(off, u, 0.9, k, p, mp)
            assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def test_sample_follows_the_distribution():
    """20000 draws of one row: each token's share within 5 standard deviations."""
    m, n = 20000, 12
    l = torch.randn(1, n, generator=gen(9))
    u = torch.rand(m, generator=gen(10))
    ids, _ = run_sample(l.expand(m, n).contiguous(), u, 0.9)
    p = torch.softmax(l[0].double() / 0.9, 0).numpy()
    share = np.bincount(ids.cpu().numpy(), minlength=n) / m
    assert np.all(np.abs(share - p) <= 5 * np.sqrt(p * (1 - p) / m))


def test_sample_refuses_wrong_parameters():
    l, u = torch.zeros(2, 8, device=DEV), torch.zeros(2, device=DEV)
    with pytest.raises(ValueError):
        wql.wql_sample(l, u, top_k=torch.zeros(2, device=DEV))              # not int32
    with pytest.raises(ValueError):
        wql.wql_sample(l, u, top_p=torch.zeros(3, device=DEV))
    with pytest.raises(ValueError):
        wql.wql_sample(l, torch.zeros(2))
    with pytest.raises(ValueError):
        wql.wql_sample(l[:, ::2], u)
    ids, logp = wql.wql_sample(l[:0], u[:0])
    assert ids.shape == (0,) and logp.shape == (0,)


# ---------------------------------------------------------------------------
# together, and on a stream of its own
# ---------------------------------------------------------------------------
def test_step_on_a_side_stream():
    m, n, k = 4, 2000, 256
    g = gen(12)
    x, r, gamma = norm_inputs(m, k, "bf16", 12)
    w = torch.randn(n, k, generator=g) * 0.1
    u = torch.rand(m, generator=g)
    dev = [v.to(DEV) for v in (x, r, gamma, w, u)]
    torch.cuda.synchronize()

    def step():
        wa = wql.wql_mx_quantize(dev[3])
        y, ro, _ = wql.wql_add_rmsnorm(dev[0], dev[2], dev[1], fmt=wql.NORM_MX_FP8)
        logits = wql.wql_mx_logits(y, wa, torch.bfloat16)
        return (ro, logits, *wql.wql_sample(logits, dev[4], top_p=par(0.9, m)))

    want = step()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = step()
    side.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)


def test_example_decodes_the_same_eagerly_and_as_a_graph():
    import importlib.util
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    spec = importlib.util.spec_from_file_location(
        "decode_step", os.path.join(root, "examples", "decode_step.py"))
    ex = importlib.util.module_from_spec(spec)
    import sys
    sys.modules["decode_step"] = ex
    spec.loader.exec_module(ex)
    eager, logp = ex.decode(3, 4099, 256, 5, graph=False)
    graph, logp2 = ex.decode(3, 4099, 256, 5, graph=True)
    assert torch.equal(eager, graph) and torch.equal(logp, logp2)
    assert eager.min() >= 0 and eager.max() < 4099 and (logp <= 0).all()
