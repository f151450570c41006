"""Argument checks of the operators around the head (norm, microscaled codes
and product, sampling) through the C ABI, on the host: a refused call launches
nothing.  And the numpy references' own pins."""
import ctypes

import numpy as np
import pytest
import torch

import ref64
import weight_only_quantized_wql_gb300 as wql

OK, EINVAL, EUNSUPPORTED, ECUDA, EWORKSPACE = 0, 1, 2, 3, 4
A = 0x7F0000100000  # an aligned fake device address: never dereferenced by the checks
F32, F16, BF16 = 0, 1, 2


@pytest.fixture(autouse=True)
def nothing_launched():
    before = wql.wql_launch_count()
    yield
    assert wql.wql_launch_count() == before


@pytest.fixture(scope="module")
def lib():
    return wql.load()


def mx(fmt=0, rows=100, k=256, codes=A, scales=A, reserved=0):
    return wql._WqlMx(fmt, reserved, rows, k, codes, scales)


def test_scale_bytes():
    assert wql.wql_mx_scale_bytes(1, 32) == 512
    assert wql.wql_mx_scale_bytes(128, 128) == 512
    assert wql.wql_mx_scale_bytes(129, 160) == 4 * 512
    assert wql.wql_mx_scale_bytes(0, 32) == 0
    assert wql.wql_mx_scale_bytes(-1, 32) == 0
    assert wql.wql_mx_scale_bytes(1, 0) == 0


def test_mx_quantize_refusals(lib):
    def call(x=A, dt=F16, rows=4, k=64, fmt=0, codes=A, scales=A):
        return lib.wql_mx_quantize(x, dt, rows, k, fmt, codes, scales, None)

    assert call(rows=-1) == EINVAL
    assert call(k=0) == EINVAL
    assert call(fmt=2) == EINVAL
    assert call(x=None) == EINVAL
    assert call(codes=None) == EINVAL
    assert call(scales=None) == EINVAL
    assert call(dt=3) == EUNSUPPORTED
    assert call(k=48) == EUNSUPPORTED
    assert call(rows=2 ** 31) == EUNSUPPORTED
    assert call(x=A + 8) == EUNSUPPORTED
    assert call(codes=A + 4) == EUNSUPPORTED
    assert call(scales=A + 4) == EUNSUPPORTED
    assert call(rows=0, x=None, codes=None, scales=None) == OK


def test_mx_dequantize_refusals(lib):
    def call(m, dt=F32, out=A):
        return lib.wql_mx_dequantize(ctypes.byref(m) if m else None, dt, out, None)

    assert call(None) == EINVAL
    assert call(mx(fmt=5)) == EINVAL
    assert call(mx(reserved=1)) == EINVAL
    assert call(mx(rows=-1)) == EINVAL
    assert call(mx(codes=None)) == EINVAL
    assert call(mx(), out=None) == EINVAL
    assert call(mx(), dt=7) == EUNSUPPORTED
    assert call(mx(k=40)) == EUNSUPPORTED
    assert call(mx(), out=A + 8) == EUNSUPPORTED
    assert call(mx(rows=0, codes=None, scales=None), out=None) == OK


def test_mx_logits_refusals(lib):
    def call(x, w, bias=None, dt=F16, out=A, ws=None, wsb=0):
        return lib.wql_mx_logits(ctypes.byref(x) if x else None, ctypes.byref(w) if w else None,
                                 bias, dt, out, ws, wsb, None)

    assert call(None, mx()) == EINVAL
    assert call(mx(rows=2), None) == EINVAL
    assert call(mx(rows=2, k=128), mx(k=256)) == EINVAL
    assert call(mx(rows=2), mx(), out=None) == EINVAL
    assert call(mx(rows=2, scales=None), mx()) == EINVAL
    assert call(mx(rows=2), mx(fmt=1)) == EUNSUPPORTED             # the weight is FP4
    assert call(mx(rows=2), mx(), dt=F32) == EUNSUPPORTED
    assert call(mx(rows=2, k=40), mx(k=40)) == EUNSUPPORTED
    assert call(mx(rows=2), mx(codes=A + 8)) == EUNSUPPORTED
    assert call(mx(rows=2), mx(), out=A + 1) == EUNSUPPORTED
    assert call(mx(rows=2), mx(), bias=A + 1) == EUNSUPPORTED
    assert call(mx(rows=2), mx(), ws=A, wsb=255) == EWORKSPACE
    assert call(mx(rows=2), mx(), ws=A + 64, wsb=256) == EWORKSPACE
    assert call(mx(rows=0), mx()) == OK
    assert call(mx(rows=2), mx(rows=0)) == OK


def test_add_rmsnorm_refusals(lib):
    def call(x=A, r=A, g=A, dt=BF16, m=2, k=64, eps=1e-6, fmt=0, out=A, sc=A, ro=A):
        return lib.wql_add_rmsnorm(x, r, g, dt, m, k, eps, fmt, out, sc, ro, None)

    assert call(m=-1) == EINVAL
    assert call(k=0) == EINVAL
    assert call(eps=-1.0) == EINVAL
    assert call(eps=float("nan")) == EINVAL
    assert call(fmt=4) == EINVAL
    assert call(fmt=-1) == EINVAL
    assert call(x=None) == EINVAL
    assert call(g=None) == EINVAL
    assert call(out=None) == EINVAL
    assert call(fmt=1, sc=None) == EINVAL
    assert call(dt=F32) == EUNSUPPORTED
    assert call(k=65537) == EUNSUPPORTED
    assert call(fmt=2, k=72) == EUNSUPPORTED
    assert call(fmt=3, x=A + 8) == EUNSUPPORTED
    assert call(x=A + 1) == EUNSUPPORTED
    assert call(fmt=1, sc=A + 2) == EUNSUPPORTED
    assert call(m=0, x=None, g=None, out=None) == OK


def test_sample_refusals(lib):
    def call(l=A, dt=F16, m=2, n=100, u=A, t=None, k=None, p=None, mp=None, ids=A, lp=A):
        return lib.wql_sample(l, dt, m, n, u, t, k, p, mp, ids, lp, None)

    assert call(m=-1) == EINVAL
    assert call(n=0) == EINVAL
    assert call(l=None) == EINVAL
    assert call(u=None) == EINVAL
    assert call(ids=None) == EINVAL
    assert call(dt=3) == EUNSUPPORTED
    assert call(n=wql.SAMPLE_MAX_N + 1) == EUNSUPPORTED
    assert call(m=1 << 27) == EUNSUPPORTED
    assert call(l=A + 1) == EUNSUPPORTED
    assert call(l=A + 2, dt=F32) == EUNSUPPORTED
    assert call(t=A + 2) == EUNSUPPORTED
    assert call(k=A + 1) == EUNSUPPORTED
    assert call(m=0, l=None, u=None, ids=None) == OK


def test_binding_refuses_host_tensors_and_wrong_shapes():
    x = torch.zeros(2, 64, dtype=torch.float16)
    for f in (lambda: wql.wql_mx_quantize(x), lambda: wql.wql_add_rmsnorm(x, x[0]),
              lambda: wql.wql_sample(x, torch.zeros(2)),
              lambda: wql.wql_mx_dequantize(
                  wql.MXMatrix(torch.zeros(2, 32, dtype=torch.uint8),
                               torch.zeros(1, 1, 512, dtype=torch.uint8), wql.MX_FP4, 2, 64))):
        with pytest.raises(ValueError, match="CUDA tensor"):
            f()


# ---------------------------------------------------------------------------
# the references
# ---------------------------------------------------------------------------
def test_fp8_table_is_torchs():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(ref64.fp8_table(), t)


def test_nearest_code_is_brute_force():
    g = ref64.grid(0)
    a = np.arange(0, 8, 1 / 64)
    want = [min(range(8), key=lambda c: (abs(v - g[c]), c % 2)) for v in a]
    np.testing.assert_array_equal(ref64.nearest_code(a, g), want)
    x = torch.cat((torch.linspace(0, 448, 9001), torch.tensor([2 ** -9, 2 ** -10, 3 * 2 ** -10])))
    np.testing.assert_array_equal(ref64.nearest_code(x.double().numpy(), ref64.grid(1)),
                                  x.to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_worked_block():
    """amax 11: e = floor(log2 11) - 2 = 1, so codes are x / 2."""
    x = np.zeros((1, 32))
    x[0, :4] = [11.0, -1.0, 0.5, 5.0]      # 5.5 -> 6, -0.5, 0.25 -> 0 (tie), 2.5 -> 2 (tie)
    codes, byte = ref64.mx_quantize(x, 0)
    assert byte[0, 0] == 128 and codes[0, 0] == 0x97 and codes[0, 1] == 0x40
    np.testing.assert_array_equal(ref64.mx_values(codes, byte, 0)[0, :4], [12.0, -1.0, 0.0, 4.0])


def test_sample_exact_worked():
    """Weights 4 : 2 : 1 : 1 (in units of 2^29): sums 4, 6, 7, 8 by rank."""
    t = float(np.float32(1.44269504088896340736))          # c = 1
    l = [3.0, 1.0, 2.0, 1.0]
    un = 1 << 29
    assert ref64.sample_exact(l, t, 0, 1.0, 0.0, 0.0) == (0, 4 * un, 8 * un)
    assert ref64.sample_exact(l, t, 0, 1.0, 0.0, 0.5) == (1, un, 8 * un)
    assert ref64.sample_exact(l, t, 0, 1.0, 0.0, 0.99) == (3, un, 8 * un)
    assert ref64.sample_exact(l, t, 3, 1.0, 0.0, 0.99) == (2, 2 * un, 7 * un)
    assert ref64.sample_exact(l, t, 0, 0.75, 0.0, 0.99) == (2, 2 * un, 6 * un)
    assert ref64.sample_exact(l, t, 0, 0.76, 0.0, 0.99) == (2, 2 * un, 7 * un)
    assert ref64.sample_exact(l, t, 0, 1.0, 0.5, 0.99) == (2, 2 * un, 6 * un)
    assert ref64.sample_exact(l, 0.0, 0, 1.0, 0.5, 0.99)[0] == 0
