"""The norm and the quantiser where a launch has many rows (several per block,
or fewer threads to a row), and the norm on tensors that start anywhere."""
import numpy as np
import pytest
import torch

import ref64
import test_gpu_operators as small
import weight_only_quantized_wql_gb300 as wql
from ref64 import f64

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.mark.parametrize("rows,k", [(2500, 96), (5003, 160), (20011, 64), (4900, 1056)])
@pytest.mark.parametrize("fmt", [wql.MX_FP4, wql.MX_FP8])
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_mx_bit_exact(rows, k, fmt, dt):
    """Two, four and eight rows per block, the last block short."""
    small.test_mx_bit_exact(fmt, rows, k, dt)


NORMS = [(305, 4099), (400, 5120), (700, 1024), (310, 16400), (304, 30001)]


@pytest.mark.parametrize("m,k", NORMS)
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_norm_same(m, k, dt):
    small.test_norm_same(m, k, dt, True)


@pytest.mark.parametrize("m,k", NORMS)
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_norm_e4m3(m, k, dt):
    small.test_norm_e4m3(m, k, dt)


@pytest.mark.parametrize("fmt", [wql.NORM_MX_FP8, wql.NORM_MX_FP4])
@pytest.mark.parametrize("m,k", [(305, 4128), (400, 5120), (700, 1024), (310, 16416)])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_norm_mx(fmt, m, k, dt):
    small.test_norm_mx(fmt, m, k, dt)


@pytest.mark.parametrize("m,k", [(5, 1003), (3, 1024), (306, 777), (2, 65536)])
@pytest.mark.parametrize("shift", [1, 3, 8])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_norm_any_alignment_against_64_bits(m, k, shift, dt):
    """Tensors that start on any element: each output by its own bound."""
    x, r, w = small.norm_inputs(m, k, dt, 9 + k)
    off = [torch.empty(t.numel() + shift, dtype=t.dtype, device=DEV)[shift:].view(t.shape)
           for t in (x, r, w)]
    for o, t in zip(off, (x, r, w)):
        o.copy_(t)
    _, want = ref64.rmsnorm(f64(x), f64(r), f64(w), 1e-6)
    rel = small.rel32(k)
    aligned = wql.wql_add_rmsnorm(x.to(DEV), w.to(DEV), r.to(DEV))[1]
    y, ro, sc = wql.wql_add_rmsnorm(off[0], off[2], off[1])
    assert sc is None and torch.equal(ro, aligned)       # does not depend on the sum's order
    assert np.all(np.abs(f64(y) - want) <=
                  (small.ULP[dt] * 1.001 + rel) * np.abs(want) + small.TINY[dt])
    y, ro, sc = wql.wql_add_rmsnorm(off[0], off[2], off[1], fmt=wql.NORM_E4M3)
    assert torch.equal(ro, aligned)
    s = np.maximum(np.abs(want).max(-1) / 448, 1e-8)
    assert np.all(np.abs(f64(sc) - s) <= (rel + 2.0 ** -22) * s)
    v = want / s[:, None]
    # half a step of e4m3 (3 bits of fraction, subnormals of 2^-9), and the fp32 steps
    tol = np.maximum(2.0 ** -4 * np.abs(v), 2.0 ** -10) + (rel + 2.0 ** -21) * np.abs(v) * 2
    assert np.all(np.abs(f64(y.float()) - v) <= tol)


@pytest.mark.parametrize("fmt", [wql.NORM_SAME, wql.NORM_E4M3])
def test_norm_leaves_the_elements_around_alone(fmt):
    """Outputs inside a larger buffer, on odd boundaries."""
    m, k = 3, 1003
    x, r, w = (t.to(DEV) for t in small.norm_inputs(m, k, "bf16", 4))
    for at in (8, 9):
        buf = torch.full((m * k + 24,), 7.0, dtype=torch.bfloat16, device=DEV)
        ro = buf[at:at + m * k].view(m, k)
        _, got, _ = wql.wql_add_rmsnorm(x, w, r, fmt=fmt, residual_out=ro)
        assert got is ro and torch.equal(ro, (x.float() + r.float()).bfloat16())
        assert torch.all(buf[:at] == 7) and torch.all(buf[at + m * k:] == 7)
