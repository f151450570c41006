"""wql_mx_logits where a block works through many vocab tiles, as on a whole
head: accumulators, ring slots and resident tokens are used again and again."""
import numpy as np
import pytest
import torch

import ref64
import weight_only_quantized_wql_gb300 as wql
from ref64 import f64

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
T = {"f16": torch.float16, "bf16": torch.bfloat16}
ULP = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}            # half an ulp, relative
TINY = {"f16": 2.0 ** -25, "bf16": 1e-38}               # half the smallest subnormal


@pytest.mark.parametrize("fmt", [wql.MX_FP8, wql.MX_FP4])
@pytest.mark.parametrize("m,n,k", [
    (1, 151936, 64),         # eight tiles a block, 64-byte stores
    (40, 151936, 256),       # two accumulators
    (33, 100003, 96),        # rows that are not 16-byte aligned, tokens and codes of odd blocks
    (20, 120000, 160),       # e4m3: the weight by cp.async
    (200, 60000, 128),       # tokens that stay, two slices of them
    (256, 59997, 512),
    (250, 40000, 2304),      # e2m1: tokens that do not stay, one accumulator of 256 columns
    (140, 40000, 2336),      # the same for rows that are not whole 128-column blocks
    (600, 30000, 96)])       # five slices
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_many_tiles_per_block(fmt, m, n, k, dt):
    g = torch.Generator().manual_seed(m + n + k)
    x = torch.randn(m, k, generator=g) * (1 + 15 * (torch.rand(k, generator=g) < 0.02))
    xa = wql.wql_mx_quantize(x.to(DEV), fmt)
    xv = torch.from_numpy(ref64.mx_values(*ref64.mx_quantize(f64(x), fmt), fmt)).to(DEV)
    # the weight: any codes, scales around 2^-7
    codes = torch.randint(0, 256, (n, k // 2), generator=g, dtype=torch.uint8)
    byte = torch.randint(117, 124, (n, k // 32), generator=g, dtype=torch.uint8)
    wa = wql.MXMatrix(codes.to(DEV), torch.from_numpy(ref64.tile(byte.numpy())).to(DEV),
                      wql.MX_FP4, n, k)
    nibble = torch.stack((codes.to(DEV) & 15, codes.to(DEV) >> 4), -1).reshape(n, k).long()
    value = torch.tensor(np.concatenate((ref64.FP4, -ref64.FP4)), device=DEV)[nibble]
    wv = value * torch.exp2(byte.to(DEV).double() - 127).repeat_interleave(32, 1)
    bias = torch.randn(n, generator=g).to(T[dt])
    ws = wql.Workspace(DEV)
    got = wql.wql_mx_logits(xa, wa, T[dt], bias=bias.to(DEV), workspace=ws)
    assert ws.error_word() == 0
    b = bias.to(DEV).double()
    worst = 0.0
    for i in range(0, n, 20000):
        part = wv[i:i + 20000]
        want = xv @ part.t() + b[i:i + 20000]
        absacc = xv.abs() @ part.abs().t() + b[i:i + 20000].abs()
        # exact products, fp32 sums (the bound of the other product tests), one rounding
        tol = k * 2.0 ** -22 * absacc + ULP[dt] * 1.001 * want.abs() + TINY[dt]
        err = (got[:, i:i + 20000].double() - want).abs()
        assert torch.isfinite(err).all()
        worst = max(worst, float((err / tol).max()))
    assert worst <= 1, f"worst {worst:.2f} of the tolerance"
    assert torch.equal(got, wql.wql_mx_logits(xa, wa, T[dt], bias=bias.to(DEV)))


@pytest.mark.parametrize("fmt", [wql.MX_FP8, wql.MX_FP4])
@pytest.mark.parametrize("m,n,k", [(5, 1000, 512), (40, 1000, 640), (200, 1000, 384)])
def test_operands_and_output_on_other_boundaries(fmt, m, n, k):
    """Codes 16 bytes into a buffer, logits two bytes into one: other copies, the
    same logits."""
    g = torch.Generator().manual_seed(n + k)
    xa = wql.wql_mx_quantize(torch.randn(m, k, generator=g).to(DEV), fmt)
    wa = wql.wql_mx_quantize(torch.randn(n, k, generator=g).to(DEV))
    want = wql.wql_mx_logits(xa, wa, torch.float16)

    def moved(a):
        codes = torch.empty(a.codes.numel() + 16, dtype=torch.uint8, device=DEV)[16:].view(a.codes.shape)
        scales = torch.empty(a.scales.numel() + 16, dtype=torch.uint8, device=DEV)[16:].view(a.scales.shape)
        codes.copy_(a.codes)
        scales.copy_(a.scales)
        return wql.MXMatrix(codes, scales, a.fmt, a.rows, a.k)

    buf = torch.full((m * n + 16,), 7.0, dtype=torch.float16, device=DEV)
    out = buf[1:1 + m * n].view(m, n)
    got = wql.wql_mx_logits(moved(xa), moved(wa), torch.float16, out=out)
    # the same products in the same order of columns, whatever brings them in
    assert torch.equal(got, want)
    assert buf[0] == 7 and torch.all(buf[1 + m * n:] == 7)
