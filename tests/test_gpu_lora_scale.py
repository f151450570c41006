"""Adapters whose scale is far above what fp16 holds."""
import pytest
import torch

import weight_only_quantized_wql_gb300 as wql

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("scale", [3e38, -3e38, 1e36])
def test_nothing_times_a_large_scale(dt, scale):
    """Where b is zero nothing is added, however large scale and u are; elsewhere the
    sum overflows with its sign."""
    x = torch.full((3, 64), 64.0, dtype=dt, device=DEV)
    a = torch.full((1, 8, 64), 2.0, dtype=dt, device=DEV)          # u = 8192
    b = torch.zeros(1, 40, 8, dtype=dt, device=DEV)
    b[0, 3], b[0, 5] = 1.0, -1.0
    y = torch.randn(3, 40, device=DEV).to(dt)
    ad = wql.LoraAdapters(a, b, torch.tensor([scale], device=DEV))
    got = wql.wql_lora_add(y, x, ad, torch.tensor([0, -1, 0], dtype=torch.int32, device=DEV))
    want = y.clone()
    up = float("inf") if scale > 0 else -float("inf")
    want[[0, 2], 3], want[[0, 2], 5] = up, -up
    assert torch.equal(got, want)
