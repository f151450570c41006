"""Bounded waits of the operators around the head, made to run out on purpose
without faulting or hanging anything (see wql_debug_set_waits): the call
returns, says so, leaves no copy in flight, and the next call is right."""
import numpy as np
import pytest
import torch

import ref64
import weight_only_quantized_wql_gb300 as wql

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BUDGET = 2_000_000                                    # SM cycles, about 1 ms
LOG2E = float(np.float32(1.44269504088896340736))    # as a temperature: c = 1


@pytest.fixture(autouse=True)
def _restore_waits():
    torch.cuda.set_device(DEV)
    wql.load()
    yield
    wql.wql_debug_set_waits(0, False)


@pytest.mark.parametrize("m,n,dt", [(1, 40001, torch.bfloat16),      # eight blocks a row
                                    (200, 3001, torch.float32)])     # one
def test_sample_wait_timeout_is_reported_and_recovers(m, n, dt):
    g = torch.Generator().manual_seed(n)
    l = torch.randint(-9, 10, (m, n), generator=g).float()
    u = torch.rand(m, generator=g)
    t = torch.full((m,), LOG2E, device=DEV)
    args = (l.to(dt).to(DEV), u.to(DEV), t)
    wql.wql_debug_set_waits(BUDGET, True)
    ids, logp = wql.wql_sample(*args)
    torch.cuda.synchronize()
    assert (ids == -2).all() and torch.isnan(logp).all()
    wql.wql_debug_set_waits(0, False)
    ids, logp = wql.wql_sample(*args)
    for i in range(0, m, 40):
        want = ref64.sample_exact(l[i].tolist(), LOG2E, 0, 1.0, 0.0, float(u[i]))
        assert int(ids[i]) == want[0]
    assert torch.isfinite(logp).all()


def test_mx_logits_without_a_workspace_reports_its_waits():
    x = wql.wql_mx_quantize(torch.randn(3, 512, device=DEV), wql.MX_FP8)
    w = wql.wql_mx_quantize(torch.randn(1000, 512, device=DEV))
    good = wql.wql_mx_logits(x, w)
    ws = wql.default_workspace(DEV)
    assert ws.error_word() == 0
    wql.wql_debug_set_waits(BUDGET, True)
    wql.wql_mx_logits(x, w)
    wql.wql_debug_set_waits(0, False)
    assert ws.error_word() == 8
    ws.clear_error()
    assert torch.equal(wql.wql_mx_logits(x, w), good) and ws.error_word() == 0
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):                     # a stream has one of its own
        assert wql.default_workspace(DEV) is not ws
        assert wql.default_workspace() is wql.default_workspace(DEV)


def test_mx_logits_refuses_a_workspace_elsewhere():
    x = wql.wql_mx_quantize(torch.randn(3, 512, device=DEV))
    w = wql.wql_mx_quantize(torch.randn(100, 512, device=DEV))
    with pytest.raises(ValueError, match="workspace"):
        wql.wql_mx_logits(x, w, workspace=wql.Workspace("cpu"))
