"""Steps of a beam search that say something: nearly all of them are compared."""
import pytest

import weight_only_quantized_wql_gb300 as wql
from test_gpu_requests import check_select, search

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("order", [wql.BEAM_RANKED, wql.BEAM_ANCHORED])
@pytest.mark.parametrize("seed", [0, 1, 2])
def test_steps_are_compared(order, seed):
    """(A step is left out where scores of two beams are nearer than their errors: one
    in hundreds.)"""
    batch, beams, n, steps = 3, 4, 1000, 6
    compared = 0
    for before, logits, parents, ended, tokens, scores, *_ in search(batch, beams, n, 128, steps, False, order,
                                                                     seed):
        compared += check_select(logits.view(batch, beams, n), before, 3, order,
                                 (tokens, parents, scores, ended))
    assert compared >= steps - 1
