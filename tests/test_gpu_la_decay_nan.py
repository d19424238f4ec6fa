"""The gradient of a decay that is not finite (la_prefill_backward's dlog_decay)."""
import numpy as np
import pytest
import torch

from gated_deltanet_hybrid_amd import hla
from gpu_util import note
from la_util import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("per_head", [False, True])
def test_a_decay_that_is_nan_has_a_gradient_that_is(dtype, per_head):
    """exp(NaN) <G, M> is NaN; only a decay that clears the state has the gradient 0."""
    note(f"dlog_decay of NaN {dtype} {per_head}")
    c = Case(2, 150, 2, 2, 64, 64, dtype, per_head=per_head, seed=35)
    r = np.random.default_rng(7)
    c.g_ = torch.from_numpy((-0.02 * (1.0 + 2.0 * r.random(tuple(c.g_.shape)))).astype(np.float32))
    run = lambda: hla.la_prefill_backward(*c.args(), c.device("dO"), dS_final=c.device("dS"), **c.kw())["dlog_decay"].cpu()  # noqa: E731
    if per_head:
        c.g_[1] = float("nan")
        got = run()
        assert torch.isfinite(got[0]) and torch.isnan(got[1])
    else:
        c.g_[0, 70, 1] = float("nan")
        c.g_[1, 70, 1] = -float("inf")
        got = run()
        assert torch.isnan(got[0, 70, 1]) and got[1, 70, 1] == 0
        assert torch.isfinite(got[:, :, 0]).all() and torch.isfinite(got[1]).all()
