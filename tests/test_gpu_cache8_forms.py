"""Which form an 8-bit decode takes: what the caller's gates save is not charged."""
import pytest
import torch

from gpu_util import note
from test_gpu_cache8 import hla, make_cache, rnd, token
from test_gpu_cache8_precision import check_close

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_gates_that_are_given_cost_no_scoring(fmt):
    """64 chunks of 256 representatives: scoring them in one workgroup takes longer than the split
    form; with the caller's gates nothing is scored and one workgroup a row is the shorter way.  The
    split form writes its workspace, the other leaves it alone; both are right."""
    note(f"cache8 form with gates {fmt}")
    h = hla()
    c = make_cache(h, 1, 2, 64, 128, 64, 256, fmt, 601)
    c.count.fill_(64)
    need = h.cache8_workspace_bytes(c)
    assert need > 0
    _, rand = rnd(602)
    gi = 0.05 + 0.9 * rand(1, 2, 64)
    tok, gates, S, A = token(1, 2, 128, 64, "bf16", False, 603)
    for given, form in ((gi, "whole"), (None, "split")):
        ws = torch.full((need,), 0xA5, dtype=torch.uint8, device="cuda")
        h.gdn_decode8(*tok, *gates, S.clone(), A.clone(), c, gates_in=given, ws=ws)
        assert bool((ws == 0xA5).all()) == (form == "whole")
        check_close(h, c, tok, gates, S.clone(), A.clone(), gates_in=given)
