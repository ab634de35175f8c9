"""Forms of the linear attention that the other GPU tests leave out: batches without
tokens under every schedule."""
import pytest
import torch

import gated_delta_rule_short_amd as kda
from tests._linattn_common import DEV, make_linattn

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    kda.load_library()


@pytest.mark.parametrize("schedule", ["auto", "one_pass", "two_pass"])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_an_empty_batch_passes_its_states_through(schedule, dtype):
    inp = make_linattn([0, 0, 0], 4, 2, 64, 128, dtype, seed=1, device=DEV)
    o, st = kda.kda_linattn_prefill(inp["q"], inp["k"], inp["v"], inp["log_decay"], cu_seqlens=inp["cu"],
                                    cu_seqlens_host=inp["cu_host"], state_in=inp["state"], state_out=True,
                                    schedule=schedule)
    assert o.shape == (0, 4, 128) and torch.equal(st, inp["state"])
