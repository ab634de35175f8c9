"""The largest calls that the gated scan accepts: 2^22 - 1 pairs of a sequence and 128 channels,
all of one channel group or all of one sequence, sampled against the recurrence in 64 bits."""
import pytest
import torch

import gated_delta_rule_short_amd as kda
from tests._scan_common import BF, DEV, F32, U32, check_scan

pytestmark = pytest.mark.gpu
MOST = (1 << 22) - 1


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    kda.load_library()


def _tensors(rows, C, dtype):
    gen = torch.Generator(device=DEV).manual_seed(rows % 1009)
    x = torch.randn(rows, C, generator=gen, device=DEV, dtype=dtype)
    g = torch.randn(rows, C, generator=gen, device=DEV, dtype=dtype)
    return x, g, torch.randn(rows, C, generator=gen, device=DEV)


@pytest.mark.parametrize("N,C", [(MOST, 8), (1, 128 * MOST), (2047, 128 * 2049)])
def test_single_steps(N, C):
    x, g, state = _tensors(N, C, BF)
    rows = torch.tensor(sorted({0, N // 2, N - 1}), device=DEV)
    cols = torch.tensor(sorted({0, 7, C // 2, C - 4, C - 1}), device=DEV)
    pick = lambda t: t[rows][:, cols]
    inp = {"x": pick(x), "gate": pick(g), "state": pick(state), "slots": None, "lengths": [1] * len(rows)}
    o = kda.kda_gated_scan_decode(x, g, state, gate_kind="sigmoid", input_kind="complement")
    check_scan(pick(o), pick(state), inp, "sigmoid", "complement")
    assert torch.isfinite(state).all() and torch.equal(o, state.to(BF))


def test_prompts_of_as_many_sequences():
    """One token each (what a chain of tiles would not hold is done in one pass)."""
    x, g, state = _tensors(MOST, 8, F32)
    rows = torch.tensor([0, 1, MOST // 2, MOST - 2, MOST - 1], device=DEV)
    inp = {"x": x[rows], "gate": g[rows], "state": state[rows], "slots": None, "lengths": [1] * len(rows)}
    o, out = kda.kda_gated_scan_prefill(x, g, gate_kind="sigmoid", num_seqs=MOST, state_in=state, state_out=True)
    check_scan(o[rows], out[rows], inp, "sigmoid", "plain")
    # Every row: o and the final state are two roundings of one h.  o = a h + x with a itself,
    # the state = P h + x with P = 2^l through the logarithm; each is off by at most the decay's
    # k of _scan_common times a |h| and 4 u32 of a |h| + |x|.
    z = g.double()
    a, l = torch.sigmoid(z), torch.nn.functional.softplus(-z) * 1.4426950408889634
    held = a * state.double().abs()
    bound = 2 * (((140 + 4 * z.abs()) * l + 8) * U32 * held + 4 * U32 * (held + x.double().abs()))
    assert ((o.double() - out.double()).abs() <= bound).all()
    with pytest.raises(kda.KdaError):
        kda.kda_gated_scan_prefill(x, g, num_seqs=MOST, schedule="chained")
