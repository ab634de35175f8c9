"""The arithmetic of the gated scan's decays, evaluated on the CPU in fp32: what a rounded
decay would cost on the gates of test_gpu_scan_memory, and that the bounds there see it."""
import numpy as np
import pytest
import torch

from tests._scan_memory import GATES, slack, steady

f32 = np.float32


@pytest.mark.parametrize("gate", ["log", "sigmoid"])
@pytest.mark.parametrize("rows", [1, 4, 6, 8, 10, 12, 14, 16])
def test_a_rounded_decay_breaks_the_bounds(gate, rows):
    """Decays handed on as the product of `rows` rounded ones, or as its logarithm, remember
    another number of tokens: twice the bound of the memory tests away."""
    la, a, c = (float(v) for v in steady(gate))
    assert float(torch.tensor(GATES[gate]).bfloat16()) == GATES[gate]
    prod = f32(1.0)
    for _ in range(rows):
        prod = f32(prod * f32(a))
    shift = abs(np.log(float(prod)) / rows - la) / c
    assert shift > 2 * max(slack(gate, False), slack(gate, True))
