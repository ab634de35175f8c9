"""The arithmetic of the gated scan's decays, evaluated on the CPU in fp32: what a rounded
decay would cost on the gates of test_gpu_scan_memory, and that the bounds there see it."""
import numpy as np
import pytest
import torch

from tests._scan_common import U32
from tests._scan_memory import GATES, slack, steady, step_slack

f32 = np.float32


def _fma(a, b, c):
    """fp32 fused multiply-add (the product of two fp32 numbers is exact in 64 bits)."""
    return (np.float64(a) * np.float64(b) + np.float64(c)).astype(f32)


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


@pytest.mark.parametrize("gate", ["log", "sigmoid"])
def test_single_steps_by_the_complement(gate):
    """h - (1 - a) h stays inside the bound of the single-step test, a h with a rounded a is
    tens of times outside."""
    la, a, c = (float(v) for v in steady(gate))
    steps, rng = 400, np.random.default_rng(2)
    first = (1.0 + rng.random(32768)).astype(f32)
    h, naive = first.copy(), first.copy()
    for _ in range(steps):
        h = (h + _fma(-f32(c), h, f32(0.0))).astype(f32)
        naive = _fma(f32(a), naive, f32(0.0))
    off = [abs(float((v.astype(np.float64) / first).mean()) * np.exp(-steps * la) - 1.0) for v in (h, naive)]
    bound = step_slack(gate, steps, first.size)
    assert off[0] <= bound and off[1] > 30 * bound, [v / U32 for v in off + [bound]]
