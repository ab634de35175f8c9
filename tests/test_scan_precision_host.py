"""The arithmetic of the gated scan's decays, evaluated on the CPU in fp32: what a rounded
decay would cost on the gates of test_gpu_scan_memory, and that the bounds there see it; and
the errors that kda_scan.h states for its series and for the logistic function."""
import os
import re

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


SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gated_delta_rule_short_amd", "csrc",
                      "kda_scan.h")


def _body(head):
    """The source of the device function whose declaration holds `head`."""
    text = open(SOURCE, encoding="utf-8").read()
    at = text.index(head)
    return text[at:text.index("}\n", at)]


def _worst(got, want):
    return float((np.abs(got.astype(np.float64) - want) / np.abs(want)).max())


def test_the_logarithm_of_1_plus_e():
    """log2_1p over 2^-30 to 1, in fp32 as the source has it: 2.1e-7 of itself."""
    body = _body("float log2_1p(float e)")
    coeff = [f32(v) for v in re.findall(r"(-?\d\.\d+)f", body)]
    assert len(coeff) == 9 and body.count("fmaf(") == 8
    e = np.concatenate([np.exp2(np.linspace(-30, 0, 200001)), np.linspace(0.25, 1.0, 200001)]).astype(f32)
    q = np.full_like(e, coeff[0])
    for k in coeff[1:]:
        q = _fma(q, e, k)
    assert 1.5e-7 < _worst((e * q).astype(f32), np.log1p(e.astype(np.float64)) / np.log(2.0)) < 2.1e-7


def test_1_minus_the_exponential_near_0():
    """near_zero over -1/8 to -1e-8: 9e-8 of itself."""
    body = _body("float near_zero(float g)")
    assert [int(v) for v in re.findall(r"1\.f / (\d+)\.f", body)] == [720, 120, 24, 6] and body.count("fmaf(") == 5
    g = -np.concatenate([np.exp2(np.linspace(-26, -3, 200001)), np.linspace(0.0625, 0.125, 200001)]).astype(f32)
    q = _fma(g, f32(1.0) / f32(720.0), f32(1.0) / f32(120.0))
    for k in (f32(1.0) / f32(24.0), f32(1.0) / f32(6.0), f32(0.5), f32(1.0)):
        q = _fma(q, g, k)
    assert 6e-8 < _worst((-g * q).astype(f32), -np.expm1(g.astype(np.float64))) < 9e-8


def test_the_logistic_function_and_its_complement():
    """a and 1 - a from one exponential, with every step rounded once: the argument's rounding
    costs 1.3 |z| u32, four roundings the rest.  (The hardware's exponential and reciprocal may
    be another u32 off, each.)"""
    z = np.linspace(-60.0, 60.0, 400001).astype(f32)
    e = np.exp2((-np.abs(z) * f32(1.4426950408889634)).astype(f32).astype(np.float64)).astype(f32)
    r = (1.0 / (f32(1.0) + e).astype(f32).astype(np.float64)).astype(f32)
    er = (e * r).astype(f32)
    z64 = z.astype(np.float64)
    for got, want in ((np.where(z > 0, r, er), 1.0 / (1.0 + np.exp(-z64))), (np.where(z > 0, er, r), 1.0 / (1.0 + np.exp(z64)))):
        off = np.abs(got.astype(np.float64) - want) / want / U32
        assert (off <= 4 + 1.3 * np.abs(z64)).all() and (off > 10).any()
