"""Steady gates that remember thousands of tokens, and what the gated scan makes of them in
64 bits: closed forms, and bounds that a decay rounded to fp32 does not keep.

With a gate value z at every token, a = 1 - c, and ones for x, the state from zero is
h_t = b (1 - a^t) / c.  A rounding of a alone, by d, is a memory of another length: h is off
by d / c of itself.  The gates here, which bf16 holds too, are ones whose a lies far from fp32:
d is half a step, 2^-25, or nearly, and d / c 1.2e-4 and 1.7e-4.

What the kernels may be off by, in units of u32 = 2^-24 of h (every term is positive):
  * 3 a tile: the exponential that makes the tile's decay (1 ulp, 2 units above 1/2) and the
    step over it.  M = 1 / c tokens count, the smallest tiles of a long sequence are 7 waves
    of 6 rows forward and 4 backward: 3 (M / 42 + 1) and 3 (M / 28 + 1);
  * inside a tile, once: 16 rows of a wave, each with its decay's and its step's rounding, 15
    waves joined with an exponential (2) and a step each, 45: 77, and 31 additions of logarithms,
    each 1 of their sum, which is 1 of the memory's length: 108 in all, and 20 for the rest;
  * the factors themselves: 1 - a, which is the memory's length, and b, each 6 + 1.3 |z| units
    (series and differences 9), twice that under a root's slope and a gradient's product:
    charged 32 + 8 |z|."""
import torch

from tests._scan_common import U32

GATES = {"log": -2.0 ** -12, "sigmoid": 8.6875}
TOKENS = 40000


def steady(gate):
    """(log a, a, c) in 64 bits."""
    z = torch.tensor(GATES[gate], dtype=torch.float64)
    la = z if gate == "log" else -torch.log1p(torch.exp(-z))
    return la, la.exp(), -torch.expm1(la)


def input_factor(a, c, inputs):
    return {"plain": torch.ones_like(a), "complement": c, "norm": (c * (1.0 + a)).sqrt()}[inputs]


def filled(gate, t):
    """1 + a + .. + a^(t - 1)."""
    la, _, c = steady(gate)
    return -torch.expm1(la * torch.as_tensor(t, dtype=torch.float64)) / c


def slack(gate, backward):
    """The bound above, relative to h."""
    tile = 28 if backward else 42
    return (3 * (1 / float(steady(gate)[2]) / tile + 1) + 160 + 8 * abs(GATES[gate])) * U32


def step_slack(gate, steps, values):
    """Of the mean over `values` states of h_n / (a^n h_0) - 1 after n single steps without an
    input: 1 - a is off by at most 9 + 1.3 |z| units each step; the step's rounding, of states
    with random digits, is as often up as down, at most half an ulp, and its root mean square
    ulp / sqrt(12), 0.58 units: eight times that of the mean of n x values of them."""
    c = float(steady(gate)[2])
    return (steps * c * (9 + 1.3 * abs(GATES[gate])) + 8 * 0.58 * (steps / values) ** 0.5) * U32
