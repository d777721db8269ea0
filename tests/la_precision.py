"""Norm-wise error of linear attention with a decay for each head, one figure for each head.

The element-wise bounds of la_model.py hold for any signs, so where a head remembers long
they are as wide as the outputs themselves; these figures see what stays inside them.

A rounding to bf16 is off by at most 2^-8 of the value and, evenly spread over a step, by
u = 2^-8 / sqrt(3) of it in the root mean square at the most (mantissa 1; 1.7e-3 over the
mantissas that occur).  An output of the bf16 path is rounded once itself: u.  Before that
each product that it sums had one factor rounded: the decayed score inside a chunk, the state
before it.  Those errors are independent, and so are the signs of the products, so together
they are u of the root of the sum of squares, which is the output's own size.  In all
sqrt(2) u = 3.2e-3; a tenth more for outputs a little smaller than their products.

An fp32 output sums, one after the other, d products (scores, or the state's row) and up to
64 tokens of its chunk, and the state it reads was added to once a token: n = T + d + 32
roundings of 2^-24 / sqrt(3) of partial sums, independent of each other: 2^-24 sqrt(n).

A state of the bf16 path is fp32: each tile of 64 or 128 tokens is 12 or 24 steps of a tensor
core, which may cut (a step of 2^-23 at most, half of it on average, of partial sums that
average two thirds of the end's): 16 x 2^-24 at the most; the additions of the tiles, rounded
to nearest, and the fp32 weights' own rounding are independent: sqrt(T / 64 + 2) 2^-24 / sqrt(3).
Weighted rows of two bf16 terms instead of three drop up to 2^-17 of every product, 2^-17 / sqrt(3)
in the root mean square: 4.4e-6 at the most, more than twice as much.
"""
import numpy as np
import torch

import la_model as lm

OUT_BF16 = 1.1 * 2 ** 0.5 * 2.0 ** -8 / 3 ** 0.5


def out_limit(dtype, T, d):
    return OUT_BF16 if dtype == torch.bfloat16 else 2.0 ** -24 * (T + d + 32) ** 0.5


def state_limit(dtype, T, d):
    if dtype == torch.bfloat16:
        return 2.0 ** -24 * (16 + ((T / 64 + 2) / 3) ** 0.5)
    return 2.0 ** -24 * (T + d + 32) ** 0.5


def rel(got, want, head_axis):
    """||got - want|| / ||want|| of each head; elements that are NaN in `want` are nobody's."""
    got = lm.to64(got) if torch.is_tensor(got) else got
    live = ~np.isnan(want)
    axes = tuple(a for a in range(want.ndim) if a != head_axis)
    size = lambda x: np.sqrt((np.where(live, x, 0.0) ** 2).sum(axis=axes))  # noqa: E731
    return size(got - want) / np.maximum(size(want), 1e-300)


def over(got, want, limit, head_axis):
    """Heads whose figure is above the limit, with it."""
    r = rel(got, want, head_axis)
    return {int(h): float(x) for h, x in enumerate(r) if not x <= limit}
