"""The error of the paged attention as one number per call: the norm of the
difference over the norm of the result, and what it may be.

An output is a weighted mean of value rows. The kernels round some of what goes
into it to bf16, each to nearest, so by at most half a step: relative at most
2^-8, evenly spread, hence with a root mean square of at most 2^-8 / sqrt(3) (where
the mantissa is 1; less elsewhere). The roundings of different positions are
independent, so each kind adds at most that much of the result's own norm for
values about zero:

- the weights (with their steps for single tokens over 4-bit pages): always;
- values and keys too in tiles of 4-bit pages. A key's rounding moves a score by
  the root of the sum of (q_d k_d)^2 over its dims / 16 times that, which is that
  much itself for queries and keys of variance 1, and the weights by as much;
- outputs in bf16.

fp32 sums add orders less, at any length. Norms over thousands of elements vary
by a few percent around their mean, so the bound is taken as it is for results of a
hundred positions or more."""
from __future__ import annotations

import numpy as np
import torch

HALF_STEP = 2.0 ** -8


def roundings(four_bits: bool, max_q: int, out_dtype) -> int:
    return (3 if four_bits and max_q > 2 else 1) + (out_dtype == torch.bfloat16)


def bound(four_bits: bool, max_q: int, out_dtype) -> float:
    return HALF_STEP * (roundings(four_bits, max_q, out_dtype) / 3) ** 0.5


def relative(got, ref) -> float:
    got = got.detach().cpu().double().numpy() if isinstance(got, torch.Tensor) else np.asarray(got)
    return float(np.linalg.norm(got - ref) / np.linalg.norm(ref))


# new tokens and contexts of the batches that are compared by norm
BATCHES = [([257], [1300]), ([513, 64], [513, 900]), ([130, 1], [200, 700]), ([3, 20, 0, 17], [1000, 131, 50, 333]),
           ([70], [1300]), ([1, 1, 1], [1025, 129, 513]), ([2, 1, 2], [900, 700, 130]), ([8, 5], [300, 2600])]
