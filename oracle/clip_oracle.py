"""fp64 CPU oracle of the gradient norm and clipping -- TEST INFRASTRUCTURE ONLY.
Shares no code with the HIP library."""

from __future__ import annotations

import math

import numpy as np


def norm(tensors):
    """The 2-norm over all elements of a list of arrays, the sum of squares exact (fsum)."""
    return math.sqrt(math.fsum(float(x) * float(x) for t in tensors for x in np.asarray(t, dtype=np.float64).ravel()))


def factor(norm, max_norm, eps=1e-6):
    if math.isnan(norm):
        return math.nan
    if math.isinf(max_norm):
        return 1.0
    return min(1.0, max_norm / (norm + eps))
