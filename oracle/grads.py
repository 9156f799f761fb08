"""Global gradient norm and clipping, from the definitions in 64 bits."""
import math

import numpy as np


def norm_and_scale(grads, max_norm, mult=1.0):
    """norm = |m| sqrt(sum of squares); scale = m where norm <= max_norm, else m max_norm / norm."""
    with np.errstate(invalid="ignore", over="ignore"):
        total = math.fsum(float(np.square(np.asarray(g, dtype=np.float64)).sum()) for g in grads) \
            if all(np.isfinite(g).all() for g in grads) else \
            float(sum(np.square(np.asarray(g, dtype=np.float64)).sum() for g in grads))
        norm = abs(mult) * math.sqrt(total) if total == total else math.nan
    if norm <= max_norm:
        return norm, mult
    return norm, mult * (max_norm / norm)
