"""Half an ulp of a result's type: what one rounding to it may add to an error
bound.  bf16 keeps 8 significant bits and float32 24, so a value in
[2^k, 2^(k+1)) rounds by at most 2^(k-8) or 2^(k-24)."""

import numpy as np
import torch


def half_ulp(dtype, ref, slack=0.0):
    """For results within ``slack`` of ``ref`` (float64 arrays)."""
    top = np.maximum(np.abs(ref) + slack, 2.0 ** -126)
    return 2.0 ** (np.floor(np.log2(top)) - (8 if dtype == torch.bfloat16 else 24))
