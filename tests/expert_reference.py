"""Plain 64-bit forms that the tests of the expert layer's calls share."""

import numpy as np
import torch

from oracle import formats as F
from oracle import mx as omx

FMTS = {"e4m3": F.E4M3, "e5m2": F.E5M2, "e2m1": F.E2M1}


def routing(rng, tokens, top, experts, pattern):
    """Routings [tokens][top]: even, skewed, one expert for all, none left, some out of range, one expert twice."""
    if pattern == "one":
        return np.full((tokens, top), experts - 1)
    if pattern == "none":
        return np.full((tokens, top), -1)
    e = rng.integers(0, experts, size=(tokens, top))
    if pattern == "skewed":
        e = np.minimum(e, rng.integers(0, experts, size=(tokens, top)) // 3)
    if pattern == "dropped":
        e = np.where(rng.random((tokens, top)) < 0.4, rng.choice([-1, experts, -(2 ** 31), 2 ** 31 - 1], size=(tokens, top)), e)
    return e


def plan_of(experts, E, align):
    """offsets, counts, slot_row, row_slot, block_expert of a routing, slot by slot."""
    tokens, top = experts.shape
    slots = tokens * top
    R = (slots + min(E, slots) * (align - 1)) // align * align
    flat = experts.reshape(-1)
    counts = np.array([(flat == e).sum() for e in range(E)], dtype=np.int64)
    offsets = np.concatenate([[0], np.cumsum((counts + align - 1) // align * align)])
    slot_row = np.full(slots, -1, dtype=np.int64)
    row_slot = np.full(R, -1, dtype=np.int64)
    block = np.full(R // align, -1, dtype=np.int64)
    for e in range(E):
        mine = np.flatnonzero(flat == e)
        slot_row[mine] = offsets[e] + np.arange(len(mine))
        row_slot[offsets[e]:offsets[e] + len(mine)] = mine
        block[offsets[e] // align:offsets[e + 1] // align] = e
    return offsets, counts, slot_row.reshape(tokens, top), row_slot, block


def decoded(q, s, fmt):
    """float64 values of codes with MMA-layout scales (tensors), as a matrix."""
    q = q.cpu().numpy()
    q = q.reshape(-1, q.shape[-1])
    k = q.shape[1] * (2 if fmt == "e2m1" else 1)
    s = omx.sf_from_mma(s.cpu().numpy().reshape(-1), q.shape[0], k // 32)
    return omx.dequantize(q, s, FMTS[fmt])


def integer_operand(rng, rows, k, fmt):
    """Codes and scales of values whose products' sums are exact in float32 in
    any order: the values are multiples of 1/4 up to 2, so terms are multiples
    of 1/16 up to 4 and sums of up to 4096 terms take 18 bits."""
    v = rng.choice([0.0, 0.5, 1.0, 1.5, -0.5, -1.0, -2.0, 2.0], size=(rows, k))
    scale = rng.choice([126, 127], size=(rows, k // 32)).astype(np.uint8)      # 1/2, 1
    code = F.encode_rne_sat(FMTS[fmt], v)
    code = F.pack_fp4(code) if fmt == "e2m1" else code
    return torch.from_numpy(np.ascontiguousarray(code)).cuda(), torch.from_numpy(omx.sf_to_mma(scale)).cuda()
