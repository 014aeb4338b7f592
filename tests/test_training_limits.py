"""The longest rows that the training-step operators take: the kernels count a
row's elements in 32 bits and step beyond its end, so the limit leaves room
for a step.  CPU only: nothing is launched."""

import os

import pytest

import block_scaled_precision_02_gb300 as mxq

P = 0x10000          # aligned, never dereferenced
LIMIT = 2 ** 31 - 2 ** 16
REFUSED, ACCEPTED = -2, -4       # bad shape; all checks passed, but no device here


@pytest.fixture(scope="module")
def so():
    from block_scaled_precision_02_gb300 import build
    if not os.path.exists(mxq.LIB_PATH):
        build.build()
    return mxq.load()


@pytest.mark.parametrize("n,want", [(LIMIT, ACCEPTED), (LIMIT + 1, REFUSED), (2 ** 31 - 1025, REFUSED), (2 ** 31 - 1008, REFUSED),
                                    (2 ** 31 - 256, REFUSED), (2 ** 31 - 16, REFUSED), (2 ** 31, REFUSED)])
def test_longest_rows(so, n, want):
    assert so.mxq_layer_norm(P, 1, n, n, 0, P, 0, P, 0, 1e-5, 0, P, P, P, None) == want
    assert so.mxq_layer_norm_backward(P, n, 0, P, n, 0, 1, n, P, P, P, 0, P, P, P, P, 1 << 40, None) == want
    assert so.mxq_policy_loss(P, 1, n, n, 0, P, 1, P, P, P, P, 0.2, 0.2, 0.1, 1.0, P, P, P, n, 0, P, 1 << 20, None) == want
    if n % 32 == 0:
        assert so.mxq_layer_norm_mx(P, 32, n, n, 0, P, 0, P, 0, 1e-5, 0, 3, 0, 0, P, P, P, P, P, P, None) == want
