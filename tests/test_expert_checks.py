"""What the calls of a mixture-of-experts layer and dropout refuse, before any
launch.  CPU only: the binding's checks raise, and the C entry points return
their status."""

import copy
import ctypes
import os
import pickle

import pytest
import torch

import block_scaled_precision_02_gb300 as mxq

BF, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
P, ODD = 0x10000, 0x10001        # never dereferenced
BAD_ARG, BAD_SHAPE, MISALIGNED, NO_DEVICE = -1, -2, -3, -4


def z(*shape, dtype=F32):
    return torch.zeros(*shape, dtype=dtype)


def plan(tokens=4, top=2, experts=3, align=128):
    """A plan in host memory: only what a call checks before it needs a device."""
    p = object.__new__(mxq.ExpertPlan)
    slots = tokens * top
    p.tokens, p.top, p.experts, p.align = tokens, top, experts, align
    p.rows = (slots + min(experts, slots) * (align - 1)) // align * align
    p._at, p._buffer, p._pointers = [0] * 6, z(1, dtype=I32), [0] * 6
    return p


@pytest.fixture(scope="module")
def so():
    from block_scaled_precision_02_gb300 import build
    if not os.path.exists(mxq.LIB_PATH):
        build.build()
    return mxq.load()


def test_sort_checks():
    e = z(4, 2, dtype=I32)
    for bad, match in ((z(4, 2), "int32 or int64"), (None, "int32 or int64"), (z(8, dtype=I32), "contiguous"),
                       (z(4, 0, dtype=I32), "contiguous"), (z(2, 4, dtype=I32).t(), "contiguous"), (e, "CUDA tensor")):
        with pytest.raises(ValueError, match=match):
            mxq.expert_sort(bad, 8)
    for n in (0, 1025):
        with pytest.raises(ValueError, match="num_experts"):
            mxq.expert_sort(e, n)
    for a in (0, 64, 512):
        with pytest.raises(ValueError, match="align"):
            mxq.expert_sort(e, 8, a)
    with pytest.raises(ValueError, match="too many"):
        mxq.expert_sort(torch.empty(2 ** 30, 2, dtype=I32, device="meta"), 8)


def test_plan_checks():
    for bad in (None, (1, 2, 3), z(4)):
        for call in (lambda: mxq.expert_gather(z(4, 8), bad), lambda: mxq.expert_combine(z(4, 8), bad),
                     lambda: mxq.mx_expert_gather(z(4, 8), bad), lambda: mxq.expert_combine_backward(z(4, 8), z(4, 8), bad, z(4, 2)),
                     lambda: mxq.mx_expert_gemm(z(4, 8), z(1), z(1), z(1), bad),
                     lambda: mxq.mx_expert_wgrad(z(4, 8), z(1), z(1), z(1), bad)):
            with pytest.raises(ValueError, match="what expert_sort returned"):
                call()


def test_row_calls_checks():
    p = plan()
    R = p.rows
    with pytest.raises(ValueError, match="x has 5 rows, the plan 4 tokens"):
        mxq.expert_gather(z(5, 8), p)
    with pytest.raises(ValueError, match="bf16 or float32"):
        mxq.expert_gather(z(4, 8, dtype=torch.float16), p)
    with pytest.raises(ValueError, match="CUDA tensor"):
        mxq.expert_gather(z(4, 8), p)
    with pytest.raises(ValueError, match="must be bf16"):
        mxq.mx_expert_gather(z(4, 128), p)
    with pytest.raises(ValueError, match="unknown orientation"):
        mxq.mx_expert_gather(z(4, 128, dtype=BF), p, orientation="both")
    with pytest.raises(ValueError, match="CUDA tensor"):
        mxq.mx_expert_gather(z(4, 128, dtype=BF), p)
    with pytest.raises(ValueError, match="rows has 4 rows"):
        mxq.expert_combine(z(4, 8), p)
    for w, match in ((z(4, 3), "weights are"), (z(8), "weights are"), (z(4, 2, dtype=torch.float64), "weights must be"),
                     (z(2, 4).t(), "weights must be")):
        with pytest.raises(ValueError, match=match):
            mxq.expert_combine(z(R, 8), p, w)
        with pytest.raises(ValueError, match=match):
            mxq.expert_combine_backward(z(4, 8), z(R, 8), p, w)
    with pytest.raises(ValueError, match="out_dtype"):
        mxq.expert_combine(z(R, 8), p, out_dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        mxq.expert_combine(z(R, 8), p, z(4, 2))
    with pytest.raises(ValueError, match="dy has 8 columns, rows 9"):
        mxq.expert_combine_backward(z(4, 8), z(R, 9), p, z(4, 2))
    with pytest.raises(ValueError, match="weights must be"):
        mxq.expert_combine_backward(z(4, 8), z(R, 8), p, None)


def test_product_checks():
    p = plan()
    R, E, N, K = p.rows, p.experts, 128, 256
    a, sa = z(R, K, dtype=U8), z(R * K // 32, dtype=U8)
    b, sb = z(E, N, K, dtype=U8), z(E * N * K // 32, dtype=U8)
    ok = dict(a_q=a, a_s=sa, b_q=b, b_s=sb, plan=p)
    for key, bad, match in (("a_q", z(R - 1, K, dtype=U8), "a_s holds"), ("a_q", z(R, K), "1-byte"), ("a_q", b, "2-D"),
                            ("a_s", z(R, dtype=U8), "a_s holds"), ("b_s", z(N, dtype=U8), "b_s holds"),
                            ("b_q", z(N, K, dtype=U8), "b_s holds"), ("b_q", z(E * N * K, dtype=U8), "2-D or 3-D"),
                            ("out_dtype", torch.float16, "out_dtype"), ("fmt", "e3m4", "unknown format"),
                            ("a_q", a, "CUDA tensor")):
        with pytest.raises(ValueError, match=match):
            mxq.mx_expert_gemm(**{**ok, key: bad})
    with pytest.raises(ValueError, match="a_q has 512 rows"):
        mxq.mx_expert_gemm(**{**ok, "a_q": z(512, K, dtype=U8), "a_s": z(512 * K // 32, dtype=U8)})
    with pytest.raises(ValueError, match="holds 2 experts"):
        mxq.mx_expert_gemm(**{**ok, "b_q": z(2, N, K, dtype=U8), "b_s": z(2 * N * K // 32, dtype=U8)})
    with pytest.raises(ValueError, match="K differs"):
        mxq.mx_expert_gemm(**{**ok, "b_q": z(E, N, 128, dtype=U8), "b_s": z(E * N * 4, dtype=U8)})
    with pytest.raises(ValueError, match="K differs.*for 3 experts"):
        mxq.mx_expert_gemm(**{**ok, "b_q": z(N, K, dtype=U8), "b_s": z(N * K // 32, dtype=U8)})
    g, sg = z(N, R, dtype=U8), z(N * R // 32, dtype=U8)
    for key, bad, match in (("a_q", b, "2-D"), ("b_s", sa, "b_s holds"), ("out_dtype", BF, "CUDA tensor")):
        with pytest.raises(ValueError, match=match):
            mxq.mx_expert_wgrad(**{**dict(a_q=g, a_s=sg, b_q=g, b_s=sg, plan=p), key: bad})
    with pytest.raises(ValueError, match="a_q holds 128 rows"):
        mxq.mx_expert_wgrad(z(N, 128, dtype=U8), z(N * 4, dtype=U8), g, sg, p)


def test_dropout_checks():
    x = z(4, 8)
    for p in (-0.1, 1.0, 2.0, float("nan")):
        with pytest.raises(ValueError, match=r"\[0, 1\)"):
            mxq.dropout(x, p, 0)
    for r in (z(4, 9), z(4, 8, dtype=BF)):
        with pytest.raises(ValueError, match="residual must have"):
            mxq.dropout(x, 0.1, 0, residual=r)
    for o in (z(1), z(2, dtype=torch.int64)):
        with pytest.raises(ValueError, match="offset must be"):
            mxq.dropout(x, 0.1, 0, o)
    with pytest.raises(ValueError, match="bf16 or float32"):
        mxq.dropout(z(4, 8, dtype=torch.float16), 0.1, 0)
    with pytest.raises(ValueError, match="CUDA tensor"):
        mxq.dropout(x, 0.1, 0)


def test_c_sort(so):
    rows = ctypes.c_int64()
    R = lambda s, e, a: (so.mxq_expert_rows(s, e, a, ctypes.byref(rows)), rows.value)
    assert R(0, 8, 128) == (0, 0)
    assert R(1, 8, 128) == (0, 128)
    assert R(9, 8, 128) == (0, 1024)              # 8 experts: 9 + 8 * 127 = 1025
    assert R(1000, 1, 256) == (0, 1024)
    for s, e, a, want in ((-1, 8, 128, BAD_SHAPE), (4, 0, 128, BAD_SHAPE), (4, 1025, 128, BAD_SHAPE), (4, 8, 64, BAD_ARG),
                          (2 ** 31, 8, 128, BAD_SHAPE), (2 ** 31 - 2 ** 16, 1024, 256, BAD_SHAPE)):
        assert R(s, e, a)[0] == want
    assert so.mxq_expert_rows(1, 1, 128, None) == BAD_ARG
    n = ctypes.c_size_t()
    assert so.mxq_expert_sort_workspace_size(100000, 64, ctypes.byref(n)) == 0 and n.value >= 64 * 4
    ok = [P, 0, 9, 8, 128, 1024, P, P, P, P, P, P, 1 << 20, None]
    assert so.mxq_expert_sort(*ok) == NO_DEVICE
    for at, bad, want in ((1, 2, BAD_ARG), (5, 1152, BAD_SHAPE), (0, None, BAD_ARG), (6, None, BAD_ARG), (9, None, BAD_ARG),
                          (11, None, BAD_ARG), (12, 8, BAD_ARG), (0, 0x10002, MISALIGNED), (8, ODD, MISALIGNED),
                          (11, 0x10008, MISALIGNED)):
        assert so.mxq_expert_sort(*[bad if i == at else v for i, v in enumerate(ok)]) == want, at


def test_c_rows(so):
    def each(fn, ok, cases):
        assert fn(*ok) == NO_DEVICE
        for at, bad, want in cases:
            assert fn(*[bad if i == at else v for i, v in enumerate(ok)]) == want, at

    each(so.mxq_expert_gather, [P, 4, 8, 8, 1, P, 2, P, P, 3, 384, P, None],
         ((4, 2, BAD_ARG), (1, -1, BAD_SHAPE), (2, 0, BAD_SHAPE), (3, 7, BAD_SHAPE), (6, 0, BAD_SHAPE), (0, None, BAD_ARG),
          (5, None, BAD_ARG), (7, None, BAD_ARG), (8, None, BAD_ARG), (9, 0, BAD_SHAPE), (9, 1025, BAD_SHAPE), (11, None, BAD_ARG),
          (0, 0x10002, MISALIGNED), (11, ODD, MISALIGNED), (7, ODD, MISALIGNED), (1, 2 ** 30, BAD_SHAPE)))
    each(so.mxq_expert_gather_mx, [P, 4, 128, 128, P, 384, 2, 0, 3, 0, 1, P, P, P, P, None],
         ((7, 3, BAD_ARG), (8, 0, BAD_ARG), (9, 2, BAD_ARG), (10, 2, BAD_ARG), (5, 32, BAD_SHAPE), (2, 160, BAD_SHAPE),
          (3, 64, BAD_SHAPE), (3, 132, MISALIGNED), (0, 0x10008, MISALIGNED), (11, 0x10008, MISALIGNED), (13, 0x10008, MISALIGNED),
          (0, None, BAD_ARG), (4, None, BAD_ARG), (12, None, BAD_ARG), (14, None, BAD_ARG),
          (12, 0x10008, MISALIGNED), (14, 0x10008, MISALIGNED)))
    each(so.mxq_expert_combine, [P, 384, 8, 8, 1, P, 4, 2, P, 1, P, 0, None],
         ((4, 2, BAD_ARG), (9, 2, BAD_ARG), (11, 2, BAD_ARG), (2, 0, BAD_SHAPE), (3, 7, BAD_SHAPE), (0, None, BAD_ARG),
          (5, None, BAD_ARG), (10, None, BAD_ARG), (8, 0x10002, MISALIGNED), (10, ODD, MISALIGNED)))
    each(so.mxq_expert_combine_backward, [P, 8, 0, P, 8, 1, 384, 8, P, 4, 2, P, P, 3, P, 1, P, P, None],
         ((1, 7, BAD_SHAPE), (4, 7, BAD_SHAPE), (2, 2, BAD_ARG), (5, 2, BAD_ARG), (15, 2, BAD_ARG), (0, None, BAD_ARG),
          (3, None, BAD_ARG), (8, None, BAD_ARG), (11, None, BAD_ARG), (12, None, BAD_ARG), (13, 0, BAD_SHAPE), (14, None, BAD_ARG),
          (16, None, BAD_ARG), (17, None, BAD_ARG), (0, ODD, MISALIGNED), (17, 0x10002, MISALIGNED)))
    each(so.mxq_dropout, [P, 4, 8, 8, 0, P, 8, 0.1, 1, 2, P, P, None],
         ((4, 2, BAD_ARG), (7, 1.0, BAD_ARG), (7, float("nan"), BAD_ARG), (1, -1, BAD_SHAPE), (2, 0, BAD_SHAPE), (3, 7, BAD_SHAPE),
          (6, 7, BAD_SHAPE), (0, None, BAD_ARG), (11, None, BAD_ARG), (0, ODD, MISALIGNED), (10, 0x10004, MISALIGNED)))
    assert so.mxq_dropout(None, 0, 8, 8, 0, None, 0, 0.1, 1, 2, None, None, None) == 0


def test_c_products(so):
    #     0  1  2  3  4  5   6    7    8   9  10  11 12 13 14 15
    ok = [P, P, 0, P, P, 0, 256, 128, 128, 3, 128, P, P, 0, P, 0, None]
    assert so.mxq_expert_gemm(*ok) == NO_DEVICE
    for at, bad, want in ((2, 3, BAD_ARG), (5, -1, BAD_ARG), (6, 200, BAD_SHAPE), (7, 64, BAD_SHAPE), (8, 130, BAD_SHAPE),
                          (9, 0, BAD_SHAPE), (9, 1025, BAD_SHAPE), (10, 64, BAD_ARG), (13, 2, BAD_ARG), (15, 2, BAD_ARG),
                          (0, None, BAD_ARG), (3, None, BAD_ARG), (11, None, BAD_ARG), (12, None, BAD_ARG), (14, None, BAD_ARG),
                          (0, 0x10008, MISALIGNED), (4, 0x10008, MISALIGNED), (14, 0x10008, MISALIGNED), (11, ODD, MISALIGNED),
                          (12, ODD, MISALIGNED), (7, 2 ** 30, BAD_SHAPE), (8, 2 ** 30, BAD_SHAPE)):
        assert so.mxq_expert_gemm(*[bad if i == at else v for i, v in enumerate(ok)]) == want, at
    fp4 = [P, P, 2, P, P, 2, 256, 128, 128, 3, 128, P, P, 0, P, 0, None]
    assert so.mxq_expert_gemm(*fp4) == BAD_SHAPE                     # both E2M1: K % 256
    assert so.mxq_expert_gemm(*[0x10010 if i == 3 else 0 if i == 2 else v for i, v in enumerate(fp4)]) == MISALIGNED
    wg = [P, P, 0, P, P, 0, 256, 128, 128, 3, 128, P, P, 0, None]
    assert so.mxq_expert_wgrad(*wg) == NO_DEVICE
    assert so.mxq_expert_wgrad(*[2 if i in (2, 5) else v for i, v in enumerate(wg)]) == BAD_SHAPE      # both E2M1: align 256
    assert so.mxq_expert_wgrad(*[None if i == 12 else v for i, v in enumerate(wg)]) == BAD_ARG
    assert so.mxq_expert_wgrad(*[200 if i == 6 else v for i, v in enumerate(wg)]) == BAD_SHAPE


def test_plan_is_not_copied():
    # a copy's addresses would be the original's, whose memory may be gone
    p = plan()
    for call in (copy.copy, copy.deepcopy, pickle.dumps):
        with pytest.raises(TypeError, match="copied or pickled"):
            call(p)


def test_c_backward_reads_the_stretches_whenever_it_runs(so):
    # tokens without rows, rows without tokens: both launch, and every launch reads offsets and counts
    none = [P, 8, 0, None, 8, 1, 0, 8, P, 4, 2, P, P, 3, P, 1, None, P, None]
    rest = [None, 8, 0, P, 8, 1, 384, 8, None, 0, 2, P, P, 3, None, 1, P, None, None]
    for ok in (none, rest):
        for at in (11, 12):
            assert so.mxq_expert_combine_backward(*[None if i == at else v for i, v in enumerate(ok)]) == BAD_ARG, at
        assert so.mxq_expert_combine_backward(*ok) == NO_DEVICE
    # nothing to do: nothing is needed
    idle = [None, 8, 0, None, 8, 1, 0, 8, None, 0, 2, None, None, 3, None, 1, None, None, None]
    assert so.mxq_expert_combine_backward(*idle) in (0, NO_DEVICE)


def test_c_stall_hook_covers_the_products(so):
    assert [so.mxq_test_stall_next_launch(w) for w in (3, 0, 4, -1)] == [0, 0, BAD_ARG, BAD_ARG]
