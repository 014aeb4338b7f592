"""Calls of a mixture-of-experts layer: tokens sorted by expert and gathered
into rows (plain or as MX operands), the experts' block-scaled products in one
call, the gradient of their weights, and the way back to tokens.  Argument
marshalling only, as in the package."""

from __future__ import annotations

from typing import Optional

import torch

from . import (_FMT, _ORIENT, _PARAM, _SCALE, _SF, _TYPE, COL, E2M1, ROW, _byte_tensor, _launch, _matrix,
               _same_device, _size)

MAX_EXPERTS = 1024
_LIMIT = 2 ** 31 - 2 ** 16
_INDEX = {torch.int32: 0, torch.int64: 1}


class ExpertPlan:
    """Where expert_sort puts every slot (slot s = token * top + j).

    tokens, top, experts, align   as given
    rows          rows of gathered tensors: enough for any routing of this size
    and int32 tensors, parts of one allocation:
    offsets       [experts + 1] first row of each expert's stretch, and the end of the last
    counts        [experts] slots of each expert
    slot_row      [tokens][top] row of each slot, -1 where it is dropped
    row_slot      [rows] slot of each row, -1 in padding and behind the last stretch
    block_expert  [rows / align] expert of each block of rows, -1 behind the last stretch

    A plan is neither copied nor pickled (its addresses are those of its own
    allocation): sort again, or keep the tensors."""

    __slots__ = ("_buffer", "_at", "_pointers", "tokens", "top", "experts", "rows", "align")

    def __init__(self, tokens: int, top: int, experts: int, align: int, device):
        slots = tokens * top
        rows = (slots + min(experts, slots) * (align - 1)) // align * align
        if rows > _LIMIT:
            raise ValueError("too many slots")
        # where each tensor starts, then the sort's workspace (at 16 bytes), then the end
        a1 = experts + 1
        a2 = a1 + experts
        a3 = a2 + slots
        a4 = a3 + rows
        a5 = (a4 + rows // align + 3) // 4 * 4
        end = a5 + (_size("mxq_expert_sort_workspace_size", device, slots, experts) + 3) // 4
        self._buffer = torch.empty(end, dtype=torch.int32, device=device)
        p = self._buffer.data_ptr()
        self._at = (0, a1, a2, a3, a4, a5, end)
        self._pointers = (p, p + 4 * a1, p + 4 * a2, p + 4 * a3, p + 4 * a4, p + 4 * a5)
        self.tokens, self.top, self.experts, self.rows, self.align = tokens, top, experts, rows, align

    def __reduce_ex__(self, protocol):
        raise TypeError("a plan cannot be copied or pickled: it holds its allocation's addresses")

    @property
    def offsets(self):
        return self._buffer.as_strided((self.experts + 1,), (1,), 0)

    @property
    def counts(self):
        return self._buffer.as_strided((self.experts,), (1,), self._at[1])

    @property
    def slot_row(self):
        return self._buffer.as_strided((self.tokens, self.top), (self.top, 1), self._at[2])

    @property
    def row_slot(self):
        return self._buffer.as_strided((self.rows,), (1,), self._at[3])

    @property
    def block_expert(self):
        return self._buffer.as_strided((self.rows // self.align,), (1,), self._at[4])


def expert_sort(experts: torch.Tensor, num_experts: int, align: Optional[int] = None) -> ExpertPlan:
    """Sort the slots of a routing ``experts`` [tokens][top] (int32 or int64) by
    expert.  An expert's slots keep their order; its rows start at a multiple
    of ``align``: 128, or 256 for the products' larger tiles (the default from
    256 slots an expert on, where they outweigh the longer padding).  An index
    outside [0, num_experts) drops the slot."""
    if not isinstance(experts, torch.Tensor) or experts.dtype not in _INDEX:
        raise ValueError("experts must be an int32 or int64 tensor")
    if experts.dim() != 2 or experts.shape[1] < 1 or not experts.is_contiguous():
        raise ValueError("experts must be a contiguous [tokens][top] tensor")
    if not 1 <= num_experts <= MAX_EXPERTS:
        raise ValueError(f"num_experts must lie in 1 .. {MAX_EXPERTS}")
    tokens, top = experts.shape
    if align is None:
        align = 256 if tokens * top >= 256 * num_experts else 128
    elif align not in (128, 256):
        raise ValueError("align must be 128 or 256")
    if tokens * top > _LIMIT:
        raise ValueError("too many slots")
    dev = _same_device("experts", experts)
    plan = ExpertPlan(tokens, top, num_experts, align, dev)
    at = plan._at
    _launch("mxq_expert_sort", dev, experts.data_ptr(), _INDEX[experts.dtype], tokens * top, num_experts, align, plan.rows,
            *plan._pointers, 4 * (at[6] - at[5]))
    return plan


def _plan(plan) -> ExpertPlan:
    if type(plan) is not ExpertPlan:
        raise ValueError("plan must be what expert_sort returned")
    return plan


def _rows_of(t: torch.Tensor, name: str, n: int, what: str):
    code, rows, cols, ld = _matrix(t, name)
    if rows != n:
        raise ValueError(f"{name} has {rows} rows, the plan {n} {what}")
    return code, cols, ld


def _gate(weights: torch.Tensor, plan: ExpertPlan):
    """(pointer, type code) of the gate's weights [tokens][top]."""
    if not isinstance(weights, torch.Tensor) or weights.dtype not in _PARAM or not weights.is_contiguous():
        raise ValueError("weights must be a contiguous float32 or bfloat16 tensor")
    if tuple(weights.shape) != (plan.tokens, plan.top):
        raise ValueError(f"weights are {tuple(weights.shape)}, the plan's slots {(plan.tokens, plan.top)}")
    return weights.data_ptr(), _TYPE[weights.dtype]


def expert_gather(x: torch.Tensor, plan: ExpertPlan) -> torch.Tensor:
    """Rows by expert [plan.rows][cols] of tokens ``x`` [tokens][cols] (bf16 or
    float32, row stride may exceed cols), every token in the row of each of its
    slots, zeros in padding.  Its backward pass is expert_combine(drows, plan)."""
    plan = _plan(plan)
    xt, cols, ld = _rows_of(x, "x", plan.tokens, "tokens")
    dev = _same_device("x plan", x, plan._buffer)
    out = torch.empty(plan.rows, cols, dtype=x.dtype, device=dev)
    at = plan._pointers
    _launch("mxq_expert_gather", dev, x.data_ptr(), plan.tokens, cols, ld, xt, at[2], plan.top, at[0], at[1], plan.experts,
            plan.rows, out.data_ptr())
    return out


def mx_expert_gather(x: torch.Tensor, plan: ExpertPlan, fmt="e4m3", orientation="row", scale_mode="floor",
                     sf_layout="canonical"):
    """expert_gather of bf16 ``x`` straight to MX operands: (q_row, s_row, q_col,
    s_col), byte for byte mx_quantize(expert_gather(x, plan), ...), without the
    bf16 rows in memory.  The row copy is mx_expert_gemm's operand, the column
    copy mx_expert_wgrad's."""
    plan = _plan(plan)
    f, o = _FMT[fmt], _ORIENT[orientation]
    sm, sf = _SCALE[scale_mode], _SF[sf_layout]
    _, cols, ld = _rows_of(x, "x", plan.tokens, "tokens")
    if x.dtype != torch.bfloat16:
        raise ValueError("x must be bf16 with a contiguous last dimension")
    dev = _same_device("x plan", x, plan._buffer)
    rows, qb = plan.rows, 2 if f == E2M1 else 1
    q_row = s_row = q_col = s_col = None
    rp = rs = cp = cs = 0
    if o & ROW:
        q_row = torch.empty(rows, cols // qb, dtype=torch.uint8, device=dev)
        s_row = torch.empty(rows, cols // 32, dtype=torch.uint8, device=dev)
        rp, rs = q_row.data_ptr(), s_row.data_ptr()
    if o & COL:
        q_col = torch.empty(cols, rows // qb, dtype=torch.uint8, device=dev)
        s_col = torch.empty(cols, rows // 32, dtype=torch.uint8, device=dev)
        cp, cs = q_col.data_ptr(), s_col.data_ptr()
    _launch("mxq_expert_gather_mx", dev, x.data_ptr(), plan.tokens, cols, ld, plan._pointers[3], rows, plan.top, f, o,
            sm, sf, rp, rs, cp, cs)
    return q_row, s_row, q_col, s_col


def expert_combine(rows: torch.Tensor, plan: ExpertPlan, weights: Optional[torch.Tensor] = None,
                   out_dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """Tokens [tokens][cols] from ``rows`` [plan.rows][cols]: the sum of a
    token's slots' rows times ``weights`` [tokens][top] (float32 or bf16; 1 where
    None), added in float32 in the slots' order and rounded once to
    ``out_dtype`` (rows' type by default).  Dropped slots add nothing."""
    plan = _plan(plan)
    t, cols, ld = _rows_of(rows, "rows", plan.rows, "rows")
    w, wt = (0, 0) if weights is None else _gate(weights, plan)
    out_dtype = rows.dtype if out_dtype is None else out_dtype
    if out_dtype not in _TYPE:
        raise ValueError("out_dtype must be torch.float32 or torch.bfloat16")
    dev = _same_device("rows plan weights", rows, plan._buffer, weights)
    y = torch.empty(plan.tokens, cols, dtype=out_dtype, device=dev)
    _launch("mxq_expert_combine", dev, rows.data_ptr(), plan.rows, cols, ld, t, plan._pointers[2], plan.tokens,
            plan.top, w, wt, y.data_ptr(), _TYPE[out_dtype])
    return y


def expert_combine_backward(dy: torch.Tensor, rows: torch.Tensor, plan: ExpertPlan, weights: torch.Tensor):
    """Backward pass of expert_combine with weights: (drows, dweights) from
    ``dy`` [tokens][cols] and the forward pass's ``rows`` and ``weights``.  drows
    [plan.rows][cols] has rows' type (zeros in padding), dweights is float32
    [tokens][top].  (Without weights it is expert_gather(dy, plan).)"""
    plan = _plan(plan)
    dt, cols, ld_dy = _rows_of(dy, "dy", plan.tokens, "tokens")
    t, rcols, ld = _rows_of(rows, "rows", plan.rows, "rows")
    if rcols != cols:
        raise ValueError(f"dy has {cols} columns, rows {rcols}")
    w, wt = _gate(weights, plan)
    dev = _same_device("rows dy plan weights", rows, dy, plan._buffer, weights)
    drows = torch.empty(plan.rows, cols, dtype=rows.dtype, device=dev)
    dw = torch.empty(plan.tokens, plan.top, dtype=torch.float32, device=dev)
    at = plan._pointers
    _launch("mxq_expert_combine_backward", dev, dy.data_ptr(), ld_dy, dt, rows.data_ptr(), ld, t, plan.rows, cols,
            at[2], plan.tokens, plan.top, at[0], at[1], plan.experts, w, wt, drows.data_ptr(), dw.data_ptr())
    return drows, dw


def _codes(q: torch.Tensor, s: torch.Tensor, name: str, fmt: int, dims) -> tuple:
    """Shape of an operand in elements (its last axis unpacked), after checking
    its codes and that its scales hold a byte for every 32 of them."""
    if not isinstance(q, torch.Tensor) or q.dim() not in dims:
        raise ValueError(f"{name}_q must be a {' or '.join(f'{d}-D' for d in dims)} tensor of codes")
    _byte_tensor(q, f"{name}_q")
    shape = (*q.shape[:-1], q.shape[-1] * (2 if fmt == E2M1 else 1))
    _byte_tensor(s, f"{name}_s", q.numel() * (2 if fmt == E2M1 else 1) // 32)
    return shape


def mx_expert_gemm(a_q: torch.Tensor, a_s: torch.Tensor, b_q: torch.Tensor, b_s: torch.Tensor, plan: ExpertPlan,
                   fmt="e4m3", b_fmt=None, out_dtype=torch.bfloat16) -> torch.Tensor:
    """C [plan.rows][N]: the rows of A [plan.rows][K] times their expert's
    weights, all experts in one launch; zeros behind the last stretch.

    B is [experts][N][K], or, for the backward pass, [N][experts * K]: the column
    copy that mx_quantize makes of the weights stacked as [experts * K][N].
    Scales in the MMA layout; formats as mx_gemm; N and K multiples of 128."""
    plan = _plan(plan)
    f = _FMT[fmt]
    fb = f if b_fmt is None else _FMT[b_fmt]
    if out_dtype not in _TYPE:
        raise ValueError("out_dtype must be torch.bfloat16 or torch.float32")
    R, K = _codes(a_q, a_s, "a", f, (2,))
    b_shape = _codes(b_q, b_s, "b", fb, (2, 3))
    if R != plan.rows:
        raise ValueError(f"a_q has {R} rows, the plan {plan.rows} rows")
    N = b_shape[-2]
    along_k = len(b_shape) == 2
    if not along_k and b_shape[0] != plan.experts:
        raise ValueError(f"b_q holds {b_shape[0]} experts, the plan {plan.experts}")
    if b_shape[-1] != (plan.experts * K if along_k else K):
        raise ValueError(f"K differs: a_q holds {K}, b_q {b_shape[-1]}" + (f" for {plan.experts} experts" if along_k else ""))
    dev = _same_device("a_q a_s b_q b_s plan", a_q, a_s, b_q, b_s, plan._buffer)
    c = torch.empty(R, N, dtype=out_dtype, device=dev)
    at = plan._pointers
    _launch("mxq_expert_gemm", dev, a_q.data_ptr(), a_s.data_ptr(), f, b_q.data_ptr(), b_s.data_ptr(), fb, R, N, K,
            plan.experts, plan.align, at[0], at[4], int(along_k), c.data_ptr(),
            int(out_dtype == torch.float32))
    return c


def mx_expert_wgrad(a_q: torch.Tensor, a_s: torch.Tensor, b_q: torch.Tensor, b_s: torch.Tensor, plan: ExpertPlan,
                    fmt="e4m3", b_fmt=None, out_dtype=torch.float32) -> torch.Tensor:
    """Gradient [experts][N][K] of the experts' weights from the column copies
    of the rows' gradients, A [N][plan.rows], and of the rows, B [K][plan.rows]
    (mx_quantize's and mx_expert_gather's q_col and s_col, MMA layout): for every
    expert the product over its own rows, zeros where it has none.  Formats as
    mx_gemm (two E2M1 operands want a plan with align 256)."""
    plan = _plan(plan)
    f = _FMT[fmt]
    fb = f if b_fmt is None else _FMT[b_fmt]
    if out_dtype not in _TYPE:
        raise ValueError("out_dtype must be torch.bfloat16 or torch.float32")
    N, ra = _codes(a_q, a_s, "a", f, (2,))
    K, rb = _codes(b_q, b_s, "b", fb, (2,))
    for n, name in ((ra, "a_q"), (rb, "b_q")):
        if n != plan.rows:
            raise ValueError(f"{name} holds {n} rows, the plan {plan.rows}")
    dev = _same_device("a_q a_s b_q b_s plan", a_q, a_s, b_q, b_s, plan._buffer)
    c = torch.empty(plan.experts, N, K, dtype=out_dtype, device=dev)
    _launch("mxq_expert_wgrad", dev, a_q.data_ptr(), a_s.data_ptr(), f, b_q.data_ptr(), b_s.data_ptr(), fb, plan.rows, N, K,
            plan.experts, plan.align, plan._pointers[0], c.data_ptr(), int(out_dtype == torch.float32))
    return c
