"""What the training-step operators refuse, before any launch.  CPU only: the
binding's checks raise, and the C entry points return their status."""

import ctypes

import pytest
import torch

import block_scaled_precision_02_gb300 as mxq

BF, F32 = torch.bfloat16, torch.float32


def z(*shape, dtype=F32):
    return torch.zeros(*shape, dtype=dtype)


def test_norm_checks():
    with pytest.raises(ValueError, match="x must be a bf16 or float32"):
        mxq.layer_norm(z(4, 8, dtype=torch.float16))
    with pytest.raises(ValueError, match="2-D with contiguous rows"):
        mxq.layer_norm(z(4))
    with pytest.raises(ValueError, match="2-D with contiguous rows"):
        mxq.layer_norm(z(4, 8).t())
    with pytest.raises(ValueError, match="2-D with contiguous rows"):
        mxq.layer_norm(z(1, 8).expand(4, 8))
    with pytest.raises(ValueError, match="at least one column"):
        mxq.layer_norm(z(4, 0))
    with pytest.raises(ValueError, match="weight holds 7 elements, expected 8"):
        mxq.layer_norm(z(4, 8), z(7))
    with pytest.raises(ValueError, match="bias must be a contiguous"):
        mxq.layer_norm(z(4, 8), z(8), z(8, dtype=torch.float64))
    with pytest.raises(ValueError, match="CUDA tensor"):
        mxq.layer_norm(z(4, 8), z(8), z(8))
    with pytest.raises(ValueError, match="unknown format"):
        mxq.mx_layer_norm(z(32, 32), fmt="e3m4")
    with pytest.raises(ValueError, match="unknown orientation"):
        mxq.mx_layer_norm(z(32, 32), orientation="both")
    with pytest.raises(ValueError, match="unknown scale layout"):
        mxq.mx_layer_norm(z(32, 32), sf_layout="tiled")
    with pytest.raises(ValueError, match="CUDA tensor"):
        mxq.mx_layer_norm(z(32, 32))


def test_norm_backward_checks():
    x = z(4, 8)
    with pytest.raises(ValueError, match=r"dy is \(4, 7\)"):
        mxq.layer_norm_backward(z(4, 7), x, z(4), z(4))
    with pytest.raises(ValueError, match="mean holds 3"):
        mxq.layer_norm_backward(x, x, z(3), z(4))
    with pytest.raises(ValueError, match="forward pass"):
        mxq.layer_norm_backward(x, x, None, z(4))
    with pytest.raises(ValueError, match="rstd must be a contiguous float32"):
        mxq.layer_norm_backward(x, x, z(4), z(4, dtype=BF))
    with pytest.raises(ValueError, match="CUDA tensor"):
        mxq.layer_norm_backward(x, x, z(4), z(4), z(8))


def test_policy_loss_checks():
    ok = dict(logits=z(4, 8), targets=z(4, dtype=torch.int64), old_logp=z(4), advantages=z(4), weights=z(4))
    for key, bad, match in (("logits", z(4, 8, dtype=torch.float16), "logits must be"),
                            ("logits", z(4, 0), "at least one column"),
                            ("targets", z(4), "targets must be"), ("targets", None, "targets is needed"),
                            ("targets", z(3, dtype=torch.int64), "targets holds 3"),
                            ("old_logp", z(4, dtype=BF), "old_logp must be"), ("old_logp", None, "old_logp is needed"),
                            ("advantages", z(5), "advantages holds 5"), ("weights", z(4, 1), "weights must be"),
                            ("weights", z(8)[::2], "weights must be"), ("beta", 0.1, "ref_logp is needed"),
                            ("clip_low", -0.1, "must not be negative"), ("clip_high", float("nan"), "must not be negative"),
                            ("grad_dtype", torch.float16, "grad_dtype"), ("logits", z(4, 8), "CUDA tensor")):
        with pytest.raises(ValueError, match=match):
            mxq.policy_loss(**{**ok, key: bad})


def test_clip_checks():
    with pytest.raises(ValueError, match="at least one"):
        mxq.grad_norm([])
    with pytest.raises(ValueError, match=r"grads\[1\] must be a bf16 or float32"):
        mxq.grad_norm([z(4), z(4, dtype=torch.float64)])
    with pytest.raises(ValueError, match="CUDA tensor"):
        mxq.grad_norm([z(4)])
    with pytest.raises(ValueError, match="fill its storage"):
        mxq.grad_norm([z(8)[::2]])
    with pytest.raises(ValueError, match=r"out\[0\] holds 5 elements, grads\[0\] 4"):
        mxq.clip_grad_norm([z(4)], 1.0, out=[z(5)])
    with pytest.raises(ValueError, match="shape and strides"):
        mxq.clip_grad_norm([z(4, 8).t()], 1.0, out=[z(8, 4)])
    with pytest.raises(ValueError, match=r"out\[1\] must be a bf16 or float32"):
        mxq.clip_grad_norm([z(4), z(4)], 1.0, out=[z(4), z(4, dtype=torch.int32)])
    with pytest.raises(ValueError, match=r"grads\[0\] must be a bf16 or float32"):
        mxq.grad_norm([3.0])
    with pytest.raises(ValueError, match="1 gradients, 2 outputs"):
        mxq.clip_grad_norm([z(4)], 1.0, out=[z(4), z(4)])
    with pytest.raises(ValueError, match="must not be negative"):
        mxq.clip_grad_norm([z(4)], -1.0)
    with pytest.raises(ValueError, match="must not be negative"):
        mxq.clip_grad_norm([z(4)], float("nan"))


P = 0x10000          # aligned, never dereferenced


@pytest.fixture(scope="module")
def so():
    import os
    from block_scaled_precision_02_gb300 import build
    if not os.path.exists(mxq.LIB_PATH):
        build.build()
    return mxq.load()


def test_c_norm_statuses(so):
    f = so.mxq_layer_norm
    #      x  rows cols ld xt  w wt  b bt  eps  yt y  mean rstd stream
    ok = [P, 4, 8, 8, 0, P, 0, P, 1, 1e-5, 0, P, P, P, None]

    def call(**kw):
        a = list(ok)
        for k, v in kw.items():
            a[int(k[1:])] = v
        return f(*a)

    assert call(_0=None) == -1 and call(_4=2) == -1 and call(_6=5) == -1 and call(_10=3) == -1
    assert call(_11=None) == -1 and call(_12=None) == -1
    assert call(_1=-1) == -2 and call(_2=0) == -2 and call(_3=7) == -2 and call(_1=1 << 40) == -2
    assert call(_0=P + 1) == -3 and call(_11=P + 1) == -3 and call(_13=P + 2) == -3
    assert call() == -4                                          # no device here

    g = so.mxq_layer_norm_mx
    ok2 = [P, 32, 64, 64, 0, P, 0, P, 0, 1e-5, 0, 3, 0, 0, P, P, P, P, P, P, None]

    def mx(**kw):
        a = list(ok2)
        for k, v in kw.items():
            a[int(k[1:])] = v
        return g(*a)

    assert mx(_10=3) == -1 and mx(_11=0) == -1 and mx(_12=2) == -1 and mx(_13=2) == -1
    assert mx(_14=None) == -1 and mx(_17=None) == -1 and mx(_11=1, _16=None, _17=None) == -4
    assert mx(_1=33) == -2 and mx(_2=48) == -2 and mx(_1=0) == -2 and mx(_13=1) == -2
    assert mx(_0=P + 8) == -3 and mx(_3=68) == -3 and mx(_14=P + 8) == -3 and mx(_5=P + 2) == -3
    assert mx() == -4


def test_c_norm_backward_statuses(so):
    f = so.mxq_layer_norm_backward
    #     dy ld dt  x ld xt rows cols mean rstd w wt dx dw db ws bytes stream
    ok = [P, 8, 0, P, 8, 0, 4, 8, P, P, P, 0, P, P, P, P, 1 << 30, None]

    def call(**kw):
        a = list(ok)
        for k, v in kw.items():
            a[int(k[1:])] = v
        return f(*a)

    assert call(_0=None) == -1 and call(_2=7) == -1 and call(_12=None) == -1 and call(_8=None) == -1
    assert call(_15=None) == -1 and call(_16=8) == -1
    assert call(_1=7) == -2 and call(_4=7) == -2 and call(_7=0) == -2
    assert call(_15=P + 8) == -3 and call(_13=P + 2) == -3
    assert call() == -4
    assert call(_13=None, _14=None, _15=None, _16=0) == -4       # dx alone needs no workspace
    assert so.mxq_layer_norm_backward_workspace_size(4, 8, None) == -1


def test_c_policy_loss_statuses(so):
    f = so.mxq_policy_loss
    #     z T  V  ld zt tgt 64 old adv w ref lo hi beta scale loss logp g ldg gt ws bytes stream
    ok = [P, 4, 8, 8, 0, P, 1, P, P, P, P, 0.2, 0.2, 0.1, 1.0, P, P, P, 8, 0, P, 1 << 20, None]

    def call(**kw):
        a = list(ok)
        for k, v in kw.items():
            a[int(k[1:])] = v
        return f(*a)

    assert call(_0=None) == -1 and call(_4=2) == -1 and call(_6=2) == -1 and call(_5=None) == -1
    assert call(_10=None) == -1 and call(_15=None) == -1 and call(_16=None) == -1 and call(_19=4) == -1
    assert call(_11=-0.1) == -1 and call(_12=float("nan")) == -1
    assert call(_20=None) == -1 and call(_21=256) == -1
    assert call(_1=-1) == -2 and call(_2=0) == -2 and call(_3=7) == -2 and call(_18=7) == -2 and call(_1=1 << 30) == -2
    assert call(_0=P + 1) == -3 and call(_5=P + 4) == -3 and call(_17=P + 1) == -3 and call(_20=P + 8) == -3
    assert call() == -4 and call(_10=None, _13=0.0) == -4 and call(_17=None, _18=0) == -4
    assert so.mxq_policy_loss_workspace_size(4, None) == -1
    n = ctypes.c_size_t(0)
    assert so.mxq_policy_loss_workspace_size(10, ctypes.byref(n)) == 0 and n.value == 296


class Grad(ctypes.Structure):
    _fields_ = [("g", ctypes.c_void_p), ("out", ctypes.c_void_p), ("n", ctypes.c_int64), ("g_type", ctypes.c_int32),
                ("out_type", ctypes.c_int32)]


def test_c_clip_statuses(so):
    def call(g=P, out=P, n=4, gt=0, ot=0, count=1, max_norm=1.0, norm=P, ws=P, size=1 << 30):
        t = (Grad * 1)(Grad(g, out, n, gt, ot))
        return so.mxq_clip_grad_norm(t, count, max_norm, norm, ws, size, None)

    assert call(g=None) == -1 and call(out=None) == -1 and call(gt=3) == -1 and call(ot=3) == -1
    assert call(count=-1) == -1 and call(max_norm=-1.0) == -1 and call(max_norm=float("nan")) == -1
    assert call(norm=None) == -1 and call(ws=None) == -1 and call(size=8) == -1
    assert call(gt=1, ot=0) == -1                                # in place needs one type
    assert call(n=-1) == -2
    assert call(g=P + 1) == -3 and call(norm=P + 2) == -3 and call(ws=P + 8) == -3
    assert call() == -4 and call(n=0, g=None, out=None) == -4
    assert so.mxq_clip_grad_norm(None, 1, 1.0, P, P, 1 << 30, None) == -1
    assert so.mxq_grad_norm((Grad * 1)(Grad(P, None, 4, 0, 0)), 1, P, P, 1 << 30, None) == -4
    assert so.mxq_grad_norm_workspace_size(4, None) == -1


def test_calls_enter_the_device_guard_only_for_another_device(monkeypatch):
    """_launch runs the call with the tensors' device current and that device's stream."""
    events = []

    class FakeDevice:
        def __init__(self, d):
            self.d = d

        def __enter__(self):
            events.append(("enter", str(self.d)))

        def __exit__(self, *a):
            events.append(("exit", str(self.d)))

    class FakeLib:
        def mxq_grad_norm(self, *args):
            events.append(("call", args[-1]))
            return 0

    monkeypatch.setattr(mxq, "_lib", FakeLib())
    monkeypatch.setattr(mxq.torch.cuda, "device", FakeDevice)
    monkeypatch.setattr(mxq.torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(mxq.torch._C, "_cuda_getCurrentRawStream", lambda i: f"stream {i}", raising=False)
    mxq._launch("mxq_grad_norm", torch.device("cuda", 0), 1, 2)
    mxq._launch("mxq_grad_norm", torch.device("cuda", 1), 1, 2)
    assert events == [("call", "stream 0"), ("enter", "cuda:1"), ("call", "stream 1"), ("exit", "cuda:1")]
