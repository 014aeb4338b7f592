"""The calls of a mixture-of-experts layer run together, forward and backward,
as a training step runs them; in CUDA graphs, on other streams and from several
host threads."""

import threading

import numpy as np
import pytest
import torch

from oracle import gemm as og
from tests.expert_reference import decoded
from tests.rounding import half_ulp

pytestmark = pytest.mark.gpu

dev = torch.device("cuda")
BF, F32 = torch.bfloat16, torch.float32
T, TOP, E, D, H, P = 384, 2, 6, 256, 512, 0.1


def data(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(*s, device=dev, generator=g)
    z = n(T, E)
    best, experts = z.topk(TOP, dim=1)
    experts[torch.rand(T, TOP, device=dev, generator=g) < 0.1] = -1
    return dict(x=n(T, D).to(BF), w1=(0.06 * n(E * H, D)).to(BF), w2=(0.04 * n(E * D, H)).to(BF), experts=experts.contiguous(),
                gate=best.softmax(1), dy=n(T, D).to(BF))


def layer(lib, d, align, seed=5):
    """One expert layer x + dropout(sum_j gate_j W2 W1 x), forward and backward."""
    o = {}
    p = lib.expert_sort(d["experts"], E, align)
    w1, s1, w1T, s1T = lib.mx_quantize(d["w1"], "e4m3", "dual", "ceil", sf_layout="mma")
    w2, s2, w2T, s2T = lib.mx_quantize(d["w2"], "e4m3", "dual", "ceil", sf_layout="mma")
    x, sx, xT, sxT = lib.mx_expert_gather(d["x"], p, "e4m3", "dual", "ceil", "mma")
    o["h"] = lib.mx_expert_gemm(x, sx, w1.view(E, H, D), s1, p)
    h, sh, hT, shT = lib.mx_quantize(o["h"], "e4m3", "dual", "ceil", sf_layout="mma")
    o["r"] = lib.mx_expert_gemm(h, sh, w2.view(E, D, H), s2, p)
    o["c"] = lib.expert_combine(o["r"], p, d["gate"])
    o["y"] = lib.dropout(o["c"], P, seed, residual=d["x"])
    o["dc"] = lib.dropout(d["dy"], P, seed)
    o["dr"], o["dgate"] = lib.expert_combine_backward(o["dc"], o["r"], p, d["gate"])
    g, sg, gT, sgT = lib.mx_quantize(o["dr"], "e5m2", "dual", "ceil", sf_layout="mma")
    o["dw2"] = lib.mx_expert_wgrad(gT, sgT, hT, shT, p, "e5m2", "e4m3")
    o["dh"] = lib.mx_expert_gemm(g, sg, w2T, s2T, p, "e5m2", "e4m3")
    k, sk, kT, skT = lib.mx_quantize(o["dh"], "e5m2", "dual", "ceil", sf_layout="mma")
    o["dw1"] = lib.mx_expert_wgrad(kT, skT, xT, sxT, p, "e5m2", "e4m3")
    o["dxr"] = lib.mx_expert_gemm(k, sk, w1T, s1T, p, "e5m2", "e4m3")
    o["dx"] = lib.expert_combine(o["dxr"], p)
    o["codes"] = dict(x=(x, sx), xT=(xT, sxT), w1=(w1, s1), w2=(w2, s2), w1T=(w1T, s1T), w2T=(w2T, s2T), h=(h, sh), hT=(hT, shT))
    o["grads"] = dict(g=(g, sg), gT=(gT, sgT), k=(k, sk), kT=(kT, skT))
    return p, o


def n64(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("align", [128, 256])
def test_every_step_of_a_layer(lib, align):
    """Each step's output against float64 arithmetic on that step's own inputs."""
    d = data(1)
    p, o = layer(lib, d, align)
    v = {k: decoded(*c, "e4m3") for k, c in o["codes"].items()}
    v.update({k: decoded(*c, "e5m2") for k, c in o["grads"].items()})
    off = p.offsets.tolist()
    seg = [slice(off[e], off[e + 1]) for e in range(E)]
    slot = p.slot_row.cpu().numpy()
    live, at = slot >= 0, np.maximum(slot, 0)

    def rows(a, b):
        c = np.zeros((p.rows, b[0].shape[0]))
        for e in range(E):
            c[seg[e]] = a[seg[e]] @ b[e].T
        return c

    gate = lambda got, ref, bf=True: og.gate_error(n64(got), ref, bf)
    assert gate(o["h"], rows(v["x"], v["w1"].reshape(E, H, D))) <= 2e-3
    assert gate(o["r"], rows(v["h"], v["w2"].reshape(E, D, H))) <= 2e-3
    assert gate(o["dh"], rows(v["g"], v["w2T"].reshape(H, E, D).transpose(1, 0, 2))) <= 2e-3
    assert gate(o["dxr"], rows(v["k"], v["w1T"].reshape(D, E, H).transpose(1, 0, 2))) <= 2e-3
    assert gate(o["dw2"], np.stack([v["gT"][:, s] @ v["hT"][:, s].T for s in seg]), False) <= 2e-3
    assert gate(o["dw1"], np.stack([v["kT"][:, s] @ v["xT"][:, s].T for s in seg]), False) <= 2e-3
    w = np.where(live, n64(d["gate"]), 0)
    for got, src, ww in ((o["c"], o["r"], w), (o["dx"], o["dxr"], live * 1.0)):
        terms = n64(src)[at] * ww[:, :, None]
        tol = TOP * 2.0 ** -24 * np.abs(terms).sum(1) * 1.01
        ref = terms.sum(1)
        assert np.all(np.abs(n64(got) - ref) <= tol + half_ulp(BF, ref, tol))
    terms = n64(o["dc"])[:, None] * np.where(live[:, :, None], n64(o["r"])[at], 0)
    assert np.all(np.abs(n64(o["dgate"]) - terms.sum(2)) <= 24 * 2.0 ** -24 * np.abs(terms).sum(2))
    # the mask of the backward pass is the forward pass's
    assert torch.equal(o["dc"] != 0, (lib.dropout(torch.ones_like(o["c"]), P, 5) != 0) & (d["dy"] != 0))


def test_gradients_of_the_layer_follow_the_formula(lib):
    """Against float64 autograd of the layer without quantization.  Every code
    is off by at most 1/16 of its value (E4M3; E5M2 1/8) or, below the smallest
    normal, by less than 2^-10 of its block's largest value; errors of different
    elements are as good as independent, so a product's error, relative to its
    norm, is below sqrt(2) times 1/8 for each of the at most three quantized
    products behind a gradient: 0.54 in all.  The cosine is then above 0.84."""
    d = data(2)
    p, o = layer(lib, d, 128)
    x, w1, w2, gate = (d[k].double().requires_grad_() for k in ("x", "w1", "w2", "gate"))
    keep = (lib.dropout(torch.ones(T, D, device=dev), P, 5) != 0).double() / (1 - P)
    e = d["experts"]
    acc = 0
    for j in range(TOP):
        idx = e[:, j].clamp(min=0)
        h = torch.einsum("td,thd->th", x, w1.view(E, H, D)[idx])
        r = torch.einsum("th,tdh->td", h, w2.view(E, D, H)[idx])
        acc = acc + r * (gate[:, j] * (e[:, j] >= 0))[:, None]
    (acc * keep * d["dy"].double()).sum().backward()
    for got, want in ((o["dx"], x.grad), (o["dw1"], w1.grad.view(E, H, D)), (o["dw2"], w2.grad.view(E, D, H)),
                      (o["dgate"], gate.grad), (o["y"].double() - d["x"].double(), (acc * keep).detach())):
        got = got.double()
        cos = float((got * want).sum() / (got.norm() * want.norm()))
        assert cos > 0.84 and abs(float(got.norm() / want.norm()) - 1) < 0.54


KEYS = ("h", "r", "c", "y", "dr", "dgate", "dw2", "dh", "dw1", "dx")


def same(a, b):
    return all(torch.equal(a[k], b[k]) for k in KEYS)


def test_layer_in_graphs_with_other_routings(lib):
    """A recorded layer, replayed on other inputs of the same sizes: the sizes
    of the experts' stretches are read on the device."""
    d = data(3)
    layer(lib, d, 256)
    graphs, outs = [], []
    for _ in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(layer(lib, d, 256)[1])
    for seed in (4, 5):
        n = data(seed)
        for k in d:
            d[k].copy_(n[k])
        want = layer(lib, n, 256)[1]
        for k in (1, 0):
            graphs[k].replay()
        torch.cuda.synchronize()
        assert same(outs[0], want) and same(outs[1], want)
    # both at once
    other = torch.cuda.Stream()
    for _ in range(5):
        graphs[0].replay()
        with torch.cuda.stream(other):
            graphs[1].replay()
    torch.cuda.synchronize()
    assert same(outs[0], want) and same(outs[1], want) and lib.last_device_status() == 0


def test_layers_from_threads_on_their_own_streams(lib):
    ds = [data(s) for s in (6, 7, 8)]
    want = [layer(lib, d, 128)[1] for d in ds]
    torch.cuda.synchronize()
    wrong = []

    def work(k):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(10):
                o = layer(lib, ds[k], 128)[1]
                torch.cuda.current_stream().synchronize()
                if not same(o, want[k]):
                    wrong.append(k)

    threads = [threading.Thread(target=work, args=(k,)) for k in range(3)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not wrong and lib.last_device_status() == 0
