"""The training-step operators in CUDA graphs, from several host threads, and
with workspaces of any contents: a call's scratch is its own, so every result
has the bits of a call made alone."""

import ctypes
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

dev = torch.device("cuda")


def tokens(T, V, seed, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    z = torch.randn(T, V, device=dev, generator=g).to(dtype)
    a = torch.randint(V, (T,), device=dev, generator=g)
    old = torch.log_softmax(z.float(), 1)[torch.arange(T, device=dev), a] - 0.05
    return z, a, old, torch.randn(T, device=dev, generator=g), torch.rand(T, device=dev, generator=g) / T


def same(got, want):
    return all(torch.equal(g, w) for g, w in zip(got, want))


# a warp, a CTA and a cluster a row; the ring
SHAPES = [(300, 64), (1500, 1000), (200, 5000), (5, 32001), (700, 12296)]


@pytest.mark.parametrize("T,V", SHAPES)
def test_graphs_replayed_in_any_order(lib, T, V):
    """Two graphs from torch's shared capture stream, the second replayed
    first, then both at once on two streams; memory that was freed since the
    captures is given new contents, which stay."""
    first, second = tokens(T, V, 1), tokens(T, V, 2)
    want = [lib.policy_loss(*t) for t in (first, second)]
    graphs, outs = [], []
    for t in (first, second):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(lib.policy_loss(*t))
    other = torch.cuda.Stream()
    for order in ((1, 0), (0, 1)):
        for o in outs:
            for x in o:
                x.fill_(float("nan"))
        for k in order:
            graphs[k].replay()
        torch.cuda.synchronize()
        assert same(outs[0], want[0]) and same(outs[1], want[1])
    # a larger call on the stream, then memory with known contents
    lib.policy_loss(*tokens(20000, 64, 3))
    torch.cuda.synchronize()
    guard = [torch.full((1 << 16,), 7, dtype=torch.uint8, device=dev) for _ in range(8)]
    torch.cuda.synchronize()
    for _ in range(20):
        graphs[0].replay()
        with torch.cuda.stream(other):
            graphs[1].replay()
    torch.cuda.synchronize()
    assert same(outs[0], want[0]) and same(outs[1], want[1])
    assert all((g == 7).all() for g in guard)


def test_every_operator_in_one_graph(lib):
    """The norms, the loss and the clip of a step, captured and replayed on new inputs."""
    T, C = 1024, 512
    x, w = torch.randn(T, C, device=dev), torch.rand(C, device=dev) + 0.5
    a = torch.arange(T, device=dev) % C
    v = torch.ones(T, device=dev)

    def step():
        y, mean, rstd = lib.layer_norm(x, w)
        q = lib.mx_layer_norm(x, w, orientation="dual", sf_layout="mma")
        loss, logp, dz = lib.policy_loss(y, a, -6 * v, v, v / T)
        grads = lib.layer_norm_backward(dz, x, mean, rstd, w)
        return (y, *q, loss, logp, dz, *grads, lib.clip_grad_norm([g.clone() for g in grads], 1.0))

    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for seed in range(3):
        x.normal_(generator=torch.Generator(device="cuda").manual_seed(seed))
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        assert same(got, step())


@pytest.mark.parametrize("T,V", SHAPES)
def test_threads_on_one_stream(lib, T, V):
    """Host threads that share the default stream: the launches of their calls interleave."""
    data = [tokens(T, V, 10 + k) for k in range(4)]
    want = [lib.policy_loss(*t) for t in data]
    torch.cuda.synchronize()
    wrong = []

    def work(k):
        got = [lib.policy_loss(*data[k]) for _ in range(30)]
        torch.cuda.synchronize()
        wrong.extend((k, i) for i, g in enumerate(got) if not same(g, want[k]))

    threads = [threading.Thread(target=work, args=(k,)) for k in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
    assert not any(t.is_alive() for t in threads) and not wrong


@pytest.mark.parametrize("T,V", SHAPES)
@pytest.mark.parametrize("fill", [0, 1, 255])
def test_workspace_of_any_contents(lib, T, V, fill):
    z, a, old, adv, w = tokens(T, V, 20)
    want = lib.policy_loss(z, a, old, adv, w)
    L = lib.load()
    n = ctypes.c_size_t(0)
    assert L.mxq_policy_loss_workspace_size(T, ctypes.byref(n)) == 0
    ws = torch.full((n.value + 64,), fill, dtype=torch.uint8, device=dev)
    out = [torch.full_like(t, float("nan")) for t in want]
    p = [t.data_ptr() for t in (z, a, old, adv, w, *out, ws)]
    for _ in range(2):
        assert L.mxq_policy_loss(p[0], T, V, V, 0, p[1], 1, p[2], p[3], p[4], None, 0.2, 0.2, 0.0, 1.0, p[5], p[6],
                                 p[7], V, 0, p[8], n.value, torch.cuda.current_stream().cuda_stream) == 0
        assert same(out, want)
    assert (ws[n.value:] == fill).all()
