"""Cases of the operators that a training step runs around its block-scaled products: the layer norm that makes an
operand (plain, or straight to MX codes) and its backward pass, the clipped policy loss on the last product's logits,
and the global gradient norm with clipping.

``run`` computes each either in its plain form (elementary torch operations in float32, rounded once at the end) or,
where ``own`` is true, through the framework's entry points."""

import torch

own = False

EPS = 1e-5
CLIP_LOW, CLIP_HIGH, BETA = 0.2, 0.2, 0.04
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
FP8_MAX = {"e4m3": 448.0, "e5m2": 57344.0}     # both 1.75 * 2^E
FP8_EXP = {"e4m3": 8, "e5m2": 15}


def listed():
    return [
        # one token's norm, as in generation: a launch and its latency
        {"name": "norm_one_token", "op": "norm", "rows": 1, "cols": 4096, "x": "bf16", "y": "bf16", "w": "bf16"},
        # a float32 residual stream of odd width, normalised to bf16: rows that start at no 16-byte boundary
        {"name": "norm_ragged_f32", "op": "norm", "rows": 1531, "cols": 2049, "x": "f32", "y": "bf16", "w": "f32"},
        # the feed-forward width over a training batch
        {"name": "norm_4096x14336", "op": "norm", "rows": 4096, "cols": 14336, "x": "bf16", "y": "bf16", "w": "bf16"},
        # the small row-wise quantize shape, norm included
        {"name": "mx_norm_row_256x512", "op": "mx_norm", "rows": 256, "cols": 512, "fmt": "e4m3", "dual": False,
         "scale": "floor", "mma": False, "w": "f32"},
        # the activations of a training batch, as both operands that its products read
        {"name": "mx_norm_dual_8192x4096", "op": "mx_norm", "rows": 8192, "cols": 4096, "fmt": "e4m3", "dual": True,
         "scale": "ceil", "mma": True, "w": "bf16"},
        # backward of a short ragged batch in float32
        {"name": "norm_bwd_ragged_f32", "op": "norm_bwd", "rows": 333, "cols": 1021, "x": "f32", "dy": "f32", "w": "f32"},
        # backward over a training batch
        {"name": "norm_bwd_8192x4096", "op": "norm_bwd", "rows": 8192, "cols": 4096, "x": "bf16", "dy": "bf16",
         "w": "bf16"},
        # a handful of tokens over a vocabulary of odd size: few rows, each long
        {"name": "policy_5x32001", "op": "policy", "tokens": 5, "vocab": 32001, "z": "bf16", "g": "bf16", "masked": 0.0},
        # float32 logits of odd width, gradient to bf16 for the quantizer, a quarter of the tokens being prompt
        {"name": "policy_515x50021_f32", "op": "policy", "tokens": 515, "vocab": 50021, "z": "f32", "g": "bf16",
         "masked": 0.25},
        # a training micro-batch over a large vocabulary
        {"name": "policy_2048x131072", "op": "policy", "tokens": 2048, "vocab": 131072, "z": "bf16", "g": "bf16",
         "masked": 0.25},
        # a small model's gradients, clipped into the optimizer's buffer: many short tensors
        {"name": "clip_small", "op": "clip", "layers": 4, "hidden": 129, "ffn": 515, "vocab": 1000, "g": "f32"},
        # a deep model's bf16 gradients into float32
        {"name": "clip_large", "op": "clip", "layers": 32, "hidden": 1024, "ffn": 3584, "vocab": 32768, "g": "bf16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def _pick(rng, *choices):
    return choices[rng.randrange(len(choices))]


def draw(rng):
    op = _pick(rng, "norm", "mx_norm", "norm_bwd", "policy", "clip")
    if op in ("norm", "norm_bwd"):
        cols = _log(rng, 8, 16384)
        if rng.random() < 0.6:
            cols = max(8, cols // 8 * 8)
        rows = _log(rng, 1, max(1, min(16384, (32 << 20) // cols)))
        c = {"op": op, "rows": rows, "cols": cols, "x": _pick(rng, "bf16", "f32"), "w": _pick(rng, "bf16", "f32")}
        c["y" if op == "norm" else "dy"] = _pick(rng, "bf16", c["x"])
        return c
    if op == "mx_norm":
        mma = rng.random() < 0.5
        unit = 128 if mma else 32
        cols = unit * _log(rng, 1, 16384 // unit)
        rows = unit * _log(rng, 1, max(1, min(8192, (32 << 20) // cols) // unit))
        return {"op": op, "rows": rows, "cols": cols, "fmt": _pick(rng, "e4m3", "e5m2"), "dual": rng.random() < 0.5,
                "scale": _pick(rng, "floor", "ceil"), "mma": mma, "w": _pick(rng, "bf16", "f32")}
    if op == "policy":
        vocab = _log(rng, 500, 131072)
        if rng.random() < 0.6:
            vocab = vocab // 8 * 8
        z = _pick(rng, "bf16", "f32")
        return {"op": op, "tokens": _log(rng, 1, min(8192, (128 << 20) // vocab)), "vocab": vocab, "z": z,
                "g": _pick(rng, "bf16", z), "masked": _pick(rng, 0.0, 0.25, 0.5)}
    hidden = _log(rng, 64, 1024)
    return {"op": op, "layers": _log(rng, 1, 32), "hidden": hidden, "ffn": int(hidden * (2 + 2 * rng.random())),
            "vocab": _log(rng, 500, 32768), "g": _pick(rng, "bf16", "f32")}


def _grad_shapes(c):
    h, f = c["hidden"], c["ffn"]
    layer = [(h,), (h,), (3 * h, h), (h, h), (h,), (h,), (f, h), (f,), (h, f)]
    return [(c["vocab"], h)] + layer * c["layers"]


def prepare(case, seed):
    """The inputs of a case on the GPU, from the seed alone."""
    c = dict(case)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    s = {"case": c}
    if c["op"] in ("norm", "mx_norm", "norm_bwd"):
        # activations: every row with an offset and a spread of its own, and a few outlier channels
        R, C = c["rows"], c["cols"]
        x = normal(R, C) * (0.5 + normal(R, 1).abs()) + normal(R, 1)
        x[:, :: 1021] *= 20.0
        s["x"] = x.to(TYPES[c.get("x", "bf16")])
        s["weight"] = (1.0 + 0.1 * normal(C)).to(TYPES[c["w"]])
        s["bias"] = (0.1 * normal(C)).to(TYPES[c["w"]])
        if c["op"] == "norm_bwd":
            s["dy"] = (0.1 * normal(R, C)).to(TYPES[c["dy"]])
            _, s["mean"], s["rstd"] = _norm(s["x"])     # kept from the forward pass
    elif c["op"] == "policy":
        # a policy that has drifted a little from the one that sampled the tokens; prompt tokens have no weight
        T, V = c["tokens"], c["vocab"]
        z = normal(T, V).mul_(2.0)
        a = torch.randint(V, (T,), device="cuda", generator=gen)
        z[torch.arange(T, device="cuda"), a] += 8.0
        z = z.to(TYPES[c["z"]])
        logp = _token_logp(z, a)
        # the drift is a multiple of 0.01: no ratio lies within rounding of the clip's edges, where the gradient jumps
        drift = (normal(T) * 12.0).round() * 0.01
        live = torch.rand(T, device="cuda", generator=gen) >= c["masked"]
        s["logits"] = z
        s["targets"] = torch.where(live, a, -100)
        s["old"] = logp - drift
        s["ref"] = logp + 0.2 * normal(T)
        s["adv"] = normal(T)
        s["weights"] = live.float() / live.sum().clamp(min=1)
    else:
        shapes = _grad_shapes(c)
        s["grads"] = [(normal(*sh) * 0.02).to(TYPES[c["g"]]) for sh in shapes]
        # the optimizer's flat float32 buffer, every tensor at a 128-byte boundary
        ends, at = [], 0
        for g in s["grads"]:
            ends.append(at)
            at += (g.numel() + 31) // 32 * 32
        s["flat"] = torch.zeros(at, device="cuda")
        s["out"] = [s["flat"][e:e + g.numel()].view(g.shape) for e, g in zip(ends, s["grads"])]
    return s


# ------------------------------------------------------------------ plain forms (float32)
def _norm(x):
    x = x.float()
    mean = x.sum(1) / x.shape[1]
    d = x - mean[:, None]
    rstd = 1.0 / ((d * d).sum(1) / x.shape[1] + EPS).sqrt()
    return d * rstd[:, None], mean, rstd


def _mx(y, fmt, scale, mma):
    R, C = y.shape
    b = y.reshape(R, C // 32, 32)
    bits = b.abs().amax(2).view(torch.int32)
    e = (bits >> 23) - 127 - FP8_EXP[fmt]
    if scale == "ceil":
        e = e + ((bits & 0x7FFFFF) > 0x600000).int()
    e = e.clamp(-127, 127)
    q = (b * torch.exp2(-e.float())[:, :, None]).clamp(-FP8_MAX[fmt], FP8_MAX[fmt]).to(FP8[fmt]).reshape(R, C)
    sf = (e + 127).to(torch.uint8)
    if mma:
        sf = sf.reshape(R // 128, 4, 32, C // 128, 4).permute(0, 3, 2, 1, 4).reshape(R, C // 32)
    return q, sf.contiguous().view(torch.float8_e8m0fnu)


def _token_logp(z, a):
    z = z.float()
    m = z.amax(1)
    return z.gather(1, a[:, None])[:, 0] - m - (z - m[:, None]).exp().sum(1).log()


def _policy(s, g):
    z = s["logits"].float()
    w, A = s["weights"], s["adv"]
    live = w != 0
    a = torch.where(live, s["targets"], 0)
    m = z.amax(1)
    p = (z - m[:, None]).exp()
    total = p.sum(1)
    logp = torch.where(live, z.gather(1, a[:, None])[:, 0] - m - total.log(), 0.0)
    ratio = (logp - s["old"]).exp()
    clipped = ratio.clamp(1 - CLIP_LOW, 1 + CLIP_HIGH)
    d = s["ref"] - logp
    each = -torch.minimum(ratio * A, clipped * A) + BETA * (d.exp() - d - 1)
    slope = torch.where(ratio * A <= clipped * A, -ratio * A, 0.0) + BETA * (1 - d.exp())
    loss = torch.where(live, w * each, 0.0).sum().reshape(1)
    k = torch.where(live, w * slope, 0.0)
    dz = p * (-k / total)[:, None]
    dz[torch.arange(z.shape[0], device=z.device), a] += k
    return loss, logp, torch.where(live[:, None], dz, 0.0).to(TYPES[g])


def _run_plain(s):
    c = s["case"]
    if c["op"] in ("norm", "mx_norm"):
        h, mean, rstd = _norm(s["x"])
        y = h * s["weight"].float() + s["bias"].float()
        if c["op"] == "norm":
            return {"y": y.to(TYPES[c["y"]]), "mean": mean, "rstd": rstd}
        q, sf = _mx(y, c["fmt"], c["scale"], c["mma"])
        out = {"q": q, "s": sf, "mean": mean, "rstd": rstd}
        if c["dual"]:
            out["qT"], out["sT"] = _mx(y.t(), c["fmt"], c["scale"], c["mma"])
        return out
    if c["op"] == "norm_bwd":
        dy, w = s["dy"].float(), s["weight"].float()
        h = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
        g = dy * w
        C = h.shape[1]
        c1, c2 = g.sum(1) / C, (g * h).sum(1) / C
        dx = (g - c1[:, None] - h * c2[:, None]) * s["rstd"][:, None]
        return {"dx": dx.to(s["x"].dtype), "dweight": (dy * h).sum(0), "dbias": dy.sum(0)}
    if c["op"] == "policy":
        loss, logp, dz = _policy(s, c["g"])
        return {"loss": loss, "logp": logp, "dlogits": dz}
    squares = torch.stack([(g.float() * g.float()).sum() for g in s["grads"]])
    norm = squares.sum().sqrt().reshape(1)
    scale = (1.0 / (norm + 1e-6)).clamp(max=1.0)
    [o.copy_(g.float() * scale) for o, g in zip(s["out"], s["grads"])]
    return {"norm": norm, "clipped": s["flat"]}


# ------------------------------------------------------------------ the framework's calls
def _run_own(s):
    import block_scaled_precision_02_gb300 as mxq
    c = s["case"]
    if c["op"] == "norm":
        y, mean, rstd = mxq.layer_norm(s["x"], s["weight"], s["bias"], EPS, out_dtype=TYPES[c["y"]])
        return {"y": y, "mean": mean, "rstd": rstd}
    if c["op"] == "mx_norm":
        q, sf, qT, sfT, mean, rstd = mxq.mx_layer_norm(
            s["x"], s["weight"], s["bias"], EPS, c["fmt"], "dual" if c["dual"] else "row", c["scale"],
            sf_layout="mma" if c["mma"] else "canonical")
        e8 = torch.float8_e8m0fnu
        out = {"q": q.view(FP8[c["fmt"]]), "s": sf.view(e8), "mean": mean, "rstd": rstd}
        if c["dual"]:
            out["qT"], out["sT"] = qT.view(FP8[c["fmt"]]), sfT.view(e8)
        return out
    if c["op"] == "norm_bwd":
        dx, dw, db = mxq.layer_norm_backward(s["dy"], s["x"], s["mean"], s["rstd"], s["weight"])
        return {"dx": dx, "dweight": dw, "dbias": db}
    if c["op"] == "policy":
        loss, logp, dz = mxq.policy_loss(s["logits"], s["targets"], s["old"], s["adv"], s["weights"],
                                         ref_logp=s["ref"], clip_low=CLIP_LOW, clip_high=CLIP_HIGH, beta=BETA,
                                         grad_dtype=TYPES[c["g"]])
        return {"loss": loss, "logp": logp, "dlogits": dz}
    norm = mxq.clip_grad_norm(s["grads"], 1.0, out=s["out"])
    return {"norm": norm, "clipped": s["flat"]}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------ the definition in float64
def exact(case, seed):
    """The outputs by definition in float64.  Quantized codes and scales have no entry: a value between two grid
    neighbours is settled by the arithmetic that makes it, not by more bits."""
    s = prepare(case, seed)
    c = s["case"]
    f8 = torch.float64
    if c["op"] in ("norm", "mx_norm", "norm_bwd"):
        x, w = s["x"].to(f8), s["weight"].to(f8)
        if c["op"] == "norm_bwd":
            mean, rstd = s["mean"].to(f8).unsqueeze(1), s["rstd"].to(f8).unsqueeze(1)
            dy = s["dy"].to(f8)
            n = (x - mean).mul_(rstd)
            wdy = dy * w
            proj = (wdy * n).mean(1, keepdim=True)
            return {"dx": (wdy - wdy.mean(1, keepdim=True) - n * proj) * rstd, "dweight": torch.einsum("rc,rc->c", dy, n),
                    "dbias": dy.sum(0)}
        mean = x.mean(1)
        rstd = (x.var(1, unbiased=False) + EPS).rsqrt()
        if c["op"] == "mx_norm":
            return {"q": None, "s": None, "mean": mean, "rstd": rstd, "qT": None, "sT": None}
        y = torch.addcmul(s["bias"].to(f8), (x - mean.unsqueeze(1)) * rstd.unsqueeze(1), w)
        return {"y": y, "mean": mean, "rstd": rstd}
    if c["op"] == "policy":
        live = s["weights"] > 0
        z = s["logits"][live].to(f8)
        a = s["targets"][live]
        old, ref, A, w = (s[k][live].to(f8) for k in ("old", "ref", "adv", "weights"))
        lp_all = torch.log_softmax(z, 1)
        lp = lp_all.take_along_dim(a.unsqueeze(1), 1).squeeze(1)
        lp.requires_grad_(True)
        r = torch.exp(lp - old)
        surrogate = torch.where(A >= 0, r.clamp(max=1 + CLIP_HIGH) * A, r.clamp(min=1 - CLIP_LOW) * A)
        kl = torch.expm1(ref - lp) - (ref - lp)
        loss = (w * (BETA * kl - surrogate)).sum()
        if lp.numel():
            loss.backward()
        k = lp.grad if lp.numel() else lp.detach()
        dz = lp_all.exp_().mul_(-k.unsqueeze(1))
        dz.scatter_add_(1, a.unsqueeze(1), k.unsqueeze(1))
        T, V = c["tokens"], c["vocab"]
        logp = torch.zeros(T, dtype=f8, device="cuda")
        logp[live] = lp.detach()
        full = torch.zeros(T, V, dtype=f8, device="cuda")
        full[live] = dz
        return {"loss": loss.detach().reshape(1), "logp": logp, "dlogits": full}
    norm = torch.linalg.vector_norm(torch.stack([torch.linalg.vector_norm(g.to(f8)) for g in s["grads"]]))
    factor = min(1.0, 1.0 / (float(norm) + 1e-6))
    flat = torch.zeros(s["flat"].numel(), dtype=f8, device="cuda")
    at = 0
    for g in s["grads"]:
        flat[at:at + g.numel()] = g.reshape(-1).to(f8) * factor
        at += (g.numel() + 31) // 32 * 32
    return {"norm": norm.reshape(1), "clipped": flat}


def work(case):
    c = case
    if c["op"] in ("norm", "mx_norm", "norm_bwd"):
        n, params = c["rows"] * c["cols"], c["cols"] * SIZE[c["w"]]
        stats = 8 * c["rows"]
        if c["op"] == "norm":
            return {"bytes": n * (SIZE[c["x"]] + SIZE[c["y"]]) + 2 * params + stats, "flops": 8 * n}
        if c["op"] == "mx_norm":
            sides = 2 if c["dual"] else 1
            return {"bytes": 2 * n + sides * (n + n // 32) + 2 * params + stats, "flops": (8 + 4 * sides) * n}
        return {"bytes": n * (2 * SIZE[c["x"]] + SIZE[c["dy"]]) + params + 8 * c["cols"] + stats, "flops": 14 * n}
    if c["op"] == "policy":
        n = c["tokens"] * c["vocab"]
        read = n * (1.0 - c["masked"])      # the logits of a token without weight are not needed
        return {"bytes": read * SIZE[c["z"]] + n * SIZE[c["g"]] + 32 * c["tokens"], "flops": 6 * read}
    n = 0
    for sh in _grad_shapes(c):
        k = 1
        for d in sh:
            k *= d
        n += k
    return {"bytes": n * (SIZE[c["g"]] + 4), "flops": 3 * n}
