"""Cases of the operators of a mixture-of-experts layer in MX precision: tokens sorted by expert and gathered into rows
(plain, or straight to MX operands), the block-scaled products of all experts in one call and their weights' gradient,
the way back with the gate's weights and its gradient, and dropout onto the residual stream.

``run`` computes each either in its plain form (elementary torch operations in float32, rounded once at the end) or,
where ``own`` is true, through the framework's entry points."""

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
MAX = {"e4m3": 448.0, "e5m2": 57344.0, "e2m1": 6.0}
EXP = {"e4m3": 8, "e5m2": 15, "e2m1": 2}            # exponents of the formats' largest values
MANTISSA = {"e4m3": 0x600000, "e5m2": 0x600000, "e2m1": 0x400000}     # and their mantissas' bits, of 23
CODE_BYTES = {"e4m3": 1.0, "e5m2": 1.0, "e2m1": 0.5}
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)     # magnitudes of E2M1, by code


def listed():
    return [
        # one token of generation: the sort's and the gather's latency
        {"name": "dispatch_one_token", "op": "dispatch", "tokens": 1, "top": 8, "experts": 64, "cols": 4096, "x": "bf16",
         "mx": False, "align": 128, "dropped": 0.0},
        # a training batch's activations, as both operands that the experts' products and their gradients read
        {"name": "dispatch_mx_8192x4096", "op": "dispatch", "tokens": 8192, "top": 2, "experts": 16, "cols": 4096,
         "x": "bf16", "mx": True, "fmt": "e4m3", "dual": True, "scale": "ceil", "mma": True, "align": 256, "dropped": 0.0},
        # float32 rows of odd width, an expert's capacity having dropped some of the tokens' choices
        {"name": "combine_ragged_f32", "op": "combine", "tokens": 515, "top": 3, "experts": 5, "cols": 2049, "x": "f32",
         "y": "bf16", "w": "f32", "align": 128, "dropped": 0.1},
        # a training batch's way back
        {"name": "combine_8192x4096", "op": "combine", "tokens": 8192, "top": 2, "experts": 16, "cols": 4096, "x": "bf16",
         "y": "bf16", "w": "f32", "align": 256, "dropped": 0.0},
        # gradients of the way back, a short ragged batch
        {"name": "combine_bwd_ragged", "op": "combine_bwd", "tokens": 333, "top": 4, "experts": 8, "cols": 1021, "x": "f32",
         "y": "f32", "w": "f32", "align": 128, "dropped": 0.1},
        # and of a training batch
        {"name": "combine_bwd_8192x4096", "op": "combine_bwd", "tokens": 8192, "top": 2, "experts": 16, "cols": 4096,
         "x": "bf16", "y": "bf16", "w": "f32", "align": 256, "dropped": 0.0},
        # a few sequences' new tokens through the experts: the weights' bytes count
        {"name": "gemm_8_tokens", "op": "gemm", "tokens": 8, "top": 2, "experts": 16, "n": 4096, "k": 4096, "a": "e4m3",
         "b": "e4m3", "align": 128, "y": "bf16"},
        # a training batch through the experts' feed-forward weights
        {"name": "gemm_8192_tokens", "op": "gemm", "tokens": 8192, "top": 2, "experts": 8, "n": 14336, "k": 4096,
         "a": "e4m3", "b": "e4m3", "align": 256, "y": "bf16"},
        # the weights' gradient of small experts, odd counts of tokens
        {"name": "wgrad_1001_tokens", "op": "wgrad", "tokens": 1001, "top": 2, "experts": 16, "n": 512, "k": 1024,
         "a": "e4m3", "b": "e4m3", "align": 128, "y": "f32"},
        # the weights' gradient of a training batch: E5M2 gradients beside E4M3 activations
        {"name": "wgrad_8192_tokens", "op": "wgrad", "tokens": 8192, "top": 2, "experts": 8, "n": 4096, "k": 4096,
         "a": "e5m2", "b": "e4m3", "align": 256, "y": "bf16"},
        # dropout of a float32 stream of odd width, as the backward pass runs it
        {"name": "dropout_ragged_f32", "op": "dropout", "rows": 1531, "cols": 2049, "x": "f32", "residual": False, "p": 0.1},
        # dropout onto the residual stream at the feed-forward width of a training batch
        {"name": "dropout_8192x14336", "op": "dropout", "rows": 8192, "cols": 14336, "x": "bf16", "residual": True, "p": 0.1},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def _pick(rng, *choices):
    return choices[rng.randrange(len(choices))]


def draw(rng):
    op = _pick(rng, "dispatch", "combine", "combine_bwd", "gemm", "wgrad", "dropout")
    if op == "dropout":
        cols = _log(rng, 8, 16384)
        if rng.random() < 0.6:
            cols = max(8, cols // 8 * 8)
        x = _pick(rng, "bf16", "f32")
        return {"op": op, "rows": _log(rng, 1, max(1, min(16384, (64 << 20) // cols))), "cols": cols, "x": x,
                "residual": rng.random() < 0.6, "p": _pick(rng, 0.0, 0.05, 0.1, 0.3, 0.5, 0.9)}
    experts = _log(rng, 1, 128)
    c = {"op": op, "tokens": 1, "top": rng.randint(1, min(8, experts)), "experts": experts, "align": _pick(rng, 128, 256),
         "dropped": 0.0}
    if op in ("gemm", "wgrad"):
        c["n"] = 128 * _log(rng, 1, 64)
        c["k"] = 128 * _log(rng, 1, 64)
        c["experts"] = max(1, min(experts, (256 << 20) // (c["n"] * c["k"])))
        c["top"] = min(c["top"], c["experts"])
        c["a"], c["b"] = _pick(rng, ("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e2m1", "e2m1"), ("e4m3", "e2m1"))
        if c["a"] == "e2m1":        # two codes a byte on both sides: 256 elements of the contraction to a step
            c["k"] = (c["k"] + 255) // 256 * 256
            c["align"] = 256
        c["tokens"] = _log(rng, 1, max(1, 16384 // c["top"]))
        c["y"] = _pick(rng, "bf16", "f32")
        del c["dropped"]
        return c
    c["dropped"] = _pick(rng, 0.0, 0.0, 0.1, 0.5)
    if op == "dispatch":
        c["mx"] = rng.random() < 0.5
        c["x"] = "bf16" if c["mx"] else _pick(rng, "bf16", "f32")
        c["cols"] = _log(rng, 8, 8192)
        if c["mx"]:
            c["mma"] = rng.random() < 0.6
            c["cols"] = (c["cols"] + 127) // 128 * 128
            c["fmt"], c["dual"] = _pick(rng, "e4m3", "e5m2"), rng.random() < 0.6
            c["scale"] = _pick(rng, "floor", "ceil")
    else:
        c["x"], c["w"] = _pick(rng, "bf16", "f32"), _pick(rng, "f32", "f32", "bf16")
        c["y"] = _pick(rng, "bf16", c["x"])
        c["cols"] = _log(rng, 8, 8192)
    if not c.get("mx") and rng.random() < 0.6:
        c["cols"] = max(8, c["cols"] // 8 * 8)
    c["tokens"] = _log(rng, 1, max(1, min(16384, (32 << 20) // (c["cols"] * c["top"]))))
    return c


def _rows(c):
    """Rows that the gathered tokens can take, every expert's stretch a multiple of ``align``."""
    s = c["tokens"] * c["top"]
    return (s + min(c["experts"], s) * (c["align"] - 1)) // c["align"] * c["align"]


# ------------------------------------------------------------------ plain forms (float32)
def _sort(experts, E, align):
    """The plan of a routing [tokens][top]: every expert's tokens in their order, each expert's stretch padded."""
    T, top = experts.shape
    s = T * top
    R = (s + min(E, s) * (align - 1)) // align * align
    e = experts.reshape(-1).long()
    live = (e >= 0) & (e < E)
    hot = (e[:, None] == torch.arange(E, device=e.device)).int()
    rank = hot.cumsum(0)
    counts = rank[-1]
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=e.device)
    offsets[1:] = ((counts + align - 1) // align * align).cumsum(0)
    at = torch.where(live, e, 0)
    row = offsets[at] + rank.gather(1, at[:, None])[:, 0] - 1
    slot_row = torch.where(live, row, -1)
    row_slot = torch.full((R + 1,), -1, dtype=torch.int64, device=e.device)
    row_slot[torch.where(live, row, R)] = torch.where(live, torch.arange(s, device=e.device), -1)
    row_slot[R] = -1
    first = torch.arange(0, R, align, device=e.device)
    block = (first[:, None] >= offsets[None, 1:]).sum(1)
    block = torch.where(first < offsets[E], block, -1)
    return {"offsets": offsets.int(), "counts": counts.int(), "slot_row": slot_row.int().reshape(T, top),
            "row_slot": row_slot[:R].int(), "block_expert": block.int()}


def _gather(x, row_slot, top):
    pad = row_slot < 0
    token = torch.where(pad, 0, row_slot) // top
    return x[token].masked_fill_(pad[:, None], 0)


def _mx(y, fmt, scale="floor", mma=True):
    """Codes and scales of the 1 x 32 blocks of float32 rows (E2M1 codes two a byte)."""
    R, C = y.shape
    b = y.reshape(R, C // 32, 32)
    bits = b.abs().amax(2).view(torch.int32)
    e = (bits >> 23) - 127 - EXP[fmt]
    if scale == "ceil":
        e = e + ((bits & 0x7FFFFF) > MANTISSA[fmt]).int()
    e = e.clamp(-127, 127)
    v = (b * torch.exp2(-e.float())[:, :, None]).clamp(-MAX[fmt], MAX[fmt]).reshape(R, C)
    if fmt == "e2m1":
        middles = torch.tensor([(lo + hi) / 2 for lo, hi in zip(GRID, GRID[1:])], device=y.device)
        code = torch.bucketize(v.abs(), middles).to(torch.uint8) | ((v < 0).to(torch.uint8) << 3)
        q = code[:, 0::2] | (code[:, 1::2] << 4)
    else:
        q = v.to(FP8[fmt])
    sf = (e + 127).to(torch.uint8)
    if mma:
        sf = sf.reshape(R // 128, 4, 32, C // 128, 4).permute(0, 3, 2, 1, 4).reshape(R, C // 32)
    return q.view(torch.uint8).contiguous(), sf.contiguous()


def _decode(q, sf, fmt):
    """Codes with scales in the products' layout, as float32."""
    if fmt == "e2m1":
        grid = torch.tensor(GRID + tuple(-g for g in GRID), device=q.device)
        v = torch.stack([grid[(q & 15).int()], grid[(q >> 4).int()]], 2).reshape(q.shape[0], -1)
    else:
        v = q.view(FP8[fmt]).float()
    R, K = v.shape
    s = sf.reshape(R // 128, K // 128, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(R, K // 32)
    scale = torch.exp2(s.float() - 127.0)
    return (v.reshape(R, K // 32, 32) * scale[:, :, None]).reshape(R, K)


def _philox(counter, seed):
    """Philox-4x32-10 of 64-bit counters (the upper two words 0) under a 64-bit key, as four columns of 32 bits."""
    m = 0xFFFFFFFF
    k0, k1 = seed & m, seed >> 32
    x0, x1 = counter & m, (counter >> 32) & m
    x2, x3 = torch.zeros_like(counter), torch.zeros_like(counter)
    for _ in range(10):
        a, b = x0 * 0xD2511F53, x2 * 0xCD9E8D57
        x0, x1, x2, x3 = ((b >> 32) & m) ^ x1 ^ k0, b & m, ((a >> 32) & m) ^ x3 ^ k1, a & m
        k0, k1 = (k0 + 0x9E3779B9) & m, (k1 + 0xBB67AE85) & m
    return torch.stack([x0, x1, x2, x3], 1)


# ------------------------------------------------------------------ inputs
def _routing(c, gen):
    """Experts and gate weights of every token: some experts are in demand, others may get none."""
    T, E, top = c["tokens"], c["experts"], c["top"]
    demand = torch.randn(E, device="cuda", generator=gen) * 0.5
    z = torch.randn(T, E, device="cuda", generator=gen) + demand
    best, experts = z.topk(top, dim=1)
    weights = best.softmax(1)
    lost = torch.rand(T, top, device="cuda", generator=gen) < c.get("dropped", 0.0)
    return experts.masked_fill(lost, -1).int(), weights


def prepare(case, seed):
    """The inputs of a case on the GPU, from the seed alone, with the plan that a layer makes once for all its steps."""
    c = dict(case)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    s = {"case": c}
    if c["op"] == "dropout":
        s["x"] = normal(c["rows"], c["cols"]).to(TYPES[c["x"]])
        s["residual"] = (4.0 * normal(c["rows"], c["cols"])).to(TYPES[c["x"]]) if c["residual"] else None
        s["seed"] = (seed * 0x9E3779B97F4A7C15 + 0x1234567) & 0xFFFFFFFFFFFFFFFF
        s["offset"] = (seed & 0xFF) * 1000003
        return s
    s["experts"], weights = _routing(c, gen)
    plan = _sort(s["experts"], c["experts"], c["align"])
    s["plan"] = plan
    if c["op"] == "dispatch":
        # activations: every row with a spread of its own, and a few outlier channels
        x = normal(c["tokens"], c["cols"]) * (0.5 + normal(c["tokens"], 1).abs())
        x[:, :: 1021] *= 20.0
        s["x"] = x.to(TYPES[c["x"]])
        return s
    if own:
        import block_scaled_precision_02_gb300 as mxq
        s["own_plan"] = mxq.expert_sort(s["experts"], c["experts"], c["align"])
    R = _rows(c)
    pad = (plan["row_slot"] < 0)[:, None]
    if c["op"] in ("combine", "combine_bwd"):
        s["rows"] = normal(R, c["cols"]).to(TYPES[c["x"]]).masked_fill_(pad, 0)
        s["weights"] = weights.to(TYPES[c["w"]])
        if c["op"] == "combine_bwd":
            s["dy"] = (0.1 * normal(c["tokens"], c["cols"])).to(TYPES[c["y"]])
        return s
    s["starts"] = plan["offsets"].tolist()
    if c["op"] == "gemm":
        s["a_q"], s["a_s"] = _mx(normal(R, c["k"]).masked_fill_(pad, 0), c["a"])
        parts = [_mx(0.02 * normal(c["n"], c["k"]), c["b"]) for _ in range(c["experts"])]
        s["b_q"], s["b_s"] = torch.stack([q for q, _ in parts]), torch.stack([f for _, f in parts])
    else:
        # column copies of the gradients and the activations: blocks of 32 rows, stored transposed
        s["a_q"], s["a_s"] = _mx((1e-3 * normal(R, c["n"])).masked_fill_(pad, 0).t().contiguous(), c["a"])
        s["b_q"], s["b_s"] = _mx(normal(R, c["k"]).masked_fill_(pad, 0).t().contiguous(), c["b"])
    return s


def _dispatch_out(plan, *arrays):
    return {**plan, **{k: v for k, v in zip(("q", "s", "qT", "sT") if len(arrays) > 1 else ("rows",), arrays)
                       if v is not None}}


def _run_plain(s):
    c = s["case"]
    if c["op"] == "dispatch":
        plan = _sort(s["experts"], c["experts"], c["align"])
        rows = _gather(s["x"], plan["row_slot"], c["top"])
        if not c["mx"]:
            return _dispatch_out(plan, rows)
        rows = rows.float()
        q, sf = _mx(rows, c["fmt"], c["scale"], c["mma"])
        qT, sT = _mx(rows.t().contiguous(), c["fmt"], c["scale"], c["mma"]) if c["dual"] else (None, None)
        f8, e8 = FP8[c["fmt"]], torch.float8_e8m0fnu
        return _dispatch_out(plan, q.view(f8), sf.view(e8), *((qT.view(f8), sT.view(e8)) if c["dual"] else ()))
    if c["op"] == "dropout":
        n = s["x"].numel()
        words = _philox(torch.arange((n + 3) // 4, device="cuda") + s["offset"], s["seed"]).reshape(-1)[:n]
        keep = (words >= min(int(round(c["p"] * 2.0 ** 32)), 2 ** 32 - 1)).reshape(s["x"].shape)
        y = torch.where(keep, s["x"].float() * (1.0 / (1.0 - c["p"])), 0.0)
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return {"y": y.to(s["x"].dtype)}
    plan = s["plan"]
    if c["op"] in ("combine", "combine_bwd"):
        slot = plan["slot_row"].long()
        live = slot >= 0
        at = torch.where(live, slot, 0)
        w = torch.where(live, s["weights"].float(), 0.0)
        if c["op"] == "combine":
            y = torch.zeros(c["tokens"], c["cols"], device="cuda")
            for j in range(c["top"]):
                y += torch.where(live[:, j, None], s["rows"][at[:, j]].float(), 0.0) * w[:, j, None]
            return {"y": y.to(TYPES[c["y"]])}
        dy = s["dy"].float()
        drows = torch.zeros(s["rows"].shape[0] + 1, c["cols"], dtype=s["rows"].dtype, device="cuda")
        dw = torch.zeros(c["tokens"], c["top"], device="cuda")
        for j in range(c["top"]):
            dw[:, j] = torch.where(live[:, j], (dy * s["rows"][at[:, j]].float()).sum(1), 0.0)
            drows[torch.where(live[:, j], slot[:, j], drows.shape[0] - 1)] = (dy * w[:, j, None]).to(drows.dtype)
        return {"drows": drows[:-1], "dweights": dw}
    st = s["starts"]
    a = _decode(s["a_q"], s["a_s"], c["a"])
    if c["op"] == "gemm":
        y = torch.zeros(a.shape[0], c["n"], dtype=TYPES[c["y"]], device="cuda")
        for e in range(c["experts"]):
            if st[e + 1] > st[e]:
                y[st[e]:st[e + 1]] = a[st[e]:st[e + 1]] @ _decode(s["b_q"][e], s["b_s"][e], c["b"]).t()
        return {"y": y}
    b = _decode(s["b_q"], s["b_s"], c["b"])
    y = torch.zeros(c["experts"], c["n"], c["k"], dtype=TYPES[c["y"]], device="cuda")
    for e in range(c["experts"]):
        y[e] = a[:, st[e]:st[e + 1]] @ b[:, st[e]:st[e + 1]].t()
    return {"dweight": y}


# ------------------------------------------------------------------ the framework's calls
def _run_own(s):
    import block_scaled_precision_02_gb300 as mxq
    c = s["case"]
    if c["op"] == "dispatch":
        p = mxq.expert_sort(s["experts"], c["experts"], c["align"])
        plan = {"offsets": p.offsets, "counts": p.counts, "slot_row": p.slot_row, "row_slot": p.row_slot,
                "block_expert": p.block_expert}
        if not c["mx"]:
            return _dispatch_out(plan, mxq.expert_gather(s["x"], p))
        q, sf, qT, sT = mxq.mx_expert_gather(s["x"], p, c["fmt"], "dual" if c["dual"] else "row", c["scale"],
                                             "mma" if c["mma"] else "canonical")
        f8, e8 = FP8[c["fmt"]], torch.float8_e8m0fnu
        return _dispatch_out(plan, q.view(f8), sf.view(e8), *((qT.view(f8), sT.view(e8)) if c["dual"] else ()))
    if c["op"] == "dropout":
        return {"y": mxq.dropout(s["x"], c["p"], s["seed"], s["offset"], residual=s["residual"])}
    p = s["own_plan"]
    if c["op"] == "combine":
        return {"y": mxq.expert_combine(s["rows"], p, s["weights"], out_dtype=TYPES[c["y"]])}
    if c["op"] == "combine_bwd":
        drows, dw = mxq.expert_combine_backward(s["dy"], s["rows"], p, s["weights"])
        return {"drows": drows, "dweights": dw}
    if c["op"] == "gemm":
        return {"y": mxq.mx_expert_gemm(s["a_q"], s["a_s"], s["b_q"], s["b_s"], p, c["a"], b_fmt=c["b"],
                                        out_dtype=TYPES[c["y"]])}
    return {"dweight": mxq.mx_expert_wgrad(s["a_q"], s["a_s"], s["b_q"], s["b_s"], p, c["a"], b_fmt=c["b"],
                                           out_dtype=TYPES[c["y"]])}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------ the definition in float64
def _bits32(w, lo, n):
    return (w >> lo) & ((1 << n) - 1)


def _mul32(a, const):
    """High and low 32 bits of a 32-bit column times a constant, from products of 16 bits."""
    a0, a1, c0, c1 = _bits32(a, 0, 16), _bits32(a, 16, 16), const & 0xFFFF, const >> 16
    low = a0 * c0
    mid = a1 * c0 + _bits32(low, 16, 48)
    mid2 = a0 * c1 + _bits32(mid, 0, 16)
    return a1 * c1 + _bits32(mid, 16, 48) + _bits32(mid2, 16, 48), _bits32(mid2, 0, 16) * 65536 + _bits32(low, 0, 16)


def _values(q, sf, fmt):
    """Codes and scales in the products' layout as float64, scale by scale."""
    if fmt == "e2m1":
        nibbles = torch.empty(q.shape[0], 2 * q.shape[1], dtype=torch.int64, device=q.device)
        nibbles[:, 0::2], nibbles[:, 1::2] = q.long() % 16, q.long() // 16
        e, m = nibbles % 8 // 2, nibbles % 2
        v = torch.where(e > 0, (1.0 + 0.5 * m.double()) * torch.exp2(e.double() - 1.0), 0.5 * m.double())
        v = torch.where(nibbles >= 8, -v, v)
    else:
        v = q.view(FP8[fmt]).double()
    R, K = v.shape
    r, k = torch.arange(R, device=q.device)[:, None], torch.arange(K // 32, device=q.device)[None, :]
    at = (r // 128 * (K // 128) + k // 4) * 512 + r % 32 * 16 + r // 32 % 4 * 4 + k % 4
    s = sf.reshape(-1)[at].double()
    return v.mul_(torch.exp2(s - 127.0).repeat_interleave(32, 1))


def exact(case, seed):
    """The outputs by definition in float64.  Quantized codes and scales have no entry: a value between two grid
    neighbours is settled by the arithmetic that makes it, not by more bits."""
    s = prepare(case, seed)
    c = s["case"]
    f8 = torch.float64
    if c["op"] == "dropout":
        x = s["x"].reshape(-1).to(f8)
        n = x.numel()
        i = torch.arange((n + 3) // 4, device="cuda") + s["offset"]
        w = [_bits32(i, 0, 32), _bits32(i, 32, 32), torch.zeros_like(i), torch.zeros_like(i)]
        for r in range(10):
            key = [(s["seed"] + r * 0x9E3779B9) % 2 ** 32, (s["seed"] // 2 ** 32 + r * 0xBB67AE85) % 2 ** 32]
            (h0, l0), (h1, l1) = _mul32(w[0], 0xD2511F53), _mul32(w[2], 0xCD9E8D57)
            w = [h1 ^ w[1] ^ key[0], l1, h0 ^ w[3] ^ key[1], l0]
        y = torch.zeros(4 * i.numel(), dtype=f8, device="cuda")
        y[:n] = x / (1.0 - c["p"])
        for j in range(4):
            y[j::4] *= (w[j].to(f8) / 2.0 ** 32 >= round(c["p"] * 2.0 ** 32) / 2.0 ** 32).to(f8)
        y = y[:n].reshape(s["x"].shape)
        return {"y": y if s["residual"] is None else y + s["residual"].to(f8)}
    T, top, E, align, R = c["tokens"], c["top"], c["experts"], c["align"], _rows(c)
    chosen = s["experts"].reshape(-1).cpu().tolist()
    slots = [[] for _ in range(E)]
    for i, e in enumerate(chosen):
        if 0 <= e < E:
            slots[e].append(i)
    offsets, row_slot, block = [0], [], []
    for e in range(E):
        size = -(-len(slots[e]) // align) * align
        row_slot += slots[e] + [-1] * (size - len(slots[e]))
        block += [e] * (size // align)
        offsets.append(offsets[-1] + size)
    row_slot += [-1] * (R - len(row_slot))
    block += [-1] * (R // align - len(block))
    slot_row = [-1] * (T * top)
    for r, i in enumerate(row_slot):
        if i >= 0:
            slot_row[i] = r

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    if c["op"] == "dispatch":
        out = {"offsets": ints(offsets), "counts": ints([len(x) for x in slots]), "slot_row": ints(slot_row).reshape(T, top),
               "row_slot": ints(row_slot), "block_expert": ints(block)}
        if c["mx"]:
            return {**out, "q": None, "s": None, **({"qT": None, "sT": None} if c["dual"] else {})}
        rows = torch.zeros(R, c["cols"], dtype=f8, device="cuda")
        at = ints(row_slot).long()
        rows[at >= 0] = s["x"].to(f8)[at[at >= 0] // top]
        return {**out, "rows": rows}
    if c["op"] in ("combine", "combine_bwd"):
        live = [i for i in range(T * top) if slot_row[i] >= 0]
        li = torch.tensor(live, dtype=torch.int64, device="cuda")
        row = ints(slot_row).long()[li]
        token = li // top
        w = s["weights"].reshape(-1)[li].to(f8)
        picked = s["rows"][row].to(f8)
        if c["op"] == "combine":
            y = torch.zeros(T, c["cols"], dtype=f8, device="cuda")
            return {"y": y.index_add_(0, token, picked * w[:, None])}
        dy = s["dy"].to(f8)[token]
        dw = torch.zeros(T * top, dtype=f8, device="cuda")
        dw[li] = torch.einsum("rc,rc->r", dy, picked)
        drows = torch.zeros(R, c["cols"], dtype=f8, device="cuda")
        drows[row] = dy * w[:, None]
        return {"drows": drows, "dweights": dw.reshape(T, top)}
    a = _values(s["a_q"], s["a_s"], c["a"])
    if c["op"] == "gemm":
        y = torch.zeros(R, c["n"], dtype=f8, device="cuda")
        for e in range(E):
            part = slice(offsets[e], offsets[e + 1])
            if slots[e]:
                y[part] = torch.einsum("rk,nk->rn", a[part], _values(s["b_q"][e], s["b_s"][e], c["b"]))
        return {"y": y}
    b = _values(s["b_q"], s["b_s"], c["b"])
    parts = [slice(offsets[e], offsets[e + 1]) for e in range(E)]
    return {"dweight": torch.stack([torch.einsum("nr,kr->nk", a[:, p], b[:, p]) for p in parts])}


def work(case):
    c = case
    if c["op"] == "dropout":
        n = c["rows"] * c["cols"]
        # a generator's call for four elements: ten rounds of two products and six other operations
        return {"bytes": n * SIZE[c["x"]] * (3 if c["residual"] else 2), "flops": 23 * n}
    slots, R, E = c["tokens"] * c["top"], _rows(c), c["experts"]
    if c["op"] in ("gemm", "wgrad"):
        a = CODE_BYTES[c["a"]] + 1 / 32
        b = CODE_BYTES[c["b"]] + 1 / 32
        flops = 2 * slots * c["n"] * c["k"]
        if c["op"] == "gemm":       # weights of experts that can have a token
            return {"bytes": int(slots * c["k"] * a + min(E, slots) * c["n"] * c["k"] * b + R * c["n"] * SIZE[c["y"]]),
                    "flops": flops}
        return {"bytes": int(slots * (c["n"] * a + c["k"] * b) + E * c["n"] * c["k"] * SIZE[c["y"]]), "flops": flops}
    kept = slots * (1.0 - c["dropped"])
    if c["op"] == "dispatch":
        plan = 4 * (2 * slots + R + 2 * E + R // c["align"])
        if not c["mx"]:
            return {"bytes": plan + (c["tokens"] + R) * c["cols"] * SIZE[c["x"]], "flops": slots}
        sides = 2 if c["dual"] else 1
        return {"bytes": plan + c["tokens"] * c["cols"] * 2 + sides * R * c["cols"] * 33 // 32,
                "flops": 4 * sides * R * c["cols"]}
    n = c["tokens"] * c["cols"]
    if c["op"] == "combine":
        return {"bytes": int(kept * c["cols"] * SIZE[c["x"]] + n * SIZE[c["y"]] + 8 * slots), "flops": 2 * kept * c["cols"]}
    return {"bytes": int((kept + R) * c["cols"] * SIZE[c["x"]] + n * SIZE[c["y"]] + 12 * slots), "flops": 3 * kept * c["cols"]}
