"""The 8-bit linear layer's operators and the gradient clipping of its training step, as cases to measure.

Three operators:

  fwd   Y = Xq Wq^T * sx * sw (+ s (X A^T) B^T): a frozen weight in 8-bit integers with one scale per output
        channel, tokens quantized to 8 bits with one scale per token, products in whole numbers.  Returns Y
        and T = X A^T (the forward's saved adapter product).
  bwd   the same layer's input gradient: the channel scales go into dY, whose tokens are quantized the same
        way; dX = Vq Wq * sv + s (dY B) A.  Returns dX and U = dY B.
  clip  the Euclidean norm of all gradients together, and the gradients scaled down to max_norm.  Returns the
        scaled gradients (one flat tensor per type) and the norm.

A row is quantized by scale = fp32(amax / 127), code = 127 x / amax rounded to the nearest whole number, ties
to even, decided exactly; a zero row has scale 0 and codes 0.

`run` computes the plain form where `own` is false, and makes the framework's calls where it is true.
"""
import math

import torch

own = False

# (out features, in features) of a LLaMA-3-8B layer's seven linear weights
LAYER_8B = ((4096, 4096), (1024, 4096), (1024, 4096), (4096, 4096), (14336, 4096), (14336, 4096), (4096, 14336))
S = 2.0          # adapter scale alpha / r
EPS = 1e-6       # added to the norm before the division, as clipping usually does


# ------------------------------------------------------------------------------------------------ the cases
def listed():
    return [
        # one token through an attention projection without an adapter: the smallest call of a decode step
        {"name": "fwd 1 token 4096x4096", "op": "fwd", "m": 1, "n": 4096, "k": 4096, "rank": 0},
        # 16 concurrent sequences through the MLP's down projection while its adapter is still separate
        {"name": "fwd 16 tokens 8B down r16", "op": "fwd", "m": 16, "n": 4096, "k": 14336, "rank": 16},
        # a prompt chunk of 512 tokens through the gate projection, its adapter merged
        {"name": "fwd 512 tokens 8B gate", "op": "fwd", "m": 512, "n": 14336, "k": 4096, "rank": 0},
        # the training step's forward (batch 4 x 1024 tokens), rank 16
        {"name": "fwd 4096 tokens 8B gate r16", "op": "fwd", "m": 4096, "n": 14336, "k": 4096, "rank": 16},
        # odd sizes: a short batch, an odd channel count, an odd rank
        {"name": "fwd 77 tokens 1001x2064 r5", "op": "fwd", "m": 77, "n": 1001, "k": 2064, "rank": 5},
        # a short fine-tuning batch's input gradient through the attention projection
        {"name": "bwd 129 tokens 4096x4096 r8", "op": "bwd", "m": 129, "n": 4096, "k": 4096, "rank": 8},
        # the training step's input gradients through large MLP weights: a long reduction and a longer one
        {"name": "bwd 4096 tokens 8B gate r16", "op": "bwd", "m": 4096, "n": 14336, "k": 4096, "rank": 16},
        {"name": "bwd 2048 tokens 70B gate r64", "op": "bwd", "m": 2048, "n": 28672, "k": 8192, "rank": 64},
        # clipping one layer's adapters (a step that trains few layers): 14 small tensors
        {"name": "clip 1 layer r16 fp32", "op": "clip", "layers": 1, "rank": 16, "dtype": "float32", "odd": False,
         "std": 1e-2, "max_norm": 0.3},
        # clipping all adapters of the 8B model: 448 tensors, 42 M values
        {"name": "clip 32 layers r16 fp32", "op": "clip", "layers": 32, "rank": 16, "dtype": "float32", "odd": False,
         "std": 1e-2, "max_norm": 0.3},
        # the same model at rank 64 with bf16 gradients: 168 M values
        {"name": "clip 32 layers r64 bf16", "op": "clip", "layers": 32, "rank": 64, "dtype": "bfloat16", "odd": False,
         "std": 1e-2, "max_norm": 0.3},
        # gradients of three types with odd sizes, so that most outputs start off the 16-byte grid
        {"name": "clip 9 layers r7 mixed odd", "op": "clip", "layers": 9, "rank": 7, "dtype": "mixed", "odd": True,
         "std": 1e-3, "max_norm": 1.0},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("fwd", "fwd", "bwd", "clip"))
    if op == "clip":
        return {"op": op, "layers": _log_int(rng, 1, 24), "rank": _log_int(rng, 1, 48),
                "dtype": rng.choice(("float32", "bfloat16", "float16", "mixed")), "odd": rng.random() < 0.5,
                "std": 10.0 ** rng.uniform(-3, 0), "max_norm": rng.choice((0.1, 0.3, 1.0, 10.0))}
    while True:
        m = _log_int(rng, 1, 4096)
        n = _log_int(rng, 64, 14336)
        k = 16 * _log_int(rng, 4, 896)
        rank = rng.choice((0, 0, 1, 4, 8, 16, 16, 33, 64))
        if op == "bwd":
            n = (n + 7) // 8 * 8
        if m * n * k <= 2.0e11:
            return {"op": op, "m": m, "n": n, "k": k, "rank": rank}


# ------------------------------------------------------------------------------------------------ the inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, std):
    return torch.randn(shape, generator=g, device="cuda").mul_(std)


def _clip_shapes(case):
    shapes = []
    for n, k in LAYER_8B:
        if case["odd"]:
            n, k = n // 3 + 2, k // 5 + 4          # 1367, 343 and 4780 by 823 and 2871: odd counts at odd ranks
        shapes += [(case["rank"], k), (n, case["rank"])]
    return shapes * case["layers"]


def _clip_types(case, count):
    if case["dtype"] != "mixed":
        return [getattr(torch, case["dtype"])] * count
    return [(torch.float32, torch.bfloat16, torch.float16)[i % 3] for i in range(count)]


def _prepare_clip(case, g):
    shapes = _clip_shapes(case)
    types = _clip_types(case, len(shapes))
    grads = [_normal(g, sh, case["std"]).to(t) for sh, t in zip(shapes, types)]
    # the optimizer reads the clipped gradients from one flat buffer per type
    flat = {t: torch.empty(sum(x.numel() for x in grads if x.dtype == t), dtype=t, device="cuda")
            for t in dict.fromkeys(types)}
    outs, at = [], dict.fromkeys(types, 0)
    for x in grads:
        outs.append(flat[x.dtype][at[x.dtype]:at[x.dtype] + x.numel()].view(x.shape))
        at[x.dtype] += x.numel()
    state = {"case": case, "grads": grads, "flat": flat, "max_norm": case["max_norm"]}
    if own:
        from qlora_quantized_linear_b200 import lbq
        state["plan"] = lbq.GradClip(grads, outs)
    return state


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] == "clip":
        return _prepare_clip(case, g)
    m, n, k, r = case["m"], case["n"], case["k"], case["rank"]
    # the weight N(0, 0.02^2) with 0.1 % of its input channels 20 times as large
    W = _normal(g, (n, k), 0.02)
    far = torch.randperm(k, generator=g, device="cuda")[:max(1, k // 1000)]
    W[:, far] *= 20.0
    W = W.to(torch.bfloat16)
    # what a user keeps of it: 8-bit codes and one scale per output channel
    amax = W.abs().amax(1, keepdim=True).double()
    codes = torch.where(amax > 0, (W.double() * 127.0 / amax).round_(), 0.0).to(torch.int8)
    scale = (amax.squeeze(1) / 127.0).float()
    del W, amax
    # activations N(0, 1) with a few outlier channels; gradients whose size differs from token to token
    if case["op"] == "fwd":
        x = _normal(g, (m, k), 1.0)
        x[:, far] *= 10.0
    else:
        x = _normal(g, (m, n), 0.1)
        x *= torch.exp(_normal(g, (m, 1), 1.5))
    state = {"case": case, "x": x.to(torch.bfloat16), "codes": codes, "scale": scale, "A": None, "B": None}
    if r:
        state["A"] = _normal(g, (r, k), 0.01).to(torch.bfloat16)
        state["B"] = _normal(g, (n, r), 0.01).to(torch.bfloat16)
    if own:
        from qlora_quantized_linear_b200 import lbq
        fwd = case["op"] == "fwd"
        state["weight"] = lbq.Int8Weight(n, k, codes=codes, scale=scale)
        state["out"] = torch.empty((m, n if fwd else k), device="cuda")
        state["saved"] = torch.empty((m, r), device="cuda") if r else None
        size = lbq.linear_i8_fwd_workspace if fwd else lbq.linear_i8_bwd_workspace
        state["workspace"] = size(m, state["weight"], r)
    return state


# ------------------------------------------------------------------------------------------------ one pass
def _quantize_rows(v):
    """(codes, scale) of the rows of v (32-bit floats); the codes as 32-bit floats."""
    amax = v.abs().amax(1, keepdim=True)
    codes = torch.round(v.double() * 127.0 / amax.double())        # next to a half in 64 bits
    codes = torch.where(amax > 0, codes, 0.0).float()
    return codes, amax / 127.0


def _plain_fwd(st):
    x = st["x"].float()
    codes, scale = _quantize_rows(x)
    y = (codes @ st["codes"].float().t()) * scale * st["scale"]
    if st["A"] is None:
        return {"Y": y}
    t = x @ st["A"].float().t()
    return {"Y": y + S * (t @ st["B"].float().t()), "T": t}


def _plain_bwd(st):
    dy = st["x"].float()
    codes, scale = _quantize_rows(dy * st["scale"])
    dx = (codes @ st["codes"].float()) * scale
    if st["A"] is None:
        return {"dX": dx}
    u = dy @ st["B"].float()
    return {"dX": dx + S * (u @ st["A"].float()), "U": u}


def _plain_clip(st):
    norm = torch.cat([x.float().flatten() for x in st["grads"]]).double().square().sum().sqrt()   # a long sum
    coef = (st["max_norm"] / (norm + EPS)).clamp(max=1.0).float()
    out = [(torch.cat([x.float().flatten() for x in st["grads"] if x.dtype == t]) * coef).to(t) for t in st["flat"]]
    return {"out": out, "norm": norm.float().reshape(1)}


def run(st):
    op = st["case"]["op"]
    if not own:
        return {"fwd": _plain_fwd, "bwd": _plain_bwd, "clip": _plain_clip}[op](st)
    from qlora_quantized_linear_b200 import lbq
    if op == "clip":
        norm = st["plan"].clip(st["max_norm"])
        return {"out": list(st["flat"].values()), "norm": norm}
    if op == "fwd":
        y, t = lbq.linear_i8_fwd(st["x"], st["weight"], st["A"], st["B"], S, Y=st["out"], T=st["saved"],
                                 workspace=st["workspace"])
        return {"Y": y} if t is None else {"Y": y, "T": t}
    dx, u = lbq.linear_i8_bwd(st["x"], st["weight"], st["A"], st["B"], S, dX=st["out"], U=st["saved"],
                              workspace=st["workspace"])
    return {"dX": dx} if u is None else {"dX": dx, "U": u}


# ------------------------------------------------------------------------------------------------ what it takes
def work(case):
    if case["op"] == "clip":
        shapes = _clip_shapes(case)
        size = {torch.float32: 4, torch.bfloat16: 2, torch.float16: 2}
        moved = sum(a * b * size[t] for (a, b), t in zip(shapes, _clip_types(case, len(shapes))))
        return {"bytes": 2 * moved + 4, "flops": 3 * sum(a * b for a, b in shapes)}
    m, n, k, r = case["m"], case["n"], case["k"], case["rank"]
    read, write = (k, n) if case["op"] == "fwd" else (n, k)
    return {"bytes": 2 * m * read + n * k + 4 * n + 4 * m * write + 2 * r * (n + k) + 4 * m * r,
            "flops": 2 * m * n * k + 2 * m * r * (n + k)}


# ------------------------------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "clip":
        norm = torch.sqrt(torch.stack([x.double().pow(2).sum() for x in st["grads"]]).sum())
        coef = min(1.0, case["max_norm"] / (norm.item() + EPS))
        parts = {t: [] for t in st["flat"]}
        for x in st["grads"]:
            parts[x.dtype].append(x.double().flatten() * coef)
        return {"out": [torch.cat(p) for p in parts.values()], "norm": norm.reshape(1)}
    f = torch.float64
    x, w, sw = st["x"].to(f), st["codes"].to(f), st["scale"].to(f)
    fwd = case["op"] == "fwd"
    # the backward's scaled gradient is rounded to 32 bits by definition; the forward takes the activations as they are
    v = x if fwd else (x * sw[None, :]).float().to(f)
    top = v.abs().max(dim=1).values
    q = torch.round((v * 127.0) / torch.where(top == 0, torch.ones_like(top), top)[:, None])
    main = torch.einsum("mk,nk->mn" if fwd else "mn,nk->mk", q, w) * (top / 127.0)[:, None]
    if fwd:
        main = main * sw[None, :]
    name, saved = ("Y", "T") if fwd else ("dX", "U")
    if st["A"] is None:
        return {name: main}
    a, b = st["A"].to(f), st["B"].to(f)
    t = torch.einsum("mk,rk->mr", x, a) if fwd else torch.einsum("mn,nr->mr", x, b)
    return {name: main + S * torch.einsum("mr,nr->mn" if fwd else "mr,rk->mk", t, b if fwd else a), saved: t}
