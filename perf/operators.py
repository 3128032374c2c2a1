"""The layer and gradient operators, as cases that can be timed and compared.

Three operators of one training step of a learner, in the order in which the
step runs them:

  linear, linear_backward        y = act(x w^T + bias) + residual, and its
                                 gradients
  gated_ffn, gated_ffn_backward  h = act(x wg^T) * (x wu^T), and its gradients
  clip, pack                     the norm over all gradient tensors, and the
                                 clipped gradients in their own types or end to
                                 end in the learner's flat binary32 layout

A case names its operator under "op".  With `own` false, `run` computes it in
elementary torch operations in 32 bits (64 for the norm's long sum), rounded
once at the end; with `own` true it calls the package.
"""

import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one token through a projection of a decoder: the weights' bytes count
        {"name": "linear one row", "op": "linear", "type": "bf16", "m": 1, "n": 4096, "k": 4096,
         "act": "gelu", "bias": True, "residual": True, "pre": False, "pad": 0},
        # a 1000-way classifier on 2048 features (ResNet-50's last layer), a ragged last batch
        {"name": "linear classifier", "op": "linear", "type": "fp16", "m": 777, "n": 1000, "k": 2048,
         "act": "none", "bias": True, "residual": False, "pre": False, "pad": 0},
        # the second projection of a feed-forward block on a long batch, with its residual
        {"name": "linear large", "op": "linear", "type": "bf16", "m": 8192, "n": 8192, "k": 8192,
         "act": "none", "bias": True, "residual": True, "pre": False, "pad": 0},
        # gate matrices of a recurrent layer of width 1280 (3 * 1280 rows), odd batch
        {"name": "linear backward gates", "op": "linear_backward", "type": "bf16", "m": 1531, "n": 3840,
         "k": 1280, "act": "gelu_tanh", "bias": True, "flat": False, "pad": 0},
        # a projection's gradients, dw in binary32 for the learner's flat gradient
        {"name": "linear backward large", "op": "linear_backward", "type": "bf16", "m": 8192, "n": 8192,
         "k": 4096, "act": "none", "bias": True, "flat": True, "pad": 0},
        # a few tokens while answering: nothing is kept for a backward pass
        {"name": "ffn three rows", "op": "gated_ffn", "type": "bf16", "m": 3, "d": 2048, "f": 8192,
         "act": "silu", "save": False, "pad": 0},
        # the forward pass of training on a long batch, gate and up kept
        {"name": "ffn large", "op": "gated_ffn", "type": "bf16", "m": 8192, "d": 4096, "f": 12288,
         "act": "silu", "save": True, "pad": 0},
        # a short ragged batch, a width that is no power of two, rows of a wider buffer
        {"name": "ffn backward ragged", "op": "gated_ffn_backward", "type": "fp16", "m": 333, "d": 1152,
         "f": 3456, "act": "gelu_tanh", "pad": 64},
        # the backward pass of training on a long batch
        {"name": "ffn backward large", "op": "gated_ffn_backward", "type": "bf16", "m": 8192, "d": 4096,
         "f": 12288, "act": "silu", "pad": 0},
        # one small layer's gradients: latency alone
        {"name": "clip few", "op": "clip", "type": "bf16", "layout": "spread", "tensors": 5, "least": 3,
         "most": 40000, "shape_seed": 1, "clip": 0.5, "norm": "l2", "unscale": 1.0},
        # ResNet-50's 161 tensors: fp16 convolutions, fp32 normalisation layers, a scaled loss
        {"name": "clip resnet50", "op": "clip", "type": "fp16", "layout": "resnet50", "tensors": 161, "least": 64,
         "most": 2359296, "shape_seed": 0, "clip": 0.5, "norm": "l2", "unscale": 0.125},
        # a billion bf16 gradients in 64 tensors into the learner's flat layout
        {"name": "pack 1b", "op": "pack", "type": "bf16", "layout": "even", "tensors": 64, "least": 1 << 24,
         "most": 1 << 24, "shape_seed": 0, "clip": 0.5, "norm": "l2", "unscale": 1.0},
    ]


def _size(rng, low, high):
    """Log-uniform in [low, high]; one third as it falls, one third a multiple of 8, one third of 64."""
    v = math.exp(rng.uniform(math.log(low), math.log(high)))
    step = rng.choice((1, 8, 64))
    v = int(min(high, max(low, round(v / step) * step)))
    return v - 8 if v == 3 << 10 else v


def draw(rng):
    op = rng.choice(("linear", "linear_backward", "gated_ffn", "gated_ffn_backward", "clip", "pack"))
    half = rng.choice(("bf16", "bf16", "fp16"))
    if op in ("clip", "pack"):
        tensors = _size(rng, 1, 300)
        most = _size(rng, 64, min(1 << 24, (1 << 30) // tensors))
        return {"op": op, "type": rng.choice(("bf16", "fp16", "fp32")), "layout": "spread", "tensors": tensors,
                "least": max(1, most // rng.choice((1, 10, 1000))), "most": most, "shape_seed": rng.randrange(1 << 20),
                "clip": rng.choice((0.5, 0.5, 1e9)), "norm": rng.choice(("l2", "l2", "max")),
                "unscale": rng.choice((1.0, 0.125))}
    act = rng.choice(("silu", "gelu", "gelu_tanh", "relu"))
    m, n, k = _size(rng, 1, 8192), _size(rng, 64, 8192), _size(rng, 64, 8192)
    pad = rng.choice((0, 0, 8, 13))
    if op == "linear":
        return {"op": op, "type": half, "m": m, "n": n, "k": k, "act": rng.choice(("none", act)),
                "bias": rng.random() < 0.5, "residual": rng.random() < 0.5, "pre": rng.random() < 0.3, "pad": pad}
    if op == "linear_backward":
        act = rng.choice(("none", act))
        return {"op": op, "type": half, "m": m, "n": n, "k": min(k, 4096), "act": act, "bias": rng.random() < 0.5,
                "flat": act == "none" and rng.random() < 0.5, "pad": pad}
    c = {"op": op, "type": half, "m": m, "d": min(k, 4096), "f": n, "act": act, "pad": pad}
    return dict(c, save=rng.random() < 0.5) if op == "gated_ffn" else c


# ------------------------------------------------------------------- inputs

def _resnet50():
    """(elements, whether a convolution or the classifier's matrix) of ResNet-50's tensors."""
    out, wide = [(64 * 3 * 49, True), (64, False), (64, False)], 64
    for p, blocks in ((64, 3), (128, 4), (256, 6), (512, 3)):
        for b in range(blocks):
            out += [(p * wide, True), (p, False), (p, False), (9 * p * p, True), (p, False), (p, False),
                    (4 * p * p, True), (4 * p, False), (4 * p, False)]
            out += [(4 * p * wide, True), (4 * p, False), (4 * p, False)] if b == 0 else []
            wide = 4 * p
    return out + [(1000 * 2048, True), (1000, False)]


def _layout(case):
    """[(elements, type name)] of the gradient tensors."""
    if case["layout"] == "resnet50":
        return [(n, case["type"] if big else "fp32") for n, big in _resnet50()]
    if case["layout"] == "even":
        return [(case["most"], case["type"])] * case["tensors"]
    r = np.random.RandomState(case["shape_seed"])
    sizes = np.exp(r.uniform(math.log(case["least"]), math.log(case["most"] + 0.5), case["tensors"]))
    vectors = r.random_sample(case["tensors"]) < 0.25  # gains and biases stay in 32 bits
    return [(max(1, int(s)), "fp32" if v else case["type"]) for s, v in zip(sizes, vectors)]


def _draws(seed, device="cuda"):
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)

    def normal(shape, dtype, scale=1.0, pad=0):
        """A normal draw; with `pad`, rows of a buffer that is `pad` columns wider."""
        wide = shape[:-1] + (shape[-1] + pad,)
        t = torch.randn(wide, generator=gen, device=device, dtype=torch.float32).mul_(scale).to(dtype)
        return t[..., :shape[-1]]
    return normal


def _grads(case, seed):
    """Gradients whose scale differs from tensor to tensor by up to 1000."""
    normal = _draws(seed)
    scales = 10.0 ** np.random.RandomState(seed % (1 << 31)).uniform(-4.5, -1.5, 4096)
    return [normal((n,), TYPES[t], float(scales[i % 4096])) for i, (n, t) in enumerate(_layout(case))]


def _inputs(case, seed):
    """The tensors of a layer's case, by name."""
    normal, t, op, pad = _draws(seed), TYPES[case["type"]], case["op"], case["pad"]
    m = case["m"]
    if op == "linear":
        n, k = case["n"], case["k"]
        return {"x": normal((m, k), t, 1.0, pad), "w": normal((n, k), t, k ** -0.5),
                "bias": normal((n,), t, 0.1) if case["bias"] else None,
                "residual": normal((m, n), t) if case["residual"] else None}
    if op == "linear_backward":
        n, k = case["n"], case["k"]
        return {"dy": normal((m, n), t), "x": normal((m, k), t, 1.0, pad), "w": normal((n, k), t, k ** -0.5),
                "pre": normal((m, n), t) if case["act"] != "none" else None}
    d, f = case["d"], case["f"]
    x, wg, wu = normal((m, d), t, 1.0, pad), normal((f, d), t, d ** -0.5), normal((f, d), t, d ** -0.5)
    if op == "gated_ffn":
        return {"x": x, "w_gate": wg, "w_up": wu}
    return {"dh": normal((m, f), t), "x": x, "w_gate": wg, "w_up": wu, "gate": normal((m, f), t), "up": normal((m, f), t)}


def prepare(case, seed):
    """Inputs and what a training program keeps beside them: output buffers, workspace, the gradient set."""
    state = {"case": case}
    if case["op"] in ("clip", "pack"):
        grads = state["grads"] = _grads(case, seed)
        if own:
            from sparsified_gradient_compression_amd import dgc
            state["set"] = dgc.GradSet([g.shape for g in grads], [g.dtype for g in grads])
        if case["op"] == "pack":
            state["flat"] = torch.empty(sum(g.numel() for g in grads), dtype=torch.float32, device="cuda")
            return state
        # clipped gradients go into one bucket per type, tensors end to end
        names = [t for _, t in _layout(case)]
        state["buckets"] = {t: torch.empty(sum(g.numel() for g, u in zip(grads, names) if u == t),
                                           dtype=TYPES[t], device="cuda") for t in sorted(set(names))}
        at, state["out"] = dict.fromkeys(names, 0), []
        for g, t in zip(grads, names):
            state["out"].append(state["buckets"][t][at[t]:at[t] + g.numel()])
            at[t] += g.numel()
        state["names"] = names
        return state
    state.update(_inputs(case, seed))
    m, t = case["m"], TYPES[case["type"]]

    def new(*shape, dtype=t):
        return torch.empty(shape, dtype=dtype, device="cuda")

    if case["op"] == "linear":
        state.update(out=new(m, case["n"]), pre=new(m, case["n"]) if case["pre"] else None)
    elif case["op"] == "linear_backward":
        g = torch.float32 if case["flat"] else t
        state.update(dx=new(m, case["k"]), dw=new(case["n"], case["k"], dtype=g),
                     dbias=new(case["n"], dtype=g) if case["bias"] else None)
    elif case["op"] == "gated_ffn":
        state.update(out=new(m, case["f"]), gate=new(m, case["f"]) if case["save"] else None,
                     up=new(m, case["f"]) if case["save"] else None)
    else:
        state.update(dx=new(m, case["d"]), dw_gate=new(case["f"], case["d"]), dw_up=new(case["f"], case["d"]))
    if own:
        from sparsified_gradient_compression_amd import dgc
        if case["op"].startswith("linear"):
            state["workspace"] = dgc.linear_workspace(m, case["n"], case["k"], backward=case["op"] != "linear")
        else:
            state["workspace"] = dgc.gated_ffn_workspace(m, case["d"], case["f"], backward=case["op"] != "gated_ffn")
    return state


# --------------------------------------------------------------- plain forms

def _act(name, z):
    if name == "relu":
        return z.clamp_min(0)
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _act_slope(name, z):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    if name == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def _run_linear(s, c):
    z = s["x"].float() @ s["w"].float().t()
    if c["bias"]:
        z = z + s["bias"].float()
    y = _act(c["act"], z)
    if c["residual"]:
        y = y + s["residual"].float()
    t = s["x"].dtype
    return {"y": y.to(t), "pre": z.to(t)} if c["pre"] else {"y": y.to(t)}


def _run_linear_backward(s, c):
    t, dz = s["x"].dtype, s["dy"].float()
    if c["act"] != "none":
        dz = dz * _act_slope(c["act"], s["pre"].float())
    g = torch.float32 if c["flat"] else t
    out = {"dx": (dz @ s["w"].float()).to(t), "dw": (dz.t() @ s["x"].float()).to(g)}
    return dict(out, dbias=dz.sum(0, dtype=torch.float64).to(g)) if c["bias"] else out


def _run_gated_ffn(s, c):
    t, x = s["x"].dtype, s["x"].float()
    a, b = x @ s["w_gate"].float().t(), x @ s["w_up"].float().t()
    out = {"h": (_act(c["act"], a) * b).to(t)}
    return dict(out, gate=a.to(t), up=b.to(t)) if c["save"] else out


def _run_gated_ffn_backward(s, c):
    t, x, dh = s["x"].dtype, s["x"].float(), s["dh"].float()
    a, b = s["gate"].float(), s["up"].float()
    da, db = dh * b * _act_slope(c["act"], a), dh * _act(c["act"], a)
    return {"dx": (da @ s["w_gate"].float() + db @ s["w_up"].float()).to(t),
            "dw_gate": (da.t() @ x).to(t), "dw_up": (db.t() @ x).to(t)}


def _norm_and_scale(s, c):
    """The norm of the unscaled gradients in 64 bits, and the factor unscale * min(1, clip / norm) in 32."""
    if c["norm"] == "max":
        norm = torch.stack([g.abs().max().double() for g in s["grads"]]).max()
    else:
        norm = torch.stack([g.double().square().sum() for g in s["grads"]]).sum().sqrt()
    norm = norm * c["unscale"]
    return norm, (torch.where(norm > c["clip"], c["clip"] / norm, torch.ones_like(norm)) * c["unscale"]).float()


def _run_clip(s, c):
    norm, scale = _norm_and_scale(s, c)
    out = [(g.float() * scale).to(g.dtype) for g in s["grads"]]
    return {"norm": norm.reshape(1), "scale": scale.reshape(1),
            "buckets": {t: torch.cat([o for o, u in zip(out, s["names"]) if u == t]) for t in s["buckets"]}}


def _run_pack(s, c):
    norm, scale = _norm_and_scale(s, c)
    return {"norm": norm.reshape(1), "scale": scale.reshape(1),
            "flat": torch.cat([g.float() for g in s["grads"]]) * scale}


PLAIN = {"linear": _run_linear, "linear_backward": _run_linear_backward, "gated_ffn": _run_gated_ffn,
         "gated_ffn_backward": _run_gated_ffn_backward, "clip": _run_clip, "pack": _run_pack}


# ------------------------------------------------------------ the package's

def _own_linear(s, c, dgc):
    dgc.linear(s["x"], s["w"], bias=s["bias"], residual=s["residual"], act=c["act"], out=s["out"], pre=s["pre"],
               workspace=s["workspace"])
    return {"y": s["out"], "pre": s["pre"]} if c["pre"] else {"y": s["out"]}


def _own_linear_backward(s, c, dgc):
    dgc.linear_backward(s["dy"], s["x"], s["w"], pre=s["pre"], act=c["act"], dx=s["dx"], dw=s["dw"],
                        dbias=s["dbias"], workspace=s["workspace"])
    out = {"dx": s["dx"], "dw": s["dw"]}
    return dict(out, dbias=s["dbias"]) if c["bias"] else out


def _own_gated_ffn(s, c, dgc):
    dgc.gated_ffn(s["x"], s["w_gate"], s["w_up"], act=c["act"], out=s["out"], gate=s["gate"], up=s["up"],
                  workspace=s["workspace"])
    return {"h": s["out"], "gate": s["gate"], "up": s["up"]} if c["save"] else {"h": s["out"]}


def _own_gated_ffn_backward(s, c, dgc):
    dgc.gated_ffn_backward(s["dh"], s["x"], s["w_gate"], s["w_up"], s["gate"], s["up"], act=c["act"], dx=s["dx"],
                           dw_gate=s["dw_gate"], dw_up=s["dw_up"], workspace=s["workspace"])
    return {"dx": s["dx"], "dw_gate": s["dw_gate"], "dw_up": s["dw_up"]}


def _own_clip(s, c, dgc):
    s["set"].clip(s["grads"], c["clip"], out=s["out"], norm=c["norm"], unscale=c["unscale"])
    return {"norm": s["set"].total, "scale": s["set"].scale, "buckets": s["buckets"]}


def _own_pack(s, c, dgc):
    s["set"].pack(s["grads"], s["flat"], c["clip"], norm=c["norm"], unscale=c["unscale"])
    return {"norm": s["set"].total, "scale": s["set"].scale, "flat": s["flat"]}


OWN = {"linear": _own_linear, "linear_backward": _own_linear_backward, "gated_ffn": _own_gated_ffn,
       "gated_ffn_backward": _own_gated_ffn_backward, "clip": _own_clip, "pack": _own_pack}


def run(state):
    case = state["case"]
    if own:
        from sparsified_gradient_compression_amd import dgc
        return OWN[case["op"]](state, case, dgc)
    return PLAIN[case["op"]](state, case)


# ------------------------------------------------------------------- exact

def _pair64(name, z):
    """act(z) and its slope in 64 bits, from the definitions: z * Phi(z), z * sigmoid(z), tanh by its exponential."""
    if name == "relu":
        return torch.where(z > 0, z, 0.0), torch.where(z > 0, 1.0, 0.0).to(z.dtype)
    if name == "silu":
        p = torch.sigmoid(z)
        return z * p, p + z * p * torch.sigmoid(-z)
    if name == "gelu":
        cdf, pdf = 0.5 * torch.erfc(-z / 2 ** 0.5), torch.exp(-z ** 2 / 2) / (2 * math.pi) ** 0.5
        return z * cdf, cdf + z * pdf
    if name == "gelu_tanh":  # (1 + tanh(q)) / 2 = sigmoid(2 q)
        q2 = 2 * (2 / math.pi) ** 0.5 * (z + 0.044715 * z ** 3)
        p = torch.sigmoid(q2)
        return z * p, p + z * p * torch.sigmoid(-q2) * 2 * (2 / math.pi) ** 0.5 * (1 + 0.134145 * z ** 2)
    return z, torch.ones_like(z)


def exact(case, seed):
    op = case["op"]
    if op in ("clip", "pack"):
        grads, names = [g.to(torch.float64) for g in _grads(case, seed)], [t for _, t in _layout(case)]
        if case["norm"] == "max":
            norm = max(torch.linalg.vector_norm(g, math.inf) for g in grads) * case["unscale"]
        else:
            norm = torch.linalg.vector_norm(torch.stack([torch.linalg.vector_norm(g) for g in grads])) * case["unscale"]
        scale = case["unscale"] * (case["clip"] / norm).clamp(max=1.0)
        out = {"norm": norm.reshape(1), "scale": scale.reshape(1)}
        if op == "pack":
            return dict(out, flat=torch.cat([g * scale for g in grads]))
        return dict(out, buckets={t: torch.cat([g * scale for g, u in zip(grads, names) if u == t])
                                  for t in sorted(set(names))})
    s = {k: v if v is None else v.to(torch.float64) for k, v in _inputs(case, seed).items()}
    if op == "linear":
        z = torch.mm(s["x"], s["w"].t()) if s["bias"] is None else torch.addmm(s["bias"], s["x"], s["w"].t())
        y = _pair64(case["act"], z)[0]
        y = y if s["residual"] is None else y + s["residual"]
        return {"y": y, "pre": z} if case["pre"] else {"y": y}
    if op == "linear_backward":
        dz = s["dy"] if s["pre"] is None else s["dy"] * _pair64(case["act"], s["pre"])[1]
        out = {"dx": torch.mm(dz, s["w"]), "dw": torch.mm(dz.t(), s["x"])}
        return dict(out, dbias=dz.sum(0)) if case["bias"] else out
    if op == "gated_ffn":
        a, b = torch.mm(s["x"], s["w_gate"].t()), torch.mm(s["x"], s["w_up"].t())
        out = {"h": _pair64(case["act"], a)[0] * b}
        return dict(out, gate=a, up=b) if case["save"] else out
    value, slope = _pair64(case["act"], s["gate"])
    da, db = s["dh"] * s["up"] * slope, s["dh"] * value
    return {"dx": torch.mm(da, s["w_gate"]) + torch.mm(db, s["w_up"]),
            "dw_gate": torch.mm(da.t(), s["x"]), "dw_up": torch.mm(db.t(), s["x"])}


# -------------------------------------------------------------------- work

def work(case):
    """Bytes that one pass cannot do without (each input read once, each output written once) and its operations."""
    op = case["op"]
    if op in ("clip", "pack"):
        layout = _layout(case)
        size = {"bf16": 2, "fp16": 2, "fp32": 4}
        read = sum(n * size[t] for n, t in layout)
        return {"bytes": read + (4 * sum(n for n, _ in layout) if op == "pack" else read),
                "flops": 3 * sum(n for n, _ in layout)}
    m = case["m"]
    if op == "linear":
        n, k = case["n"], case["k"]
        words = m * k + n * k + m * n * (1 + case["residual"] + case["pre"]) + n * case["bias"]
        return {"bytes": 2 * words, "flops": 2 * m * n * k}
    if op == "linear_backward":
        n, k = case["n"], case["k"]
        g = 4 if case["flat"] else 2
        read = 2 * (m * n * (1 if case["act"] == "none" else 2) + m * k + n * k)
        return {"bytes": read + 2 * m * k + g * n * (k + case["bias"]), "flops": 4 * m * n * k}
    d, f = case["d"], case["f"]
    if op == "gated_ffn":
        return {"bytes": 2 * (m * d + 2 * f * d + m * f * (3 if case["save"] else 1)), "flops": 4 * m * d * f}
    return {"bytes": 2 * (3 * m * f + 2 * m * d + 4 * f * d), "flops": 8 * m * d * f}
