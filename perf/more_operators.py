"""The token operators, as cases that can be timed and compared.

What a learner's language or speech model needs around its layers, in the
order in which a step runs it:

  embedding, embedding_backward    y[i] = scale * table[ids[i]], and the table's
                                   gradient over the tokens of each id
  dropout, dropout_backward        y = keep * x / P(keep) + residual; `keep` comes
                                   from a counter and is never stored
  layer_norm, layer_norm_backward  rows brought to mean 0 and variance 1, and the
                                   gradients of rows, gain and bias
  recurrence, recurrence_backward  h[t] = f[t] h[t-1] + (1 - f[t]) x[t] along
                                   sequences, f = sigmoid(gate), and its gradients

A case names its operator under "op".  With `own` false, `run` computes it in
elementary torch operations in 32 bits (64 for sums over many rows), rounded
once at the end; with `own` true it calls the package.
"""

import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32,
         "int32": torch.int32, "int64": torch.int64}


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one token while answering: latency alone
        {"name": "norm one row", "op": "layer_norm", "type": "bf16", "m": 1, "d": 4096, "weight": "bf16", "save": False,
         "pad": 0},
        # the forward pass of training on a long batch, gain and bias in 32 bits, mean and rstd kept
        {"name": "norm large", "op": "layer_norm", "type": "bf16", "m": 16384, "d": 4096, "weight": "fp32", "save": True,
         "pad": 0},
        # a short ragged batch, a recurrent layer's width, rows of a wider buffer
        {"name": "norm backward ragged", "op": "layer_norm_backward", "type": "fp16", "m": 777, "d": 1152, "weight": "fp16",
         "grad": "fp16", "residual": False, "pad": 13},
        # the backward pass of training: joined by the residual's gradient, gain and bias into the flat gradient
        {"name": "norm backward large", "op": "layer_norm_backward", "type": "bf16", "m": 16384, "d": 4096,
         "weight": "fp32", "grad": "fp32", "residual": True, "pad": 0},
        # a few tokens while answering
        {"name": "embedding three tokens", "op": "embedding", "type": "bf16", "m": 3, "vocab": 32000, "d": 2048,
         "ids": "int64", "spread": "zipf", "padding": 0.0, "scale": True, "pad": 0},
        # the table's gradient, all rows of it, in the learner's flat gradient
        {"name": "embedding backward large", "op": "embedding_backward", "type": "bf16", "m": 32768, "vocab": 50000,
         "d": 2048, "ids": "int64", "spread": "zipf", "padding": 0.0, "scale": True, "grad": "fp32",
         "accumulate": False, "pad": 0},
        # a short padded batch added to the gradient of a table that is the output layer's weight too
        {"name": "embedding backward tied", "op": "embedding_backward", "type": "fp16", "m": 1531, "vocab": 10000,
         "d": 1152, "ids": "int32", "spread": "zipf", "padding": 0.2, "scale": True, "grad": "fp16",
         "accumulate": True, "pad": 0},
        # a small classifier's ragged last batch
        {"name": "dropout ragged", "op": "dropout", "type": "fp16", "m": 777, "d": 1001, "p": 0.5, "residual": False,
         "pad": 0},
        # a block's output on its way into the residual stream
        {"name": "dropout large", "op": "dropout", "type": "bf16", "m": 16384, "d": 4096, "p": 0.1, "residual": True,
         "pad": 0},
        # one token for each of 32 answers, the states kept in 32 bits
        {"name": "recurrence one token", "op": "recurrence", "type": "bf16", "layout": "even", "batch": 32, "length": 1,
         "d": 1280, "tail": 0, "shape_seed": 0, "state": True, "fused": True},
        # utterances of 1 to 1500 frames end to end, gate and candidate from one product
        {"name": "recurrence ragged", "op": "recurrence", "type": "fp16", "layout": "ragged", "batch": 24, "length": 1500,
         "d": 1152, "tail": 3, "shape_seed": 4, "state": False, "fused": True},
        # the backward pass of training on a few long texts
        {"name": "recurrence backward large", "op": "recurrence_backward", "type": "bf16", "layout": "even", "batch": 4,
         "length": 8192, "d": 4096, "tail": 0, "shape_seed": 0, "state": False, "fused": False},
    ]


def _size(rng, low, high):
    """Log-uniform in [low, high]; one third as it falls, one third a multiple of 8, one third of 64."""
    v = math.exp(rng.uniform(math.log(low), math.log(max(low, high))))
    step = rng.choice((1, 8, 64))
    return int(min(high, max(low, round(v / step) * step)))


def draw(rng):
    op = rng.choice(("layer_norm", "layer_norm_backward", "embedding", "embedding_backward", "dropout",
                     "dropout_backward", "recurrence", "recurrence_backward"))
    t = rng.choice(("bf16", "bf16", "fp16", "fp32"))
    most = 1 << (25 if t == "fp32" else 26)
    pad = rng.choice((0, 0, 8, 13))
    c = {"op": op, "type": t}
    if op.startswith("layer_norm"):
        d = _size(rng, 64, 16384)
        c.update(m=_size(rng, 1, min(65536, most // d)), d=d, weight=rng.choice((t, "fp32", "none")), pad=pad)
        if op == "layer_norm":
            return dict(c, save=rng.random() < 0.5)
        return dict(c, grad=rng.choice((t, "fp32")), residual=rng.random() < 0.5)
    if op.startswith("embedding"):
        d = _size(rng, 64, 4096)
        c.update(m=_size(rng, 1, min(65536, most // d)), vocab=_size(rng, 100, min(131072, most // d)), d=d,
                 ids=rng.choice(("int32", "int64")), spread=rng.choice(("zipf", "zipf", "even")),
                 padding=rng.choice((0.0, 0.0, 0.2, 0.9)), scale=rng.random() < 0.5, pad=pad)
        if op == "embedding":
            return c
        return dict(c, grad=rng.choice((t, "fp32")), accumulate=rng.random() < 0.4)
    if op.startswith("dropout"):
        d = _size(rng, 64, 16384)
        c.update(m=_size(rng, 1, min(65536, most // d)), d=d, p=rng.choice((0.0, 0.1, 0.1, 0.37, 0.5, 0.9)), pad=pad)
        return dict(c, residual=rng.random() < 0.5) if op == "dropout" else dict(c, residual=False)
    d = _size(rng, 64, 8192)
    rows = _size(rng, 1, min(65536, most // d))
    length = _size(rng, 1, rows)
    layout = rng.choice(("even", "ragged"))
    # ragged lengths lie between 1 and `length`, about a third of it
    batch = max(1, rows // length)
    return dict(c, layout=layout, batch=batch, length=length, d=d,
                tail=rng.choice((0, 5)) if layout == "ragged" else 0, shape_seed=rng.randrange(1 << 20),
                state=rng.random() < 0.5, fused=rng.random() < 0.5)


# ------------------------------------------------------------------- inputs

def _offsets(case):
    """Where sequences begin, and the end of the last: batch + 1 row numbers, as a list."""
    if case["layout"] == "even":
        return [case["length"] * b for b in range(case["batch"] + 1)]
    r = np.random.RandomState(case["shape_seed"])
    lengths = np.exp(r.uniform(0.0, math.log(case["length"] + 0.5), case["batch"])).astype(np.int64)
    lengths[r.random_sample(case["batch"]) < 0.05] = 0  # nothing was said
    lengths[0] = case["length"]
    return [0] + np.cumsum(lengths).tolist()


def _draws(seed, device="cuda"):
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)

    def normal(shape, dtype, scale=1.0, shift=0.0, pad=0):
        """A normal draw; with `pad`, rows of a buffer that is `pad` columns wider."""
        wide = shape[:-1] + (shape[-1] + pad,)
        t = torch.randn(wide, generator=gen, device=device, dtype=torch.float32).mul_(scale).add_(shift).to(dtype)
        return t[..., :shape[-1]]

    def uniform(n):
        return torch.rand(n, generator=gen, device=device, dtype=torch.float64)
    return normal, uniform


def _ids(case, uniform):
    """Token numbers: small ones are common (number v with a probability near 1 / v), some are padding."""
    v, u = case["vocab"], uniform(case["m"])
    ids = torch.floor(torch.exp(u * math.log(v + 1))) - 1 if case["spread"] == "zipf" else torch.floor(u * v)
    ids = ids.clamp(0, v - 1).to(TYPES[case["ids"]])
    return torch.where(uniform(case["m"]) < case["padding"], torch.full_like(ids, -1), ids)


def _scale(case):
    return float(math.sqrt(case["d"])) if case["scale"] else 1.0


def _inputs(case, seed):
    """What a call reads, by name."""
    (normal, uniform), t, op = _draws(seed), TYPES[case["type"]], case["op"]
    if op.startswith("layer_norm"):
        m, d, pad = case["m"], case["d"], case["pad"]
        # rows of a residual stream: off centre, of different sizes
        x = normal((m, d), torch.float32).mul_(normal((m, 1), torch.float32).mul_(0.5).exp_()).add_(0.3).to(t)
        s = {"x": torch.nn.functional.pad(x, (0, pad))[:, :d]}
        w = case["weight"]
        s["weight"] = None if w == "none" else normal((d,), TYPES[w], 0.2, 1.0)
        if op == "layer_norm":
            s["bias"] = None if w == "none" else normal((d,), TYPES[w], 0.1)
            return s
        wide = s["x"].double()
        mean = wide.mean(1)
        s.update(dy=normal((m, d), t, 0.01, 0.0, pad), mean=mean.float(),
                 rstd=(wide.sub_(mean[:, None]).square_().mean(1) + 1e-5).rsqrt().float(),
                 residual=normal((m, d), t, 0.01) if case["residual"] else None)
        return s
    if op.startswith("embedding"):
        m, v, d = case["m"], case["vocab"], case["d"]
        s = {"ids": _ids(case, uniform)}
        if op == "embedding":
            return dict(s, table=normal((v, d), t, d ** -0.5, 0.0, case["pad"]))
        s["dy"] = normal((m, d), t, 0.01, 0.0, case["pad"])
        g = TYPES[case["grad"]]
        s["dtable"] = normal((v, d), g, 0.01) if case["accumulate"] else torch.empty((v, d), dtype=g, device="cuda")
        return s
    if op.startswith("dropout"):
        m, d = case["m"], case["d"]
        s = {"x": normal((m, d), t, 1.0, 0.0, case["pad"]), "residual": normal((m, d), t) if case["residual"] else None}
        r = np.random.RandomState(seed % (1 << 32))
        return dict(s, seed=int(r.randint(0, 1 << 62)), offset=int(r.randint(0, 1 << 40)))
    at, d = _offsets(case), case["d"]
    m = at[-1] + case["tail"]
    if case["fused"]:
        both = normal((m, 2 * d), t)
        s = {"gate": both[:, :d], "x": both[:, d:]}
    else:
        s = {"gate": normal((m, d), t), "x": normal((m, d), t)}
    # memories of a few to a few hundred steps
    s["gate"].mul_(1.5).add_(torch.linspace(0.0, 4.0, d, device="cuda").to(t))
    s["h0"] = normal((case["batch"], d), torch.float32, 0.5) if case["state"] else None
    s["at"] = at
    if op == "recurrence_backward":
        s["h"] = _plain_recurrence(s["gate"], s["x"], s["h0"], at).to(t)
        s["dh"] = normal((m, d), t, 0.01)
        s["dstate"] = normal((case["batch"], d), torch.float32, 0.01) if case["state"] else None
    return s


def prepare(case, seed):
    """Inputs and what a training program keeps beside them: output buffers, offsets on the device, workspace."""
    op, t = case["op"], TYPES[case["type"]]
    state = dict(_inputs(case, seed), case=case)

    def new(*shape, dtype=t):
        return torch.empty(shape, dtype=dtype, device="cuda")

    if own:
        from sparsified_gradient_compression_amd import dgc
    if op.startswith("layer_norm"):
        m, d = case["m"], case["d"]
        if op == "layer_norm":
            keep = {"mean": new(m, dtype=torch.float32), "rstd": new(m, dtype=torch.float32)} if case["save"] else {}
            state.update(out=new(m, d), keep=keep)
        else:
            g = TYPES[case["grad"]]
            gain = case["weight"] != "none"
            state.update(dx=new(m, d), dweight=new(d, dtype=g) if gain else None,
                         dbias=new(d, dtype=g) if gain else None)
            if own:
                state["workspace"] = dgc.layer_norm_workspace(m, d, backward=True)
    elif op == "embedding":
        state["out"] = new(case["m"], case["d"])
    elif op == "embedding_backward":
        if own:
            state["workspace"] = dgc.embedding_workspace(case["m"], case["vocab"], case["d"])
    elif op.startswith("dropout"):
        state["out"] = new(case["m"], case["d"])
    else:
        m, d, at, b = state["x"].shape[0], case["d"], state["at"], case["batch"]
        even = case["layout"] == "even"
        state["rows"] = {"batch": b} if even else {"offsets": torch.tensor(at, dtype=torch.int32, device="cuda")}
        # rows behind the last sequence stay as they are
        outs = ("out",) if op == "recurrence" else ("dgate", "dx")
        state.update({name: torch.zeros((m, d), dtype=t, device="cuda") for name in outs})
        name = "state" if op == "recurrence" else "dh0"
        state[name] = new(b, d, dtype=torch.float32) if case["state"] else None
        if own:
            state["workspace"] = dgc.recurrence_workspace(m, d, b, backward=op == "recurrence_backward")
    return state


# --------------------------------------------------------------- plain forms

def _run_layer_norm(s, c):
    x = s["x"].float()
    mean = x.mean(1, keepdim=True)
    off = x - mean
    rstd = 1 / torch.sqrt((off * off).mean(1, keepdim=True) + 1e-5)
    y = off * rstd
    if s["weight"] is not None:
        y = y * s["weight"].float() + s["bias"].float()
    out = {"y": y.to(s["x"].dtype)}
    return dict(out, mean=mean.reshape(-1), rstd=rstd.reshape(-1)) if c["save"] else out


def _run_layer_norm_backward(s, c):
    t, dy, rstd = s["x"].dtype, s["dy"].float(), s["rstd"][:, None]
    n = (s["x"].float() - s["mean"][:, None]) * rstd
    g = dy if s["weight"] is None else dy * s["weight"].float()
    dx = rstd * (g - g.mean(1, keepdim=True) - n * (g * n).mean(1, keepdim=True))
    if s["residual"] is not None:
        dx = dx + s["residual"].float()
    out = {"dx": dx.to(t)}
    if s["weight"] is None:
        return out
    u = TYPES[c["grad"]]
    return dict(out, dweight=(dy * n).sum(0, dtype=torch.float64).to(u), dbias=dy.sum(0, dtype=torch.float64).to(u))


def _run_embedding(s, c):
    ids, v = s["ids"].long(), c["vocab"]
    known = (ids >= 0) & (ids < v)
    y = s["table"].float()[ids.clamp(0, v - 1)] * _scale(c)
    return {"y": torch.where(known[:, None], y, torch.zeros_like(y)).to(s["table"].dtype)}


def _run_embedding_backward(s, c):
    ids, v = s["ids"].long(), c["vocab"]
    known = ((ids >= 0) & (ids < v)).nonzero().reshape(-1)
    total = torch.zeros((v, c["d"]), dtype=torch.float64, device="cuda")
    total.index_add_(0, ids[known], s["dy"].double()[known])
    total *= _scale(c)
    if c["accumulate"]:
        total += s["dtable"]
    s["dtable"].copy_(total)
    return {"dtable": s["dtable"]}


def _bits32(case, seed, offset):
    """16 random bits for each element [m, d]: Philox4x32-10 (Salmon, Moraes, Dror, Shaw, 2011) of the counter
    (column / 8, row, offset) and the key `seed`, its four words cut in halves, the low one first."""
    m, groups = case["m"], (case["d"] + 7) // 8
    low = 0xFFFFFFFF
    c = [torch.arange(groups, device="cuda")[None, :], torch.arange(m, device="cuda")[:, None],
         torch.full((1, 1), offset & low, device="cuda"), torch.full((1, 1), offset >> 32 & low, device="cuda")]
    k = [seed & low, seed >> 32 & low]
    for _ in range(10):
        p, q = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57  # modulo 2^64
        c = [(q >> 32) & low ^ c[1] ^ k[0], q & low, (p >> 32) & low ^ c[3] ^ k[1], p & low]
        k = [(k[0] + 0x9E3779B9) & low, (k[1] + 0xBB67AE85) & low]
    halves = [h for w in c for h in ((w & 0xFFFF), (w >> 16 & 0xFFFF))]
    return torch.stack([h.expand(m, groups) for h in halves], 2).reshape(m, groups * 8)[:, :case["d"]]


def _kept(p):
    """How many of 65536 equally likely draws keep an element."""
    return int(math.floor((1 - p) * 65536 + 0.5))


def _run_dropout(s, c):
    kept = _kept(c["p"])
    x = s["x"].float()
    keep = _bits32(c, s["seed"], s["offset"]) < kept
    y = torch.where(keep, x * (65536 / kept), torch.zeros_like(x))
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return {"y": y.to(s["x"].dtype)}


def _scan(a, b, longest):
    """In place: b[t] = a[t] b[t-1] + b[t] along the rows, by doubling; a[t] = 0 where nothing comes before."""
    step = 1
    while step < longest:
        b[step:] += a[step:] * b[:-step]
        a[step:] = a[step:] * a[:-step]
        step *= 2
    return b


def _sigmoid(z):
    return 1 / (1 + torch.exp(-z))


def _rows_of(at, filled):
    """The first (or last) rows of the sequences that have any, and which these are."""
    first = torch.tensor([at[b] for b in filled], dtype=torch.int64, device="cuda")
    last = torch.tensor([at[b + 1] - 1 for b in filled], dtype=torch.int64, device="cuda")
    return first, last, torch.tensor(filled, dtype=torch.int64, device="cuda")


def _plain_recurrence(gate, x, h0, at):
    """All rows of h in binary32; 0 behind the last sequence."""
    filled = [b for b in range(len(at) - 1) if at[b + 1] > at[b]]
    first, _, which = _rows_of(at, filled)
    z = gate.float()
    f, b = _sigmoid(z), _sigmoid(-z) * x.float()
    if h0 is not None:
        b[first] += f[first] * h0[which]
    f[first] = 0
    f[at[-1]:] = 0
    b[at[-1]:] = 0
    return _scan(f, b, max([at[i + 1] - at[i] for i in range(len(at) - 1)]))


def _run_recurrence(s, c):
    h = _plain_recurrence(s["gate"], s["x"], s["h0"], s["at"])
    out = {"h": h.to(s["x"].dtype)}
    if not c["state"]:
        return out
    filled = [b for b in range(c["batch"]) if s["at"][b + 1] > s["at"][b]]
    _, last, which = _rows_of(s["at"], filled)
    state = s["h0"].clone()
    state[which] = h[last]
    return dict(out, state=state)


def _run_recurrence_backward(s, c):
    """g[t] = dh[t] + f[t+1] g[t+1]; dx = (1 - f) g; dgate = g (h[t-1] - x) f (1 - f); dh0 = f[0] g[0]."""
    at, t = s["at"], s["x"].dtype
    filled = [b for b in range(c["batch"]) if at[b + 1] > at[b]]
    first, last, which = _rows_of(at, filled)
    z = s["gate"].float()
    f, r = _sigmoid(z), _sigmoid(-z)
    g = s["dh"].float()
    if s["dstate"] is not None:
        g[last] += s["dstate"][which]
    g[at[-1]:] = 0
    after = torch.zeros_like(f)
    after[:-1] = f[1:]
    after[last] = 0
    after[at[-1]:] = 0
    g = _scan(after.flip(0), g.flip(0), max([at[i + 1] - at[i] for i in range(len(at) - 1)])).flip(0)
    before = torch.zeros_like(f)
    before[1:] = s["h"][:-1]
    before[first] = 0 if s["h0"] is None else s["h0"][which]
    out = {"dgate": (g * (before - s["x"].float()) * f * r).to(t), "dx": (g * r).to(t)}
    if not c["state"]:
        return out
    dh0 = s["dstate"].clone()
    dh0[which] = f[first] * g[first]
    return dict(out, dh0=dh0)


PLAIN = {"layer_norm": _run_layer_norm, "layer_norm_backward": _run_layer_norm_backward, "embedding": _run_embedding,
         "embedding_backward": _run_embedding_backward, "dropout": _run_dropout, "dropout_backward": _run_dropout,
         "recurrence": _run_recurrence, "recurrence_backward": _run_recurrence_backward}


# ------------------------------------------------------------ the package's

def _own_layer_norm(s, c, dgc):
    dgc.layer_norm(s["x"], s["weight"], s["bias"], eps=1e-5, out=s["out"], **s["keep"])
    return dict(s["keep"], y=s["out"])


def _own_layer_norm_backward(s, c, dgc):
    dgc.layer_norm_backward(s["dy"], s["x"], s["mean"], s["rstd"], s["weight"], residual=s["residual"], dx=s["dx"],
                            dweight=s["dweight"], dbias=s["dbias"], workspace=s["workspace"])
    if s["weight"] is None:
        return {"dx": s["dx"]}
    return {"dx": s["dx"], "dweight": s["dweight"], "dbias": s["dbias"]}


def _own_embedding(s, c, dgc):
    return {"y": dgc.embedding(s["ids"], s["table"], scale=_scale(c), out=s["out"])}


def _own_embedding_backward(s, c, dgc):
    dgc.embedding_backward(s["dy"], s["ids"], s["dtable"], scale=_scale(c), accumulate=c["accumulate"],
                           workspace=s["workspace"])
    return {"dtable": s["dtable"]}


def _own_dropout(s, c, dgc):
    return {"y": dgc.dropout(s["x"], c["p"], s["seed"], s["offset"], residual=s["residual"], out=s["out"])}


def _own_dropout_backward(s, c, dgc):
    return {"y": dgc.dropout_backward(s["x"], c["p"], s["seed"], s["offset"], dx=s["out"])}


def _own_recurrence(s, c, dgc):
    dgc.recurrence(s["gate"], s["x"], s["h0"], out=s["out"], state=s["state"], workspace=s["workspace"], **s["rows"])
    return {"h": s["out"], "state": s["state"]} if c["state"] else {"h": s["out"]}


def _own_recurrence_backward(s, c, dgc):
    dgc.recurrence_backward(s["dh"], s["gate"], s["x"], s["h"], s["h0"], dstate=s["dstate"], dgate=s["dgate"],
                            dx=s["dx"], dh0=s["dh0"], workspace=s["workspace"], **s["rows"])
    out = {"dgate": s["dgate"], "dx": s["dx"]}
    return dict(out, dh0=s["dh0"]) if c["state"] else out


OWN = {"layer_norm": _own_layer_norm, "layer_norm_backward": _own_layer_norm_backward, "embedding": _own_embedding,
       "embedding_backward": _own_embedding_backward, "dropout": _own_dropout, "dropout_backward": _own_dropout_backward,
       "recurrence": _own_recurrence, "recurrence_backward": _own_recurrence_backward}


def run(state):
    case = state["case"]
    if own:
        from sparsified_gradient_compression_amd import dgc
        return OWN[case["op"]](state, case, dgc)
    return PLAIN[case["op"]](state, case)


# ------------------------------------------------------------------- exact

def _bits64(case, seed, offset):
    """The same bits by numpy's whole numbers, group by group of eight columns."""
    m, groups = case["m"], (case["d"] + 7) // 8
    u = np.uint64
    mask, half = u(0xFFFFFFFF), u(32)
    x0 = np.broadcast_to(np.arange(groups, dtype=u), (m, groups))
    x1 = np.broadcast_to(np.arange(m, dtype=u)[:, None], (m, groups))
    x2, x3 = u(offset & 0xFFFFFFFF), u(offset >> 32 & 0xFFFFFFFF)
    for i in range(10):
        key0 = u((seed + i * 0x9E3779B9) & 0xFFFFFFFF)
        key1 = u(((seed >> 32) + i * 0xBB67AE85) & 0xFFFFFFFF)
        first, second = x0 * u(0xD2511F53), x2 * u(0xCD9E8D57)
        x0, x1, x2, x3 = (second >> half) ^ x1 ^ key0, second & mask, (first >> half) ^ x3 ^ key1, first & mask
    words = np.stack([np.broadcast_to(w, (m, groups)) for w in (x0, x1, x2, x3)], 2).astype("<u4")
    return words.view("<u2").reshape(m, groups * 8)[:, :case["d"]]


def _side_by_side(s, c):
    """Row numbers of the sequences [batch, longest], and which of these places hold one."""
    at = torch.tensor(s["at"], device="cuda")
    step = torch.arange(max(1, int((at[1:] - at[:-1]).max())), device="cuda")
    valid = step < (at[1:] - at[:-1])[:, None]
    return torch.where(valid, at[:-1, None] + step, 0), valid


def _exact_recurrence(s, c):
    """Step by step, all sequences side by side; behind its end a sequence keeps its state."""
    row, valid = _side_by_side(s, c)
    hold = valid[:, :, None]
    gate = s["gate"].double()
    keep = torch.where(hold, torch.sigmoid(gate)[row], 1.0)
    take = torch.where(hold, (torch.sigmoid(-gate) * s["x"])[row], 0.0)
    now = torch.zeros((c["batch"], c["d"]), dtype=torch.float64, device="cuda")
    if s["h0"] is not None:
        now += s["h0"]
    for i in range(row.shape[1]):
        now = torch.addcmul(take[:, i], keep[:, i], now)
        take[:, i] = now
    h = torch.zeros_like(gate)
    h[row[valid]] = take[valid]
    return {"h": h, "state": now} if c["state"] else {"h": h}


def _exact_recurrence_backward(s, c):
    row, valid = _side_by_side(s, c)
    hold = valid[:, :, None]
    x, gate = s["x"].double(), s["gate"].double()
    keep = torch.where(hold, torch.sigmoid(gate)[row], 1.0)
    dh = torch.where(hold, s["dh"].double()[row], 0.0)
    start, now = (torch.zeros((c["batch"], c["d"]), dtype=torch.float64, device="cuda") for _ in range(2))
    if s["h0"] is not None:
        start += s["h0"]
    if s["dstate"] is not None:
        now += s["dstate"]
    for i in reversed(range(row.shape[1])):
        dh[:, i] += now  # the gradient of the state behind this row
        now = keep[:, i] * dh[:, i]
    before = torch.cat([start[:, None], torch.where(hold, s["h"].double()[row], 0.0)[:, :-1]], 1)
    g, previous = torch.zeros_like(x), torch.zeros_like(x)
    g[row[valid]] = dh[valid]
    previous[row[valid]] = before[valid]
    slope = torch.sigmoid(gate) * torch.sigmoid(-gate)
    out = {"dgate": g * slope * (previous - x), "dx": g * torch.sigmoid(-gate)}
    return dict(out, dh0=now) if c["state"] else out


def exact(case, seed):
    op, s = case["op"], _inputs(case, seed)
    if op.startswith("layer_norm"):
        x, w = s["x"].double(), None if s["weight"] is None else s["weight"].double()
        if op == "layer_norm":
            var, mean = torch.var_mean(x, 1, unbiased=False)
            rstd = (var + 1e-5) ** -0.5
            y = (x - mean[:, None]) * rstd[:, None]
            y = y if w is None else torch.addcmul(s["bias"].double(), y, w)
            return {"y": y, "mean": mean, "rstd": rstd} if case["save"] else {"y": y}
        dy, mean, r = s["dy"].double(), s["mean"].double()[:, None], s["rstd"].double()[:, None]
        off, g = x - mean, s["dy"].double() if w is None else s["dy"].double() * w
        dots = torch.einsum("md,md->m", g, off)[:, None] / case["d"]
        dx = r * g - r * g.mean(1, keepdim=True) - r ** 3 * dots * off
        dx = dx if s["residual"] is None else dx + s["residual"]
        return {"dx": dx} if w is None else {"dx": dx, "dweight": (r * off * dy).sum(0), "dbias": dy.sum(0)}
    if op == "embedding":
        padded = torch.cat([s["table"].double(), torch.zeros((1, case["d"]), dtype=torch.float64, device="cuda")])
        return {"y": padded[s["ids"].long()] * _scale(case)}  # -1 is the last row
    if op == "embedding_backward":
        total = torch.zeros((case["vocab"] + 1, case["d"]), dtype=torch.float64, device="cuda")
        ids, order = torch.sort(torch.where(s["ids"] < 0, case["vocab"], s["ids"].long()), stable=True)
        total.index_put_((ids,), s["dy"].double()[order], accumulate=True)
        total = total[:-1] * _scale(case)
        return {"dtable": total + s["dtable"] if case["accumulate"] else total}
    if op.startswith("dropout"):
        bits = torch.from_numpy(_bits64(case, s["seed"], s["offset"]).astype(np.int32)).cuda()
        kept = _kept(case["p"])
        y = torch.where(bits < kept, s["x"].double() * 65536 / max(kept, 1), 0.0)
        return {"y": y if s["residual"] is None else y + s["residual"]}
    return _exact_recurrence(s, case) if op == "recurrence" else _exact_recurrence_backward(s, case)


# -------------------------------------------------------------------- work

def _different(case):
    """How many of the table's rows a batch is expected to name."""
    v, n = case["vocab"], case["m"] * (1 - case["padding"])
    at = np.arange(1, v + 1, dtype=np.float64)
    p = np.log1p(1 / at) / math.log(v + 1) if case["spread"] == "zipf" else np.full(v, 1 / v)
    return float(-np.expm1(n * np.log1p(-np.minimum(p, 1 - 1e-15))).sum())


def work(case):
    """Bytes that one pass cannot do without (each input read once, each output written once) and its operations."""
    op, t = case["op"], TYPES[case["type"]].itemsize
    if op.startswith("layer_norm"):
        n, d = case["m"] * case["d"], case["d"]
        w = 0 if case["weight"] == "none" else TYPES[case["weight"]].itemsize
        if op == "layer_norm":
            return {"bytes": 2 * t * n + 2 * w * d + (8 * case["m"] if case["save"] else 0), "flops": 8 * n}
        g = TYPES[case["grad"]].itemsize if w else 0
        return {"bytes": (3 + case["residual"]) * t * n + 8 * case["m"] + (w + 2 * g) * d, "flops": 14 * n}
    if op.startswith("embedding"):
        m, d, i = case["m"], case["d"], TYPES[case["ids"]].itemsize
        named, rows = m * (1 - case["padding"]), _different(case)
        if op == "embedding":
            return {"bytes": i * m + t * d * (rows + m), "flops": m * d}
        g = TYPES[case["grad"]].itemsize
        out = 2 * rows if case["accumulate"] else case["vocab"]
        return {"bytes": i * m + t * d * named + g * d * out, "flops": 2 * named * d}
    if op.startswith("dropout"):
        n = case["m"] * case["d"]
        return {"bytes": (2 + case["residual"]) * t * n, "flops": 2 * n}
    n, b = _offsets(case)[-1] * case["d"], case["batch"] * case["d"] if case["state"] else 0
    if op == "recurrence":
        return {"bytes": 3 * t * n + 8 * b, "flops": 8 * n}
    return {"bytes": 6 * t * n + 12 * b, "flops": 14 * n}
