"""What is measured of the norm before a layer, the 8-bit projections and the gated linear recurrence.

Five calls: the root-mean-square norm with the residual's addition and an
output in 8 bits (``kda_rmsnorm``, ``kda_rmsnorm_i8``), the projection in 8-bit
integers with a scale per token and per channel (``kda_linear_i8``), and the gated
linear recurrence, one decay per channel, over packed sequences
(``kda_glr_scan``), with its gradient (``kda_glr_scan_backward``) and over a few tokens
of many sequences (``kda_glr_step``).  ``run`` makes the library's calls where ``own`` is
set, and computes the same with elementary torch operations where it is not.

    norm:        s = x + residual;  n = s / sqrt(mean s^2 + eps) * w
                 8 bits: scale = max |n| / 127 per token, q = n / scale to the nearest integer
    projection:  y = act(sx_m sw_n sum_k x_mk w_nk + bias_n) + residual
    recurrence:  g = min(la, 0), or -A softplus(la + b), or -A sigmoid(la + b);  a = e^g
                 u = c sigmoid(i) x,  c = 1, or 1 - a, or sqrt(1 - a^2)
                 h_t = a_t h_{t-1} + u_t,  y_t = h_t
"""
import math
import random

import torch

own = False

CHUNK = 64
EPS = 1e-6
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh", "sigmoid")
DECAYS = ("log", "softplus", "sigmoid")
SCALES = ("none", "complement", "normalized")
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # the next token of 64 users on its way into 8-bit projections: latency
        {"name": "norm decode batch", "op": "norm", "M": 64, "D": 4096, "res": True, "i8": True,
         "dtype": "bf16"},
        # the tokens of some packed prompts, an odd number of them, residual stream carried on
        {"name": "norm prefill", "op": "norm", "M": 12001, "D": 4096, "res": True, "i8": False,
         "dtype": "bf16"},
        # one token through a layer's output projection onto the residual stream
        {"name": "product one token", "op": "product", "M": 1, "K": 4096, "N": 4096, "bias": False,
         "act": "none", "res": True, "dtype": "bf16"},
        # a decode batch of 64 sequences: 96 heads of 128 channels back to the model width
        {"name": "product decode batch", "op": "product", "M": 64, "K": 12288, "N": 4096,
         "bias": True, "act": "none", "res": True, "dtype": "bf16"},
        # a ragged prefill batch through a small biased, activated projection, odd sizes
        {"name": "product ragged", "op": "product", "M": 333, "K": 1000, "N": 1499, "bias": True,
         "act": "silu", "res": False, "dtype": "f32"},
        # 4096 tokens into 96 heads of 128 channels
        {"name": "product prefill", "op": "product", "M": 4096, "K": 4096, "N": 12288, "bias": True,
         "act": "gelu_tanh", "res": True, "dtype": "bf16"},
        # a serving batch: prompts of ragged lengths, one of them empty, states in a pool
        {"name": "scan packed prompts", "op": "scan", "T": 12000, "seqs": 9, "cut": 5, "D": 4096,
         "decay": "sigmoid", "input": "normalized", "gate": True, "pool": True, "dtype": "bf16"},
        # one long document
        {"name": "scan long", "op": "scan", "T": 32768, "seqs": 1, "cut": 0, "D": 4096,
         "decay": "softplus", "input": "complement", "gate": False, "pool": False, "dtype": "bf16"},
        # a training step of a layer: four sequences of uneven lengths, forward and backward
        {"name": "train batch", "op": "train", "T": 16384, "seqs": 4, "cut": 12, "D": 4096,
         "decay": "sigmoid", "input": "normalized", "gate": True, "dtype": "bf16"},
        # the 32-bit path: a small layer of an odd width as tests and checks of a model use it
        {"name": "train f32", "op": "train", "T": 777, "seqs": 3, "cut": 8, "D": 1001,
         "decay": "log", "input": "none", "gate": False, "dtype": "f32"},
        # one user's next token
        {"name": "step one user", "op": "step", "N": 1, "L": 1, "D": 4096, "decay": "sigmoid",
         "input": "normalized", "gate": True, "dtype": "bf16"},
        # the next token of 256 users
        {"name": "step batch", "op": "step", "N": 256, "L": 1, "D": 4096, "decay": "softplus",
         "input": "complement", "gate": False, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def _width(rng, lo, hi):
    """Most widths are multiples of 8, some are not."""
    n = _log(rng, lo, hi)
    return (n + 7) // 8 * 8 if rng.random() < 0.6 else n


def draw(rng):
    op = rng.choice(("norm", "norm", "product", "product", "scan", "train", "step"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    if op == "norm":
        M, D = _log(rng, 1, 16384), _width(rng, 32, 16384)
        while M * D > 6000 * 4096:
            M = (M + 1) // 2
        return {"op": op, "M": M, "D": D, "res": rng.random() < 0.6, "i8": rng.random() < 0.5,
                "dtype": dtype}
    if op == "product":
        M, K, N = _log(rng, 1, 4096), _width(rng, 64, 12288), _width(rng, 64, 12288)
        while M * K * N > 4096 * 4096 * 6144:
            M = (M + 1) // 2
        return {"op": op, "M": M, "K": K, "N": N, "bias": rng.random() < 0.5,
                "act": rng.choice(ACTS), "res": rng.random() < 0.5, "dtype": dtype}
    form = {"decay": rng.choice(DECAYS), "input": rng.choice(SCALES), "gate": rng.random() < 0.5,
            "dtype": dtype}
    D = _width(rng, 32, 8192)
    if op == "step":
        N, L = _log(rng, 1, 512), rng.choice((1, 1, 1, 2, 4, 7))
        return {"op": op, "N": N, "L": L, "D": D, **form}
    T = _log(rng, 1, 32768 if op == "scan" else 16384)
    while T * D > (16384 if op == "scan" else 8192) * 4096:
        T = T // 2 + 1
    c = {"op": op, "T": T, "seqs": _log(rng, 1, 16), "cut": rng.randrange(1, 1 << 20), "D": D, **form}
    return c | {"pool": rng.random() < 0.5} if op == "scan" else c


def _lengths(c):
    """The case's T tokens cut into `seqs` sequences: the lengths, one of them empty from three on."""
    n, r = c["seqs"], random.Random(c["cut"])
    if n == 1:
        return [c["T"]]
    at = sorted(r.randrange(0, c["T"] + 1) for _ in range(n - 1))
    if n > 2:
        at[n // 2] = at[n // 2 - 1]
    return [b - a for a, b in zip([0] + at, at + [c["T"]])]


# ------------------------------------------------------------------ what a program has in hand
def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    t = TYPES[c["dtype"]]

    def normal(*shape, std=1.0, dtype=t):
        return (torch.randn(shape, generator=g, device=dev) * std).to(dtype)

    def eight_bits(rows, width, std=1.0):  # each row by its largest value
        v = normal(rows, width, std=std, dtype=torch.float32)
        scale = v.abs().amax(1) / 127
        return torch.round(v / scale[:, None]).to(torch.int8), scale

    if c["op"] == "norm":
        M, D = c["M"], c["D"]
        return {"case": c, "x": normal(M, D), "res": normal(M, D, std=3.0) if c["res"] else None,
                "w": 1 + normal(D, std=0.1, dtype=torch.float32)}
    if c["op"] == "product":
        M, K, N = c["M"], c["K"], c["N"]
        x, sx = eight_bits(M, K)
        w, sw = eight_bits(N, K, K ** -0.5)
        return {"case": c, "x": x, "sx": sx, "w": w, "sw": sw,
                "bias": normal(N, std=0.5) if c["bias"] else None,
                "res": normal(M, N) if c["res"] else None}
    D, step = c["D"], c["op"] == "step"
    rows, n = ((c["N"], c["L"]), c["N"]) if step else ((c["T"],), c["seqs"])
    s = {"case": c, "x": normal(*rows, D), "gate": normal(*rows, D) if c["gate"] else None,
         "A": None, "b": None}
    if not step:
        lens = _lengths(c)
        at = [0]
        for x in lens:
            at.append(at[-1] + x)
        s |= {"lens": lens, "cu": torch.tensor(at, dtype=torch.int32, device=dev)}
    if c["decay"] == "log":  # decays of e^-0.05, ten times more or less
        s["la"] = -torch.exp(normal(*rows, D, dtype=torch.float32) - 3).to(t)
    else:
        s["la"] = normal(*rows, D)
        r = torch.rand(D, generator=g, device=dev)
        if c["decay"] == "sigmoid":  # with the gate open, a state fades by 0.9 to 0.999 per token
            s["A"], s["b"] = -torch.log(0.9 + 0.099 * r), normal(D, std=0.5, dtype=torch.float32)
        else:  # rates in [1, 4], steps of 0.001 to 0.1
            s["A"] = 1 + 3 * r
            u = torch.rand(D, generator=g, device=dev)
            s["b"] = torch.log(torch.expm1(torch.exp(math.log(1e-3) + math.log(100.0) * u)))
    if step or c.get("pool"):
        s["h"] = normal(n + 2, D, dtype=torch.float32)
        s["slots"] = torch.randperm(n + 2, generator=g, device=dev)[:n].to(torch.int32)
    if c["op"] == "train":
        s |= {"h0": normal(n, D, dtype=torch.float32), "dy": normal(*rows, D),
              "dh": normal(n, D, dtype=torch.float32)}
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _own_norm, "product": _own_product, "scan": _own_scan, "train": _own_train,
                "step": _own_step}[op](state)
    return {"norm": _plain_norm, "product": _plain_product, "scan": _plain_scan,
            "train": _plain_train, "step": _plain_step}[op](state)


def _own_norm(s):
    from linear_attention_recurrence_prefill_gb300 import kda
    if not s["case"]["i8"]:
        return kda.kda_rmsnorm(s["x"], s["w"], s["res"])
    q, scale, *total = kda.kda_rmsnorm_i8(s["x"], s["w"], s["res"])
    return (torch.mul(q, scale[:, None]), scale, *total)  # the values that the integers stand for


def _own_product(s):
    from linear_attention_recurrence_prefill_gb300 import kda
    c = s["case"]
    return kda.kda_linear_i8(s["x"], s["sx"], s["w"], s["sw"], s["bias"], s["res"], act=c["act"],
                             dtype=TYPES[c["dtype"]])


def _form(s):
    c = s["case"]
    return dict(decay_from=c["decay"], decay_scale=s["A"], decay_bias=s["b"],
                input_scale=c["input"], input_gate=s["gate"])


def _own_scan(s):
    from linear_attention_recurrence_prefill_gb300 import kda
    more = dict(max_seqlen=max(s["lens"]), **_form(s))
    if s["case"]["pool"]:
        return kda.kda_glr_scan(s["x"], s["la"], s["h"], s["cu"], h_T=s["h"], slots=s["slots"],
                                **more)
    return kda.kda_glr_scan(s["x"], s["la"], None, s["cu"], **more)


def _own_train(s):
    from linear_attention_recurrence_prefill_gb300 import kda
    more = dict(max_seqlen=max(s["lens"]), **_form(s))
    y, h, saved = kda.kda_glr_scan(s["x"], s["la"], s["h0"], s["cu"], checkpoints=True, **more)
    grads = kda.kda_glr_scan_backward(s["dy"], s["dh"], s["x"], s["la"], saved, s["cu"], **more)
    return [y, h] + [d for d in grads if d is not None]


def _own_step(s):
    from linear_attention_recurrence_prefill_gb300 import kda
    return kda.kda_glr_step(s["x"], s["la"], s["h"], slots=s["slots"], **_form(s)), s["h"]


def _plain_norm(s):
    c, t = s["case"], s["x"].dtype
    # values next to the middle between two integers: 64 bits
    x = s["x"].double() if c["i8"] else s["x"].float()
    if c["res"]:
        x = x + s["res"]
    # a mean of up to 16384 squares: 64 bits
    r = torch.rsqrt((x * x).sum(-1, keepdim=True, dtype=torch.float64) / c["D"] + EPS)
    n = (x * r.to(x.dtype)) * s["w"]
    total = (x.to(t),) if c["res"] else ()
    if not c["i8"]:
        return (n.to(t), *total) if c["res"] else n.to(t)
    scale = n.abs().amax(-1) / 127
    q = torch.round(n / scale[:, None]).float()
    scale = scale.float()
    return (q * scale[:, None], scale, *total)


def _act(y, act):
    if act == "relu":
        return y.clamp_min(0.0)
    if act == "silu":
        return y / (1 + torch.exp(-y))
    if act == "sigmoid":
        return 1 / (1 + torch.exp(-y))
    if act == "gelu":
        return 0.5 * y * (1 + torch.erf(y * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * y * (1 + torch.tanh(math.sqrt(2 / math.pi) * (y + 0.044715 * y * y * y)))
    return y


def _plain_product(s):
    y = (s["x"].float() @ s["w"].float().T) * s["sx"][:, None] * s["sw"]
    if s["bias"] is not None:
        y = y + s["bias"].float()
    y = _act(y, s["case"]["act"])
    if s["res"] is not None:
        y = y + s["res"].float()
    return y.to(TYPES[s["case"]["dtype"]])


def _gates(s, t=torch.float32):
    """(x, v = la + b, log decay, decay, input scale, gate) of every token."""
    c = s["case"]
    x, v = s["x"].to(t), s["la"].to(t)
    if s["b"] is not None:
        v = v + s["b"]
    if c["decay"] == "log":
        g = v.clamp_max(0.0)
    elif c["decay"] == "softplus":
        g = -s["A"] * (v.clamp_min(0.0) + torch.log1p(torch.exp(-v.abs())))
    else:
        g = -s["A"] / (1 + torch.exp(-v))
    if c["input"] == "none":
        scale = torch.ones_like(g)
    elif c["input"] == "complement":
        scale = -torch.expm1(g)
    else:
        scale = torch.sqrt(-torch.expm1(2 * g))
    gate = 1 / (1 + torch.exp(-s["gate"].to(t))) if c["gate"] else torch.ones_like(g)
    return x, v, g, torch.exp(g), scale, gate


def _linear_scan(a, u):
    """h_t = a_t h_{t-1} + u_t over the first axis: inside chunks, then over their ends."""
    T, D = a.shape
    n = -(-T // CHUNK)
    pad = n * CHUNK - T
    if pad:
        a, u = (torch.cat([x, x.new_zeros(pad, D)]) for x in (a, u))
    a, h = a.reshape(n, CHUNK, D).clone(), u.reshape(n, CHUNK, D).clone()
    for i in range(1, CHUNK):
        h[:, i] += a[:, i] * h[:, i - 1]
        a[:, i] *= a[:, i - 1]
    carry = torch.zeros(n, D, dtype=a.dtype, device=a.device)
    for i in range(1, n):
        carry[i] = h[i - 1, -1] + a[i - 1, -1] * carry[i - 1]
    return (h + a * carry[:, None]).reshape(n * CHUNK, D)[:T]


def _some(lens):
    """The sequences that have tokens, and their first and last ones."""
    some, first, last, at = [], [], [], 0
    for i, n in enumerate(lens):
        if n:
            some.append(i)
            first.append(at)
            last.append(at + n - 1)
        at += n
    return some, first, last


def _plain_forward(s, h0):
    """(all states, the final ones, the gates, the decays cut at the sequences' first tokens), in h0's type"""
    x, v, g, a, scale, gate = _gates(s, h0.dtype)
    some, first, last = _some(s["lens"])
    u = scale * gate * x
    u[first] += a[first] * h0[some]
    cut = a.clone()
    cut[first] = 0
    h = _linear_scan(cut, u)
    end = h0.clone()
    end[some] = h[last]
    return h, end, (x, v, g, a, scale, gate), cut


def _plain_scan(s):
    c, t = s["case"], s["x"].dtype
    if c["pool"]:
        slots = s["slots"].long()
        h, end, _, _ = _plain_forward(s, s["h"][slots])
        s["h"][slots] = end
        return h.to(t), s["h"]
    h, end, _, _ = _plain_forward(s, torch.zeros(c["seqs"], c["D"], device=s["x"].device))
    return h.to(t), end


def _plain_train(s):
    # 64 bits: a parameter's gradient is a sum over all tokens of terms that nearly cancel, each of
    # them from a sum over the thousand tokens that a slow decay remembers
    c, t = s["case"], s["x"].dtype
    h0, dh = s["h0"].double(), s["dh"].double()
    h, end, (x, v, g, a, scale, gate), cut = _plain_forward(s, h0)
    some, first, last = _some(s["lens"])
    before = torch.cat([h[:1], h[:-1]])
    before[first] = h0[some]
    d = s["dy"].double()
    d[last] += dh[some]
    after = torch.cat([cut[1:], cut[:1]])  # the next token's decay, zero at a sequence's end
    after[last] = 0
    G = _linear_scan(after.flip(0), d.flip(0)).flip(0)
    dh0 = dh.clone()
    dh0[some] = a[first] * G[first]
    dh0 = dh0.float()
    dx = G * scale * gate
    dgate = [(dx * x * (1 - gate)).to(t)] if c["gate"] else []
    dg = G * a * before
    if c["input"] == "complement":
        dg = dg - a * gate * x * G
    elif c["input"] == "normalized":
        dg = dg - a * a / scale * gate * x * G
    out = [h.to(t), end.float(), dx.to(t)]
    if c["decay"] == "log":
        return out + [(dg * (v <= 0)).to(t)] + dgate + [dh0]
    sig = 1 / (1 + torch.exp(-v))
    if c["decay"] == "softplus":
        value, slope = v.clamp_min(0.0) + torch.log1p(torch.exp(-v.abs())), sig
    else:
        value, slope = sig, sig * (1 - sig)
    dla = -s["A"] * slope * dg
    dA = -(value * dg).sum(0).float()
    return out + [dla.to(t)] + dgate + [dh0, dA, dla.sum(0).float()]


def _plain_step(s):
    x, v, g, a, scale, gate = _gates(s)
    u = scale * gate * x
    slots = s["slots"].long()
    h, y = s["h"][slots], []
    for i in range(s["case"]["L"]):
        h = a[:, i] * h + u[:, i]
        y.append(h)
    s["h"][slots] = h
    return torch.stack(y, 1).to(s["x"].dtype), s["h"]


# ------------------------------------------------------------------ 64 bits, by the definition
def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "norm":
        x = s["x"].to(torch.float64)
        if c["res"]:
            x = x + s["res"].to(torch.float64)
        n = x / torch.sqrt(x.pow(2).mean(dim=1, keepdim=True) + EPS) * s["w"].to(torch.float64)
        if not c["i8"]:
            return (n, x) if c["res"] else n
        scale = n.abs().max(dim=1).values / 127
        q = torch.round(n / scale[:, None]) * scale[:, None]
        return (q, scale, x) if c["res"] else (q, scale)
    if c["op"] == "product":
        z = torch.einsum("mk,nk->mn", s["x"].to(torch.float64), s["w"].to(torch.float64))
        z = z * torch.outer(s["sx"].to(torch.float64), s["sw"].to(torch.float64))
        if s["bias"] is not None:
            z = z + s["bias"].to(torch.float64)
        f = {"none": lambda t: t,
             "relu": lambda t: torch.where(t > 0, t, torch.zeros_like(t)),
             "silu": lambda t: t * torch.special.expit(t),
             "sigmoid": torch.special.expit,
             "gelu": lambda t: t * torch.special.ndtr(t),
             "gelu_tanh": lambda t: t * torch.special.expit(2 * math.sqrt(2 / math.pi) * (t + 0.044715 * t ** 3))}
        z = f[c["act"]](z)
        return z if s["res"] is None else z + s["res"].to(torch.float64)
    return _exact_recurrence(c, s)


def _exact_recurrence(c, s):
    """Token by token, all sequences side by side; the gradient by differentiating that."""
    train, step = c["op"] == "train", c["op"] == "step"

    def leaf(name):
        t = s.get(name)
        return None if t is None else t.detach().to(torch.float64).requires_grad_(train)

    x, la, i, A, b, h0 = (leaf(k) for k in ("x", "la", "gate", "A", "b", "h0"))
    g = la if b is None else la + b
    if c["decay"] == "log":
        g = torch.clamp(g, max=0.0)
    elif c["decay"] == "softplus":
        g = -A * torch.logaddexp(g, torch.zeros((), dtype=torch.float64, device=g.device))
    else:
        g = -A * torch.special.expit(g)
    a = torch.exp(g)
    u = x if i is None else x * torch.special.expit(i)
    if c["input"] == "complement":
        u = u * -torch.expm1(g)
    elif c["input"] == "normalized":
        u = u * torch.sqrt(-torch.expm1(2 * g))
    a, u = (t.reshape(-1, c["D"]) for t in (a, u))
    lens = [c["L"]] * c["N"] if step else s["lens"]
    start = [sum(lens[:n]) for n in range(len(lens))]
    pooled = step or c.get("pool")
    if pooled:
        h0 = s["h"].to(torch.float64)[s["slots"].long()]
    elif h0 is None:
        h0 = torch.zeros(len(lens), c["D"], device="cuda", dtype=torch.float64)
    order = sorted(range(len(lens)), key=lambda n: -lens[n])  # longest first: those still running come first
    at = torch.tensor([start[n] for n in order], device="cuda")
    h, ends, rows, where = h0[order], [], [], []
    for t in range(max(lens)):
        n = sum(m > t for m in lens)
        if n < h.shape[0]:
            ends.insert(0, h[n:])
            h = h[:n]
        h = a[at[:n] + t] * h + u[at[:n] + t]
        rows.append(h)
        where.append(at[:n] + t)
    y = torch.cat(rows)[torch.argsort(torch.cat(where))]
    end = torch.cat([h] + ends)[torch.argsort(torch.tensor(order, device="cuda"))]
    if not train:
        if pooled:
            pool = s["h"].to(torch.float64)
            pool[s["slots"].long()] = end
            end = pool
        return y.reshape(s["x"].shape), end
    value = (y * s["dy"].to(torch.float64)).sum() + (end * s["dh"].to(torch.float64)).sum()
    wanted = [t for t in (x, la, i, h0, A, b) if t is not None]
    grads = torch.autograd.grad(value, wanted)
    return [y.detach(), end.detach(), *grads]


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "norm":
        M, D = c["M"], c["D"]
        return {"bytes": M * D * (e * (3 if c["res"] else 1) + (1 if c["i8"] else e)) + 4 * D + (4 * M if c["i8"] else 0),
                "flops": 8 * M * D}
    if c["op"] == "product":
        M, K, N = c["M"], c["K"], c["N"]
        return {"bytes": M * K + N * K + 4 * (M + N) + e * (M * N * (2 if c["res"] else 1) + (N if c["bias"] else 0)),
                "flops": 2 * M * K * N}
    D = c["D"]
    T = c["N"] * c["L"] if c["op"] == "step" else c["T"]
    n = c["N"] if c["op"] == "step" else c["seqs"]
    arrays = 4 if c["gate"] else 3  # x, la, (gate), y
    states = 2 if c["op"] != "scan" or c["pool"] else 1
    if c["op"] == "train":  # x, la, (gate), dy; dx, dla, (dgate); dh_T, dh_0; both parameters, read and their gradients written
        arrays += 7 if c["gate"] else 5
        states += 2
    # a multiplication and an addition for the state; the gates: an exponential each, products and sums
    return {"bytes": T * D * arrays * e + states * n * D * 4, "flops": T * D * (24 if c["op"] == "train" else 10)}
