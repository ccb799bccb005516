"""What is measured of the gated delta rule and the projections around it.

Three operators of a gated-delta-rule layer: the rule over packed sequences in
chunks (``kda_gdr_prefill``), the same rule as a recurrence over a few tokens
per sequence (``kda_gdr_decode_step``), and the matrix product with bias,
activation and residual that makes its inputs and takes its output
(``kda_linear``).  ``run`` makes the library's calls where ``own`` is set, and
computes the same with elementary torch operations where it is not.

The rule, per sequence and value head h (query / key head h // (H_v / H_k)):

    q, k <- q / sqrt(|q|^2 + eps), k / sqrt(|k|^2 + eps)
    b    =  sigmoid(beta)
    la   =  min(log_alpha, 0), or -A_h softplus(z + bias_h) from the logit z
    S_t  =  (I - b k k^T) e^la S_{t-1} + b k v^T        [d_k x d_v]
    o_t  =  S_t^T q
"""
import math
import random

import torch

own = False

CHUNK = 64
EPS = 1e-6
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh", "sigmoid")
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one token through a layer's output projection onto the residual stream
        {"name": "linear one token", "op": "linear", "M": 1, "K": 4096, "N": 4096, "bias": False,
         "act": "none", "res": True, "dtype": "bf16"},
        # a decode batch of 64 sequences: 96 heads of 128 channels back to the model width
        {"name": "linear decode batch", "op": "linear", "M": 64, "K": 12288, "N": 4096,
         "bias": True, "act": "none", "res": True, "dtype": "bf16"},
        # a ragged prefill batch through a small biased, activated projection, odd sizes
        {"name": "linear ragged", "op": "linear", "M": 333, "K": 1000, "N": 1499, "bias": True,
         "act": "silu", "res": False, "dtype": "bf16"},
        # 4096 tokens into 96 heads of 128 channels
        {"name": "linear prefill", "op": "linear", "M": 4096, "K": 4096, "N": 12288, "bias": True,
         "act": "gelu_tanh", "res": True, "dtype": "bf16"},
        # the 32-bit path: a small projection as tests and checks of a model use it
        {"name": "linear f32", "op": "linear", "M": 200, "K": 512, "N": 640, "bias": True,
         "act": "sigmoid", "res": False, "dtype": "f32"},
        # one short prompt, where a call's latency counts
        {"name": "rule short prompt", "op": "prefill", "T": 77, "seqs": 1, "cut": 0, "Hk": 4,
         "Hv": 8, "dk": 128, "dv": 128, "logit": False, "pool": False, "dtype": "bf16"},
        # a serving batch: prompts of ragged lengths, one of them empty, states in a pool
        {"name": "rule packed prompts", "op": "prefill", "T": 12000, "seqs": 9, "cut": 5, "Hk": 16,
         "Hv": 32, "dk": 128, "dv": 128, "logit": True, "pool": True, "dtype": "bf16"},
        # 4096 tokens through 96 heads of 128 channels
        {"name": "rule long prompt", "op": "prefill", "T": 4096, "seqs": 1, "cut": 0, "Hk": 48,
         "Hv": 96, "dk": 128, "dv": 128, "logit": False, "pool": False, "dtype": "bf16"},
        # the 32-bit path, small heads, wider values than keys
        {"name": "rule f32", "op": "prefill", "T": 300, "seqs": 2, "cut": 3, "Hk": 4, "Hv": 4,
         "dk": 64, "dv": 128, "logit": False, "pool": False, "dtype": "f32"},
        # one user's next token
        {"name": "step one user", "op": "step", "N": 1, "L": 1, "Hk": 16, "Hv": 32, "dk": 128,
         "dv": 128, "logit": False, "snap": False, "dtype": "bf16"},
        # the next token of 64 users, 96 heads
        {"name": "step batch", "op": "step", "N": 64, "L": 1, "Hk": 48, "Hv": 96, "dk": 128,
         "dv": 128, "logit": True, "snap": False, "dtype": "bf16"},
        # four proposed tokens for each of 24 users, the state after each kept until some are taken
        {"name": "step proposed tokens", "op": "step", "N": 24, "L": 4, "Hk": 16, "Hv": 32,
         "dk": 128, "dv": 128, "logit": False, "snap": True, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(("linear", "linear", "prefill", "prefill", "step"))
    dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
    if op == "linear":
        small = dtype == "f32"
        M = _log(rng, 1, 1024 if small else 4096)
        K, N = (_log(rng, 64, 1024 if small else 12288) for _ in range(2))
        if rng.random() < 0.6:  # most widths are multiples of 8, some are not
            K, N = (K + 7) // 8 * 8, (N + 7) // 8 * 8
        while M * K * N > 4096 * 4096 * 12288:
            M = (M + 1) // 2
        return {"op": op, "M": M, "K": K, "N": N, "bias": rng.random() < 0.5,
                "act": rng.choice(ACTS), "res": rng.random() < 0.5, "dtype": dtype}
    small = dtype == "f32"
    Hk = rng.choice((1, 2, 4, 8) if small else (1, 2, 4, 8, 16, 32))
    Hv = Hk * rng.choice((1, 2, 3, 4))
    dk, dv = rng.choice((32, 64, 128, 128)), rng.choice((32, 64, 128, 128, 256))
    cost = 4096 * 96 * 128 * 128 // (16 if small else 1)
    if op == "prefill":
        T = _log(rng, 1, 2048 if small else 16384)
        while T * Hv * dk * dv > cost:
            T = T // 2 + 1
        return {"op": op, "T": T, "seqs": _log(rng, 1, 16), "cut": rng.randrange(1, 1 << 20),
                "Hk": Hk, "Hv": Hv, "dk": dk, "dv": dv, "logit": rng.random() < 0.5,
                "pool": rng.random() < 0.5, "dtype": dtype}
    N, L = _log(rng, 1, 128), rng.choice((1, 1, 2, 3, 4, 7))
    while N * Hv * dk * dv > 64 * 96 * 128 * 128:
        N = (N + 1) // 2
    return {"op": op, "N": N, "L": L, "Hk": Hk, "Hv": Hv, "dk": dk, "dv": dv,
            "logit": rng.random() < 0.5, "snap": L > 1 and N * Hv * L <= 4096, "dtype": dtype}


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

    if c["op"] == "linear":
        M, K, N = c["M"], c["K"], c["N"]
        return {"case": c, "x": normal(M, K), "w": normal(N, K, std=K ** -0.5),
                "bias": normal(N, std=0.5) if c["bias"] else None,
                "res": normal(M, N) if c["res"] else None}
    Hk, Hv, dk, dv = c["Hk"], c["Hv"], c["dk"], c["dv"]
    if c["op"] == "prefill":
        lens = _lengths(c)
        rows, n = (c["T"],), len(lens)
        at = [0]
        for x in lens:
            at.append(at[-1] + x)
        s = {"lens": lens, "cu": torch.tensor(at, dtype=torch.int32, device=dev)}
    else:
        rows, n = (c["N"], c["L"]), c["N"]
        s = {}
    s |= {"case": c, "q": normal(*rows, Hk, dk), "k": normal(*rows, Hk, dk),
          "v": normal(*rows, Hv, dv), "beta": normal(*rows, Hv)}
    # decays as such layers start out: rates A in [1, 16], steps of 0.001 to 0.1
    A = 1 + 15 * torch.rand(Hv, generator=g, device=dev)
    step = torch.exp(math.log(1e-3) + math.log(100.0) * torch.rand(Hv, generator=g, device=dev))
    z, bias = normal(*rows, Hv, dtype=torch.float32), torch.log(torch.expm1(step))
    s["A"], s["bias"] = (A, bias) if c["logit"] else (None, None)
    s["la"] = z if c["logit"] else -A * torch.nn.functional.softplus(z + bias)
    if c["op"] == "step":
        s["S"] = normal(n, Hv, dk, dv, std=0.1, dtype=torch.float32)
        s["slots"] = torch.randperm(n, generator=g, device=dev).to(torch.int32)
    elif c["pool"]:
        s["S"] = normal(n + 2, Hv, dk, dv, std=0.1, dtype=torch.float32)
        s["slots"] = torch.randperm(n + 2, generator=g, device=dev)[:n].to(torch.int32)
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return {"linear": _own_linear, "prefill": _own_prefill, "step": _own_step}[op](state)
    return {"linear": _plain_linear, "prefill": _plain_prefill, "step": _plain_step}[op](state)


def _own_linear(s):
    from linear_attention_recurrence_prefill_gb300 import kda
    return kda.kda_linear(s["x"], s["w"], s["bias"], s["res"], act=s["case"]["act"])


def _own_prefill(s):
    from linear_attention_recurrence_prefill_gb300 import kda
    c = s["case"]
    form = dict(beta_is_logit=True, max_seqlen=max(s["lens"]), decay_from_logit=c["logit"],
                decay_scale=s["A"], decay_bias=s["bias"])
    if c["pool"]:
        return kda.kda_gdr_prefill(s["q"], s["k"], s["v"], s["la"], s["beta"], s["S"], s["cu"],
                                   S_T=s["S"], slots=s["slots"], **form)
    return kda.kda_gdr_prefill(s["q"], s["k"], s["v"], s["la"], s["beta"], None, s["cu"], **form)


def _own_step(s):
    from linear_attention_recurrence_prefill_gb300 import kda
    c = s["case"]
    got = kda.kda_gdr_decode_step(s["q"], s["k"], s["v"], s["la"], s["beta"], s["S"],
                                  slots=s["slots"], beta_is_logit=True,
                                  decay_from_logit=c["logit"], decay_scale=s["A"],
                                  decay_bias=s["bias"], snapshots=c["snap"])
    return (*got, s["S"]) if c["snap"] else (got, s["S"])


def _plain_linear(s):
    y = s["x"].float() @ s["w"].float().T
    if s["bias"] is not None:
        y = y + s["bias"].float()
    act = s["case"]["act"]
    if act == "relu":
        y = y.clamp_min(0.0)
    elif act == "silu":
        y = y / (1 + torch.exp(-y))
    elif act == "sigmoid":
        y = 1 / (1 + torch.exp(-y))
    elif act == "gelu":
        y = 0.5 * y * (1 + torch.erf(y * math.sqrt(0.5)))
    elif act == "gelu_tanh":
        y = 0.5 * y * (1 + torch.tanh(math.sqrt(2 / math.pi) * (y + 0.044715 * y * y * y)))
    if s["res"] is not None:
        y = y + s["res"].float()
    return y.to(s["x"].dtype)


def _unit(x):
    return x * torch.rsqrt((x * x).sum(-1, keepdim=True) + EPS)


def _plain_inputs(s):
    """q, k (one row per value head), v, log alpha and beta, in 32 bits."""
    c = s["case"]
    q, k, v, la, beta = (s[x].float() for x in ("q", "k", "v", "la", "beta"))
    if c["logit"]:
        x = la + s["bias"]
        la = -s["A"] * (x.clamp_min(0.0) + torch.log1p(torch.exp(-x.abs())))
    G = c["Hv"] // c["Hk"]
    q, k = (_unit(x).repeat_interleave(G, dim=-2) for x in (q, k))
    return q, k, v, la.clamp_max(0.0), torch.sigmoid(beta)


def _plain_prefill(s):
    c, cu, C = s["case"], s["cu"], CHUNK
    N, nc = len(s["lens"]), max(1, -(-max(s["lens"]) // C))
    q, k, v, la, beta = _plain_inputs(s)
    # sequences side by side, each in nc chunks: rows behind a sequence's end have k = v = beta = la = 0
    t = torch.arange(nc * C, device=cu.device)
    inside = t < (cu[1:] - cu[:-1])[:, None]
    row = (cu[:-1, None] + t).clamp_max(c["T"] - 1).long()

    def chunks(x):  # [T, Hv, ...] -> [nc, N, Hv, C, ...]
        x = x[row] * inside.reshape(N, nc * C, *([1] * (x.dim() - 1)))
        return x.reshape(N, nc, C, *x.shape[2:]).transpose(0, 1).transpose(2, 3)

    q, k, v, la, beta = (chunks(x) for x in (q, k, v, la, beta))
    # sums of up to 64 log decays, of which differences are taken: 64 bits
    g = la.double().cumsum(-1)
    D = torch.exp((g[..., :, None] - g[..., None, :]).clamp_max(0.0)).float()
    eg, eG, rest = torch.exp(g).float(), torch.exp(g[..., -1:]).float(), torch.exp(g[..., -1:] - g).float()
    A = torch.tril(k @ k.transpose(-1, -2) * D, -1) * beta[..., None]
    P = torch.tril(q @ k.transpose(-1, -2) * D)
    X = torch.eye(C, device=cu.device).expand(A.shape).clone()  # (I + A)^-1, row by row
    for i in range(1, C):
        X[..., i, :i] = -(A[..., i:i + 1, :i] @ X[..., :i, :i]).squeeze(-2)
    X = X * beta[..., None, :]
    pool = c["pool"]
    slots = s["slots"].long() if pool else None
    S = s["S"][slots] if pool else torch.zeros(N, c["Hv"], c["dk"], c["dv"], device=cu.device)
    o = torch.empty(nc, N, c["Hv"], C, c["dv"], device=cu.device)
    for i in range(nc):
        U = X[i] @ (v[i] - eg[i][..., None] * (k[i] @ S))
        o[i] = eg[i][..., None] * (q[i] @ S) + P[i] @ U
        S = eG[i][..., None] * S + (rest[i][..., None] * k[i]).transpose(-1, -2) @ U
    # each token's sequence and place in it (an empty sequence owns no token)
    at = torch.arange(c["T"], device=cu.device, dtype=cu.dtype)
    seq = torch.searchsorted(cu, at, right=True) - 1
    place = at.long() - cu[seq].long()
    out = o[place // C, seq, :, place % C].to(s["q"].dtype)
    if pool:
        s["S"][slots] = S
        return out, s["S"]
    return out, S


def _plain_step(s):
    c = s["case"]
    q, k, v, la, beta = _plain_inputs(s)
    slots = s["slots"].long()
    S, o, snaps = s["S"][slots], [], []
    for i in range(c["L"]):
        S = S * torch.exp(la[:, i])[..., None, None]
        u = (k[:, i, :, None, :] @ S).squeeze(-2)
        w = beta[:, i, :, None] * (v[:, i] - u)
        S = S + k[:, i, :, :, None] * w[:, :, None, :]
        o.append((q[:, i, :, None, :] @ S).squeeze(-2))
        snaps.append(S)
    s["S"][slots] = S
    o = torch.stack(o, 1).to(s["q"].dtype)
    return (o, torch.stack(snaps, 1), s["S"]) if c["snap"] else (o, s["S"])


# ------------------------------------------------------------------ 64 bits, by the definition
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "linear":
        x, w = s["x"].to(torch.float64), s["w"].to(torch.float64)
        z = torch.einsum("mk,nk->mn", x, w)
        if s["bias"] is not None:
            z += s["bias"].to(torch.float64)
        f = {"none": lambda t: t,
             "relu": lambda t: torch.where(t > 0, t, torch.zeros_like(t)),
             "silu": lambda t: t * torch.special.expit(t),
             "sigmoid": torch.special.expit,
             "gelu": lambda t: t * torch.special.ndtr(t),
             "gelu_tanh": lambda t: t * torch.special.expit(2 * math.sqrt(2 / math.pi) * (t + 0.044715 * t ** 3))}
        z = f[case["act"]](z)
        return z if s["res"] is None else z + s["res"].to(torch.float64)
    return _exact_rule(case, s)


def _exact_rule(c, s):
    """Token by token: the state fades, what k finds in it is replaced by a mix with v, q reads it."""
    d = {x: s[x].to(torch.float64) for x in ("q", "k", "v", "la", "beta")}
    G, step = c["Hv"] // c["Hk"], c["op"] == "step"
    head = torch.arange(c["Hv"], device="cuda") // G
    for x in ("q", "k"):
        d[x] = (d[x] / torch.sqrt(d[x].pow(2).sum(-1, keepdim=True) + EPS))[..., head, :]
    if c["logit"]:
        d["la"] = -s["A"].double() * torch.logaddexp(d["la"] + s["bias"].double(), torch.zeros((), device="cuda", dtype=torch.float64))
    alpha, b = torch.exp(torch.minimum(d["la"], torch.zeros_like(d["la"]))), torch.special.expit(d["beta"])
    lens = [c["L"]] * c["N"] if step else s["lens"]
    start = [i * c["L"] for i in range(c["N"])] if step else [sum(lens[:i]) for i in range(len(lens))]
    q, k, v, alpha, b = (x.reshape(-1, *x.shape[2 if step else 1:]) for x in (d["q"], d["k"], d["v"], alpha, b))
    pooled = step or c["pool"]
    pool = s["S"].double() if pooled else torch.zeros(len(lens), c["Hv"], c["dk"], c["dv"], device="cuda", dtype=torch.float64)
    slot = s["slots"].tolist() if pooled else list(range(len(lens)))
    o = torch.zeros(q.shape[0], c["Hv"], c["dv"], device="cuda", dtype=torch.float64)
    order = sorted(range(len(lens)), key=lambda i: -lens[i])  # longest first: those still running come first
    at, slot = (torch.tensor([x[i] for i in order], device="cuda") for x in (start, slot))
    S, snaps = pool[slot], []
    for t in range(max(lens)):
        n = sum(x > t for x in lens)
        r, live = at[:n] + t, S[:n]
        live *= alpha[r][..., None, None]
        found = torch.einsum("nhk,nhkv->nhv", k[r], live)
        live += torch.einsum("nhk,nhv->nhkv", k[r], b[r][..., None] * (v[r] - found))
        o[r] = torch.einsum("nhk,nhkv->nhv", q[r], live)
        if step and c["snap"]:
            snaps.append(S.clone())
    pool[slot] = S
    if not step:
        return o, pool
    o = o.reshape(c["N"], c["L"], c["Hv"], c["dv"])
    if not c["snap"]:
        return o, pool
    back = torch.argsort(torch.tensor(order, device="cuda"))
    return o, torch.stack(snaps, 1)[back], pool


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "linear":
        M, K, N = c["M"], c["K"], c["N"]
        return {"bytes": e * (M * K + N * K + M * N * (2 if c["res"] else 1) + (N if c["bias"] else 0)),
                "flops": 2 * M * K * N}
    Hk, Hv, dk, dv = c["Hk"], c["Hv"], c["dk"], c["dv"]
    step = c["op"] == "step"
    T = c["N"] * c["L"] if step else c["T"]
    token = e * (2 * Hk * dk + 2 * Hv * dv + Hv) + 4 * Hv
    n = c["N"] if step else c["seqs"]
    states = n * (2 if step or c["pool"] else 1) + (T if step and c["snap"] else 0)
    # per token and head: k and q against the state, and the rank-one update, 2 d_k d_v each
    return {"bytes": T * token + states * Hv * dk * dv * 4, "flops": 6 * T * Hv * dk * dv}
