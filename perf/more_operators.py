"""The operators of a block with a residual path and of training on a policy's
own tokens, as measured cases: one pass through each operator, its plain form
in elementary torch operations and its value in 64 bits.

Operators (T is the number of logical shards):

  norm         y = (x - mean) / sqrt(var + eps) * w + b, row by row
  norm_grad    gradients of x (with the residual path's gradient added), w, b
  linear       column split: Y = act(X W + b) + R, W's columns in T shards;
               row split: Y = sum_r X_r W_r + b + R, W's rows in T shards
  linear_grad  its other direction: gradients of X, W and b
  policy       clipped policy loss of given tokens with a KL term, and its
               gradient, in one call ("fused") or as a loss call and a
               gradient call
"""

import math

import torch

own = False   # true: `run` calls the package's operators

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f32": 4}
_EPS = 1e-5


def _pkg():
    import tensor_transformer_mlp_columnparallel_gb300 as tp
    return tp


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one decoding step of one request: launch latency
        dict(name="norm_n1", op="norm", dt="bf16", wdt="bf16", N=1, D=12288, pad=0, offset=0.0),
        # a training step's tokens
        dict(name="norm_n8192", op="norm", dt="bf16", wdt="f32", N=8192, D=8192, pad=0, offset=0.0),
        # the same step's other direction, the residual path's gradient added
        dict(name="norm_grad_n8192", op="norm_grad", dt="bf16", wdt="f32", N=8192, D=8192, pad=0,
             offset=0.0, residual=True),
        # odd sizes in padded rows, a mean well away from zero
        dict(name="norm_grad_odd_f32", op="norm_grad", dt="f32", wdt="f32", N=4099, D=1030, pad=7,
             offset=4.0, residual=False),
        # the exact-fp32 projection
        dict(name="linear_f32", op="linear", split="column", dt="f32", N=64, D=256, F=1024, T=2,
             act="relu", bias=True, residual=False, save_z=True, pad=0),
        # the block end of one decoding step: the weights' reads bound it
        dict(name="linear_row_n16", op="linear", split="row", dt="bf16", N=16, D=12288, F=49152, T=8,
             act=None, bias=True, residual=True, save_z=False, pad=0),
        # a training step's projections: up with its activation, and down onto the residual path
        dict(name="linear_up_n4096", op="linear", split="column", dt="bf16", N=4096, D=4096, F=16384,
             T=4, act="gelu_tanh", bias=True, residual=False, save_z=True, pad=0),
        dict(name="linear_down_n4096", op="linear", split="row", dt="bf16", N=4096, D=4096, F=16384,
             T=4, act=None, bias=True, residual=True, save_z=False, pad=0),
        # gradients of a few tokens: the weights' reads and writes bound them
        dict(name="linear_grad_n16", op="linear_grad", split="row", dt="bf16", N=16, D=4096, F=16384,
             T=4, act=None, bias=True, pad=0),
        # a training step's
        dict(name="linear_grad_n4096", op="linear_grad", split="column", dt="bf16", N=4096, D=4096,
             F=16384, T=4, act="gelu_tanh", bias=True, pad=0),
        # a training step on sampled answers, a quarter of the positions prompt
        # or padding, loss and gradient together
        dict(name="policy_n4096", op="policy", dt="bf16", N=4096, V=128000, T=8, pad=0, fused=True,
             tau=1.0, kl=0.02, low=0.2, high=0.28, empty=0.25),
        # fp32 logits of an odd vocabulary in padded rows; the gradient is
        # asked for later, with weights per token
        dict(name="policy_odd_f32", op="policy", dt="f32", N=1003, V=50001, T=7, pad=15, fused=False,
             tau=0.7, kl=0.0, low=0.2, high=0.2, empty=0.1),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "linear", "linear_grad", "policy"])
    dt = rng.choice(["bf16", "f32"])
    if op in ("norm", "norm_grad"):
        D = _log_int(rng, 8, 12288)
        if rng.random() < 0.6:
            D = (D + 7) // 8 * 8
        # bounded by the listed cases' elements
        N = _log_int(rng, 1, max(1, min(8192, 8192 * 8192 * 2 // (D * _SIZE[dt]))))
        case = dict(op=op, dt=dt, wdt=rng.choice([dt, "f32"]), N=N, D=D,
                    pad=rng.choice([0, 0, rng.randint(1, 64)]), offset=rng.choice([0.0, 0.0, 4.0]))
        if op == "norm_grad":
            case["residual"] = rng.random() < 0.6
        return case
    if op in ("linear", "linear_grad"):
        split = rng.choice(["column", "row"])
        if dt == "f32":
            T = rng.choice([1, 2, 3])
            N, D, F = _log_int(rng, 1, 64), _log_int(rng, 16, 256), T * max(1, _log_int(rng, 32, 1024) // T)
            pad = rng.choice([0, rng.randint(1, 9)])
        else:
            T = rng.choice([1, 2, 4, 8])
            N, D = _log_int(rng, 1, 4096), 8 * _log_int(rng, 32, 512)
            F = 8 * T * max(1, _log_int(rng, 128, 2048) // T)
            pad = rng.choice([0, 8 * rng.randint(1, 9)])
        act = rng.choice([None, "relu", "gelu_tanh", "gelu_erf", "gelu_sigmoid"]) if split == "column" else None
        case = dict(op=op, split=split, dt=dt, N=N, D=D, F=F, T=T, act=act, bias=rng.random() < 0.6, pad=pad)
        if op == "linear":
            case.update(residual=rng.random() < 0.6, save_z=act is not None and rng.random() < 0.5)
        return case
    T = rng.choice([1, 2, 3, 4, 7, 8, 16])
    V = max(_log_int(rng, 1000, 128000) // T, 1) * T
    N = _log_int(rng, 1, max(1, min(4096, 4096 * 128000 * 2 // (V * _SIZE[dt]))))
    return dict(op=op, dt=dt, N=N, V=V, T=T, pad=rng.choice([0, 0, rng.randint(1, 64)]),
                fused=rng.choice([True, True, False]), tau=rng.choice([0.7, 1.0, 1.0, 1.5]),
                kl=rng.choice([0.0, 0.02, 0.1]), low=0.2, high=rng.choice([0.2, 0.28]),
                empty=rng.choice([0.0, 0.25, 0.6]))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _matrix(g, N, C, pad, dt, std, dev):
    """[N, C] normal values in rows of C + pad elements."""
    z = torch.empty((N, C + pad), dtype=dt, device=dev)
    step = max(1, (1 << 27) // (C + pad))
    for i in range(0, N, step):
        n = min(step, N - i)
        z[i:i + n] = (torch.randn((n, C + pad), generator=g, device=dev) * std).to(dt)
    return z[:, :C]


def _policy_inputs(case, g, dev):
    """Tokens sampled from the rows' own distribution (half the rows are sure
    of one token), log probabilities of a policy a step older and of a
    reference, advantages of sequences, some of which are exactly zero."""
    N, V, tau = case["N"], case["V"], case["tau"]
    z = _matrix(g, N, V, case["pad"], _TYPES[case["dt"]], 2.0, dev)
    sure = torch.nonzero(torch.rand(N, generator=g, device=dev) < 0.5).flatten()
    token = torch.randint(0, V, (sure.numel(),), generator=g, device=dev)
    z[sure, token] = (8.0 + 17.0 * torch.rand(sure.numel(), generator=g, device=dev)).to(z.dtype)
    t = torch.empty(N, dtype=torch.int64, device=dev)
    lp = torch.empty(N, dtype=torch.float64, device=dev)
    step = max(1, (1 << 26) // V)
    for i in range(0, N, step):
        r = z[i:i + step].float() / tau
        u = torch.rand(r.shape, generator=g, device=dev).clamp_(min=1e-30, max=1.0 - 1e-7)
        t[i:i + step] = (r - torch.log(-torch.log(u))).argmax(dim=1)
        lp[i:i + step] = (r.gather(1, t[i:i + step, None])[:, 0].double()
                          - torch.logsumexp(r.double(), dim=1))
    far = torch.rand(N, generator=g, device=dev) < 0.05
    move = torch.randn(N, generator=g, device=dev) * torch.where(far, 1.0, 0.12)
    old = (lp + move).float()
    # the loss has a kink where the ratio meets a border of the clip range: no
    # derivative there, so none of the tokens lies within 1e-4 of it
    for border in (1.0 - case["low"], 1.0 + case["high"]):
        near = (torch.exp(lp - old.double()) - border).abs() < 1e-4
        old = torch.where(near, old + 1e-3, old)
    sequence = torch.arange(N, device=dev) // 64
    gain = torch.randn(N // 64 + 1, generator=g, device=dev)
    gain = torch.where(torch.rand(N // 64 + 1, generator=g, device=dev) < 0.1, torch.zeros_like(gain), gain)
    empty = torch.rand(N, generator=g, device=dev) < case["empty"]
    return {"logits": z, "targets": torch.where(empty, torch.full_like(t, -1), t), "old": old,
            "adv": gain[sequence].contiguous(),
            "ref": (lp + 0.3 * torch.randn(N, generator=g, device=dev)).float(),
            "weights": torch.rand(N, generator=g, device=dev) + 0.5}


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed) + 1)
    op, N, dt = case["op"], case["N"], _TYPES[case["dt"]]
    s = {"case": case}
    if op == "policy":
        s.update(_policy_inputs(case, g, dev))
        return s
    if op in ("norm", "norm_grad"):
        D, pad, wdt = case["D"], case["pad"], _TYPES[case["wdt"]]
        # a residual stream: unit variance, a few channels many times larger
        loud = torch.where(torch.rand(D, generator=g, device=dev) < 0.002, 20.0, 1.0)
        scale = torch.exp(0.3 * torch.randn((N, 1), generator=g, device=dev))
        x = _matrix(g, N, D, pad, torch.float32, 1.0, dev)
        s["x"] = torch.empty((N, D + pad), dtype=dt, device=dev)[:, :D]
        s["x"].copy_(x * loud * scale + case["offset"])
        s["w"] = (1.0 + 0.1 * torch.randn(D, generator=g, device=dev)).to(wdt)
        s["b"] = (0.1 * torch.randn(D, generator=g, device=dev)).to(wdt)
        if op == "norm_grad":
            s["dy"] = _matrix(g, N, D, pad, dt, 1.0, dev)
            s["dres"] = _matrix(g, N, D, pad, dt, 1.0, dev) if case["residual"] else None
            x = s["x"].double()   # what the forward kept
            mean = x.mean(dim=1, keepdim=True)
            var = ((x - mean) ** 2).mean(dim=1)
            s["mean"], s["rstd"] = mean[:, 0].float(), (1.0 / torch.sqrt(var + _EPS)).float()
        return s
    D, F, T, pad = case["D"], case["F"], case["T"], case["pad"]
    column = case["split"] == "column"
    n_in, n_out = (D, F) if column else (F, D)
    s["X"] = _matrix(g, N, n_in, pad, dt, 1.0, dev)
    shape = (D, F // T) if column else (F // T, D)
    s["W"] = [_matrix(g, *shape, 0, dt, 0.02, dev) for _ in range(T)]
    if op == "linear":
        s["b"] = None
        if case["bias"]:
            b = (torch.randn(n_out, generator=g, device=dev) * 0.02).to(dt)
            s["b"] = [x.clone() for x in b.chunk(T)] if column else b
        s["R"] = _matrix(g, N, n_out, pad, dt, 1.0, dev) if case["residual"] else None
    else:
        s["dY"] = _matrix(g, N, n_out, pad, dt, 1.0, dev)
        s["Z"] = _matrix(g, N, n_out, 0, dt, 0.02 * math.sqrt(n_in), dev) if case["act"] else None
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    return _PLAIN[op](state)


def _own_norm(s):
    y, mean, rstd = _pkg().layernorm(s["x"], s["w"], s["b"], eps=_EPS)
    return {"y": y, "mean": mean, "rstd": rstd}


def _own_norm_grad(s):
    dx, dw, db = _pkg().layernorm_backward(s["dy"], s["x"], s["w"], s["mean"], s["rstd"],
                                           dresidual=s["dres"])
    return {"dx": dx, "dw": dw, "db": db}


def _own_linear(s):
    c, tp = s["case"], _pkg()
    if c["split"] == "row":
        return {"Y": tp.row_linear(s["X"], s["W"], s["b"], residual=s["R"])}
    Y, Z = tp.column_linear(s["X"], s["W"], s["b"], act=c["act"], residual=s["R"], save_z=c["save_z"])
    return {"Y": Y, "Z": Z} if c["save_z"] else {"Y": Y}


def _own_linear_grad(s):
    c, tp = s["case"], _pkg()
    if c["split"] == "row":
        dX, dW, db = tp.row_linear_backward(s["X"], s["W"], s["dY"], bias_grads=c["bias"])
    else:
        dX, dW, db = tp.column_linear_backward(s["X"], s["W"], s["dY"], Z=s["Z"], act=c["act"],
                                               bias_grads=c["bias"])
    out = {"dX": dX, "dW": dW}
    if c["bias"]:
        out["db"] = db
    return out


def _own_policy(s):
    c, tp = s["case"], _pkg()
    args = (s["logits"], s["targets"], s["old"], s["adv"], c["T"])
    opt = dict(ref_logprobs=s["ref"], kl_coef=c["kl"], clip_low=c["low"], clip_high=c["high"],
               temperature=c["tau"])
    if c["fused"]:
        loss, mean, logprob, kl, d = tp.vocab_policy_with_grad(*args, **opt, grad_scale=1.0 / c["N"])
    else:
        loss, mean, logprob, kl = tp.vocab_policy(*args, **opt)
        d = tp.vocab_policy_backward(*args, logprob, **opt, grad_scale=1.0 / c["N"],
                                     grad_tokens=s["weights"])
    return {"loss": loss, "mean": mean, "logprob": logprob, "kl": kl, "dlogits": d}


def _plain_norm(s):
    x = s["x"].float()
    mean = x.mean(dim=1, keepdim=True)
    c = x - mean
    rstd = 1.0 / torch.sqrt((c * c).mean(dim=1, keepdim=True) + _EPS)
    y = c * rstd * s["w"].float() + s["b"].float()
    return {"y": y.to(s["x"].dtype), "mean": mean[:, 0], "rstd": rstd[:, 0]}


def _plain_norm_grad(s):
    x, dy = s["x"].float(), s["dy"].float()
    h = (x - s["mean"][:, None]) * s["rstd"][:, None]
    u = dy * s["w"].float()
    dx = s["rstd"][:, None] * (u - u.mean(dim=1, keepdim=True) - h * (u * h).mean(dim=1, keepdim=True))
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    wdt = s["w"].dtype
    return {"dx": dx.to(s["x"].dtype), "dw": (dy * h).sum(dim=0).to(wdt), "db": dy.sum(dim=0).to(wdt)}


def _act(name, z):
    if name is None:
        return z
    if name == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if name == "gelu_sigmoid":
        return z / (1.0 + torch.exp(-1.702 * z))
    if name == "gelu_erf":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))


def _act_slope(name, z):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "gelu_sigmoid":
        p = 1.0 / (1.0 + torch.exp(-1.702 * z))
        return p * (1.0 + 1.702 * z * (1.0 - p))
    if name == "gelu_erf":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    a = math.sqrt(2.0 / math.pi)
    t = torch.tanh(a * (z + 0.044715 * z * z * z))
    return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * a * (1.0 + 3.0 * 0.044715 * z * z)


def _plain_linear(s):
    c, dt = s["case"], s["X"].dtype
    X = s["X"].float()
    if c["split"] == "column":
        z = torch.cat([X @ w.float() for w in s["W"]], dim=1)
        if s["b"] is not None:
            z = z + torch.cat(s["b"]).float()
    else:
        z = sum(x @ w.float() for x, w in zip(X.chunk(c["T"], dim=1), s["W"]))
        if s["b"] is not None:
            z = z + s["b"].float()
    y = _act(c["act"], z)
    if s["R"] is not None:
        y = y + s["R"].float()
    return {"Y": y.to(dt), "Z": z.to(dt)} if c["save_z"] else {"Y": y.to(dt)}


def _plain_linear_grad(s):
    c, dt, T = s["case"], s["X"].dtype, s["case"]["T"]
    X, dZ = s["X"].float(), s["dY"].float()
    if c["act"]:
        dZ = dZ * _act_slope(c["act"], s["Z"].float())
    out = {}
    if c["split"] == "column":
        parts = dZ.chunk(T, dim=1)
        out["dX"] = sum(d @ w.float().t() for d, w in zip(parts, s["W"])).to(dt)
        out["dW"] = [(X.t() @ d).to(dt) for d in parts]
        if c["bias"]:
            out["db"] = [d.sum(dim=0).to(dt) for d in parts]
    else:
        out["dX"] = torch.cat([dZ @ w.float().t() for w in s["W"]], dim=1).to(dt)
        out["dW"] = [(x.t() @ dZ).to(dt) for x in X.chunk(T, dim=1)]
        if c["bias"]:
            out["db"] = dZ.sum(dim=0).to(dt)
    return out


def _plain_policy(s):
    c = s["case"]
    tau, N = c["tau"], c["N"]
    live = s["targets"] >= 0
    t = s["targets"].clamp(min=0)[:, None]
    z = s["logits"].float() / tau
    m = z.amax(dim=1, keepdim=True)
    e = torch.exp(z - m)
    total = e.sum(dim=1, keepdim=True)
    lp = (z.gather(1, t) - m - torch.log(total))[:, 0]
    ratio = torch.exp(lp - s["old"])
    a = s["adv"]
    held = torch.minimum(torch.maximum(ratio, torch.full_like(ratio, 1.0 - c["low"])),
                         torch.full_like(ratio, 1.0 + c["high"]))
    x = torch.exp(s["ref"] - lp)
    kl = x - (s["ref"] - lp) - 1.0
    zero = torch.zeros_like(lp)
    loss = torch.where(live, -torch.minimum(ratio * a, held * a) + c["kl"] * kl, zero)
    moves = torch.where(a > 0, ratio <= 1.0 + c["high"], ratio >= 1.0 - c["low"])
    slope = torch.where(moves, -a * ratio, zero) + c["kl"] * (1.0 - x)
    w = slope / (tau * N)
    if not c["fused"]:
        w = w * s["weights"]
    w = torch.where(live, w, zero)[:, None]
    d = e / total * -w
    d.scatter_add_(1, t, w)
    return {"loss": loss, "mean": loss.sum().reshape(1) / N, "logprob": torch.where(live, lp, zero),
            "kl": torch.where(live, kl, zero), "dlogits": d.to(s["logits"].dtype)}


_OWN = {"norm": _own_norm, "norm_grad": _own_norm_grad, "linear": _own_linear,
        "linear_grad": _own_linear_grad, "policy": _own_policy}
_PLAIN = {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "linear": _plain_linear,
          "linear_grad": _plain_linear_grad, "policy": _plain_policy}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    op, N, es = case["op"], case["N"], _SIZE[case["dt"]]
    if op in ("norm", "norm_grad"):
        D, ws = case["D"], _SIZE[case["wdt"]]
        if op == "norm":
            return {"bytes": 2.0 * N * D * es + 2.0 * D * ws + 8.0 * N, "flops": 8.0 * N * D}
        rows = 4.0 if case["residual"] else 3.0
        return {"bytes": rows * N * D * es + 3.0 * D * ws + 8.0 * N, "flops": 14.0 * N * D}
    if op == "policy":
        V = case["V"]
        read = (1.0 - case["empty"]) * N * V * es
        return {"bytes": read + N * V * es + N * (8 + 12 + 12) + 4 + (0 if case["fused"] else 4 * N),
                "flops": 6.0 * N * V}
    D, F = case["D"], case["F"]
    n_in, n_out = (D, F) if case["split"] == "column" else (F, D)
    if op == "linear":
        more = (case["residual"] + case["save_z"]) * N * n_out + case["bias"] * n_out
        return {"bytes": es * (1.0 * N * n_in + D * F + N * n_out + more), "flops": 2.0 * N * D * F}
    more = (N * n_out if case["act"] else 0) + case["bias"] * n_out
    return {"bytes": es * (2.0 * N * n_in + 2.0 * D * F + N * n_out + more), "flops": 4.0 * N * D * F}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    return _EXACT[case["op"]](case, prepare(case, seed))


def _exact_norm(case, s):
    var, mean = torch.var_mean(s["x"].double(), dim=1, unbiased=False, keepdim=True)
    rstd = torch.rsqrt(var + _EPS)
    y = torch.addcmul(s["b"].double(), (s["x"].double() - mean) * rstd, s["w"].double())
    return {"y": y, "mean": mean.flatten(), "rstd": rstd.flatten()}


def _exact_norm_grad(case, s):
    """By the chain rule: through the quotient, then through the variance and
    the mean; the statistics are those of the rows themselves."""
    D = case["D"]
    x, dy = s["x"].double(), s["dy"].double()
    var, mean = torch.var_mean(x, dim=1, unbiased=False, keepdim=True)
    rstd = torch.rsqrt(var + _EPS)
    out = {"dw": torch.einsum("nd,nd->d", dy, (x - mean) * rstd), "db": torch.einsum("nd->d", dy)}
    up = dy * s["w"].double()
    dvar = -0.5 * rstd ** 3 * torch.einsum("nd,nd->n", up, x - mean)[:, None]
    dc = up * rstd + 2.0 / D * dvar * (x - mean)
    out["dx"] = dc - torch.einsum("nd->n", dc)[:, None] / D
    if s["dres"] is not None:
        out["dx"] += s["dres"].double()
    return {k: out[k] for k in ("dx", "dw", "db")}


def _exact_act(name, z):
    f = torch.nn.functional
    if name == "gelu_sigmoid":
        return z * torch.sigmoid(1.702 * z)
    return {"relu": f.relu, "gelu_erf": f.gelu,
            "gelu_tanh": lambda v: f.gelu(v, approximate="tanh")}[name](z)


def _exact_linear(case, s):
    X = s["X"].double()
    if case["split"] == "column":
        z = torch.einsum("nd,df->nf", X, torch.cat([w.double() for w in s["W"]], dim=1))
        if s["b"] is not None:
            z += torch.cat([b.double() for b in s["b"]])
    else:
        z = torch.einsum("nf,fd->nd", X, torch.cat([w.double() for w in s["W"]], dim=0))
        if s["b"] is not None:
            z += s["b"].double()
    y = _exact_act(case["act"], z) if case["act"] else z.clone()
    if s["R"] is not None:
        y += s["R"].double()
    return {"Y": y, "Z": z} if case["save_z"] else {"Y": y}


def _exact_linear_grad(case, s):
    T, column = case["T"], case["split"] == "column"
    X, dZ = s["X"].double(), s["dY"].double()
    if case["act"]:
        z = s["Z"].double().requires_grad_()
        dZ, = torch.autograd.grad(_exact_act(case["act"], z), z, dZ)
    W = torch.cat([w.double() for w in s["W"]], dim=1 if column else 0)
    dW = torch.einsum("ni,no->io", X, dZ).chunk(T, dim=1 if column else 0)
    out = {"dX": torch.einsum("no,io->ni", dZ, W), "dW": list(dW)}
    if case["bias"]:
        db = torch.einsum("no->o", dZ)
        out["db"] = list(db.chunk(T)) if column else db
    return out


def _exact_policy(case, s):
    N, V, tau, beta = case["N"], case["V"], case["tau"], case["kl"]
    dev = s["logits"].device
    out = {k: torch.zeros(N, dtype=torch.float64, device=dev) for k in ("loss", "logprob", "kl")}
    d = torch.zeros((N, V), dtype=torch.float64, device=dev)
    step = max(1, (1 << 26) // V)
    for i in range(0, N, step):
        r = torch.arange(i, min(N, i + step), device=dev)
        r = r[s["targets"][r] >= 0]
        t = s["targets"][r]
        logp = torch.log_softmax(s["logits"][r].double() / tau, dim=1)
        at = torch.arange(r.numel(), device=dev)
        lp = logp[at, t]
        gone, adv = lp - s["old"][r].double(), s["adv"][r].double()
        ratio = torch.exp(gone)
        back = s["ref"][r].double() - lp
        out["logprob"][r] = lp
        out["kl"][r] = torch.expm1(back) - back
        out["loss"][r] = beta * (torch.expm1(back) - back) - torch.minimum(
            ratio * adv, ratio.clamp(1.0 - case["low"], 1.0 + case["high"]) * adv)
        stuck = ((adv > 0) & (ratio > 1.0 + case["high"])) | ((adv < 0) & (ratio < 1.0 - case["low"]))
        slope = -adv * ratio * ~stuck - beta * torch.expm1(back)
        if not case["fused"]:
            slope = slope * s["weights"][r].double()
        slope = slope / (tau * N)
        grad = torch.exp(logp)
        grad[at, t] = torch.zeros_like(lp)
        rest = grad.sum(dim=1)   # one minus the token's own probability
        grad *= -slope[:, None]
        grad[at, t] = slope * rest
        d[r] = grad
    return {"loss": out["loss"], "mean": out["loss"].mean().reshape(1), "logprob": out["logprob"],
            "kl": out["kl"], "dlogits": d}


_EXACT = {"norm": _exact_norm, "norm_grad": _exact_norm_grad, "linear": _exact_linear,
          "linear_grad": _exact_linear_grad, "policy": _exact_policy}
