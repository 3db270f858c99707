"""The operators of a language model's vocabulary side and its gated block, as
measured cases: one pass through each operator, its plain form in elementary
torch operations and its value in 64 bits.

Operators (T is the number of logical vocabulary or column shards):

  logprobs     log probabilities of given tokens, their rank, the entropy of
               the distribution and its K most likely tokens
  distill      distillation from a teacher's top K tokens: loss and gradient,
               in one call ("fused") or as a loss call and a gradient call
  embed        embedding rows times a factor
  embed_grad   its other direction: the table's gradient, by sorted tokens
  gated_grad   gradients of Y = sum_r (SiLU(X Wg^r) * (X Wu^r)) Wd^r
"""

import math

import numpy as np
import torch

own = False   # true: `run` calls the package's operators

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f32": 4}
_NEG = float("-inf")


def _pkg():
    import tensor_transformer_mlp_columnparallel_gb300 as tp
    return tp


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one decoding step of one request that asks for its tokens' log
        # probabilities: launch latency
        dict(name="logprobs_n1", op="logprobs", dt="f32", N=1, V=32000, T=4, K=1, pad=0, masked=0.0),
        # one decoding step of a batch, twenty alternatives, a quarter of the
        # requests held to a grammar by a mask
        dict(name="logprobs_n48", op="logprobs", dt="bf16", N=48, V=128000, T=8, K=20, pad=0,
             masked=0.25),
        # scoring a batch of prompts
        dict(name="logprobs_n2048", op="logprobs", dt="bf16", N=2048, V=128000, T=8, K=5, pad=0,
             masked=0.0),
        # a training step's tokens, padding among them, loss and gradient together
        dict(name="distill_n4096", op="distill", dt="bf16", N=4096, V=128000, T=8, K=64, pad=0,
             fused=True, tau=2.0, empty=0.1),
        # fp32 logits of an odd vocabulary in padded rows; the gradient is
        # asked for later, with weights per token
        dict(name="distill_odd_f32", op="distill", dt="f32", N=1003, V=50001, T=7, K=33, pad=15,
             fused=False, tau=1.5, empty=0.05),
        # the tokens of one decoding step
        dict(name="embed_n5", op="embed", dt="f32", N=5, V=32000, H=4096, T=4, scale=64.0),
        # embedding a long prompt
        dict(name="embed_n8192", op="embed", dt="bf16", N=8192, V=32000, H=8192, T=4, scale=90.5),
        # the embedding's gradient of a training step, fp32 table gradient
        dict(name="embed_grad_n8192", op="embed_grad", dt="bf16", grad="f32", N=8192, V=128000,
             H=4096, T=8, scale=64.0, spread="zipf"),
        # odd sizes, a padding token that most positions hold
        dict(name="embed_grad_odd", op="embed_grad", dt="f32", grad="f32", N=4099, V=9999, H=1030,
             T=3, scale=1.0, spread="pad"),
        # gradient of a few tokens' block: the weights' reads and writes bound it
        dict(name="gated_grad_n16", op="gated_grad", dt="bf16", N=16, D=4096, F=16384, T=4),
        # a training step's block
        dict(name="gated_grad_n4096", op="gated_grad", dt="bf16", N=4096, D=4096, F=16384, T=4),
        # the exact-fp32 block
        dict(name="gated_grad_f32", op="gated_grad", dt="f32", N=64, D=256, F=1024, T=2),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["logprobs", "distill", "embed", "embed_grad", "gated_grad"])
    dt = rng.choice(["bf16", "f32"])
    T = rng.choice([1, 2, 3, 4, 7, 8, 16])
    if op in ("logprobs", "distill"):
        Vs = _log_int(rng, 1000, 128000) // T
        V = max(Vs, 1) * T
        top = (2048 if op == "logprobs" else 4096) * 128000 * 2 // _SIZE[dt]
        N = _log_int(rng, 1, max(1, min(4096, top // V)))
        pad = rng.choice([0, 0, rng.randint(1, 64)])
        if op == "logprobs":
            return dict(op=op, dt=dt, N=N, V=V, T=T, K=rng.choice([0, 1, 5, 20, rng.randint(1, 64)]),
                        pad=pad, masked=rng.choice([0.0, 0.0, 0.25]))
        return dict(op=op, dt=dt, N=N, V=V, T=T, K=_log_int(rng, 1, 128), pad=pad,
                    fused=rng.choice([True, True, False]), tau=rng.choice([1.0, 1.5, 2.0, 4.0]),
                    empty=rng.choice([0.0, 0.1, 0.3]))
    if op in ("embed", "embed_grad"):
        V = max(1, _log_int(rng, 1000, 128000) // T) * T
        H = _log_int(rng, 64, 8192)
        if rng.random() < 0.7:
            H = (H + 7) // 8 * 8
        H = min(H, (128000 * 4096) // V)
        grad = dt if rng.random() < 0.5 else "f32"
        # bounded by the listed cases' work: the token rows and the table
        tokens = max(1, min(8192, 8192 * (8192 if op == "embed" else 4096) * 2 // (H * _SIZE[dt])))
        N = _log_int(rng, 1, tokens)
        case = dict(op=op, dt=dt, N=N, V=V, H=H, T=T, scale=rng.choice([1.0, math.sqrt(H)]))
        if op == "embed_grad":
            case.update(grad=grad, spread=rng.choice(["zipf", "zipf", "pad", "flat"]))
        return case
    if dt == "f32":
        T = rng.choice([1, 2, 3])
        return dict(op=op, dt=dt, N=_log_int(rng, 1, 64), D=_log_int(rng, 16, 256),
                    F=T * max(1, _log_int(rng, 32, 1024) // T), T=T)
    T = rng.choice([1, 2, 4, 8])
    D = 8 * _log_int(rng, 32, 512)
    F = 8 * T * max(1, _log_int(rng, 128, 2048) // T)
    return dict(op=op, dt=dt, N=_log_int(rng, 1, 4096), D=D, F=F, T=T)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _rows(g, N, V, pad, dt, std, dev):
    """[N, V] logits, in rows of V + pad elements."""
    z = torch.empty((N, V + pad), dtype=_TYPES[dt], device=dev)
    step = max(1, (1 << 27) // (V + pad))
    for i in range(0, N, step):
        n = min(step, N - i)
        z[i:i + n] = (torch.randn((n, V + pad), generator=g, device=dev) * std).to(z.dtype)
    return z[:, :V]


def _token_ids(g, N, V, spread, dev):
    """Token ids: word frequencies falling as 1 / rank ("zipf"), the same
    with four positions of five holding one padding token ("pad"), or every
    token alike ("flat")."""
    u = torch.rand(N, generator=g, device=dev, dtype=torch.float64)
    if spread == "flat":
        return (u * V).long().clamp_(max=V - 1)
    rank = (torch.exp(u * math.log(V + 1.0)) - 1.0).long().clamp_(max=V - 1)
    ids = (rank * 7919 + 11) % V if V % 7919 else rank
    if spread == "pad":
        keep = torch.rand(N, generator=g, device=dev) < 0.2
        ids = torch.where(keep, ids, torch.full_like(ids, min(2, V - 1)))
    return ids


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed) + 1)
    op, N, T = case["op"], case["N"], case["T"]
    dt = _TYPES[case["dt"]]
    s = {"case": case}
    if op in ("logprobs", "distill"):
        V, K = case["V"], case["K"]
        s["logits"] = _rows(g, N, V, case["pad"], case["dt"], 2.0, dev)
    if op == "logprobs":
        t = torch.randint(0, V, (N,), generator=g, device=dev)
        held = torch.nonzero(torch.rand(N, generator=g, device=dev) < case["masked"]).flatten().tolist()
        for n in held:   # a grammar leaves about one token in 200, the given one among them
            drop = torch.rand(V, generator=g, device=dev) > 0.005
            drop[t[n]] = False
            s["logits"][n].masked_fill_(drop, _NEG)
        s["targets"] = t
    elif op == "distill":
        # the teacher's K tokens, distinct in a row, its logits in falling order
        first = torch.randint(0, V, (N, 1), generator=g, device=dev)
        step = torch.randint(1, max(2, V // K), (N, 1), generator=g, device=dev)
        ids = (first + step * torch.arange(K, device=dev)) % V
        s["ids"] = ids.to(torch.int32)
        s["teacher"] = (torch.randn((N, K), generator=g, device=dev) * 2.0 + 6.0).sort(
            dim=1, descending=True).values.contiguous()
        none = torch.rand(N, generator=g, device=dev) < case["empty"]   # padding positions
        s["ids"][none] = -1
        short = torch.rand(N, generator=g, device=dev) < 0.1            # a shorter list
        if K > 2:
            s["ids"][short, K // 2:] = -1
        s["weights"] = torch.rand(N, generator=g, device=dev) + 0.5
    elif op in ("embed", "embed_grad"):
        V, H = case["V"], case["H"]
        s["ids"] = _token_ids(g, N, V, case.get("spread", "zipf"), dev)
        if op == "embed":
            s["table"] = [(torch.randn((V // T, H), generator=g, device=dev) * 0.02).to(dt)
                          for _ in range(T)]
        else:
            s["dout"] = torch.randn((N, H), generator=g, device=dev).to(dt)
    else:
        D, Fs = case["D"], case["F"] // T

        def normal(r, c, std):
            return (torch.randn((r, c), generator=g, device=dev) * std).to(dt)

        s["X"], s["dY"] = normal(N, D, 1.0), normal(N, D, 1.0)
        s["Wg"] = [normal(D, Fs, 0.02) for _ in range(T)]
        s["Wu"] = [normal(D, Fs, 0.02) for _ in range(T)]
        s["Wd"] = [normal(Fs, D, 0.02) for _ in range(T)]
        std = 0.02 * math.sqrt(D)
        s["G"] = [normal(N, Fs, std) for _ in range(T)]
        s["U"] = [normal(N, Fs, std) for _ in range(T)]
        s["H"] = [(a.float() / (1.0 + torch.exp(-a.float())) * b.float()).to(dt)
                  for a, b in zip(s["G"], s["U"])]
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    return _PLAIN[op](state)


def _own_logprobs(s):
    c = s["case"]
    lp, rank, ent, ids, top = _pkg().vocab_logprobs(s["logits"], s["targets"], c["T"], top_k=c["K"])
    return {"logprob": lp, "rank": rank, "entropy": ent, "top_ids": ids, "top_logprobs": top}


def _own_distill(s):
    c, tp = s["case"], _pkg()
    z, ids, t, T, tau, N = s["logits"], s["ids"], s["teacher"], c["T"], c["tau"], c["N"]
    if c["fused"]:
        loss, mean, _, d = tp.vocab_distill_with_grad(z, ids, t, T, temperature=tau, grad_scale=1.0 / N)
    else:
        loss, mean, lse = tp.vocab_distill(z, ids, t, T, temperature=tau)
        d = tp.vocab_distill_backward(z, ids, t, T, lse, temperature=tau, grad_scale=1.0 / N,
                                      grad_tokens=s["weights"])
    return {"loss": loss, "mean": mean, "dlogits": d}


def _own_embed(s):
    return _pkg().vocab_embedding_scaled(s["ids"], s["table"], s["case"]["scale"])


def _own_embed_grad(s):
    c = s["case"]
    return _pkg().vocab_embedding_backward(s["ids"], s["dout"], c["V"], c["T"], scale=c["scale"],
                                           grad_dtype=_TYPES[c["grad"]])


def _own_gated(s):
    dX, dWg, dWu, dWd = _pkg().swiglu_backward(s["X"], s["Wg"], s["Wu"], s["Wd"], s["H"], s["G"],
                                               s["U"], s["dY"])
    return {"dX": dX, "dWg": dWg, "dWu": dWu, "dWd": dWd}


def _plain_logprobs(s):
    z, t, K = s["logits"].float(), s["targets"], s["case"]["K"]
    V = z.shape[1]
    m = z.amax(dim=1, keepdim=True)
    lse = m + torch.log(torch.exp(z - m).sum(dim=1, keepdim=True))
    lp = z - lse
    zero = torch.zeros((), device=z.device)
    entropy = -torch.where(lp == _NEG, zero, torch.exp(lp) * lp).sum(dim=1)
    zt = z.gather(1, t[:, None])
    col = torch.arange(V, device=z.device)
    rank = 1 + (z > zt).sum(dim=1) + ((z == zt) & (col < t[:, None])).sum(dim=1)
    # one whole number per entry that falls with the logit, then rises with the index
    bits = (z + 0.0).view(torch.int32)
    order = torch.where(bits >= 0, bits, bits ^ 0x7fffffff).long() * (1 << 32) + ((1 << 32) - 1 - col)
    ids = torch.topk(order, K, dim=1).indices
    return {"logprob": lp.gather(1, t[:, None])[:, 0], "rank": rank.to(torch.int32),
            "entropy": entropy, "top_ids": ids.to(torch.int32), "top_logprobs": lp.gather(1, ids)}


def _plain_distill(s):
    c = s["case"]
    tau, N = c["tau"], c["N"]
    z = s["logits"].float() / tau
    live = s["ids"] >= 0
    ids = s["ids"].long().clamp(min=0)
    some = live.any(dim=1)
    t = torch.where(live, s["teacher"] / tau, torch.full_like(s["teacher"], _NEG))
    tm = torch.where(some[:, None], t.amax(dim=1, keepdim=True), torch.zeros_like(t[:, :1]))
    e = torch.exp(t - tm)
    total = e.sum(dim=1, keepdim=True)
    q = torch.where(live, e / total, torch.zeros_like(e))
    logq = t - tm - torch.log(total)
    m = z.amax(dim=1, keepdim=True)
    ez = torch.exp(z - m)
    sz = ez.sum(dim=1, keepdim=True)
    logp = z.gather(1, ids) - m - torch.log(sz)
    zero = torch.zeros_like(q)
    loss = tau * tau * torch.where(q > 0, q * (logq - logp), zero).sum(dim=1)
    w = torch.full((N,), 1.0 / N, device=z.device)
    if not c["fused"]:
        w = w * s["weights"]
    w = torch.where(some, w * tau, torch.zeros_like(w))[:, None]
    d = ez / sz * w
    d.scatter_add_(1, ids, -q * w)
    return {"loss": loss, "mean": loss.sum().reshape(1) / N, "dlogits": d.to(s["logits"].dtype)}


def _plain_embed(s):
    ids, T = s["ids"], s["case"]["T"]
    out = None
    Vs = s["table"][0].shape[0]
    for k in range(T):   # each shard's rows, zeros for other shards' tokens
        mine = (ids >= k * Vs) & (ids < (k + 1) * Vs)
        rows = s["table"][k][(ids - k * Vs).clamp(0, Vs - 1)].float()
        rows = torch.where(mine[:, None], rows, torch.zeros((), device=rows.device))
        out = rows if out is None else out + rows
    return (out * s["case"]["scale"]).to(s["table"][0].dtype)


def _plain_embed_grad(s):
    c = s["case"]
    order = torch.argsort(s["ids"], stable=True)
    d = torch.zeros((c["V"], c["H"]), dtype=torch.float32, device=s["dout"].device)
    d.index_add_(0, s["ids"][order], s["dout"][order].float())
    d = (d * c["scale"]).to(_TYPES[c["grad"]])
    return [x.contiguous() for x in d.chunk(c["T"], dim=0)]


def _plain_gated(s):
    dt = s["X"].dtype
    X, dY = s["X"].float(), s["dY"].float()
    dX = torch.zeros_like(X)
    out = {"dX": None, "dWg": [], "dWu": [], "dWd": []}
    for Wg, Wu, Wd, H, G, U in zip(s["Wg"], s["Wu"], s["Wd"], s["H"], s["G"], s["U"]):
        G, U = G.float(), U.float()
        dH = dY @ Wd.float().t()
        sg = 1.0 / (1.0 + torch.exp(-G))
        dU = dH * (G * sg)
        dG = dH * U * (sg * (1.0 + G * (1.0 - sg)))
        out["dWd"].append((H.float().t() @ dY).to(dt))
        out["dWg"].append((X.t() @ dG).to(dt))
        out["dWu"].append((X.t() @ dU).to(dt))
        dX = dX + dG @ Wg.float().t() + dU @ Wu.float().t()
    out["dX"] = dX.to(dt)
    return out


_OWN = {"logprobs": _own_logprobs, "distill": _own_distill, "embed": _own_embed,
        "embed_grad": _own_embed_grad, "gated_grad": _own_gated}
_PLAIN = {"logprobs": _plain_logprobs, "distill": _plain_distill, "embed": _plain_embed,
          "embed_grad": _plain_embed_grad, "gated_grad": _plain_gated}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def _different(N, V, spread):
    """Expected number of different ids among N (see _token_ids)."""
    r = np.arange(V, dtype=np.float64)
    if spread == "flat":
        p = np.full(V, 1.0 / V)
    else:
        p = np.log((r + 2.0) / (r + 1.0)) / math.log(V + 1.0)
        if spread == "pad":
            p = p * 0.2
    return float(np.sum(-np.expm1(N * np.log1p(-p))))


def work(case):
    op, N = case["op"], case["N"]
    es = _SIZE[case["dt"]]
    if op == "logprobs":
        V, K = case["V"], case["K"]
        # subtract, exp, add; multiply and add for the entropy
        return {"bytes": N * V * es + N * 8 + N * (12 + 8 * K), "flops": 5.0 * N * V}
    if op == "distill":
        V, K = case["V"], case["K"]
        read = (1.0 - case["empty"]) * N * V * es
        return {"bytes": read + N * V * es + N * K * 8 + N * 4 + 4 + (0 if case["fused"] else 4 * N),
                "flops": 6.0 * N * V}
    if op == "embed":
        H = case["H"]
        rows = _different(N, case["V"], "zipf")
        return {"bytes": rows * H * es + N * H * es + 8 * N, "flops": 1.0 * N * H}
    if op == "embed_grad":
        H = case["H"]
        return {"bytes": N * H * es + 8 * N + case["V"] * H * _SIZE[case["grad"]],
                "flops": 1.0 * N * H}
    D, F = case["D"], case["F"]
    # X, dY, dX; H, G, U; the three weights and their gradients
    return {"bytes": es * (3.0 * N * D + 3.0 * N * F + 6.0 * D * F), "flops": 12.0 * N * D * F}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    if case["op"] == "gated_grad" and 12.0 * case["N"] * case["D"] * case["F"] > 6e12:
        return None
    return _EXACT[case["op"]](case, prepare(case, seed))


def _exact_logprobs(case, s):
    K = case["K"]
    out = {"logprob": [], "rank": [], "entropy": [], "top_ids": [], "top_logprobs": []}
    for row, t in zip(s["logits"], s["targets"].tolist()):
        z = row.double()
        lse = torch.logsumexp(z, dim=0)
        lp = z - lse
        out["logprob"].append(lp[t])
        out["entropy"].append(-(torch.special.xlogy(torch.exp(lp), torch.exp(lp))).sum())
        out["rank"].append((z > z[t]).sum() + (z[:t] == z[t]).sum() + 1)
        if K:
            first = torch.sort(z, descending=True, stable=True).indices[:K]
            out["top_ids"].append(first)
            out["top_logprobs"].append(lp[first])
    dev = s["logits"].device
    res = {k: torch.stack(v) if v else torch.zeros((case["N"], 0), dtype=torch.float64, device=dev)
           for k, v in out.items()}
    res["rank"] = res["rank"].to(torch.int32)
    res["top_ids"] = res["top_ids"].to(torch.int32)
    return res


def _exact_distill(case, s):
    N, V, tau = case["N"], case["V"], case["tau"]
    dev = s["logits"].device
    loss = torch.zeros(N, dtype=torch.float64, device=dev)
    d = torch.zeros((N, V), dtype=torch.float64, device=dev)
    up = torch.full((N,), 1.0 / N, dtype=torch.float64, device=dev)
    if not case["fused"]:
        up = up * s["weights"].double()
    step = max(1, (1 << 26) // V)
    for i in range(0, N, step):
        r = slice(i, min(N, i + step))
        ids = s["ids"][r].long()
        live = ids >= 0
        row, slot = torch.nonzero(live, as_tuple=True)
        teacher = s["teacher"][r].double() / tau
        teacher = teacher.masked_fill(~live, _NEG)
        some = live.any(dim=1)
        logq = torch.log_softmax(teacher.masked_fill(~some[:, None], 0.0), dim=1)
        logp = torch.log_softmax(s["logits"][r].double() / tau, dim=1)
        q = torch.exp(logq[row, slot])
        term = q * (logq[row, slot] - logp[row, ids[row, slot]])
        loss[r] = torch.zeros(logp.shape[0], dtype=torch.float64, device=dev).index_add_(0, row, term)
        grad = torch.exp(logp)
        grad.index_put_((row, ids[row, slot]), -q, accumulate=True)
        d[r] = grad * (up[r] * some * tau)[:, None]
    loss *= tau * tau
    return {"loss": loss, "mean": loss.mean().reshape(1), "dlogits": d}


def _exact_embed(case, s):
    whole = torch.cat(s["table"], dim=0)
    return torch.stack([whole[i].double() for i in s["ids"].tolist()]) * case["scale"]


def _exact_embed_grad(case, s):
    d = torch.zeros((case["V"], case["H"]), dtype=torch.float64, device=s["dout"].device)
    for a in range(0, case["H"], 512):   # one-hot times rows, a column block at a time
        d[:, a:a + 512].index_put_((s["ids"],), s["dout"][:, a:a + 512].double(), accumulate=True)
    return list((d * case["scale"]).chunk(case["T"], dim=0))


def _exact_gated(case, s):
    """By the chain rule in 64 bits, the shards side by side."""
    def wide(ts, dim):
        return torch.cat([t.double() for t in ts], dim=dim)

    X, dY = s["X"].double(), s["dY"].double()
    G, U, H = wide(s["G"], 1), wide(s["U"], 1), wide(s["H"], 1)
    dH = torch.einsum("nd,fd->nf", dY, wide(s["Wd"], 0))
    sig = torch.sigmoid(G)
    dU = dH * G * sig
    dG = dH * U * (sig + G * sig * (1.0 - sig))
    T = case["T"]
    return {"dX": torch.einsum("nf,df->nd", dG, wide(s["Wg"], 1))
                  + torch.einsum("nf,df->nd", dU, wide(s["Wu"], 1)),
            "dWg": list(torch.einsum("nd,nf->df", X, dG).chunk(T, dim=1)),
            "dWu": list(torch.einsum("nd,nf->df", X, dU).chunk(T, dim=1)),
            "dWd": list(torch.einsum("nf,nd->fd", H, dY).chunk(T, dim=0))}


_EXACT = {"logprobs": _exact_logprobs, "distill": _exact_distill, "embed": _exact_embed,
          "embed_grad": _exact_embed_grad, "gated_grad": _exact_gated}
