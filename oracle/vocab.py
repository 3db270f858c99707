"""Vocabulary-side operators in float64: the plain definitions.

logprobs: lse_n = ln sum_v exp(z[n, v]); logprob_n = z[n, t_n] - lse_n; rank_n =
  1 + #{v: z_v > z_t} + #{v < t: z_v = z_t}; entropy_n = -sum_{p > 0} p ln p;
  the first K tokens by falling logit, equal logits by rising index.
distill: q = softmax over a row's live slots of teacher / tau, p = softmax(z / tau),
  loss_n = tau^2 sum_{q_k > 0} q_k (ln q_k - ln p_{id_k}),
  dloss_n / dz_v = tau (p_v - sum_{k: id_k = v} q_k).
  A row without a live slot (id -1 or teacher -inf everywhere) has loss and gradient 0.
embedding_backward: dE[v] = scale * sum_{n: ids[n] = v} dout[n]; ids outside [0, V) drop out.

-inf logits are masked tokens (p = 0); a row with nothing else has lse = -inf.
"""

import numpy as np

from .mlp import as_f64


def _ints(a):
    return np.asarray(a.cpu() if hasattr(a, "cpu") else a, dtype=np.int64)


def _lse(z):
    m = z.max()
    if m == -np.inf:
        return -np.inf
    return m + np.log(np.exp(z - m).sum())


def _ln_p(z):
    """ln p; relative to the maximum, since z - lse loses ln S where |z| is huge
    (rows masked by the type's lowest value)."""
    m = z.max()
    if m == -np.inf:
        return np.full_like(z, -np.inf)
    return (z - m) - np.log(np.exp(z - m).sum())


def logprobs(logits, targets, K):
    z_all, t_all = as_f64(logits), _ints(targets)
    N = z_all.shape[0]
    out = {"logprob": np.empty(N), "rank": np.empty(N, dtype=np.int64), "entropy": np.empty(N),
           "lse": np.empty(N), "top_ids": np.empty((N, K), dtype=np.int64),
           "top_logprobs": np.empty((N, K))}
    for n in range(N):
        z, t = z_all[n], t_all[n]
        lp = _ln_p(z)
        p = np.exp(lp)
        out["lse"][n] = _lse(z)
        out["entropy"][n] = -np.sum(p[p > 0] * lp[p > 0]) + 0.0
        if 0 <= t < z.size:
            out["logprob"][n] = lp[t]
            out["rank"][n] = 1 + np.sum(z > z[t]) + np.sum(z[:t] == z[t])
        else:
            out["logprob"][n], out["rank"][n] = np.nan, 0
        first = np.argsort(-z, kind="stable")[:K]
        out["top_ids"][n], out["top_logprobs"][n] = first, lp[first]
    return out


def _teacher(ids, teacher, tau):
    """(live slots, ln q over them) of one row; no slots if nothing is live."""
    live = np.flatnonzero((ids != -1) & (teacher != -np.inf))
    t = teacher[live] / tau
    return live, _ln_p(t) if live.size else t


def distill(logits, teacher_ids, teacher_logits, tau):
    z_all, ids, tl = as_f64(logits), _ints(teacher_ids), as_f64(teacher_logits)
    N = z_all.shape[0]
    loss, lse_out = np.zeros(N), np.zeros(N)
    for n in range(N):
        live, lnq = _teacher(ids[n], tl[n], tau)
        if live.size == 0:
            continue
        z = z_all[n] / tau
        lse_out[n] = _lse(z)
        lp = _ln_p(z)[ids[n][live]]
        q = np.exp(lnq)
        loss[n] = tau * tau * np.sum((q * (lnq - lp))[q > 0])
    return {"loss": loss, "lse": lse_out, "mean": loss.mean() if N else float("nan")}


def distill_backward(logits, teacher_ids, teacher_logits, tau, grad):
    """d(sum_n grad[n] loss[n]) / dlogits; grad is a number or one per token."""
    z_all, ids, tl = as_f64(logits), _ints(teacher_ids), as_f64(teacher_logits)
    N, V = z_all.shape
    g = np.broadcast_to(as_f64(grad), (N,))
    d = np.zeros((N, V))
    for n in range(N):
        live, lnq = _teacher(ids[n], tl[n], tau)
        if live.size == 0:
            continue
        z = z_all[n] / tau
        d[n] = np.exp(_ln_p(z))
        np.add.at(d[n], ids[n][live], -np.exp(lnq))
        d[n] *= g[n] * tau
    return d


def embedding_backward(ids, dout, V, scale):
    ids, dout = _ints(ids), as_f64(dout)
    d = np.zeros((V, dout.shape[1]))
    ok = (ids >= 0) & (ids < V)
    np.add.at(d, ids[ok], dout[ok])
    return scale * d


def _policy_row(z, t, old, adv, ref, kl, low, high, tau):
    """(loss, l, k, dloss / dl) of one token; ref None: no KL term."""
    l = _ln_p(z / tau)[t]
    with np.errstate(over="ignore", invalid="ignore"):
        rho = np.exp(l - old)
        loss = slope = 0.0
        if adv != 0:
            held = rho > 1 + high if adv > 0 else rho < 1 - low
            loss = -adv * ((1 + high if adv > 0 else 1 - low) if held else rho)
            slope = 0.0 if held else -adv * rho
        k = 0.0
        if ref is not None:
            r = ref - l
            k = np.inf if r == np.inf else np.expm1(r) - r
            if kl:
                loss += kl * k
                slope -= kl * np.expm1(r)
    return loss, l, k, slope


def policy(logits, targets, old, adv, ref, kl, low, high, tau):
    """Clipped policy loss with a KL term; see tpmlp_vocab_policy. A negative target
    is no token: zeros."""
    z_all, t_all, old, adv = as_f64(logits), _ints(targets), as_f64(old), as_f64(adv)
    ref = None if ref is None else as_f64(ref)
    N = z_all.shape[0]
    out = {k: np.zeros(N) for k in ("loss", "logprob", "kl")}
    for n in range(N):
        if t_all[n] >= 0:
            out["loss"][n], out["logprob"][n], out["kl"][n], _ = _policy_row(
                z_all[n], t_all[n], old[n], adv[n], None if ref is None else ref[n], kl, low, high, tau)
    out["mean"] = out["loss"].mean() if N else float("nan")
    return out


def policy_backward(logits, targets, old, adv, ref, kl, low, high, tau, grad):
    """d(sum_n grad[n] loss[n]) / dlogits; grad is a number or one per token."""
    z_all, t_all, old, adv = as_f64(logits), _ints(targets), as_f64(old), as_f64(adv)
    ref = None if ref is None else as_f64(ref)
    N, V = z_all.shape
    g = np.broadcast_to(as_f64(grad), (N,))
    d = np.zeros((N, V))
    for n in range(N):
        t = t_all[n]
        if t < 0:
            continue
        slope = _policy_row(z_all[n], t, old[n], adv[n], None if ref is None else ref[n], kl, low, high, tau)[3]
        w = g[n] * slope / tau
        if w == 0:
            continue
        p = np.exp(_ln_p(z_all[n] / tau))
        d[n] = -w * p
        p[t] = 0.0
        d[n, t] = w * p.sum()   # 1 - p_t, with its digits
    return d
