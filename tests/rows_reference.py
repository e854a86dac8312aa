"""Plain fp64 implementations of the operators on rows of logits (top logits, beam selection, distillation), for the
tests: numpy and torch on the CPU, row by row, no code of the product.

Tolerances.  The kernels sum a row's terms in fp32 per thread and in fp64 across threads.  With N columns per thread a
sum's relative error is at most SUM(V) = (N + 40) * 2^-24: N - 1 additions of half a step each, 2^-22 for an
exponential, and the rounding of its argument, 2^-24 of |argument| * ln 2 averaged over the row's distribution (at most
log2 V + 1 bits < 22).  N is at most ceil(V / 512) + 32 at every launch shape (512 threads or more share a row, each
in pieces of at most 32 columns).  An fp32 result adds half a step, 2^-24 of its value; bf16 2^-9 ... 2^-8."""
import math

import numpy as np
import torch

BIG = 1e6


def sum_tol(V: int) -> float:
    return (math.ceil(V / 512) + 72) * 2.0 ** -24


def clean(z):
    """fp64 logits with barred tokens at -inf and magnitudes as the operators take them."""
    z = np.asarray(z, dtype=np.float64)
    return np.where(np.isnan(z) | (z == -np.inf), -np.inf, np.clip(z, -BIG, BIG))


def lse_rows(z, T):
    x = clean(z) / T
    m = x.max(-1, keepdims=True)
    m0 = np.where(np.isfinite(m), m, 0.0)
    with np.errstate(divide="ignore"):
        return (m0 + np.log(np.exp(x - m0).sum(-1, keepdims=True)))[..., 0]


def top(z, k):
    """values, ids of the k largest of each row of z [R, V], the lower column first among equals."""
    z = np.asarray(z, dtype=np.float64)
    R, V = z.shape
    vals, ids = np.full((R, k), -np.inf), np.full((R, k), -1, np.int32)
    for r in range(R):
        key = np.where(np.isnan(z[r]), -np.inf, z[r]) + 0.0
        order = np.argsort(-key, kind="stable")
        order = order[key[order] > -np.inf][:k]
        vals[r, :len(order)], ids[r, :len(order)] = key[order], order
    return vals, ids


def beam(z, scores, n, states=None, history=None, pos=0, finished=None, eos=-1):
    """One selection step over z [B, W, V]; dict of fp64 / int arrays."""
    z, scores = np.asarray(z, np.float64), np.asarray(scores, np.float64)
    B, W, V = z.shape
    out = {"scores": np.full((B, n), -np.inf), "parents": np.zeros((B, n), np.int32),
           "tokens": np.zeros((B, n), np.int32), "finished": np.zeros((B, n), np.uint8)}
    lse = lse_rows(z, 1.0)
    c = clean(z)
    vals, ids = top(z.reshape(B * W, V), min(n, V))
    ids = ids.reshape(B, W, -1)
    for b in range(B):
        cand = []
        for w in range(W):
            if not scores[b, w] > -np.inf:
                continue
            if finished is not None and finished[b, w]:
                cand.append((scores[b, w], w, eos))
                continue
            for v in ids[b, w]:
                if v >= 0:
                    cand.append((scores[b, w] + (c[b, w, v] - lse[b, w]), w, int(v)))
        cand.sort(key=lambda t: -t[0])  # stable: beam, then the order within the beam
        for j, (s, w, v) in enumerate(cand[:n]):
            out["scores"][b, j], out["parents"][b, j], out["tokens"][b, j] = s, w, v
            out["finished"][b, j] = bool(finished is not None and finished[b, w]) or (eos >= 0 and v == eos)
    at = out["parents"]
    if states is not None:
        out["states"] = np.stack([np.asarray(states)[b][at[b]] for b in range(B)])
    if history is not None:
        out["history"] = np.stack([np.asarray(history)[b][at[b]] for b in range(B)])
        out["history"][:, :, pos] = out["tokens"]
    return out


def distill_row(z, ids, tops, lse_t, T, w):
    """Loss and gradient of one row (fp64 numpy); also the sum of magnitudes that its gradient is a difference of."""
    z = clean(z)
    V = len(z)
    zero = 0.0, np.zeros(V), np.zeros(V)
    if w == 0.0 or not (z > -np.inf).any() or (lse_t is not None and not np.isfinite(lse_t)):
        return zero
    ok = (ids >= 0) & (ids < V)
    ids, y = ids[ok], clean(tops[ok]) / T
    if lse_t is None:
        if not (y > -np.inf).any():
            return zero
        p = np.exp(y - y.max())
        p = p / p.sum()
    else:
        p = np.exp(y - lse_t)
    if not p.sum() > 0:
        return zero
    x = z / T
    lse = lse_rows(z[None], T)[0]
    q = np.exp(x - lse)
    outside = np.ones(V, bool)
    outside[ids] = False
    tau = q[outside].sum()
    rho = max(0.0, 1.0 - p.sum()) if lse_t is not None and tau > 0 else 0.0
    pos = p > 0
    loss = float((p[pos] * (np.log(p[pos]) - (x[ids[pos]] - lse))).sum())
    if rho > 0:
        loss += rho * (math.log(rho) - math.log(tau))
    P = p.sum() + rho
    pv = np.zeros(V)
    np.add.at(pv, ids, p)
    rest = outside * q * (rho / tau if rho > 0 else 0.0)
    return w * loss, w / T * (P * q - rest - pv), abs(w) / T * (P * q + rest + pv)


def distill(z, ids, tops, lse_t, T, weights):
    """Rows of distill_row: loss [R], grad [R, V], scale [R, V]."""
    R = len(z)
    rows = [distill_row(np.asarray(z[r], np.float64), np.asarray(ids[r]), np.asarray(tops[r], np.float64),
                        None if lse_t is None else float(lse_t[r]), T,
                        1.0 if weights is None else float(weights[r])) for r in range(R)]
    return (np.array([r[0] for r in rows]), np.stack([r[1] for r in rows]), np.stack([r[2] for r in rows]))


def padded(t, extra=0, fill=float("nan"), device="cuda"):
    """t [..., V] as a view of rows `extra` vectors of 8 longer than V rounded up, the rest filled."""
    V = t.shape[-1]
    ld = (V + 7) // 8 * 8 + 8 * extra
    full = torch.full(t.shape[:-1] + (ld,), fill, dtype=t.dtype, device=device)
    full[..., :V] = t.to(device)
    return full[..., :V]
