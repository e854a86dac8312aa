"""Cases of the vocabulary-row operators: the top logits of every row, one beam selection step, and the distillation
loss against a teacher's top logits with its gradient.

``run`` computes a case in elementary torch operations, or, with ``own`` set, by the calls a user makes of
:mod:`draft_block_causal_b200.domino`.  Logits are [B, L, V] (beam selection: [B, W, V]), fp32 or bf16; a vocabulary
that is no multiple of 8 lies in rows padded to one.
"""
import math

import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}
NINF = float("-inf")


def listed():
    return [
        # the teacher's next-token row of one sequence: latency counts
        dict(name="top-one-row", op="top", B=1, L=1, V=151936, k=8, dtype="fp32", temperature=1.0, masked=False),
        # what a distillation run stores of the target's logits: 32 blocks of 16 positions
        dict(name="top-32-blocks", op="top", B=32, L=16, V=151936, k=64, dtype="fp32", temperature=1.0, masked=False),
        # a smaller vocabulary of odd size with barred tokens, logits in bf16 (many exact ties)
        dict(name="top-odd-bf16", op="top", B=11, L=7, V=32003, k=20, dtype="bf16", temperature=2.0, masked=True),
        # one sequence drafting four beams: latency counts
        dict(name="beam-one-by-4", op="beam", B=1, W=4, beams=4, V=151936, dtype="fp32", Hs=1024, L=16, pos=5,
             ended=False, masked=False),
        # a serving batch in the middle of its blocks
        dict(name="beam-32-by-8", op="beam", B=32, W=8, beams=8, V=151936, dtype="fp32", Hs=1024, L=16, pos=9,
             ended=False, masked=False),
        # the first position of a block: one row opens eight beams
        dict(name="beam-open-128", op="beam", B=128, W=1, beams=8, V=151936, dtype="bf16", Hs=1024, L=16, pos=0,
             ended=False, masked=False),
        # odd everything: ended and dead beams, barred tokens, fewer beams than before
        dict(name="beam-odd", op="beam", B=5, W=7, beams=3, V=20011, dtype="bf16", Hs=264, L=13, pos=12,
             ended=True, masked=True),
        # one block's training step (loss and gradient in one call): latency counts
        dict(name="distill-one-block", op="distill", call="step", B=1, L=16, V=151936, K=16, dtype="bf16", tail=False,
             temperature=1.0, padded=False, masked=False),
        # a training batch with bf16 logits, the rest of the vocabulary as one class
        dict(name="distill-64-blocks", op="distill", call="step", B=64, L=16, V=151936, K=64, dtype="bf16", tail=True,
             temperature=1.0, padded=True, masked=False),
        # fp32 logits at a raised temperature
        dict(name="distill-fp32", op="distill", call="step", B=20, L=16, V=151936, K=32, dtype="fp32", tail=True,
             temperature=2.0, padded=False, masked=True),
        # an evaluation pass: the loss alone
        dict(name="distill-eval", op="distill", call="eval", B=32, L=16, V=151936, K=64, dtype="fp32", tail=True,
             temperature=1.0, padded=True, masked=False),
        # a step through autograd, an upstream gradient for every position, an odd vocabulary
        dict(name="distill-autograd", op="distill", call="train", B=24, L=15, V=50001, K=21, dtype="bf16", tail=True,
             temperature=1.5, padded=True, masked=True),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    V = _spread(rng, 1000, 262144)
    if rng.random() < 0.5:
        V -= V % 8
    dtype = rng.choice(["fp32", "bf16"])
    most = (64 << 20) // V  # rows
    op = rng.choice(["top", "beam", "distill", "distill"])
    if op == "beam":
        W, beams = rng.choice([1, 2, 3, 4, 5, 8, 12, 16]), rng.choice([1, 2, 3, 4, 6, 8, 16])
        B = _spread(rng, 1, max(1, min(256, most // W)))
        L = rng.randint(2, 24)
        return dict(op=op, B=B, W=W, beams=beams, V=V, dtype=dtype, Hs=8 * rng.randint(1, 160), L=L,
                    pos=rng.randrange(L), ended=rng.random() < 0.5, masked=rng.random() < 0.5)
    L = rng.randint(1, 24)
    B = _spread(rng, 1, max(1, min(256, most // L)))
    T = rng.choice([0.5, 1.0, 1.0, 1.7, 3.0])
    if op == "top":
        return dict(op=op, B=B, L=L, V=V, k=_spread(rng, 1, 128), dtype=dtype, temperature=T,
                    masked=rng.random() < 0.5)
    return dict(op=op, call=rng.choice(["step", "step", "eval", "train"]), B=B, L=L, V=V, K=_spread(rng, 1, 128),
                dtype=dtype, tail=rng.random() < 0.6, temperature=T, padded=rng.random() < 0.5,
                masked=rng.random() < 0.5)


def _rows(case):
    return case["B"] * (case["W"] if case["op"] == "beam" else case["L"])


def work(case):
    R, V = _rows(case), case["V"]
    es = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "top":
        return {"bytes": R * V * es + R * (8 * case["k"] + 4), "flops": 4 * R * V}
    if case["op"] == "beam":
        B, W, n = case["B"], case["W"], case["beams"]
        if case["ended"]:  # beams that ended or died are not read (see _beam_flags)
            ended, dead = _beam_flags(case)
            R = B * W - int((ended | dead).sum())
        moved = (W if n >= W else n) * B * (4 * case["Hs"] + 4 * case["L"]) + B * n * (4 * case["Hs"] + 4 * case["L"])
        return {"bytes": R * V * es + moved + B * W * 8 + B * n * 16, "flops": 4 * R * V}
    live = R - _padded_rows(case)
    small = R * (12 * case["K"] + 16)
    if case["call"] == "eval":
        return {"bytes": live * V * es + small, "flops": 4 * live * V}
    return {"bytes": (live + R) * V * es + small, "flops": 8 * live * V}


def _padded_rows(case):
    """Positions behind a block's end, whose weight is zero: the last quarter of every second block."""
    return (case["B"] // 2) * (case["L"] // 4) if case["padded"] else 0


def _beam_flags(case):
    """Which beams have ended and which are dead, [B, W] each: every fifth, and every seventh but no first one."""
    i = torch.arange(case["B"] * case["W"]).view(case["B"], case["W"])
    return i % 5 == 3, (i % 7 == 6) & (i % case["W"] != 0) & (i % 5 != 3)


def _padded(x):
    """x [..., V] as a view of rows padded to a multiple of 8 values."""
    V = x.shape[-1]
    if V % 8 == 0:
        return x
    y = torch.zeros(x.shape[:-1] + ((V + 7) // 8 * 8,), dtype=x.dtype, device=x.device)
    y[..., :V] = x
    return y[..., :V]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")
    rand = lambda *s: torch.rand(*s, generator=g, device="cuda")
    randint = lambda hi, *s: torch.randint(hi, s, generator=g, device="cuda")
    B, V = case["B"], case["V"]
    n = case["W"] if case["op"] == "beam" else case["L"]
    z = randn(B, n, V).mul_(2.5)
    # a few likely tokens in every row
    z.scatter_add_(2, randint(V, B, n, 6), 3.0 + 6.0 * rand(B, n, 6))
    barred = randint(V, max(1, V // 10)) if case["masked"] else None
    st = {"case": case}
    if case["op"] == "distill":
        K, T = min(case["K"], V), case["temperature"]
        t = z + randn(B, n, V).mul_(0.7)
        if barred is not None:
            t[..., barred] = NINF
        top, ids = torch.topk(t, K, dim=-1)
        st["top_logits"], st["top_ids"] = top.contiguous(), ids.int().contiguous()
        st["teacher_lse"] = torch.logsumexp(t / T, -1) if case["tail"] else None
        del t, top, ids
        w = 0.5 + rand(B, n)
        if case["padded"]:
            w[1::2, n - n // 4:] = 0.0
        st["row_weights"] = w
        st["upstream"] = 0.1 + rand(B, n)
    if barred is not None:
        z[..., barred] = NINF
    st["logits"] = _padded(z.to(DTYPES[case["dtype"]]))
    if case["op"] == "beam":
        W, L = n, case["L"]
        scores = -30.0 * rand(B, W) - 1.0
        st["states"], st["history"] = randn(B, W, case["Hs"]).mul_(0.3), randint(V, B, W, L).int()
        st["finished"] = None
        if case["ended"]:
            ended, dead = (x.cuda() for x in _beam_flags(case))
            scores = scores.masked_fill(dead, NINF)
            st["finished"] = ended.to(torch.uint8)
        st["scores"] = scores.contiguous()
        st["eos"] = V - 1 if case["ended"] else -1
    return st


# ---- the plain forms ----

def _plain_top(z, k):
    """The k largest of every row of z [R, V] fp32 in descending order, ties to the lowest index; nothing where a value
    is -inf.  Value and index make one 64-bit key, so that no two are equal."""
    R, V = z.shape
    k_in = min(k, V)
    b = (z + 0.0).contiguous().view(torch.int32)  # -0 becomes +0
    b = torch.where(b < 0, b ^ 0x7FFFFFFF, b).long()
    key = b * (1 << 32) + (0xFFFFFFFF - torch.arange(V, device=z.device))
    ids = 0xFFFFFFFF - (torch.topk(key, k_in, dim=-1).values & 0xFFFFFFFF)
    val = z.gather(1, ids)
    ids = torch.where(val == NINF, -1, ids).int()
    if k_in < k:
        val = torch.cat([val, val.new_full((R, k - k_in), NINF)], 1)
        ids = torch.cat([ids, ids.new_full((R, k - k_in), -1)], 1)
    return val, ids


def _plain_lse(z, T):
    """log sum exp(z / T) of every row in 64 bits, from terms in 32 bits; -inf for a row without a value."""
    m = z.amax(-1, keepdim=True)
    m = torch.where(m == NINF, 0.0, m)
    s = torch.exp((z - m) / T).sum(-1, dtype=torch.float64)
    return m[:, 0].double() / T + torch.log(s)


def _plain_beam(st):
    c = st["case"]
    B, W, n = c["B"], c["W"], c["beams"]
    z = st["logits"].float().reshape(B * W, -1)
    val, ids = _plain_top(z, n)
    # the order between beams in 64 bits: two beams' candidates can lie close together
    score = st["scores"].reshape(-1, 1).double() + (val.double() - _plain_lse(z, 1.0)[:, None])
    score = torch.where(val == NINF, NINF, score)
    if st["finished"] is not None:  # an ended beam stays as it is
        f = st["finished"].reshape(-1, 1) != 0
        first = torch.arange(n, device=z.device)[None] == 0
        score = torch.where(f, torch.where(first, st["scores"].reshape(-1, 1).double(), NINF), score)
        ids = torch.where(f, st["eos"], ids)
    score = torch.where(st["scores"].reshape(-1, 1) == NINF, NINF, score)
    best, at = torch.sort(score.view(B, W * n), dim=1, descending=True, stable=True)
    best, at = best[:, :n], at[:, :n]
    none = best == NINF
    parents = torch.where(none, 0, at // n)
    tokens = torch.where(none, 0, ids.view(B, W * n).gather(1, at)).int()
    states = st["states"].gather(1, parents[..., None].expand(-1, -1, c["Hs"]))
    history = st["history"].gather(1, parents[..., None].expand(-1, -1, c["L"]))
    history[:, :, c["pos"]] = tokens
    out = {"scores": best.float(), "parents": parents.int(), "tokens": tokens, "states": states, "history": history}
    if st["finished"] is not None:
        out["finished"] = (~none & ((st["finished"].gather(1, parents) != 0) | (tokens == st["eos"]))).to(torch.uint8)
    return out


def _plain_distill(st, upstream, want_grad):
    c = st["case"]
    T, V = c["temperature"], c["V"]
    shape = st["logits"].shape[:2]
    z = st["logits"].float().reshape(-1, V)
    ids = st["top_ids"].reshape(z.shape[0], -1).long()
    w = st["row_weights"].reshape(-1, 1)
    y = st["top_logits"].reshape(ids.shape).double() / T
    x = z / T
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - m)
    x_top, e_top = x.gather(1, ids).double(), e.gather(1, ids).double()
    rest = e.scatter(1, ids, 0.0).sum(-1, keepdim=True, dtype=torch.float64)
    s = rest + e_top.sum(-1, keepdim=True)
    lse = m.double() + torch.log(s)
    if st["teacher_lse"] is None:
        p = torch.exp(y - y.amax(-1, keepdim=True))
        p = p / p.sum(-1, keepdim=True)
        rho = torch.zeros_like(s)
    else:
        p = torch.exp(y - st["teacher_lse"].reshape(-1, 1).double())
        rho = (1.0 - p.sum(-1, keepdim=True)).clamp_min(0.0)
        rho = torch.where(rest > 0.0, rho, 0.0)
    term = torch.where(p > 0.0, p * (torch.log(p) - (x_top - lse)), 0.0).sum(-1, keepdim=True)
    term = term + torch.where(rho > 0.0, rho * (torch.log(rho) - torch.log(rest / s)), 0.0)
    loss = (w * term).float().view(shape)
    if not want_grad:
        return {"loss": loss}
    total = p.sum(-1, keepdim=True) + rho
    scale = (w if upstream is None else w * upstream.reshape(-1, 1)).double() / T
    of_rest = torch.where(rest > 0.0, scale * (total / s - rho / rest), 0.0)
    grad = (e * of_rest.float()).scatter(1, ids, (scale * (total * e_top / s - p)).float())
    return {"loss": loss, "grad": grad.to(st["logits"].dtype).view(shape + (V,))}


def _plain(st):
    c = st["case"]
    if c["op"] == "top":
        z = st["logits"].float().reshape(-1, c["V"])
        val, ids = _plain_top(z, c["k"])
        lse = _plain_lse(z, c["temperature"]).float()
        shape = st["logits"].shape[:2]
        return {"values": val.view(*shape, -1), "ids": ids.view(*shape, -1), "lse": lse.view(shape)}
    if c["op"] == "beam":
        return _plain_beam(st)
    return _plain_distill(st, st["upstream"] if c["call"] == "train" else None, c["call"] != "eval")


def run(st):
    if not own:
        return _plain(st)
    from draft_block_causal_b200 import domino
    c = st["case"]
    if c["op"] == "top":
        values, ids, lse = domino.top_logits(st["logits"], c["k"], temperature=c["temperature"])
        return {"values": values, "ids": ids, "lse": lse}
    if c["op"] == "beam":
        r = domino.beam_select(st["logits"], st["scores"], c["beams"], states=st["states"], history=st["history"],
                               pos=c["pos"], finished=st["finished"], eos=st["eos"])
        out = {"scores": r.scores, "parents": r.parents, "tokens": r.tokens, "states": r.states, "history": r.history}
        if r.finished is not None:
            out["finished"] = r.finished
        return out
    teacher = dict(teacher_lse=st["teacher_lse"], temperature=c["temperature"], row_weights=st["row_weights"])
    if c["call"] == "train":
        z = st["logits"].detach().requires_grad_()
        loss = domino.distill_loss(z, st["top_ids"], st["top_logits"], **teacher)
        (grad,) = torch.autograd.grad(loss, z, st["upstream"])
        return {"loss": loss.detach(), "grad": grad}
    loss, grad, _ = domino.distill(st["logits"], st["top_ids"], st["top_logits"], grad_out=c["call"] == "step",
                                   **teacher)
    return {"loss": loss} if grad is None else {"loss": loss, "grad": grad}


# ---- the definitions in 64 bits ----

def exact(case, seed):
    st = prepare(case, seed)
    z = st["logits"].double()
    if case["op"] == "top":
        lse = torch.logsumexp(z / case["temperature"], -1)
        k = min(case["k"], case["V"])
        top = torch.sort(z, dim=-1, descending=True).values[..., :k]
        top = torch.nn.functional.pad(top, (0, case["k"] - k), value=NINF)
        return {"values": top, "ids": None, "lse": lse}
    if case["op"] == "beam":
        B, W, V, n = case["B"], case["W"], case["V"], case["beams"]
        total = torch.log_softmax(z, -1) + st["scores"].double()[..., None]
        if st["finished"] is not None:
            f = st["finished"].bool()
            total[f] = NINF
            total[..., st["eos"]] = torch.where(f, st["scores"].double(), total[..., st["eos"]])
        best, at = torch.topk(total.view(B, W * V), n, dim=1)
        parent = torch.where(best == NINF, 0, at // V)
        states = torch.stack([st["states"][b][parent[b]] for b in range(B)])
        out = {"scores": best, "parents": None, "tokens": None, "states": states, "history": None}
        if st["finished"] is not None:
            out["finished"] = None
        return out
    T, w = case["temperature"], st["row_weights"].double()
    ids, y = st["top_ids"].long(), st["top_logits"].double() / T
    logq = torch.log_softmax(z / T, -1)
    q = logq.exp()
    outside = torch.ones_like(q).scatter_(-1, ids, 0.0)
    tau = (q * outside).sum(-1)
    if case["tail"]:
        p = torch.exp(y - st["teacher_lse"].double()[..., None])
        rho = torch.clamp(1.0 - p.sum(-1), min=0.0)
    else:
        p, rho = torch.softmax(y, -1), torch.zeros_like(tau)
    loss = w * (torch.special.xlogy(p, p).sum(-1) - (p * logq.gather(-1, ids)).sum(-1)
                + torch.special.xlogy(rho, rho) - torch.special.xlogy(rho, tau))
    if case["call"] == "eval":
        return {"loss": loss}
    up = w * st["upstream"].double() if case["call"] == "train" else w
    mass = (p.sum(-1) + rho)[..., None]
    grad = mass * q - q * outside * (rho / tau)[..., None]
    grad.scatter_add_(-1, ids, -p)
    return {"loss": loss, "grad": grad * (up / T)[..., None]}
