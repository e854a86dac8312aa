"""The operators on rows of logits as they are used together with the head: a distillation step from a target's logits
to the gradient of the base logits, and beam drafting of a block through teacher-forced steps, against the fp64 oracle.

The head's logits are within 1e-2 + 1e-2 |z| of the oracle's (gpu_common).  A difference of e in every logit moves a
log-probability by at most 2e and a probability by the factor exp(2e)."""
import numpy as np
import pytest
import torch

import oracle
from draft_block_causal_b200 import domino, synth
from tests import rows_reference as R

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from tests import gpu_common as G
else:
    G = None


def _case(B, L, seed, dtype=synth.BF16):
    wl = dict(B=B, L=L, d=256, Hs=128, r=128, V=2000, dtype=dtype, weight_seed=seed, input_seed=seed + 1, s0_std=0.3,
              peak=2.0, name="rows")
    return synth.make_workload(wl, with_tokens=True)


@pytest.mark.parametrize("logits_dtype", [torch.float32, torch.bfloat16])
def test_distillation_step_of_the_head(logits_dtype):
    B, L, K, T = 5, 6, 12, 1.5
    data = _case(B, L, 700)
    w, lb, h, S0 = G.device_inputs(data)
    V = data["shape"]["V"]
    y = torch.from_numpy(data["tokens"]).cuda()
    target = torch.randn(B, L, V, generator=torch.Generator().manual_seed(1)).cuda() + lb.float()
    weights = torch.ones(B, L, device="cuda")
    weights[3, 4:] = 0.0  # behind a block's end
    top, ids, lse = domino.top_logits(target, K, temperature=T)
    logits, _ = domino.teacher_forced(w, lb, h, S0, y, logits_dtype=logits_dtype)
    z = logits.requires_grad_()
    loss = domino.distill_loss(z, ids, top, lse, T, weights)
    loss.sum().backward()
    fused, grad, _ = domino.distill(z, ids, top, lse, T, weights, grad_out=True)
    torch.cuda.synchronize()
    # the loss alone and the loss with its gradient add a row's terms in different orders, each within
    # 4 SUM(V) + 2^-23 |loss| of the definition: they differ by at most twice that
    near = 2 * (4 * R.sum_tol(V) + 2.0 ** -23 * loss.detach().abs())
    assert ((fused - loss.detach()).abs() <= near).all()
    # the operators on the head's own logits
    zz = logits.detach().double().cpu().numpy().reshape(-1, V)
    args = (ids.cpu().numpy().reshape(-1, K), top.double().cpu().numpy().reshape(-1, K),
            lse.double().cpu().numpy().reshape(-1), T, weights.cpu().numpy().reshape(-1))
    want, gwant, scale = R.distill(zz, *args)
    assert (np.abs(loss.detach().double().cpu().numpy().reshape(-1) - want)
            <= 4 * R.sum_tol(V) + 2.0 ** -23 * np.abs(want)).all()
    half = torch.finfo(logits_dtype).eps / 2
    for g in (z.grad, grad):
        err = np.abs(g.double().cpu().numpy().reshape(-1, V) - gwant)
        # log2 q stays above -100 here: (16 + 100) * 2^-24 in place of the value's own bits
        assert (err <= 2 * (R.sum_tol(V) + 116 * 2.0 ** -24) * scale + half * 1.01 * np.abs(gwant) + 1e-30).all()
    # and the whole chain against the oracle's logits
    ref = oracle.head(data["shape"], data["weights"], data["base_logits"], data["hidden"], data["S0"],
                      tokens=data["tokens"])["logits"].reshape(-1, V)
    lref, gref, sref = R.distill(ref, *args)
    e = (1e-2 + 1e-2 * np.abs(ref).max()) / T
    assert (np.abs(loss.detach().double().cpu().numpy().reshape(-1) - lref) <= 2 * e * args[4] + 1e-5).all()
    err = np.abs(z.grad.double().cpu().numpy().reshape(-1, V) - gref)
    # q moves by exp(2e), rho q / tau by exp(4e)
    assert (err <= sref * (np.exp(4 * e) - 1) + half * 1.01 * np.abs(gref) + 1e-6).all()


def _draft_beams(w, lb, h, S0, W):
    """Beam drafting of one block: per position one teacher-forced step of the beams' last tokens, then a selection."""
    B, L, V = lb.shape
    logits, _ = domino.teacher_forced(w, lb[:, :1].contiguous(), h[:, :1].contiguous(), S0,
                                      torch.zeros(B, 1, dtype=torch.int32, device="cuda"))
    step = domino.beam_select(logits, torch.zeros(B, 1, device="cuda"), W, states=S0[:, None].contiguous(),
                              history=torch.zeros(B, 1, L, dtype=torch.int32, device="cuda"), pos=0)
    for i in range(1, L):
        rows = lambda t: t[:, i - 1:i + 1].repeat_interleave(W, 0).contiguous()
        toks = torch.stack([step.tokens.reshape(-1), torch.zeros(B * W, dtype=torch.int32, device="cuda")], 1)
        logits, states = domino.teacher_forced(w, rows(lb), rows(h), step.states.view(B * W, -1), toks.contiguous(),
                                               states_out=True)
        step = domino.beam_select(logits[:, 1].view(B, W, V), step.scores, W,
                                  states=states[:, 1].contiguous().view(B, W, -1), history=step.history, pos=i)
    return step


@pytest.mark.parametrize("dtype", [synth.F32, synth.BF16])
def test_beam_drafting_of_a_block(dtype):
    B, L, W = 3, 5, 4
    data = _case(B, L, 720, dtype)
    w, lb, h, S0 = G.device_inputs(data)
    step = _draft_beams(w, lb, h, S0, W)
    torch.cuda.synchronize()
    hist = np.ascontiguousarray(step.history.cpu().numpy())
    scores = step.scores.double().cpu().numpy()
    sh = dict(data["shape"])

    def logprobs(tokens):  # [n, B, L] -> the oracle's log-probabilities of every position, [n, B, L, V]
        out = []
        for t in tokens:
            z = oracle.head(sh, data["weights"], data["base_logits"], data["hidden"], data["S0"],
                            tokens=np.ascontiguousarray(t))["logits"]
            out.append(z - R.lse_rows(z, 1.0)[..., None])
        return np.stack(out)

    # every hypothesis has the oracle's score of its own path
    lp = logprobs([hist[:, j] for j in range(W)])
    tol = L * 2 * (1e-2 + 1e-2 * 12)
    for j in range(W):
        path = np.take_along_axis(lp[j], hist[:, j][..., None].astype(np.int64), -1)[..., 0].sum(-1)
        assert (np.abs(path - scores[:, j]) <= tol).all()
    assert (np.diff(scores, axis=1) <= 0).all()
    # a beam search on the oracle's logits ends with the same scores
    ref_hist = np.zeros((B, 1, L), np.int32)
    ref_sc = np.zeros((B, 1))
    for i in range(L):
        n = ref_hist.shape[1]
        z = np.stack([logprobs([ref_hist[:, j]])[0][:, i] for j in range(n)], 1)
        r = R.beam(z, ref_sc, W, history=ref_hist, pos=i)
        ref_sc, ref_hist = r["scores"], r["history"]
    assert (np.abs(scores - ref_sc) <= tol).all()
    firm = np.abs(np.diff(ref_sc, axis=1)).min(1) > 2 * tol
    for b in np.flatnonzero(firm):
        np.testing.assert_array_equal(hist[b], ref_hist[b])
