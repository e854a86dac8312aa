"""Beam drafting of a block, every selection against an fp64 one on the head's own logits: parents, tokens, states and
histories exactly, the scores within the log-sum-exp's tolerance.  The head's logits and states of every beam are then
compared with the fp64 oracle's along that beam's history, so that a state or a history that followed another beam's
parent would show."""
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


def _case(B, L, V, dtype):
    """A head whose beams' states lie far apart: embeddings and W2 16 times the synthetic ones (exact in bf16)."""
    wl = dict(B=B, L=L, d=256, Hs=128, r=128, V=V, dtype=dtype, weight_seed=740, input_seed=741, s0_std=0.3, peak=0.5,
              name="beams")
    data = synth.make_workload(wl)
    data["weights"] = dict(data["weights"])
    for name in ("embed", "W2"):
        x = synth.to_f32(data["weights"][name], dtype) * np.float32(16)
        data["weights"][name] = x if dtype == synth.F32 else synth.f32_to_bf16_bits(x)
    return data


@pytest.mark.parametrize("dtype", [synth.F32, synth.BF16])
@pytest.mark.parametrize("B,L,W,V", [(3, 6, 4, 2000), (2, 5, 7, 3000)])
def test_every_step_selects_as_fp64_does(B, L, W, V, dtype):
    data = _case(B, L, V, dtype)
    w, lb, h, S0 = G.device_inputs(data)
    step = None
    crossed = 0
    for i in range(L):
        if i == 0:
            logits, _ = domino.teacher_forced(w, lb[:, :1].contiguous(), h[:, :1].contiguous(), S0,
                                              torch.zeros(B, 1, dtype=torch.int32, device="cuda"))
            z, sc, st = logits, torch.zeros(B, 1, device="cuda"), S0[:, None].contiguous()
            hi = torch.zeros(B, 1, L, dtype=torch.int32, device="cuda")
        else:
            n = step.scores.shape[1]
            rows = lambda t: t[:, i - 1:i + 1].repeat_interleave(n, 0).contiguous()
            toks = torch.stack([step.tokens.reshape(-1), torch.zeros(B * n, dtype=torch.int32, device="cuda")], 1)
            logits, states = domino.teacher_forced(w, rows(lb), rows(h), step.states.view(B * n, -1),
                                                   toks.contiguous(), states_out=True)
            z, sc, hi = logits[:, 1].view(B, n, V), step.scores, step.history
            st = states[:, 1].contiguous().view(B, n, -1)  # what position i has read
            _against_the_oracle(data, z, st, hi, i)
        step = domino.beam_select(z, sc, W, states=st, history=hi, pos=i)
        torch.cuda.synchronize()
        want = R.beam(z.double().cpu().numpy(), sc.double().cpu().numpy(), W, states=st.cpu().numpy(),
                      history=hi.cpu().numpy(), pos=i)
        for name in ("parents", "tokens", "states", "history"):
            np.testing.assert_array_equal(getattr(step, name).cpu().numpy(), want[name])
        err = np.abs(step.scores.double().cpu().numpy() - want["scores"])
        assert (err <= R.sum_tol(V) + 2.0 ** -23 * np.abs(want["scores"])).all()
        crossed += int((want["parents"] != np.arange(W)).sum()) if i else 0
    assert crossed > 0  # beams did change places


def _against_the_oracle(data, z, st, hi, i):
    """The head's logits at position i and the states that it has read, along each beam's history."""
    hist = hi.cpu().numpy()
    B, n, L = hist.shape
    want = []
    for j in range(n):
        ref = oracle.head(data["shape"], data["weights"], data["base_logits"], data["hidden"], data["S0"],
                          tokens=np.ascontiguousarray(hist[:, j]))
        got = z[:, j].double().cpu().numpy()
        # logits are within 1e-2 + 1e-2 |z| of the oracle's for the synthetic W2 (gpu_common); they are L_base + W2 a,
        # and what a is off by (a rounding to bf16 of each of its entries) enters through W2: 16 times as much here
        assert (np.abs(got - ref["logits"][:, i]) <= 16e-2 + 1e-2 * np.abs(ref["logits"][:, i])).all()
        assert (np.abs(st[:, j].double().cpu().numpy() - ref["states"][:, i]) <= 5e-3).all()
        want.append(ref["states"][:, i])
    # beams of different last tokens are further apart than the tolerance
    for j in range(1, n):
        apart = hist[:, j, i - 1] != hist[:, 0, i - 1]
        assert (np.abs(want[j] - want[0]).max(-1)[apart] > 0.05).all()
