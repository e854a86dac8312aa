"""Distillation's entries in 64 bits: a peaked teacher's rest, and rows whose loss and gradient come from the entries
alone, so that no sum in fp32 takes part and a result is off by its own rounding."""
import numpy as np
import pytest
import torch

from draft_block_causal_b200 import domino
from tests import rows_reference as R
from tests.test_gpu_distill import DT, check, expected

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("peak", [12.0, 16.0, 20.0, 22.0])
def test_a_peaked_teacher_keeps_its_rest(peak, dtype):
    """1e-2 to 1e-6 of the teacher's mass lies outside its entries: the gradient there is P q - rho q / tau, and rho is
    what the given log-sum-exp leaves of one, to the last bit that matters."""
    rows, V, K = 12, 3000, 8
    g = torch.Generator().manual_seed(int(peak))
    t = torch.randn(rows, V, generator=g)
    t[torch.arange(rows), torch.randint(V, (rows,), generator=g)] += peak
    val, ids = torch.topk(t, K, dim=-1)
    lse = torch.logsumexp(t.double(), -1).float()
    z = t + 0.5 * torch.randn(rows, V, generator=g)   # a student that has learnt the peak
    z[::4] = torch.randn(rows, V, generator=g)[::4]   # and one that has not
    p = torch.exp(val.double() - lse.double()[:, None]).sum(-1)
    assert ((1 - p) > 0).sum() >= rows // 2
    check(R.padded(z.to(DT[dtype])), ids.int().cuda(), val.cuda(), lse.cuda())


@pytest.mark.parametrize("tail", [False, True], ids=["entries", "rest"])
@pytest.mark.parametrize("V,T", [(5, 1.0), (64, 0.5), (128, 2.0)])
def test_every_token_an_entry(V, T, tail):
    """No column is left to the sums in fp32.  What is computed in 64 bits is off by at most 1e-12 of the terms'
    magnitudes (some hundred operations of 2^-53); the loss and the fused gradient are then rounded once, 2^-24 of
    their value; the backward call has two factors of its terms in fp32, 2^-24 of each term, and its own rounding."""
    rows = 8
    g = torch.Generator().manual_seed(V)
    z = torch.randn(rows, V, generator=g) * 4
    t = torch.randn(rows, V, generator=g) * 4
    ids = torch.stack([torch.randperm(V, generator=g) for _ in range(rows)]).int()
    val = t.gather(1, ids.long()).contiguous()
    lse = torch.logsumexp(t.double() / T, -1).float().cuda() if tail else None
    ids, val, w = ids.cuda(), val.cuda(), (0.5 + torch.rand(rows, generator=g)).cuda()
    x = R.padded(z)
    want, gwant, scale = expected(x, ids, val, lse, T, w)
    kw = dict(teacher_lse=lse, temperature=T, row_weights=w)
    loss, _, stats = domino.distill(x, ids, val, **kw)
    fused, grad, _ = domino.distill(x, ids, val, grad_out=True, **kw)
    back = domino.distill_backward(x, ids, val, stats, **kw)
    terms = 1e-12 * 50 * np.abs(w.double().cpu().numpy())  # p (y, x, L) of at most 50 each
    for l in (loss, fused):
        assert (np.abs(l.double().cpu().numpy() - want) <= 2.0 ** -24 * np.abs(want) + terms).all()
    e = np.abs(grad.double().cpu().numpy() - gwant)
    assert (e <= 2.0 ** -24 * np.abs(gwant) * (1 + 2.0 ** -20) + 1e-12 * scale + 1e-44).all()
    e = np.abs(back.double().cpu().numpy() - gwant)
    assert (e <= 2.0 ** -24 * (np.abs(gwant) + scale) * (1 + 2.0 ** -20) + 1e-12 * scale + 1e-44).all()


def test_masses_below_2_to_minus_1022():
    """exp(-740) is a positive number: the row's loss is that of the rest, as at any other mass."""
    rows, V = 3, 400
    g = torch.Generator().manual_seed(3)
    val, ids = torch.topk(torch.randn(rows, V, generator=g), 4, dim=-1)
    z = torch.randn(rows, V, generator=g)
    check(R.padded(z), ids.int().cuda(), val.cuda(), (val[:, 0] + 740.0).cuda())


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_a_student_far_from_an_entry(dtype):
    """Where q is nothing the gradient at an entry is -w p / T, rounded once."""
    rows, V, K, T = 5, 2000, 16, 2.0
    g = torch.Generator().manual_seed(4)
    val, ids = torch.topk(torch.randn(rows, V, generator=g) * 2, K, dim=-1)
    z = torch.randn(rows, V, generator=g)
    z.scatter_(1, ids, -300.0)
    x = R.padded(z.to(DT[dtype]))
    ids, val, w = ids.int().cuda(), val.cuda(), (0.5 + torch.rand(rows, generator=g)).cuda()
    _, grad, _ = domino.distill(x, ids, val, temperature=T, row_weights=w, grad_out=torch.empty(rows, V, device="cuda"))
    p = torch.softmax(val.double() / T, -1)
    want = -w.double()[:, None] * p / T
    got = grad.double().gather(1, ids.long())
    assert ((got - want).abs() <= 2.0 ** -24 * want.abs() * (1 + 2.0 ** -20)).all()
