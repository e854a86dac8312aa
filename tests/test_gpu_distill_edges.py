"""Distillation where single values decide: stretches of NaN logits, references beyond 2^24, and teachers whose
entries hold next to nothing.  Every call of `check` compares the loss alone, the fused gradient, the backward call and
autograd with the fp64 definition, within the tolerances that test_gpu_distill derives."""
import numpy as np
import pytest
import torch

from draft_block_causal_b200 import domino
from tests import rows_reference as R
from tests.test_gpu_distill import DT, check, teacher

pytestmark = pytest.mark.gpu


def nan_rows(rows, V, dtype, K=6, seed=0):
    """Logits [rows, V] on the host, with a random teacher's entries."""
    g = torch.Generator().manual_seed(seed + V)
    ids, val, lse = teacher(rows, V, K, 1.0, g)
    return (torch.randn(rows, V, generator=g) * 2).to(DT[dtype]), ids, val, lse


def check_in_place(z, ids, val, lse):
    """The fused call over the logits themselves gives what it gives beside them."""
    _, want, _ = domino.distill(R.padded(z), ids, val, lse, grad_out=True)
    x = R.padded(z)
    domino.distill(x, ids, val, lse, grad_out=x)
    assert torch.equal(x, want) and not torch.isnan(want).any()


@pytest.mark.parametrize("tail", [False, True], ids=["entries", "rest"])
@pytest.mark.parametrize("dtype,V", [("fp32", 800), ("bf16", 1600), ("fp32", 803), ("bf16", 1605)])
def test_nan_vectors(V, dtype, tail):
    """A vector of NaN is all that one of the threads sees of such a row."""
    n = 4 if dtype == "fp32" else 8
    z, ids, val, lse = nan_rows(6, V, dtype)
    z[0, :n] = np.nan                                  # one vector
    z[1, V // 2 // n * n:] = np.nan                    # the second half
    z[2, 3 * n:5 * n] = np.nan                         # NaN and barred tokens
    z[2, 3 * n + 1:5 * n:2] = -np.inf
    at = int(ids[3, 0]) // n * n                       # NaN round an entry's column
    keep = z[3, int(ids[3, 0])].clone()
    z[3, at:at + n] = np.nan
    z[3, int(ids[3, 0])] = keep
    z[4, int(ids[4, 1])] = np.nan                      # at an entry's column: barred
    z[5, :] = np.nan                                   # one value is left
    z[5, int(ids[5, 0])] = 1.0
    lse = lse if tail else None
    check(R.padded(z), ids, val, lse)
    check_in_place(z, ids, val, lse)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_nan_in_long_rows(dtype):
    """Stretches longer than a thread's tiles, in the middle and at the end of the blocks' slices."""
    V = 151936
    z, ids, val, lse = nan_rows(3, V, dtype)
    z[0, V // 2:] = np.nan
    z[1, -3000:] = np.nan
    z[2, 30000:90000] = np.nan
    z[2, 40000:50000] = -np.inf
    check(R.padded(z), ids, val, lse)
    check_in_place(z, ids, val, lse)


def test_nan_in_more_rows_than_run_at_once():
    """A block a row: its threads walk several tiles, some of them without a value."""
    z, ids, val, lse = nan_rows(700, 9000, "fp32")
    z[::2, 7200:] = np.nan
    z[1::2, :3600] = np.nan
    check(R.padded(z), ids, val, lse, grad_dtype=torch.float32)


@pytest.mark.parametrize("tail", [False, True], ids=["entries", "rest"])
@pytest.mark.parametrize("T", [float(np.float32(0.05)), 2.0 ** -10])
def test_references_beyond_24_bits(T, tail):
    """log2(e) z / T of an entry above 2^24, where not every whole number is a float."""
    rows, V, K = 24, 500, 5
    g = torch.Generator().manual_seed(7)
    # logits a few steps of T apart about a level at which the reference has more than 24 bits
    level = 1.2 * 2 ** 24 * T / 1.4427 + 37.3 * T * torch.arange(rows)[:, None]
    t = level + T * 2 * torch.randn(rows, V, generator=g)
    val, ids = torch.topk(t.float(), K, dim=-1)
    lse = torch.logsumexp(t.float().double() / T, -1).float().cuda()
    z = level + T * 2 * torch.randn(rows, V, generator=g)
    z[::3] = -level[::3] + T * torch.randn(rows, V, generator=g)[::3]
    check(R.padded(z.float()), ids.int().cuda(), val.cuda(), lse if tail else None, T=T)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("K", [1, 3])
@pytest.mark.parametrize("T", [float(np.float32(0.05)), 2.0 ** -10, float(np.float32(0.07))])
def test_infinite_logit_at_an_entry(T, K, dtype):
    g = torch.Generator().manual_seed(8)
    z = torch.randn(4, 300, generator=g)
    val, ids = torch.topk(torch.randn(4, 300, generator=g), K, dim=-1)
    z[0, ids[0, 0]] = np.inf
    z[1, ids[1]] = np.inf
    z[2, ids[2, 0]] = 9e5
    z[3, 17] = np.inf                      # ... as here, outside the entries
    if K > 1:
        val[0, 1:] = val[2, 1:] = -np.inf  # a positive mass there would cost 1e6 / T
    check(R.padded(z.to(DT[dtype])), ids.int().cuda(), val.cuda(), None, T=T)


@pytest.mark.parametrize("below", [90.0, 104.0, 200.0, 600.0])
def test_entries_far_below_the_teachers_sum(below):
    """A positive mass that fp32 does not hold: loss and gradient are those of the rest of the vocabulary."""
    rows, V, K = 4, 1000, 6
    g = torch.Generator().manual_seed(9)
    ids, val, lse = teacher(rows, V, K, 1.0, g)
    z = torch.randn(rows, V, generator=g) * 2
    check(R.padded(z), ids, val, (val[:, 0] + below).contiguous())
    _, grad, _ = domino.distill(R.padded(z), ids, val, (val[:, 0] + below).contiguous(), grad_out=True)
    assert (grad != 0).any(-1).all()


def test_entries_far_below_at_a_low_temperature():
    rows, V, K = 3, 700, 4
    T = float(np.float32(0.05))
    g = torch.Generator().manual_seed(10)
    ids, val, lse = teacher(rows, V, K, T, g)
    check(R.padded(torch.randn(rows, V, generator=g) * 0.1), ids, val, ((val[:, 0] + 5.5) / T).contiguous(), T=T)
