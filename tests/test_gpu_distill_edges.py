"""Distillation where single values decide: stretches of NaN logits.  Every call of `check` compares the loss alone, the
fused gradient, the backward call and autograd with the fp64 definition, within the tolerances that test_gpu_distill
derives."""
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
