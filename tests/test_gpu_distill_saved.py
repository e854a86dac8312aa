"""distill_loss with the tensors that it saves: laid out anew by a saved-tensor hook."""
import pytest
import torch

from draft_block_causal_b200 import domino
from tests import rows_reference as R
from tests.test_gpu_distill import DT, teacher

pytestmark = pytest.mark.gpu


def inputs(rows, V, K, dtype="fp32", seed=0):
    g = torch.Generator().manual_seed(seed + V)
    ids, val, lse = teacher(rows, V, K, 1.0, g)
    return R.padded((torch.randn(rows, V, generator=g) * 2).to(DT[dtype])), ids, val, lse


def moved(t):
    """t in memory that starts 4 bytes past an aligned place, contiguous."""
    flat = torch.empty(t.numel() + 8, dtype=t.dtype, device=t.device)
    out = flat[4 // t.element_size():][:t.numel()].view(t.shape)
    return out.copy_(t)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("V", [1203, 1200, 7])
@pytest.mark.parametrize("how", ["host", "moved", "clone"])
def test_saved_tensors_in_another_layout(V, dtype, how):
    z, ids, val, lse = inputs(5, V, 6, dtype)
    x = z.detach().requires_grad_()
    (want,) = torch.autograd.grad(domino.distill_loss(x, ids, val, lse).sum(), x)
    hooks = {"host": torch.autograd.graph.save_on_cpu(),
             "moved": torch.autograd.graph.saved_tensors_hooks(moved, lambda t: t),
             "clone": torch.autograd.graph.saved_tensors_hooks(
                 lambda t: t.clone(memory_format=torch.contiguous_format), lambda t: t)}[how]
    with hooks:
        loss = domino.distill_loss(x, ids, val, lse)
    (got,) = torch.autograd.grad(loss.sum(), x)
    assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("pack", [lambda t: t.half() if t.dtype == torch.float32 else t, lambda t: t[:1],
                                  lambda t: t if t.shape[-1] == 400 else t.cpu(),
                                  lambda t: t.float() if t.dtype == torch.bfloat16 else t.double(),
                                  lambda t: t.cpu()],
                         ids=["half", "part", "host", "wider", "all-host"])
def test_saved_tensors_of_another_type_size_or_device_are_refused(pack, dtype):
    z, ids, val, lse = inputs(3, 400, 4, dtype)
    x = z.detach().requires_grad_()
    with torch.autograd.graph.saved_tensors_hooks(pack, lambda t: t):
        loss = domino.distill_loss(x, ids, val, lse)
    with pytest.raises(ValueError, match="came back"):
        loss.sum().backward()
    torch.cuda.synchronize()
