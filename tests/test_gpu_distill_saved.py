"""distill_loss with the tensors that it saves: laid out anew by a saved-tensor hook; and the status word of the
backward call."""
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


@pytest.mark.parametrize("V,K", [(600, 5), (151936, 128)])
def test_the_backward_call_reports_bad_tokens(V, K):
    z, ids, val, lse = inputs(4, V, K)
    for bad in (V, -2, 2 ** 31 - 1):
        bad_ids, ok_ids = ids.clone(), ids.clone()
        bad_ids[2, K - 1], ok_ids[2, K - 1] = bad, -1
        _, _, stats = domino.distill(z, ok_ids, val, lse)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        want = domino.distill_backward(z, ok_ids, val, stats, teacher_lse=lse, status=status)
        assert int(status.item()) == 0
        got = domino.distill_backward(z, bad_ids, val, stats, teacher_lse=lse, status=status)
        assert int(status.item()) == domino.STATUS_BAD_TOKEN and torch.equal(got, want)
        domino.distill_backward(z, bad_ids, val, stats, teacher_lse=lse)  # without a status word
        # a row that has no gradient for want of an entry reports as the forward call does
        bad_ids[2] = bad
        for call in ("forward", "backward"):
            status.zero_()
            if call == "forward":
                _, _, stats = domino.distill(z, bad_ids, val, status=status)
            else:
                domino.distill_backward(z, bad_ids, val, stats, status=status)
            assert int(status.item()) == domino.STATUS_BAD_TOKEN
        # rows that are not read report nothing
        w, up = torch.ones(4, device="cuda"), torch.ones(4, device="cuda")
        w[2] = 0.0
        status.zero_()
        _, _, stats = domino.distill(z, bad_ids, val, row_weights=w, status=status)
        domino.distill_backward(z, bad_ids, val, stats, row_weights=w, status=status)
        up[2] = 0.0
        _, _, stats = domino.distill(z, bad_ids, val)
        domino.distill_backward(z, bad_ids, val, stats, up, status=status)
        assert int(status.item()) == 0
