"""distill_loss with the tensors it saves: laid out anew by a hook, or overwritten before the backward pass; and the
status word of the backward call."""
import pytest
import torch

from draft_block_causal_b200 import domino, synth
from tests import rows_reference as R
from tests.test_gpu_distill import DT, teacher

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from tests import gpu_common as G
else:
    G = None


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


def test_a_call_that_fills_a_saved_tensor_is_seen_by_autograd():
    """An output buffer that holds what an earlier loss has saved: its backward pass is refused, as after a torch
    operation in place."""
    z, ids, val, lse = inputs(6, 1200, 5)
    x = z.detach().requires_grad_()
    top = domino.top_logits(z, 5)
    loss = domino.distill_loss(x, top[1], top[0], top[2])
    domino.top_logits(-z, 5, values_out=top[0], ids_out=top[1], lse_out=top[2])
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.sum().backward()
    for call in (lambda y: domino.distill(y, ids, val, lse, grad_out=y),
                 lambda y: domino.distill_backward(y, ids, val, stats, teacher_lse=lse, grad_out=y)):
        _, _, stats = domino.distill(z, ids, val, lse)
        y = z.clone()
        loss = domino.distill_loss(y.view(6, 1200).requires_grad_() * 1.0, ids, val, lse)
        loss.sum().backward()               # its own logits are untouched
        z1 = z.clone().requires_grad_() * 1.0
        loss = domino.distill_loss(z1, ids, val, lse)
        call(z1.detach())
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.sum().backward()
    # one entry a row: [6, 1] is as large as the losses of 6 rows and the scores of 2 x 3 beams
    one, first = ids[:, :1].contiguous(), val[:, :1].contiguous()
    loss = domino.distill_loss(x, one, first)
    domino.distill(z, ids, val, lse, loss_out=first.view(6))
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.sum().backward()
    first = val[:, :1].contiguous()
    loss = domino.distill_loss(x, one, first)
    beams = domino.beam_select(z.view(2, 3, 1200), torch.zeros(2, 3, device="cuda"), 3)
    domino.beam_select(z.view(2, 3, 1200), torch.zeros(2, 3, device="cuda"), 3,
                       out=beams._replace(scores=first.view(2, 3)))
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.sum().backward()
    # row weights and the teacher's log-sum-exp are read by the forward call alone
    w, row = torch.rand(6, device="cuda"), lse.clone()
    want = torch.autograd.grad(domino.distill_loss(x, ids, val, row, row_weights=w).sum(), x)[0]
    loss = domino.distill_loss(x, ids, val, row, row_weights=w)
    domino.top_logits(z, 5, lse_out=w)
    row.zero_()
    assert torch.equal(torch.autograd.grad(loss.sum(), x)[0], want)
    # the head's logits, refilled by its next call
    data = synth.make_workload(dict(B=2, L=3, d=128, Hs=64, r=64, V=1000, dtype=synth.BF16, weight_seed=1, input_seed=2,
                                    s0_std=0.1, peak=2.0, name="saved"), with_tokens=True)
    w, lb, h, S0 = G.device_inputs(data)
    toks = torch.from_numpy(data["tokens"]).cuda()
    logits, states = domino.teacher_forced(w, lb, h, S0, toks, states_out=True)
    top = domino.top_logits(lb, 5)
    for refill in (lambda: domino.teacher_forced(w, lb, h, S0, toks, logits_out=logits),
                   lambda: domino.draft_greedy(w, lb, h, S0, logits_out=logits)):
        bias = torch.zeros(1000, device="cuda", requires_grad=True)
        (bias * logits).sum().backward()    # in time
        loss = (bias * logits).sum() + domino.distill_loss(logits + bias, top[1], top[0], top[2]).sum()
        refill()
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()
    with torch.inference_mode():            # no versions there
        top = domino.top_logits(z, 5)
        domino.top_logits(z, 5, values_out=top[0], ids_out=top[1], lse_out=top[2])
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
