"""domino_distill and domino_distill_backward on the GPU against a plain fp64 implementation, and the gradient against
differences of the loss.

A gradient value is a difference of terms whose magnitudes add up to `scale` (rows_reference.distill): each carries the
relative error of a sum, of an exponential at log2 q, and a few roundings, 2 * (SUM(V) + (16 + |log2 q|) * 2^-24) in
all, and the result half a step of its type.  The loss carries the log-sum-exp's error times the teacher's mass, twice
for the others' class."""
import numpy as np
import pytest
import torch

from draft_block_causal_b200 import domino
from tests import rows_reference as R

pytestmark = pytest.mark.gpu

DT = {"fp32": torch.float32, "bf16": torch.bfloat16}


def teacher(rows, V, K, T, g, top=True):
    """Entries of a random teacher: ids, logits, log-sum-exp (fp32, on the GPU)."""
    t = torch.randn(rows, V, generator=g) * 2.5
    val, ids = torch.topk(t, min(K, V), dim=-1)
    if K > V:  # rows with fewer than K entries
        val = torch.nn.functional.pad(val, (0, K - V), value=float("-inf"))
        ids = torch.nn.functional.pad(ids, (0, K - V), value=-1)
    return ids.int().cuda(), val.float().cuda(), torch.logsumexp(t.double() / T, -1).float().cuda()


def expected(logits, ids, val, lse, T, weights):
    V = logits.shape[-1]
    f = lambda t: None if t is None else t.double().cpu().numpy().reshape(-1)
    return R.distill(logits.double().cpu().numpy().reshape(-1, V), ids.cpu().numpy().reshape(-1, ids.shape[-1]),
                     val.double().cpu().numpy().reshape(-1, ids.shape[-1]), f(lse), T, f(weights))


def check_loss(loss, want, V, weights):
    got = loss.double().cpu().numpy().reshape(-1)
    w = 1.0 if weights is None else np.abs(weights.double().cpu().numpy().reshape(-1))
    same = got == want
    np.testing.assert_array_equal(np.isfinite(got), np.isfinite(want))
    ok = np.isfinite(want)
    err = np.where(ok, np.abs(np.where(ok, got, 0) - np.where(ok, want, 0)), 0.0)
    assert (same | ~ok | (err <= 4 * w * R.sum_tol(V) + 2.0 ** -23 * np.abs(np.where(ok, want, 0)))).all(), err.max()


def check_grad(grad, want, scale, up, logits, T):
    V = logits.shape[-1]
    z = R.clean(logits.double().cpu().numpy().reshape(-1, V))
    lse = R.lse_rows(z, T)[:, None]
    with np.errstate(invalid="ignore"):
        bits = np.where(z > -np.inf, np.minimum(np.abs(z / T - np.where(np.isfinite(lse), lse, 0)) / np.log(2), 200), 0)
    u = 1.0 if up is None else up.double().cpu().numpy().reshape(-1, 1)
    got = grad.double().cpu().numpy().reshape(-1, V)
    ref = want * u
    tol = 2 * (R.sum_tol(V) + (16 + bits) * 2.0 ** -24) * scale * np.abs(u) + \
        torch.finfo(grad.dtype).eps / 2 * np.abs(ref) * (1 + 2.0 ** -8) + 1e-36
    err = np.abs(got - ref)
    assert (err <= tol).all(), (err / tol).max()


def check(logits, ids, val, lse, T=1.0, weights=None, up=None, grad_dtype=None):
    """The loss alone, the loss with its gradient, the backward call and autograd."""
    V = logits.shape[-1]
    kw = dict(teacher_lse=lse, temperature=T, row_weights=weights)
    want, gwant, scale = expected(logits, ids, val, lse, T, weights)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    loss, none, stats = domino.distill(logits, ids, val, status=status, **kw)
    assert none is None
    check_loss(loss, want, V, weights)
    for dt in ([grad_dtype] if grad_dtype else [torch.float32, torch.bfloat16]):
        grad = R.padded(torch.full(logits.shape, float("nan"), dtype=dt, device="cuda"), fill=7.0)
        loss2, g2, _ = domino.distill(logits, ids, val, grad_out=grad, status=status, **kw)
        assert g2 is grad
        check_loss(loss2, want, V, weights)
        check_grad(grad, gwant, scale, None, logits, T)
        back = domino.distill_backward(logits, ids, val, stats, up, grad_out=torch.empty_like(grad), status=status,
                                       **kw) if V % 8 == 0 else \
            domino.distill_backward(logits, ids, val, stats, up, status=status, **kw)
        check_grad(back, gwant, scale, up, logits, T)
    x = logits.detach().requires_grad_()
    loss3 = domino.distill_loss(x, ids, val, **kw)
    check_loss(loss3.detach(), want, V, weights)
    (g3,) = torch.autograd.grad(loss3, x, torch.ones_like(loss3) if up is None else up)
    assert g3.dtype == logits.dtype
    check_grad(g3, gwant, scale, up, logits, T)
    torch.cuda.synchronize()
    assert int(status.item()) == 0


@pytest.mark.parametrize("tail", [False, True], ids=["entries", "rest"])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("rows,V,K", [(1, 1, 1), (2, 7, 9), (3, 8, 3), (4, 100, 100), (5, 1003, 128), (17, 5000, 20),
                                      (2, 16384, 64), (1, 151936, 16), (6, 151936, 64), (160, 3001, 7),
                                      (2, 262144, 33), (1, 1 << 20, 5)])
def test_random_rows(rows, V, K, dtype, tail):
    g = torch.Generator().manual_seed(rows + V + K)
    ids, val, lse = teacher(rows, V, K, 1.0, g)
    z = R.padded((torch.randn(rows, V, generator=g) * 2.5).to(DT[dtype]))
    w, up = (0.5 + torch.rand(rows, generator=g)).cuda(), (0.1 + torch.rand(rows, generator=g)).cuda()
    check(z, ids, val, lse if tail else None, weights=w, up=up)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("rows,V,K", [(593, 2051, 128), (1300, 1504, 33), (160, 32003, 1)])
def test_more_rows_than_run_at_once(rows, V, K, dtype):
    g = torch.Generator().manual_seed(rows)
    ids, val, lse = teacher(rows, V, K, 1.0, g)
    z = R.padded((torch.randn(rows, V, generator=g) * 2.5).to(DT[dtype]))
    w = torch.rand(rows, generator=g)
    w[::7] = 0
    check(z, ids, val, lse, weights=w.cuda())


@pytest.mark.parametrize("tail", [False, True], ids=["entries", "rest"])
@pytest.mark.parametrize("T", [0.25, 2.0, 31.0])
def test_temperatures(T, tail):
    g = torch.Generator().manual_seed(9)
    ids, val, lse = teacher(6, 2000, 12, T, g)
    check(R.padded(torch.randn(6, 2000, generator=g) * 2), ids, val, lse if tail else None, T=T)


@pytest.mark.parametrize("tail", [False, True], ids=["entries", "rest"])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("V", [2003, 70003])
def test_ignored_rows_barred_tokens_and_unusual_entries(V, dtype, tail):
    rows, K = 16, 10
    g = torch.Generator().manual_seed(21)
    ids, val, lse = teacher(rows, V, K, 1.0, g)
    z = torch.randn(rows, V, generator=g) * 2
    low = torch.finfo(DT[dtype]).min
    w = torch.ones(rows, device="cuda")
    z[0] = -np.inf                                    # no student mass
    w[1] = 0.0                                        # padding: not read
    z[1] = np.nan
    z[2, int(ids[2, 3])] = -np.inf                    # the student bars an entry: infinite loss
    z[3] = -np.inf                                    # the student's mass on the entries alone
    z[3, ids[3].long().cpu()] = torch.randn(K, generator=g)
    ids[4] = -1                                       # no entry
    ids[5, 2:] = -1                                   # two entries
    val[6, 4:] = -np.inf                              # entries without mass
    val[7] = -np.inf
    ids[8, 5] = ids[8, 2]                             # a token given twice
    ids[9, :] = ids[9, 0]                             # one token K times
    z[10, 50:] = low                                  # a mask of the type's lowest value
    z[11] = low                                       # ... everywhere: a uniform row
    z[12, ::3] = np.nan
    z[13, int(ids[13, 0])] += 60.0                    # almost no mass outside the entries
    lse[14] = -np.inf if tail else lse[14]
    val[15] += 40.0                                   # p would sum to more than one
    if tail:
        lse[15] = torch.logsumexp(val[15].double(), -1).float()
    check(R.padded(z.to(DT[dtype])), ids, val, lse if tail else None, weights=w)


@pytest.mark.parametrize("peak", [31.0, 200.0])
def test_a_peaked_student_keeps_its_rest(peak):
    """1e-9, or 1e-82, of the student's mass lies outside the entries: as a difference of sums, or as terms about the
    row's maximum, it would be lost."""
    g = torch.Generator().manual_seed(31)
    ids, val, lse = teacher(4, 30000, 8, 1.0, g)
    z = torch.randn(4, 30000, generator=g)
    z.scatter_(1, ids.long().cpu(), peak + torch.rand(4, 8, generator=g))
    check(R.padded(z), ids, val, lse)


@pytest.mark.parametrize("tail", [False, True], ids=["entries", "rest"])
def test_gradient_against_differences(tail):
    """(loss(z + h u) - loss(z - h u)) / 2h along random directions u of unit length.  Each loss is off by at most
    4 SUM(V) + 2^-23 |loss| (< 2^-15 here, with V = 500 and losses below 8), so the quotient by 2^-15 / h; the third
    derivative along a unit direction is at most 6 in magnitude, h^2 more."""
    g = torch.Generator().manual_seed(41)
    rows, V, h = 5, 500, 2.0 ** -4
    ids, val, lse = teacher(rows, V, 6, 1.0, g)
    z = torch.randn(rows, V, generator=g).cuda()
    kw = dict(teacher_lse=lse if tail else None)
    _, grad, _ = domino.distill(R.padded(z), ids, val, grad_out=True, **kw)
    for _ in range(4):
        u = torch.randn(rows, V, generator=g).cuda()
        u = u / u.norm(dim=-1, keepdim=True)
        lp = domino.distill(R.padded(z + h * u), ids, val, **kw)[0].double()
        lm = domino.distill(R.padded(z - h * u), ids, val, **kw)[0].double()
        slope = (grad.double() * u.double()).sum(-1)
        assert float(lp.max()) < 8
        assert ((lp - lm) / (2 * h) - slope).abs().max().item() <= 2.0 ** -15 / h + h * h


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("V", [1003, 151936])
def test_in_place_and_untouched_padding(V, dtype):
    g = torch.Generator().manual_seed(51)
    ids, val, lse = teacher(7, V, 9, 1.0, g)
    z = (torch.randn(7, V, generator=g) * 2).to(DT[dtype])
    w = torch.tensor([1.0, 0.0, 2.0, 1.0, 0.5, 0.0, 1.0]).cuda()
    kw = dict(teacher_lse=lse, row_weights=w)
    _, want, stats = domino.distill(R.padded(z), ids, val, grad_out=True, stats_out=True, **kw)
    a = R.padded(z, extra=1, fill=5.0)
    domino.distill(a, ids, val, grad_out=a, **kw)
    assert torch.equal(a, want)
    base = torch.as_strided(a, (7, a.stride(0)), (a.stride(0), 1))
    assert (base[:, V:] == 5.0).all()
    b = R.padded(z, extra=1, fill=5.0)
    domino.distill_backward(b, ids, val, stats, grad_out=b, **kw)
    base = torch.as_strided(b, (7, b.stride(0)), (b.stride(0), 1))
    assert (base[:, V:] == 5.0).all()
    again = domino.distill_backward(R.padded(z), ids, val, stats, **kw)
    assert torch.equal(b, again)


def test_upstream_zero_and_three_dimensions():
    g = torch.Generator().manual_seed(61)
    ids, val, lse = teacher(12, 1000, 5, 1.0, g)
    z = torch.randn(3, 4, 1000, generator=g).cuda()
    up = torch.rand(3, 4, generator=g).cuda()
    up[1, 2] = 0.0
    check(z, ids.view(3, 4, 5), val.view(3, 4, 5), lse.view(3, 4), up=up)
    # a broadcast upstream gradient, as from .sum() and .mean()
    x = z.clone().requires_grad_()
    domino.distill_loss(x, ids.view(3, 4, 5), val.view(3, 4, 5), lse.view(3, 4)).mean().backward()
    _, whole, _ = domino.distill(z, ids.view(3, 4, 5), val.view(3, 4, 5), lse.view(3, 4), grad_out=True)
    assert torch.allclose(x.grad * 12, whole, rtol=2.0 ** -21, atol=1e-12)


def test_bad_token_sets_status_and_counts_as_none():
    g = torch.Generator().manual_seed(71)
    ids, val, lse = teacher(4, 600, 5, 1.0, g)
    z = torch.randn(4, 600, generator=g).cuda()
    for bad in (600, -2, 2 ** 31 - 1):
        bad_ids, ok_ids = ids.clone(), ids.clone()
        bad_ids[2, 1], ok_ids[2, 1] = bad, -1
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        a = domino.distill(z, bad_ids, val, grad_out=True, status=status)
        b = domino.distill(z, ok_ids, val, grad_out=True)
        torch.cuda.synchronize()
        assert int(status.item()) == domino.STATUS_BAD_TOKEN
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        domino.distill(z, bad_ids, val)  # without a status word
    torch.cuda.synchronize()


def test_repeats_bit_for_bit_on_streams_and_in_graphs():
    g = torch.Generator().manual_seed(81)
    ids, val, lse = teacher(40, 20000, 30, 1.0, g)
    z = (torch.randn(40, 20000, generator=g) * 2).bfloat16().cuda()
    want = domino.distill(z, ids, val, lse, grad_out=True, stats_out=True)
    back = domino.distill_backward(z, ids, val, want[2], teacher_lse=lse)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    late = torch.zeros_like(z)
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        late.copy_(z)
    got = domino.distill(late, ids, val, lse, grad_out=True, stats_out=True, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    buf = torch.zeros_like(z)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = domino.distill(buf, ids, val, lse, grad_out=True, stats_out=True)
        gb = domino.distill_backward(buf, ids, val, out[2], teacher_lse=lse)
    for _ in range(2):
        buf.copy_(z)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)) and torch.equal(gb, back)


def test_a_graph_captured_training_step_replays():
    """forward and backward through autograd inside a capture, after a warm-up on a side stream."""
    g = torch.Generator().manual_seed(91)
    ids, val, lse = teacher(10, 4000, 8, 1.0, g)
    x = torch.randn(10, 4000, generator=g).cuda().requires_grad_()

    def step():
        x.grad = None
        domino.distill_loss(x, ids, val, lse).sum().backward()

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    want = x.grad.clone()
    graph = torch.cuda.CUDAGraph()
    x.grad = None
    with torch.cuda.graph(graph):
        domino.distill_loss(x, ids, val, lse).sum().backward()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(x.grad, want)


def test_offsets_beyond_32_bits():
    rows, V = 16400, 131072  # 2^31 values and more, 4.3 GB, the gradient in their place
    z = torch.empty(rows, V, dtype=torch.bfloat16, device="cuda").normal_()
    last = z[-3:].clone()
    g = torch.Generator().manual_seed(3)
    ids, val, lse = teacher(4, V, 6, 1.0, g)
    ids, val, lse = (t.repeat(rows // 4, *([1] * (t.dim() - 1))).contiguous() for t in (ids, val, lse))
    loss, _, stats = domino.distill(z, ids, val, lse)
    back = domino.distill_backward(last, ids[-3:].contiguous(), val[-3:].contiguous(), stats[-3:].contiguous(),
                                   teacher_lse=lse[-3:].contiguous())
    fused, _, _ = domino.distill(z, ids, val, lse, grad_out=z)
    torch.cuda.synchronize()
    want, gwant, scale = expected(last, ids[-3:], val[-3:], lse[-3:], 1.0, None)
    for l in (loss, fused):
        check_loss(l[-3:], want, V, None)
    for x in (back, z[-3:]):
        check_grad(x, gwant, scale, None, last, 1.0)


def test_autograd_contract():
    g = torch.Generator().manual_seed(101)
    ids, val, lse = teacher(6, 1200, 5, 1.0, g)
    x = torch.randn(6, 1200, generator=g).cuda().requires_grad_()
    loss = domino.distill_loss(x * 1.0, ids, val, lse)      # a non-leaf
    (g1,) = torch.autograd.grad(loss.sum(), x, retain_graph=True)
    (g2,) = torch.autograd.grad(loss.sum(), x)               # twice from one graph
    assert torch.equal(g1, g2)
    with torch.no_grad():
        assert not domino.distill_loss(x, ids, val, lse).requires_grad
    # second derivatives are refused, and so is a backward pass over logits that were changed
    loss = domino.distill_loss(x, ids, val, lse)
    (g3,) = torch.autograd.grad(loss.sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(g3.sum(), x)
    y = x.detach().clone().requires_grad_()
    z = y * 1.0
    loss = domino.distill_loss(z, ids, val, lse)
    z.add_(1.0)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.sum().backward()
    # saved tensors that come back from the host
    with torch.autograd.graph.save_on_cpu():
        loss = domino.distill_loss(x, ids, val, lse)
    (g4,) = torch.autograd.grad(loss.sum(), x)
    assert torch.equal(g4, g1)
