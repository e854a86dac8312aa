"""domino_beam_select on the GPU against a plain fp64 implementation: parents, tokens, states, histories exactly, the
scores within the log-sum-exp's tolerance (rows_reference) and half a step of fp32."""
import numpy as np
import pytest
import torch

from draft_block_causal_b200 import domino
from tests import rows_reference as R

pytestmark = pytest.mark.gpu

DT = {"fp32": torch.float32, "bf16": torch.bfloat16}


def check(logits, scores, n, **kw):
    B, W, V = logits.shape
    got = domino.beam_select(logits, scores, n, **kw)
    torch.cuda.synchronize()
    host = {k: (v.cpu().numpy() if isinstance(v, torch.Tensor) else v) for k, v in kw.items() if k != "workspace"}
    want = R.beam(logits.double().cpu().numpy(), scores.double().cpu().numpy(), n, **host)
    np.testing.assert_array_equal(got.parents.cpu().numpy(), want["parents"])
    np.testing.assert_array_equal(got.tokens.cpu().numpy(), want["tokens"])
    for name in ("states", "history"):
        if kw.get(name) is not None:
            np.testing.assert_array_equal(getattr(got, name).cpu().numpy(), want[name])
        else:
            assert getattr(got, name) is None
    if kw.get("eos", -1) >= 0:
        np.testing.assert_array_equal(got.finished.cpu().numpy(), want["finished"])
    s, w = got.scores.double().cpu().numpy(), want["scores"]
    np.testing.assert_array_equal(s == -np.inf, w == -np.inf)
    live = w > -np.inf
    assert (np.abs(s - np.where(live, w, 0))[live] <= (R.sum_tol(V) + 2.0 ** -23 * np.abs(w))[live]).all()
    return got


def inputs(B, W, V, dtype, Hs=24, hist=9, seed=0):
    g = torch.Generator().manual_seed(seed * 1000 + B * 100 + W)
    z = (torch.randn(B, W, V, generator=g) * 2.5).to(DT[dtype])
    return (R.padded(z), (-20 * torch.rand(B, W, generator=g)).cuda(), torch.randn(B, W, Hs, generator=g).cuda(),
            torch.randint(0, V, (B, W, hist), generator=g, dtype=torch.int32).cuda())


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("B,W,n,V", [(1, 1, 1, 1), (1, 1, 8, 5), (2, 3, 32, 4), (1, 4, 4, 151936), (5, 7, 3, 20011),
                                     (40, 1, 8, 5000), (3, 32, 32, 3000), (64, 8, 8, 2500), (2, 32, 1, 1003),
                                      (2, 17, 9, 30001), (1, 16, 32, 9000), (3, 3, 5, 70000), (1, 5, 2, 40000),
                                      (300, 2, 4, 1500), (1, 1, 32, 151936), (32, 8, 8, 40000), (4, 32, 32, 70000),
                                      (70, 1, 9, 151936)])
def test_random_beams(B, W, n, V, dtype):
    z, sc, st, hi = inputs(B, W, V, dtype)
    check(z, sc, n, states=st, history=hi, pos=4)
    check(z, sc, n)


@pytest.mark.parametrize("Hs,hist,pos", [(4, 1, 0), (1024, 64, 63), (1000, 17, 0)])
def test_state_and_history_sizes(Hs, hist, pos):
    z, sc, st, hi = inputs(3, 4, 700, "fp32", Hs, hist)
    check(z, sc, 6, states=st, history=hi, pos=pos)
    check(z, sc, 6, states=st)
    check(z, sc, 6, history=hi, pos=pos)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("B,V", [(6, 1203), (90, 40003)], ids=["one-kernel", "two-kernels"])
def test_finished_and_dead_beams(B, V, dtype):
    W, eos = 5, V - 1
    code = {"fp32": torch.float32, "bf16": torch.bfloat16}[dtype]
    assert (domino.beam_workspace_bytes(B, W, 6, V, code) > 0) == (B == 90)
    z, sc, st, hi = inputs(B, W, V, dtype)
    sc[0, :] = -np.inf                   # a dead group
    sc[1, 1:] = -np.inf                  # one beam alive
    sc[2, 3] = np.nan                    # NaN: dead
    fin = torch.zeros(B, W, dtype=torch.uint8, device="cuda")
    fin[1, 0] = 1                        # the only beam has finished
    fin[3] = 1                           # all have
    fin[4, ::2] = 1
    fin[0, 2] = 1                        # finished and dead: dead
    z[5, :, eos] = 30.0                  # every beam finishes now
    z[3] = float("nan")                  # a finished beam's logits are not read
    z[2, 4] = float("-inf")              # a live beam without a token
    got = check(z, sc, 6, states=st, history=hi, pos=8, finished=fin, eos=eos)
    assert (got.scores[0] == -np.inf).all() and (got.finished[3, :5] == 1).all()
    check(z, sc, 6, states=st, history=hi, pos=8, eos=eos)


@pytest.mark.parametrize("B,V", [(2, 64), (400, 8192)], ids=["one-kernel", "two-kernels"])
def test_equal_scores_go_to_the_lower_beam_and_token(B, V):
    z = torch.zeros(B, 4, V, device="cuda")
    z[1] = 1.0 + torch.arange(V, device="cuda") % 2
    sc = torch.full((B, 4), -1.5, device="cuda")
    got = check(z, sc, 10)
    assert got.parents[0].tolist() == [0] * 10 and got.tokens[0].tolist() == list(range(10))
    assert got.tokens[1].tolist() == list(range(1, 21, 2))


@pytest.mark.parametrize("B,V", [(2, 900), (2, 70000), (60, 50000)], ids=["one-kernel", "parts", "two-kernels"])
def test_barred_and_extreme_logits(B, V):
    W = 3
    z, sc, st, hi = inputs(B, W, V, "fp32")
    z[0, 0, 5:] = float("-inf")
    z[0, 1, :] = torch.finfo(torch.float32).min
    z[0, 2, 77] = float("inf")
    z[1, 0, ::2] = float("nan")
    z[1, 1, 3:] = torch.finfo(torch.float32).min
    check(z, sc, 8, states=st, history=hi, pos=2)


def test_given_outputs_workspace_and_strides():
    z, sc, st, hi = inputs(4, 3, 2000, "bf16")
    want = domino.beam_select(z, sc, 5, states=st, history=hi, pos=1)
    out = domino.BeamStep(*(None if t is None else torch.zeros_like(t) for t in want))
    assert domino.beam_workspace_bytes(4, 3, 5, 2000, torch.bfloat16) == 0
    got = domino.beam_select(z, sc, 5, states=st, history=hi, pos=1, out=out)
    torch.cuda.synchronize()
    assert got is out
    for a, b in zip(got, want):
        assert (a is None and b is None) or torch.equal(a, b)
    z, sc, st, hi = inputs(20, 4, 151936, "fp32")  # in two kernels
    ws = domino.alloc_workspace(domino.beam_workspace_bytes(20, 4, 5, 151936))
    assert ws.numel() > 0
    ws.fill_(255)
    check(z, sc, 5, states=st, history=hi, pos=1, workspace=ws)
    sc, st, hi = (t[:4, :3].contiguous() for t in (sc, st, hi))
    wide = torch.randn(4, 3, 4096, device="cuda")
    check(wide[..., 24:2023], sc, 5, states=st)
    check(torch.randn(4, 6, 1000, device="cuda")[:, :1], sc[:, :1].contiguous(), 5)


@pytest.mark.parametrize("B,V", [(8, 6000), (40, 70000)], ids=["one-kernel", "two-kernels"])
def test_on_another_stream_and_in_two_graphs(B, V):
    z, sc, st, hi = inputs(B, 4, V, "fp32")
    assert (domino.beam_workspace_bytes(B, 4, 4, V) > 0) == (B == 40)
    want = domino.beam_select(z, sc, 4, states=st, history=hi, pos=3)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    late = torch.zeros_like(z)
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        late.copy_(z)
    got = domino.beam_select(late, sc, 4, states=st, history=hi, pos=3, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got[:5], want[:5]))
    graphs = []
    for sign in (1.0, -1.0):
        buf = z * sign
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = domino.beam_select(buf, sc, 4, states=st, history=hi, pos=3)
        graphs.append((g, out, domino.beam_select(buf, sc, 4, states=st, history=hi, pos=3), buf))
    for _ in range(2):
        for g, _, _, _ in graphs:
            g.replay()
    torch.cuda.synchronize()
    for _, out, ref, _ in graphs:
        assert all(torch.equal(a, b) for a, b in zip(out[:5], ref[:5]))
