"""Host-side checks of the operators on rows of logits: the C ABI's refusals (never dereferenced pointers, so nothing can
be launched), and the binding's refusals on CPU tensors."""
import ctypes

import pytest
import torch

from draft_block_causal_b200 import build, domino
from tests import rows_reference as R

P = 0x10000000  # 16- and 256-byte aligned, never dereferenced
STEP = 0x10000000


@pytest.fixture(scope="module")
def L():
    build.build()
    return domino.lib()


def top(L, **kw):
    a = dict(rows=4, V=1000, ld=1000, dtype=0, logits=P, k=8, T=1.0, values=P + STEP, ids=P + 2 * STEP,
             lse=P + 3 * STEP)
    a.update(kw)
    return L.domino_top_logits(a["rows"], a["V"], a["ld"], a["dtype"], a["logits"], a["k"], a["T"], a["values"], a["ids"],
                               a["lse"], None)


@pytest.mark.parametrize("bad", [dict(rows=0), dict(rows=-1), dict(V=0), dict(V=(1 << 20) + 1, ld=1 << 21), dict(ld=999),
                                 dict(ld=1001), dict(ld=992), dict(dtype=2), dict(dtype=-1), dict(logits=None),
                                 dict(logits=P + 8), dict(k=0), dict(k=129), dict(T=0.0), dict(T=-1.0), dict(T=1e-4),
                                 dict(T=1025.0), dict(T=float("nan")), dict(T=float("inf")), dict(values=None),
                                 dict(ids=None), dict(values=P + 4 * 3999), dict(ids=P), dict(lse=P + 4),
                                 dict(values=P + STEP + 2), dict(ids=P + 2 * STEP + 1), dict(lse=P + 3 * STEP + 3), dict(lse=P + STEP + 16),
                                 dict(ids=P + STEP + 4)])
def test_top_logits_refusals(L, bad):
    assert top(L, **bad) == domino.ERR_INVALID_ARGUMENT


def test_top_logits_row_limit(L):
    assert top(L, rows=(1 << 22) + 1, V=8, ld=8) == domino.ERR_UNSUPPORTED


def beam(L, ws=P + 20 * STEP, ws_bytes=1 << 40, **kw):
    a = dict(B=2, W_in=3, W_out=4, V=1000, ld=1000, dtype=1, eos=-1, Hs=64, hist_len=16, pos=3, logits=P,
             scores=P + STEP, finished=None, states=P + 2 * STEP, history=P + 3 * STEP, scores_out=P + 4 * STEP,
             parents_out=P + 5 * STEP, tokens_out=P + 6 * STEP, finished_out=None, states_out=P + 7 * STEP,
             history_out=P + 8 * STEP)
    a.update(kw)
    s = domino.BeamArgs(*(a[n] for n, _ in domino.BeamArgs._fields_))
    return L.domino_beam_select(ctypes.byref(s), ws, ws_bytes, None)


@pytest.mark.parametrize("bad", [dict(B=0), dict(W_in=0), dict(W_out=0), dict(W_in=33), dict(W_out=33), dict(V=0),
                                 dict(ld=996), dict(dtype=3), dict(logits=None), dict(scores=None),
                                 dict(scores_out=None), dict(parents_out=None), dict(tokens_out=None), dict(eos=-2),
                                 dict(eos=1000), dict(finished=P + 9 * STEP, finished_out=P + 10 * STEP),
                                 dict(finished=P + 9 * STEP, eos=5), dict(finished_out=P + 10 * STEP),
                                 dict(states_out=None), dict(states=None), dict(history_out=None), dict(history=None),
                                 dict(Hs=62), dict(Hs=0), dict(states=P + 2 * STEP + 4), dict(hist_len=0), dict(pos=-1),
                                 dict(pos=16), dict(states_out=P + 2 * STEP), dict(history_out=P + 3 * STEP + 64),
                                 dict(scores_out=P + STEP), dict(tokens_out=P + 3 * STEP),
                                 dict(scores=P + STEP + 2),
                                 dict(tokens_out=P + 6 * STEP + 1), dict(history=P + 3 * STEP + 2),
                                 dict(tokens_out=P + 5 * STEP), dict(scores_out=P + 7 * STEP + 4)])
def test_beam_select_refusals(L, bad):
    assert beam(L, **bad) == domino.ERR_INVALID_ARGUMENT


def test_beam_select_limits(L):
    assert L.domino_beam_select(None, None, 0, None) == domino.ERR_INVALID_ARGUMENT
    assert L.domino_beam_workspace_bytes(2, 3, 4, 1000, 1) == 0  # small: none is needed
    n = L.domino_beam_workspace_bytes(200, 3, 4, 100000, 0)
    assert n > 0 and n % 256 == 0 and domino.beam_workspace_bytes(200, 3, 4, 100000) == n
    with pytest.raises(ValueError, match="dtype"):
        domino.beam_workspace_bytes(200, 3, 4, 100000, torch.float16)
    big = dict(B=200, V=100000, ld=100000, dtype=0, states=None, states_out=None, history=None, history_out=None,
               scores=P + 21 * STEP)
    far = {k: P + i * 1000 * STEP for i, k in enumerate(("scores", "scores_out", "parents_out", "tokens_out"), 1)}
    big.update(far)
    for w, b in ((None, n), (P + 9000 * STEP + 16, n), (P + 9000 * STEP, n - 1)):
        assert beam(L, ws=w, ws_bytes=b, **big) == domino.ERR_WORKSPACE
    assert beam(L, ws=far["tokens_out"], ws_bytes=n, **big) == domino.ERR_INVALID_ARGUMENT
    for bad in ((0, 3, 4, 100000, 0), (2, 0, 4, 100000, 0), (2, 3, 33, 100000, 0), (1 << 22, 3, 4, 100000, 0),
                (200, 3, 4, 0, 0)):
        assert L.domino_beam_workspace_bytes(*bad) == 0
    assert beam(L, Hs=(1 << 20) + 4) == domino.ERR_UNSUPPORTED
    assert beam(L, hist_len=(1 << 20) + 1) == domino.ERR_UNSUPPORTED
    assert beam(L, B=1 << 21, V=8, ld=8, states=None, states_out=None, history=None,
                history_out=None) == domino.ERR_UNSUPPORTED


def distill(L, call="forward", **kw):
    a = dict(rows=4, V=1000, ld=1000, dtype=1, K=8, logits=P, top_ids=P + STEP, top_logits=P + 2 * STEP,
             teacher_lse=P + 3 * STEP, row_weights=P + 4 * STEP, temperature=1.0, loss=P + 5 * STEP,
             stats=P + 6 * STEP, grad=P + 7 * STEP, grad_ld=1000, grad_dtype=1, grad_loss=P + 8 * STEP)
    a.update(kw)
    s = domino.DistillArgs(*(a[n] for n, _ in domino.DistillArgs._fields_))
    if call == "forward":
        return L.domino_distill(ctypes.byref(s), a["loss"], a["stats"], a["grad"], a["grad_ld"], a["grad_dtype"], None,
                                None)
    return L.domino_distill_backward(ctypes.byref(s), a["stats"], a["grad_loss"], a["grad"], a["grad_ld"],
                                     a["grad_dtype"], None, None)


BOTH = [dict(rows=0), dict(V=0), dict(ld=1004), dict(ld=992), dict(dtype=5), dict(logits=None), dict(logits=P + 8),
        dict(K=0), dict(K=129), dict(top_ids=None), dict(top_logits=None), dict(temperature=0.0),
        dict(temperature=float("nan")), dict(temperature=2000.0), dict(stats=P + 6 * STEP + 8), dict(grad_ld=996),
        dict(grad_ld=0), dict(grad_dtype=2), dict(grad=P + 7 * STEP + 2), dict(grad=P + 16), dict(grad=P, grad_dtype=0),
        dict(grad=P, grad_ld=1008), dict(grad=P + STEP), dict(grad=P + 2 * STEP), dict(grad=P + 3 * STEP),
        dict(grad=P + 4 * STEP), dict(grad=P + 6 * STEP), dict(top_ids=P + STEP + 2), dict(top_logits=P + 2 * STEP + 1),
        dict(teacher_lse=P + 3 * STEP + 3), dict(row_weights=P + 4 * STEP + 2)]


@pytest.mark.parametrize("bad", BOTH + [dict(loss=None), dict(loss=P), dict(stats=P),
                                        dict(stats=P + 5 * STEP), dict(grad=P + 5 * STEP), dict(loss=P + STEP),
                                        dict(loss=P + 5 * STEP + 2)])
def test_distill_refusals(L, bad):
    assert distill(L, **bad) == domino.ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("bad", BOTH + [dict(stats=None), dict(grad=None), dict(grad=P + 8 * STEP),
                                        dict(grad_loss=P + 8 * STEP + 1)])
def test_distill_backward_refusals(L, bad):
    assert distill(L, "backward", **bad) == domino.ERR_INVALID_ARGUMENT


def test_distill_limits(L):
    assert L.domino_distill(None, P, P, None, 0, 0, None, None) == domino.ERR_INVALID_ARGUMENT
    assert distill(L, rows=(1 << 22) + 1, V=8, ld=8) == domino.ERR_UNSUPPORTED
    assert distill(L, "backward", rows=(1 << 22) + 1, V=8, ld=8) == domino.ERR_UNSUPPORTED


def test_binding_checks_rows():
    ok = torch.zeros(2, 3, 16)
    with pytest.raises(ValueError, match="CUDA"):
        domino.top_logits(ok, 4)
    for bad, msg in ((torch.zeros(16), "at least one row"), (torch.zeros(0, 16), "at least one row"),
                     (torch.zeros(2, 0), "at least one row"), (ok.half(), "has dtype"),
                     (torch.zeros(2, 3, 15), "multiple of 8"), (torch.zeros(16, 2).t(), "contiguous"),
                     (torch.zeros(3, 1, 16).expand(3, 2, 16), "stride"),
                     (torch.zeros(1, 16).expand(2, 16), "stride"),
                     (torch.zeros(4, 8, 16)[:, ::2][:, :3], "fixed stride"),
                     (torch.as_strided(torch.zeros(24), (1, 23), (24, 1), 1), "followed by storage")):
        with pytest.raises(ValueError, match=msg):
            domino.top_logits(bad, 4)
    for k in (0, 129):
        with pytest.raises(ValueError, match="k is"):
            domino.top_logits(ok, k)
    with pytest.raises(TypeError):
        domino.top_logits([[1.0]], 1)


def test_binding_checks_beams():
    z, sc = torch.zeros(2, 3, 16), torch.zeros(2, 3)
    st, hi = torch.zeros(2, 3, 8), torch.zeros(2, 3, 4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        domino.beam_select(z, sc, 2, states=st, history=hi)
    with pytest.raises(ValueError, match="B, W, V"):
        domino.beam_select(z[0], sc[0], 2)
    for kw, msg in ((dict(scores=sc[:, :2].contiguous()), "scores has shape"), (dict(scores=sc.double()), "scores has"),
                    (dict(states=st[:1]), "states has shape"), (dict(states=st[0]), "states must be"),
                    (dict(history=hi.long()), "history has dtype"), (dict(history=hi[0]), "history must be"),
                    (dict(finished=torch.zeros(2, 3, dtype=torch.bool)), "finished has dtype"),
                    (dict(beams=0), "expected 1 to"), (dict(beams=33), "expected 1 to")):
        a = dict(logits=z, scores=sc, beams=2, states=st, history=hi)
        a.update(kw)
        with pytest.raises(ValueError, match=msg):
            domino.beam_select(**a)


def test_binding_checks_distillation():
    z, ids, val = torch.zeros(2, 3, 16), torch.zeros(2, 3, 4, dtype=torch.int32), torch.zeros(2, 3, 4)
    row = torch.zeros(2, 3)
    for call in (domino.distill, domino.distill_loss):
        with pytest.raises(ValueError, match="CUDA"):
            call(z, ids, val, row, 1.0, row)
    with pytest.raises(ValueError, match="stats has shape"):
        domino.distill_backward(z, ids, val, torch.zeros(2, 3, 4))
    for kw, msg in ((dict(top_ids=ids.long()), "top_ids has dtype"), (dict(top_ids=ids[0]), "over the rows"),
                    (dict(top_logits=val[..., :3].contiguous()), "top_logits has shape"),
                    (dict(teacher_lse=row[0]), "teacher_lse has shape"), (dict(row_weights=row.double()), "row_weights"),
                    (dict(top_ids=torch.zeros(2, 3, 129, dtype=torch.int32)), "entries per row")):
        a = dict(logits=z, top_ids=ids, top_logits=val)
        a.update(kw)
        with pytest.raises(ValueError, match=msg):
            domino.distill(**a)
    for name in ("top_logits", "teacher_lse", "row_weights"):
        a = dict(top_logits=val, teacher_lse=row, row_weights=row)
        a[name] = a[name].clone().requires_grad_()
        with pytest.raises(ValueError, match="requires a gradient"):
            domino.distill_loss(z, ids, **a)


def test_the_plain_gradient_is_that_of_the_plain_loss():
    """rows_reference.distill_row against central differences of its own loss (fp64, h = 1e-5: the difference's error is
    about 1e-10)."""
    import numpy as np
    rng = np.random.default_rng(1)
    V = 12
    for lse_on in (False, True):
        t = rng.standard_normal(V) * 2
        ids = np.argsort(-t)[:4].astype(np.int32)
        T = 1.3
        lse = float(np.log(np.exp(t / T).sum())) if lse_on else None
        z = rng.standard_normal(V)
        _, g, _ = R.distill_row(z, ids, t[ids], lse, T, 0.7)
        for v in range(V):
            e = np.zeros(V)
            e[v] = 1e-5
            d = (R.distill_row(z + e, ids, t[ids], lse, T, 0.7)[0] - R.distill_row(z - e, ids, t[ids], lse, T, 0.7)[0]) / 2e-5
            assert abs(d - g[v]) < 1e-8
