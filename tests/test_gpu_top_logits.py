"""domino_top_logits on the GPU against a plain fp64 implementation: values and tokens exactly, the log-sum-exp within
the tolerance derived in rows_reference."""
import numpy as np
import pytest
import torch

from draft_block_causal_b200 import domino
from tests import rows_reference as R

pytestmark = pytest.mark.gpu

DT = {"fp32": torch.float32, "bf16": torch.bfloat16}


def check(logits, k, T=1.0):
    """logits [..., V] on the GPU."""
    V = logits.shape[-1]
    values, ids, lse = domino.top_logits(logits, k, temperature=T)
    torch.cuda.synchronize()
    z = logits.double().cpu().numpy().reshape(-1, V)
    want_v, want_i = R.top(z, k)
    np.testing.assert_array_equal(ids.cpu().numpy().reshape(-1, k), want_i)
    np.testing.assert_array_equal(values.double().cpu().numpy().reshape(-1, k), want_v)
    want = R.lse_rows(z, T)
    got = lse.double().cpu().numpy().reshape(-1)
    empty = want == -np.inf
    np.testing.assert_array_equal(got == -np.inf, empty)
    err = np.abs(got[~empty] - want[~empty])
    assert (err <= R.sum_tol(V) + 2.0 ** -23 * np.abs(want[~empty])).all(), err.max()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("rows,V,k", [(1, 1, 1), (3, 7, 9), (2, 8, 8), (5, 100, 128), (4, 1000, 1), (33, 5003, 20),
                                      (2, 16384, 64), (3, 16392, 5), (1, 151936, 8), (7, 151936, 128),
                                      (150, 30001, 33), (320, 20000, 64), (1, 1 << 20, 16), (400, 151936, 10)])
def test_random_rows(rows, V, k, dtype):
    g = torch.Generator().manual_seed(rows * 7 + V)
    z = (torch.randn(rows, V, generator=g) * 2.5).to(DT[dtype])
    check(R.padded(z), k)


@pytest.mark.parametrize("T", [2.0 ** -10, 0.3, 1.7, 1024.0])
def test_temperatures(T):
    z = torch.randn(6, 3001, generator=torch.Generator().manual_seed(5)) * 4
    x = R.padded(z)
    _, _, lse = domino.top_logits(x, 4, temperature=T)
    want = R.lse_rows(z.double().numpy(), T)
    # in units of 1/T the argument c z is rounded at its own size, up to |z| / T * 2^-24 in the exponent
    tol = R.sum_tol(3001) + 2.0 ** -23 * np.abs(want)
    assert (np.abs(lse.double().cpu().numpy() - want) <= tol).all()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("V", [40, 2056, 40003])
@pytest.mark.parametrize("kind", ["constant", "ascending", "descending", "few-levels", "one-thread", "sawtooth",
                                  "zeros-of-both-signs"])
def test_orders_and_ties(kind, V, dtype):
    i = torch.arange(V, dtype=torch.float32)
    z = {"constant": torch.full((V,), -3.5), "ascending": i / 64, "descending": -i / 64, "few-levels": (i * 7919) % 5,
         # every large value in the columns of one 32-byte or 16-byte piece of each 512-piece stretch
         "one-thread": torch.where((i // 8) % 512 == 3, 100.0 + i / V, -i / V),
         "sawtooth": i % 128, "zeros-of-both-signs": torch.where(i % 3 == 1, -0.0, 0.0)}[kind]
    x = R.padded(z.to(DT[dtype]).expand(3, V).contiguous())
    for k in (1, 5, 32, 128):
        check(x, k)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("V", [3001, 70001])
def test_barred_and_unusual_rows(V, dtype):
    g = torch.Generator().manual_seed(11)
    z = torch.randn(12, V, generator=g) * 2
    low = torch.finfo(DT[dtype]).min
    z[0] = -np.inf                       # nothing to select
    z[1] = -np.inf
    z[1, 2999] = 0.25                    # one token
    z[2] = np.nan
    z[3, ::2] = np.nan
    z[4, :] = low                        # a mask of the type's lowest value everywhere: a uniform row
    z[5, 100:] = low
    z[6, 17] = np.inf                    # takes all the mass
    z[7, [5, 9]] = np.inf
    z[8, :] = -np.inf
    z[8, -3:] = torch.tensor([1.0, 1.0, 2.0])
    z[9] = z[9] * 1e6
    z[10, 40:] = -np.inf
    z[11] = np.inf
    check(R.padded(z.to(DT[dtype])), 64)


def test_views_with_row_strides_and_three_dimensions():
    g = torch.Generator().manual_seed(3)
    full = torch.randn(4, 6, 1064, generator=g).cuda()
    check(full[..., :1000], 7)           # a padded vocabulary
    check(full[..., 16:1015], 7)         # a slice of columns
    check(full[:, 2], 7)                 # one position of every block
    check(full[1:2, :, :1001], 7)
    check(full[:1, :1], 7)


def test_given_outputs_repeat_and_rows_do_not_touch_each_other():
    z = (torch.randn(9, 20000, generator=torch.Generator().manual_seed(4)) * 3).bfloat16().cuda()
    a = domino.top_logits(z, 16)
    outs = (torch.full((11, 16), 7.0, device="cuda"), torch.full((11, 16), 7, dtype=torch.int32, device="cuda"),
            torch.full((11,), 7.0, device="cuda"))
    domino.top_logits(z, 16, values_out=outs[0][1:10], ids_out=outs[1][1:10], lse_out=outs[2][1:10])
    for x, y in zip(outs, a):
        assert torch.equal(x[1:10], y) and (x[0] == 7).all() and (x[10] == 7).all()
    one = domino.top_logits(z[4:5], 16)
    for x, y in zip(one[:2], a[:2]):
        assert torch.equal(x[0], y[4])


def test_on_another_stream_and_in_a_graph():
    z = torch.randn(30, 9000, device="cuda")
    want = domino.top_logits(z, 12)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    late = torch.zeros_like(z)
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        late.copy_(z)
    got = domino.top_logits(late, 12, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    buf = torch.zeros_like(z)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = domino.top_logits(buf, 12)
    for x in (z, -z):
        buf.copy_(x)
        graph.replay()
        ref = domino.top_logits(x, 12)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, ref))


def test_offsets_beyond_32_bits():
    rows, V = 16400, 131072  # 2^31 values and more, 4.3 GB
    z = torch.empty(rows, V, dtype=torch.bfloat16, device="cuda").normal_()
    values, ids, lse = domino.top_logits(z, 5)
    torch.cuda.synchronize()
    last = z[-3:].double().cpu().numpy()
    want_v, want_i = R.top(last, 5)
    np.testing.assert_array_equal(ids[-3:].cpu().numpy(), want_i)
    np.testing.assert_array_equal(values[-3:].double().cpu().numpy(), want_v)
    want = R.lse_rows(last, 1.0)
    assert (np.abs(lse[-3:].double().cpu().numpy() - want) <= R.sum_tol(V) + 2.0 ** -23 * np.abs(want)).all()


def test_two_calls_at_once():
    """Calls from two host threads on two streams, of different sizes, give what they give alone."""
    import threading
    jobs = []
    for i, (rows, V, k) in enumerate(((3, 151936, 20), (200, 9000, 64))):
        z = torch.randn(rows, V, generator=torch.Generator().manual_seed(i)).cuda()
        jobs.append((z, k, torch.cuda.Stream(), domino.top_logits(z, k)))
    torch.cuda.synchronize()
    got = [[], []]

    def work(i):
        z, k, s, _ = jobs[i]
        for _ in range(40):
            got[i].append(domino.top_logits(z, k, stream=s))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for i, (_, _, _, want) in enumerate(jobs):
        assert len(got[i]) == 40
        assert all(torch.equal(a, b) for out in got[i] for a, b in zip(out, want))
