"""The calls for candidate continuations as a program makes them: workspaces of its own, several threads, the same call
again; and the scores of a selection against the roundings that it makes."""
import math

import pytest
import torch

from test_gpu_candidates import Tree, check, pkv  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


def test_a_workspace_of_any_shape_counts_by_its_bytes(pkv):  # noqa: F811
    b = Tree(40, [70, 900], [5, 3], 8, 2)
    want, tol = b.expected()
    check(b.run(pkv, workspace=torch.empty(64, 1 << 20, dtype=torch.uint8, device="cuda")), want, tol)
    check(b.run(pkv, workspace=torch.empty(1 << 26, 1, dtype=torch.uint8, device="cuda")), want, tol)
    for small in ((16, 16), (4, 0), (0,)):
        with pytest.raises(pkv.PkvError) as e:
            b.run(pkv, workspace=torch.empty(small, dtype=torch.uint8, device="cuda"))
        assert e.value.status in (pkv.PKV_ERR_NO_MEMORY, pkv.PKV_ERR_INVALID_ARG)
    with pytest.raises(ValueError, match="workspace"):
        b.run(pkv, workspace=torch.zeros((), dtype=torch.uint8, device="cuda"))


def test_threads_with_inputs_of_their_own(pkv):  # noqa: F811
    """Calls from several threads on one stream, each thread with sizes and values of its own: scratch that grows
    meanwhile, or a result handed out twice, would show as another thread's values."""
    import threading
    sizes = [(2, 3, 5000, 6), (1, 4, 60000, 6), (5, 2, 900, 6), (2, 3, 200000, 6)]
    gen = torch.Generator(device="cuda").manual_seed(3)
    inputs = [(torch.randn((n, w, v), generator=gen, device="cuda"), torch.randn((n, w), generator=gen, device="cuda"), k)
              for n, w, v, k in sizes]
    want = [pkv.pkv_beam_select(*i) for i in inputs]
    trees = [Tree(50 + i, [60 + 500 * i, 9], [4, 1 + i], 8, 2) for i in range(4)]
    right = [(t, *t.expected()) for t in trees]
    got, beams, errors = [[] for _ in sizes], [[] for _ in sizes], []
    start = threading.Barrier(len(sizes))

    def work(i):
        try:
            start.wait()
            for _ in range(100):
                beams[i].append(pkv.pkv_beam_select(*inputs[i]))
                if len(beams[i]) % 10 == 0:
                    got[i].append(trees[i].run(pkv))
        except Exception as e:  # noqa: BLE001
            errors.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(sizes))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    pointers = [t.data_ptr() for calls in beams for r in calls for t in r] + [t.data_ptr() for calls in got for t in calls]
    assert len(set(pointers)) == len(pointers) == 4 * (300 + 10)
    for i, (t, w, tol) in enumerate(right):
        assert all(torch.equal(a, b) for r in beams[i] for a, b in zip(r, want[i])), i
        for g in got[i]:
            check(g, w, tol)


@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 128), (torch.float32, 64), (torch.float32, 128)])
def test_trees_repeat_themselves_bit_by_bit(pkv, dtype, d):  # noqa: F811
    """The same batch gives the same bits, whatever ran before and whichever part of a unit is done first."""
    b = Tree(60, [9000, 3, 700, 300, 0, 40], [16, 1, 40, 61, 2, 5], 12, 4, dtype=dtype, d=d)
    first = b.run(pkv)
    for i in range(6):
        Tree(61 + i, [5000], [7 + i], 12, 4, dtype=dtype, d=d).run(pkv)
        assert torch.equal(b.run(pkv), first), i


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,w,v,k", [(3, 4, 1000, 8), (2, 3, 50257, 12), (4, 4, 128256, 8), (1, 1, 1024, 64)])
@pytest.mark.parametrize("spread", [0.1, 3.0, 40.0])
def test_beam_scores_within_the_roundings_of_their_sums(pkv, dtype, n, w, v, k, spread):  # noqa: F811
    """Relative errors of the sum of exponents, in units of 2^-24 (all terms are positive, so they do not grow):
    a lane's 17 additions and the warp's 5; ex2.approx 4; its argument (x - m) log2 e, rounded once, with log2 e in 32
    bits: 1.7 |x - m|, of which the mean over the weights of 1024 values is at most ln 1024 (12); what rounding m log2 e
    left, an exp2f and a product: 5.  Blocks joined: an exp2f and a product, 5, its argument's three roundings
    2.7 |m_b - m|, on average at most ln V; their sum keeps what it rounds off.  The logarithm: 2.  The returned score: half
    a step of itself.  Ranks are not looked at."""
    gen = torch.Generator(device="cuda").manual_seed(v + k)
    x = (torch.randn((n, w, v), generator=gen, device="cuda") * spread).to(dtype)
    cum = -5 * torch.rand((n, w), generator=gen, device="cuda")
    s, p, t = pkv.pkv_beam_select(x, cum, k)
    full = torch.log_softmax(x.double(), -1) + cum.double()[:, :, None]
    want = full.view(n, -1).gather(1, p.long() * v + t.long())
    tol = (50 + 2.7 * math.log(v)) * 2.0**-24 + want.abs() * 2.0**-24
    assert ((s.double() - want).abs() <= tol).all(), float(((s.double() - want).abs() / tol).max())
