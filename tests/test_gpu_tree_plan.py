"""How drafted trees are cut into runs: any number of row tiles, and requests that bring nothing beside others."""
import numpy as np
import pytest
import torch

from test_gpu_candidates import Tree, check, dev, pkv  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


def expected(b):
    """candidates_ref.tree_attention (values and bounds) for many rows: a request at a time in 64 bits on the GPU."""
    T, hq, d = b.q.shape
    hkv = b.k.shape[1]
    out, tol = (torch.zeros(T, hq, d, dtype=torch.float64, device="cuda") for _ in range(2))
    half = torch.finfo(b.q.dtype).eps / 2
    k_all, v_all = b.k.cuda(), b.v.cuda()
    for i in range(len(b.lens)):
        n, t0, t1 = int(b.lens[i]), int(b.qsl[i]), int(b.qsl[i + 1])
        m = t1 - t0
        ids = dev(b.tables[i, :(n + 15) // 16].astype(np.int64))
        k, v = (x[ids].double().transpose(0, 1).reshape(hkv, -1, d)[:, :n].repeat_interleave(hq // hkv, 0) for x in (k_all, v_all))
        q = b.q[t0:t1].cuda().double().transpose(0, 1)
        words = dev(b.mask[t0:t1].view(np.int64))
        bits = (words[:, :, None] >> torch.arange(64, device="cuda") & 1).bool().flatten(1)[:, :m]
        seen = torch.cat([torch.ones(m, n - m, dtype=torch.bool, device="cuda"), bits], 1)
        s = (q @ k.transpose(1, 2) * b.scale).masked_fill(~seen, -torch.inf)
        p = torch.softmax(s, 2)
        out[t0:t1] = (p @ v).transpose(0, 1)
        size = (q.abs() @ k.abs().transpose(1, 2)).masked_fill(~seen, 0).amax(2) * abs(b.scale)
        rel = 2 * torch.expm1((d + 8) * 2.0**-24 * size) + (2 * n + 64) * 2.0**-24 + 2.0**-8
        tol[t0:t1] = ((rel[:, :, None] * (p @ v.abs())) * (1 + half)).transpose(0, 1) + half * out[t0:t1].abs()
    return out.cpu(), tol.cpu()


def run(m, b, lens, qsl, tables):
    return m.paged_attention_tree(b.q.cuda(), b.k.cuda(), b.v.cuda(), dev(tables), dev(lens.astype(np.int32)),
                                  dev(qsl.astype(np.int32)), dev(b.mask.view(np.int64)), b.scale, b.max_q, int(b.lens.max()))


@pytest.mark.parametrize("seqs,nodes,ctx,hq,hkv", [(3, 40, 5000, 16, 1), (2, 64, 9000, 16, 2), (150, 40, 700, 16, 1)])
def test_empty_requests_do_not_change_the_cut(pkv, seqs, nodes, ctx, hq, hkv):  # noqa: F811
    """Units that go side by side without an empty request do so with it: the same parts, the same bits."""
    b = Tree(seqs + nodes, [ctx + 37 * i for i in range(seqs)], [nodes] * seqs, hq, hkv)
    got = run(pkv, b, b.lens, b.qsl, b.tables)
    check(got, *expected(b))
    for at in (0, seqs // 2, seqs):
        for held in (0, 50):
            with_empty = run(pkv, b, np.insert(b.lens, at, held), np.insert(b.qsl, at, b.qsl[at]), np.insert(b.tables, at, 0, 0))
            assert torch.equal(got, with_empty), (at, held)


@pytest.mark.parametrize("units", [19, 38, 51, 60, 75, 80, 100, 128, 151, 152, 153])
def test_many_units_of_one_request(pkv, units):  # noqa: F811
    """Side by side and one after the other: any number of row tiles that divides the SMs evenly, badly or not at all."""
    b = Tree(units, [600], [units * 16 - 3], 16, 1)
    check(b.run(pkv), *expected(b))
