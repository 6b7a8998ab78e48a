"""Candidate continuations on the GPU against the 64-bit references: drafted trees over the
paged cache, the accepted path, beam selection and forked tables, each where it can go
wrong, and runs of them together."""
import math

import numpy as np
import pytest
import torch

import candidates_ref as ref

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def pkv():
    import paged_kv_cache_248_gb300 as m
    m.lib()
    assert m.pkv_get_last_error() == 0
    return m


@pytest.fixture(autouse=True)
def no_error_left(pkv):
    yield
    assert pkv.pkv_get_last_error() == 0


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


# ----------------------------------------------------------------------------- drafted trees
class Tree:
    """A batch of drafted trees: host tensors and their device copies."""

    def __init__(self, seed, ctx, nodes, hq, hkv, d=128, dtype=BF, chain=0.5, mask=None, words=None, scale=None):
        rng = np.random.default_rng(seed)
        gen = torch.Generator().manual_seed(seed)
        self.nodes = np.asarray(nodes)
        self.lens = (np.asarray(ctx) + self.nodes).astype(np.int32)
        self.qsl = np.concatenate([[0], np.cumsum(self.nodes)]).astype(np.int32)
        self.tables, pool = ref.tables_for(rng, self.lens, junk=0x7ffffff0)  # what lies behind is not read
        n = lambda *s: torch.randn(s, generator=gen).to(dtype)  # noqa: E731
        self.q, self.k, self.v = n(int(self.qsl[-1]), hq, d), n(pool, hkv, 16, d), n(pool, hkv, 16, d)
        self.max_q = int(max(1, self.nodes.max()))
        words = words or (self.max_q + 63) // 64
        self.parents = np.concatenate([ref.random_parents(rng, int(m), chain) for m in self.nodes] or [[]]).astype(np.int32)
        self.mask = ref.tree_mask(self.parents, self.qsl, words)[0] if mask is None else mask(rng, self, words)
        self.scale = scale if scale is not None else 1 / math.sqrt(d)
        # slots past a request's length hold what a freed block may hold
        for i, n_ in enumerate(self.lens):
            if n_ % 16:
                self.k[self.tables[i, n_ // 16], :, n_ % 16:] = float("nan")
                self.v[self.tables[i, n_ // 16], :, n_ % 16:] = float("inf")

    def run(self, pkv, **kw):
        return pkv.paged_attention_tree(self.q.cuda(), self.k.cuda(), self.v.cuda(), dev(self.tables), dev(self.lens),
                                        dev(self.qsl), dev(self.mask.view(np.int64)), self.scale,
                                        kw.pop("max_q", self.max_q), int(max(1, self.lens.max())), **kw)

    def expected(self):
        return ref.tree_attention(self.q, self.k, self.v, self.tables, self.lens, self.qsl, self.mask, self.scale)


def check(got, want, tol, what=""):
    got = got.double().cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what + ": NaN in other places"
    off = torch.where(torch.isfinite(want), (got - want).abs(), torch.zeros(()).double())
    bad = off > tol
    assert not bad.any(), f"{what}: {int(bad.sum())} values off, worst {float((off - tol).max()):.3e} over its bound, " \
                          f"first at {torch.nonzero(bad)[0].tolist()}"


HEADS = [(32, 8), (8, 8), (12, 4), (16, 1), (14, 2), (5, 1)]


@pytest.mark.parametrize("hq,hkv", HEADS)
def test_tree_head_layouts(pkv, hq, hkv):
    b = Tree(hq, [0, 1, 15, 16, 17, 127, 128, 300], [1, 2, 7, 16, 33, 5, 1, 13], hq, hkv)
    check(b.run(pkv), *b.expected())


@pytest.mark.parametrize("ctx,nodes", [(0, 1), (0, 5), (0, 64), (1, 1), (127, 1), (128, 1), (129, 2), (120, 16), (128, 64),
                                       (500, 65), (700, 130), (37, 200), (2100, 9), (5000, 3)])
def test_tree_lengths(pkv, ctx, nodes):
    b = Tree(ctx + nodes, [ctx], [nodes], 8, 2)
    check(b.run(pkv), *b.expected())


@pytest.mark.parametrize("seqs,nodes,hq,hkv,top", [(3, 64, 16, 1, 9000), (2, 33, 32, 2, 3000), (150, 33, 8, 1, 90),
                                                   (130, 17, 16, 1, 500), (1, 600, 16, 1, 700)])
def test_tree_units_side_by_side(pkv, seqs, nodes, hq, hkv, top):
    """Requests whose kv heads have equally many row tiles, above two: their units go through the keys together."""
    ctx = [(top * (i + 1) // seqs) for i in range(seqs)]
    b = Tree(seqs + nodes, ctx, [nodes] * seqs, hq, hkv)
    check(b.run(pkv), *b.expected())
    mixed = Tree(seqs, ctx + [50], [nodes] * seqs + [1], hq, hkv)  # one that has fewer: one after the other again
    check(mixed.run(pkv), *mixed.expected())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(8, 2), (3, 3), (16, 1), (11, 1)])
def test_tree_fp32(pkv, d, hq, hkv):
    b = Tree(d + hq, [0, 3, 64, 333, 40], [3, 1, 17, 70, 8], hq, hkv, d=d, dtype=F32)
    check(b.run(pkv), *b.expected())


def test_tree_one_token_rows_match_paged_attention(pkv):
    b = Tree(3, [0, 5, 40, 700, 3000], [1, 1, 1, 1, 1], 16, 4)
    got = b.run(pkv)
    check(got, *b.expected())
    plain = pkv.paged_attention(b.q.cuda(), b.k.cuda(), b.v.cuda(), dev(b.tables), dev(b.lens), dev(b.qsl), b.scale, 1,
                                int(b.lens.max()))
    check(plain, *b.expected())


def test_tree_chain_matches_chunked_prefill(pkv):
    b = Tree(4, [100, 0, 260], [20, 9, 40], 8, 2, chain=1.0)
    check(b.run(pkv), *b.expected())
    plain = pkv.paged_attention(b.q.cuda(), b.k.cuda(), b.v.cuda(), dev(b.tables), dev(b.lens), dev(b.qsl), b.scale,
                                b.max_q, int(b.lens.max()))
    check(plain, *b.expected())


@pytest.mark.parametrize("dtype,d,far", [(BF, 128, 0), (BF, 128, 600), (F32, 64, 0)])
def test_tree_any_mask_and_rows_that_see_nothing(pkv, dtype, d, far):
    def mask(rng, b, words):  # any bits at all, bits past the draft among them, and empty rows
        m = rng.integers(0, 1 << 63, (int(b.qsl[-1]), words), dtype=np.uint64)
        m[rng.random(len(m)) < 0.3] = 0
        return m
    b = Tree(5, [0, 0, 33, 130 + far, 0], [40, 1, 70, 20, 100], 8, 2, mask=mask, words=3, dtype=dtype, d=d)
    want, tol = b.expected()
    assert (want == 0).flatten(1).all(1).sum() > 5
    check(b.run(pkv), want, tol)
    # mask words beyond the draft change nothing
    wide = np.concatenate([b.mask, np.full((len(b.mask), 2), (1 << 64) - 1, np.uint64)], 1)
    got = b.run(pkv)
    b.mask = wide
    assert torch.equal(got, b.run(pkv))


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 128)])
@pytest.mark.parametrize("where", ["k", "v", "both"])
def test_tree_nan_and_inf_in_unseen_nodes(pkv, where, dtype, d):
    b = Tree(6, [0, 50, 128, 250, 1000], [6, 16, 64, 30, 3], 8, 2, dtype=dtype, d=d, chain=0.2)
    want, tol = b.expected()
    hit = set()
    rng = np.random.default_rng(9)
    for i in range(5):  # every other node holds what a model that went wrong writes
        for u in range(0, int(b.nodes[i]), 2):
            p = int(b.lens[i] - b.nodes[i]) + u
            for name, x in (("k", b.k), ("v", b.v)):
                if where in (name, "both"):
                    x[b.tables[i, p // 16], :, p % 16] = [float("nan"), float("inf"), -float("inf")][int(rng.integers(3))]
            hit.add((i, u))
    got = b.run(pkv).double().cpu()
    clean = 0
    for i in range(5):
        for j in range(int(b.nodes[i])):
            t = int(b.qsl[i]) + j
            sees = any(int(b.mask[t, u // 64]) >> (u % 64) & 1 for (r, u) in hit if r == i)
            if sees:
                assert not torch.isfinite(got[t]).any(), (i, j)
            else:
                clean += 1
                assert ((got[t] - want[t]).abs() <= tol[t]).all(), (i, j)
    assert clean >= 5


def test_tree_scores_that_are_large_equal_or_infinite(pkv):
    # a scale of 0 gives the mean of the seen values; a negative one and large scores stay right
    for scale in (0.0, -0.2, 3.0):
        b = Tree(7, [0, 70, 300], [4, 9, 40], 8, 2, scale=scale)
        if scale == 3.0:
            b.q[:, 0] *= 20
        check(b.run(pkv), *b.expected(), what=str(scale))


def test_tree_many_requests_of_all_lengths(pkv):
    rng = np.random.default_rng(8)
    n = 400
    b = Tree(8, rng.integers(0, 60, n), rng.integers(1, 5, n), 4, 2)
    check(b.run(pkv), *b.expected())


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 64), (F32, 128)])
def test_tree_split_over_a_long_axis(pkv, dtype, d):
    b = Tree(9, [20000, 3, 9000], [4, 2, 2], 4, 1, dtype=dtype, d=d)
    want, tol = b.expected()
    check(b.run(pkv), want, tol)
    # one part of many: a bad block id makes the request's rows zero, a NaN its rows NaN
    b.tables[2, 300] = -1
    b.k[b.tables[0, 700], :, 5] = float("nan")
    got = b.run(pkv)
    assert pkv.pkv_get_last_error() == pkv.PKV_ERR_INDEX
    assert torch.isnan(got[:4]).all() and (got[6:] == 0).all()
    check(got[4:6], want[4:6], tol[4:6])


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 64)])
def test_tree_bounds_far_above_the_batch(pkv, dtype, d):
    b = Tree(21, [0, 40, 300], [1, 20, 3], 8, 2, dtype=dtype, d=d)
    wide = np.zeros((len(b.mask), 1 << 14), np.uint64)  # room for 2^20 nodes
    wide[:, :b.mask.shape[1]] = b.mask
    for longest in (300, 2**31 - 1):
        got = pkv.paged_attention_tree(b.q.cuda(), b.k.cuda(), b.v.cuda(), dev(b.tables), dev(b.lens), dev(b.qsl),
                                       dev(wide.view(np.int64)), b.scale, 1 << 20, longest)
        check(got, *b.expected())
    assert pkv.pkv_get_last_error() == 0


def test_tree_shared_blocks_and_empty_requests(pkv):
    b = Tree(10, [100, 64, 64, 0], [3, 2, 0, 0], 8, 2)
    b.tables[2] = b.tables[1]                    # a request that brings nothing, on another's blocks
    b.tables[1, :4] = b.tables[0, :4]            # and one that shares a prefix
    check(b.run(pkv), *b.expected())


@pytest.mark.parametrize("dtype,d,more", [(BF, 128, 0), (BF, 128, 130), (F32, 64, 0)])
def test_tree_bad_data_is_flagged_and_zeroed(pkv, dtype, d, more):
    b = Tree(11, [100, 40, 30, 64] + [20] * more, [3, 4, 5, 2] + [2] * more, 8, 2, dtype=dtype, d=d)
    want, tol = b.expected()
    tables, lens = b.tables.copy(), b.lens.copy()
    b.tables[0, 2], b.tables[3, 1] = -1, 10**6    # ids outside of the pool
    b.lens[1] = 2                                 # shorter than its draft
    got = b.run(pkv, out=torch.full(b.q.shape, float("nan"), dtype=dtype, device="cuda"))
    assert pkv.pkv_peek_error_bits() == 0b101
    assert pkv.pkv_get_last_error() == pkv.PKV_ERR_INDEX
    sl = [slice(b.qsl[i], b.qsl[i + 1]) for i in range(4)]
    for i in (0, 1, 3):
        assert (got[sl[i]] == 0).all(), i
    check(got[sl[2]], want[sl[2]], tol[sl[2]])
    b.tables, b.lens = tables, lens
    for wrong in (16 * b.tables.shape[1] + 1, 2**31 - 5):  # more keys than the table has room for
        b.lens[2] = wrong
        got = b.run(pkv)
        assert pkv.pkv_get_last_error() == pkv.PKV_ERR_INDEX
        assert (got[sl[2]] == 0).all()
    b.lens[2] = lens[2]
    got = b.run(pkv, max_q=4)                     # a draft past the caller's bound
    assert pkv.pkv_get_last_error() == pkv.PKV_ERR_INDEX
    assert (got[sl[2]] == 0).all()
    for i in (0, 1, 3):
        check(got[sl[i]], want[sl[i]], tol[sl[i]])


def test_tree_offsets_past_32_bits(pkv):
    # 150000 blocks of 8 heads are 2.5 G values a pool; the requests' blocks sit at its far end
    b = Tree(12, [200, 90], [5, 12], 16, 8)
    far = 150000 - b.k.shape[0]
    k = torch.empty(150000, 8, 16, 128, dtype=BF, device="cuda")
    v = torch.empty_like(k)
    k[far:], v[far:] = b.k.cuda(), b.v.cuda()
    tables = np.where(b.tables < 10**6, b.tables + far, b.tables).astype(np.int32)
    got = pkv.paged_attention_tree(b.q.cuda(), k, v, dev(tables), dev(b.lens), dev(b.qsl), dev(b.mask.view(np.int64)),
                                   b.scale, b.max_q, int(b.lens.max()))
    check(got, *b.expected())


def test_tree_streams_graphs_and_two_calls_at_once(pkv):
    batches = [Tree(20 + i, [50 + 900 * i, 300], [9, 3 + i], 8, 2) for i in range(2)]
    args = [(b.q.cuda(), b.k.cuda(), b.v.cuda(), dev(b.tables), dev(b.lens), dev(b.qsl), dev(b.mask.view(np.int64)),
             b.scale, b.max_q, int(b.lens.max())) for b in batches]
    eager = [pkv.paged_attention_tree(*a) for a in args]
    for b, e in zip(batches, eager):
        check(e, *b.expected())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in batches]
    outs = [torch.empty_like(e) for e in eager]
    for _ in range(20):  # overlapping calls, each with its own scratch
        for s, a, o in zip(streams, args, outs):
            pkv.paged_attention_tree(*a, out=o, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, e) for o, e in zip(outs, eager))
    graphs = []
    for s, a, o in zip(streams, args, outs):
        o.fill_(float("nan"))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            pkv.paged_attention_tree(*a, out=o)
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(20):  # two captured graphs replayed side by side
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, e) for o, e in zip(outs, eager))


def test_tree_rows_behind_the_last_sequence_stay(pkv):
    b = Tree(13, [70], [5], 8, 2)
    out = torch.full((9, 8, 128), 7.0, dtype=BF, device="cuda")
    b.run(pkv, out=out[:5])
    check(out[:5], *b.expected())
    assert (out[5:] == 7).all()


def test_tree_workspace_refusals(pkv):
    b = Tree(14, [70], [5], 8, 2)
    with pytest.raises(pkv.PkvError) as e:
        b.run(pkv, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == pkv.PKV_ERR_NO_MEMORY
    with pytest.raises(pkv.PkvError) as e:
        b.run(pkv, workspace=torch.empty(1 << 28, dtype=torch.uint8, device="cuda")[8:])
    assert e.value.status == pkv.PKV_ERR_INVALID_ARG
    with pytest.raises(ValueError, match="current CUDA device"):
        pkv.paged_attention_tree(b.q, b.k, b.v, torch.from_numpy(b.tables), torch.from_numpy(b.lens),
                                 torch.from_numpy(b.qsl), torch.from_numpy(b.mask.view(np.int64)), 1.0, 5, 80)


# ----------------------------------------------------------------------------- masks
def test_tree_mask(pkv):
    rng = np.random.default_rng(1)
    nodes = [1, 2, 64, 65, 0, 200, 7]
    qsl = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
    parents = np.concatenate([ref.random_parents(rng, m) for m in nodes])
    depths = torch.empty(len(parents), dtype=torch.int32, device="cuda")
    got = pkv.pkv_tree_mask(dev(parents), dev(qsl), 200, depths=depths)
    want, deep = ref.tree_mask(parents, qsl, 4)
    assert np.array_equal(got.cpu().numpy().view(np.uint64), want)
    assert np.array_equal(depths.cpu().numpy(), deep)
    for at, bad in ((3, 5), (10, 7), (0, -2)):  # a later node, the node itself, no node at all
        p = parents.copy()
        p[qsl[2] + at if at else 0] = bad if at != 10 else 10
        got = pkv.pkv_tree_mask(dev(p), dev(qsl), 200, depths=depths)
        assert pkv.pkv_get_last_error() == pkv.PKV_ERR_INDEX
        row = qsl[2] + at if at else 0
        assert (got[row] == 0).all() and depths[row] == 0
    pkv.pkv_tree_mask(dev(parents), dev(qsl), 64)  # the largest draft does not fit its row
    assert pkv.pkv_get_last_error() == pkv.PKV_ERR_INDEX


# ----------------------------------------------------------------------------- accepted path
@pytest.mark.parametrize("layers,hkv,d,dtype", [(1, 8, 128, BF), (3, 2, 128, BF), (2, 3, 64, F32), (2, 1, 128, F32)])
def test_compact_path(pkv, layers, hkv, d, dtype):
    rng = np.random.default_rng(layers)
    nodes = np.array([1, 5, 16, 64, 300, 9, 4, 0])
    ctx = np.array([0, 14, 31, 100, 7, 16, 20, 33])
    lens = (ctx + nodes).astype(np.int32)
    qsl = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
    tables, pool = ref.tables_for(rng, lens)
    shape = (layers, pool, hkv, 16, d) if layers > 1 else (pool, hkv, 16, d)
    k, v = (torch.randn(shape, generator=torch.Generator().manual_seed(s)).to(dtype) for s in (1, 2))
    path = np.full((8, 280), 10**6, np.int32)
    path_lens = np.array([1, 2, 16, 11, 270, 0, 1, 0], np.int32)
    for i in range(8):
        path[i, :path_lens[i]] = np.sort(rng.permutation(nodes[i])[:path_lens[i]])
    path[6, 0] = 3
    lay = lambda x: x if layers > 1 else x[None]  # noqa: E731
    wk, wv, wl = ref.compact(path, path_lens, tables, lens, qsl, lay(k), lay(v))
    kg, vg = k.cuda(), v.cuda()
    got = pkv.pkv_compact_path(dev(path), dev(path_lens), dev(tables), dev(lens), dev(qsl), kg, vg)
    assert got.cpu().numpy().tolist() == wl.tolist()
    assert torch.equal(lay(kg.cpu()), wk) and torch.equal(lay(vg.cpu()), wv)


def test_compact_refuses_bad_paths_and_leaves_their_requests(pkv):
    rng = np.random.default_rng(3)
    nodes = np.full(9, 8)
    lens = np.arange(20, 29).astype(np.int32)
    qsl = (np.arange(10) * 8).astype(np.int32)
    tables, pool = ref.tables_for(rng, lens)
    path = np.tile(np.array([1, 3, 4, 7], np.int32), (9, 1))
    path_lens = np.full(9, 4, np.int32)
    path[1] = [1, 3, 3, 7]        # the same node twice
    path[2] = [3, 1, 4, 7]        # descending
    path[3, 3] = 8                # past the draft
    path[4, 0] = -1
    path_lens[5], path_lens[6] = 5, -1
    tables[7, 1] = pool           # no such block
    lens2 = lens.copy()
    lens2[8] = 3                  # shorter than its draft
    good = np.array([True] + [False] * 8)
    k = torch.randn(pool, 2, 16, 128).to(BF)
    v = torch.randn(pool, 2, 16, 128).to(BF)
    wk, wv, wl = ref.compact(path, np.where(good, path_lens, 0), tables, lens, qsl, k[None], v[None])
    kg, vg = k.cuda(), v.cuda()
    got = pkv.pkv_compact_path(dev(path), dev(path_lens), dev(tables), dev(lens2), dev(qsl), kg, vg)
    assert pkv.pkv_peek_error_bits() == 0b101
    assert pkv.pkv_get_last_error() == pkv.PKV_ERR_INDEX
    assert got.cpu().numpy().tolist() == np.where(good, wl, lens2).tolist()
    assert torch.equal(kg.cpu()[None], wk) and torch.equal(vg.cpu()[None], wv)
    # no paths at all, and no requests
    none = pkv.pkv_compact_path(dev(path[:, :0]), dev(path_lens * 0), dev(tables), dev(lens), dev(qsl), kg, vg)
    assert none.cpu().numpy().tolist() == (lens - nodes).tolist()
    z = torch.zeros(0, dtype=torch.int32, device="cuda")
    assert pkv.pkv_compact_path(z.view(0, 4), z, z.view(0, 4), z, dev(np.zeros(1, np.int32)), kg, vg).numel() == 0


# ----------------------------------------------------------------------------- beams
def beams_equal(pkv, x, cum, k, finished=None, eos=0, call=None):
    """Ranks, and scores within the sums' rounding: the kernel adds V exponents in 32 bits, as
    partial sums of at most 32 terms a thread and chunk, each off by half a step, over at most
    V / 8192 + 1 chunks and 256 threads' joins; (64 + V / 8192) 2^-23 on the sum bounds that, which
    is the same on its logarithm, plus half a step of the returned score."""
    want = ref.beam_select(x.cpu(), cum.cpu(), k, None if finished is None else finished.cpu(), eos)
    got = (call or pkv.pkv_beam_select)(x, cum, k, finished=finished, eos_token=eos)
    s, p, t = (a.cpu().numpy() for a in got)
    assert np.array_equal(p, want[1]), np.argwhere(p != want[1])[:4]
    assert np.array_equal(t, want[2]), np.argwhere(t != want[2])[:4]
    live = np.isfinite(want[0])
    assert np.array_equal(np.isfinite(s), live) and (s[~live] == -np.inf).all()
    tol = (64 + x.shape[2] / 8192) * 2.0**-23 + np.abs(want[0][live]) * 2.0**-24
    assert (np.abs(s[live] - want[0][live]) <= tol).all()
    return got


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,w,v,k", [(1, 1, 1, 1), (1, 1, 5, 5), (2, 3, 7, 21), (1, 4, 1000, 8), (5, 2, 8191, 4), (3, 4, 8192, 64),
                                     (2, 16, 8193, 33), (1, 4, 32000, 8), (3, 5, 50257, 10), (1, 64, 4097, 64),
                                     (70, 8, 2000, 16), (2, 2, 300001, 7)])
def test_beam_sizes(pkv, dtype, n, w, v, k):
    gen = torch.Generator(device="cuda").manual_seed(v + k)
    x = (torch.randn((n, w, v), generator=gen, device="cuda") * 3).to(dtype)
    cum = -5 * torch.rand((n, w), generator=gen, device="cuda")
    beams_equal(pkv, x, cum, k)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("v", [4096, 5001, 40000])
def test_beam_ties_sorted_and_equal_logits(pkv, dtype, v):
    cum = torch.zeros(1, 3, device="cuda")
    flat = torch.zeros(1, 3, v, device="cuda", dtype=dtype)
    got = beams_equal(pkv, flat, cum, 64)                     # all candidates equal: in order of their index
    assert got[2].cpu().tolist() == [list(range(64))]
    up = torch.arange(v, device="cuda").float().expand(1, 3, v) * 1e-3
    beams_equal(pkv, up.to(dtype).contiguous(), cum, 64)      # rising: the last is the best
    beams_equal(pkv, (-up).to(dtype).contiguous(), cum, 64)
    few = torch.full((1, 3, v), -float("inf"), device="cuda", dtype=dtype)
    few[:, 1, 17], few[:, 2, v - 1], few[:, 1, v // 2] = 1.0, 0.5, 1.0
    beams_equal(pkv, few, cum, 8)                             # masked: candidates run out
    beams_equal(pkv, few[:, :1].contiguous(), cum[:, :1].contiguous(), 4)
    lowest = torch.full((1, 3, v), torch.finfo(dtype).min, device="cuda", dtype=dtype)
    lowest[:, 1, 9] = 2.0
    beams_equal(pkv, lowest, cum, 12)                         # masks of the type's lowest value
    twin = torch.randn(1, 1, v, device="cuda").to(dtype).expand(1, 3, v).contiguous()
    beams_equal(pkv, twin, cum, 16)                           # beams alike: ties go to the lower beam


def test_beam_values_that_are_not_finite(pkv):
    x = torch.randn(2, 4, 9000, device="cuda")
    x[0, 1, 5], x[0, 2, 8500], x[1, 3, 0] = float("nan"), float("inf"), float("nan")
    x[1, 0] = float("nan")
    x[1, 1] = -float("inf")
    x[1, 2, ::3] = -float("inf")
    x[0, 0, 3] = -0.0
    x[0, 0, 2] = 0.0
    cum = torch.zeros(2, 4, device="cuda")
    beams_equal(pkv, x, cum, 20)
    cum[0, 0], cum[1, 2] = -float("inf"), float("nan")       # a first step: one beam is alive
    beams_equal(pkv, x, cum, 20)


def test_beam_finished_beams(pkv):
    x = torch.randn(3, 4, 700, device="cuda")
    cum = torch.tensor([[-1.0, -2, -3, -4], [-1, -20, -3, -4], [-5, -5, -5, -5]], device="cuda")
    fin = torch.tensor([[1, 0, 1, 0], [0, 1, 0, 0], [1, 1, 1, 1]], device="cuda").bool()
    beams_equal(pkv, x, cum, 9, finished=fin, eos=699)
    beams_equal(pkv, x, cum, 9, finished=fin.to(torch.uint8) * 2, eos=0)


def test_beam_strided_rows_streams_and_graphs(pkv):
    pad = torch.randn(4, 3, 1031, device="cuda").to(BF)
    cum = torch.randn(4, 3, device="cuda")
    for cut in (1031, 1024, 1000, 1):
        beams_equal(pkv, pad[:, :, :cut], cum, min(16, 3 * cut))   # a slice of a padded vocabulary
    beams_equal(pkv, pad[:, :, 7:], cum, 16)
    beams_equal(pkv, pad[1:2, :1, 3:], cum[1:2, :1].contiguous(), 16)
    want = pkv.pkv_beam_select(pad, cum, 12)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = tuple(torch.empty_like(t) for t in want)
    pkv.pkv_beam_select(pad, cum, 12, out=out, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    for t in out:
        t.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkv.pkv_beam_select(pad, cum, 12, out=out)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))


# ----------------------------------------------------------------------------- forked tables
def fork_case(seed, rows, prompt, tails, blocks=None, slack=50, holders=0):
    """Rows that share `prompt` tokens' full blocks and hold their own tails, their counts (with
    `holders` other users of the shared blocks) and a pool."""
    rng = np.random.default_rng(seed)
    lens = (prompt + np.resize(tails, rows)).astype(np.int32)
    shared = prompt // 16
    held = (lens + 15) // 16
    pool = blocks or int(shared + (held - shared).sum() + slack)
    ids = rng.permutation(pool).astype(np.int32)
    tables = np.full((rows, int(held.max()) + 3), -1, np.int32)
    at = shared
    for b in range(rows):
        tables[b, :shared] = ids[:shared]
        tables[b, shared:held[b]] = ids[at:at + held[b] - shared]
        at += held[b] - shared
    refs = np.bincount(tables[tables >= 0], minlength=pool).astype(np.int32)
    refs[ids[:shared]] += holders
    return rng, tables, lens, refs


def run_fork(pkv, tables, lens, parents, refs, new, layers=1, hkv=2, d=128, dtype=BF, caches=True, **kw):
    pool = len(refs)
    shape = (layers, pool, hkv, 16, d)
    k, v = (torch.randn(shape, generator=torch.Generator().manual_seed(s)).to(dtype) for s in (3, 4))
    kg, vg = (k.cuda(), v.cuda()) if caches else (None, None)
    rg = dev(refs)
    out = pkv.pkv_fork_tables(dev(tables), dev(lens), dev(np.asarray(parents, np.int32)), rg,
                              kg if layers > 1 or not caches else kg[0], vg if layers > 1 or not caches else vg[0],
                              new_tokens=new, **kw)

    def copy_block(dst, src):
        k[:, dst], v[:, dst] = k[:, src], v[:, src]
    want = ref.fork(tables, lens, parents, refs, new, copy_block)
    return out, rg, want, (kg, vg, k, v)


@pytest.mark.parametrize("rows,prompt,new,layers,hkv,d,dtype", [
    (1, 5, 1, 1, 2, 128, BF), (4, 64, 1, 1, 8, 128, BF), (5, 100, 1, 3, 2, 64, F32), (33, 40, 20, 2, 1, 128, BF),
    (8, 0, 1, 1, 2, 128, F32), (700, 32, 1, 1, 1, 128, BF), (12, 16, 0, 1, 2, 128, BF),
    (32, 300, 3, 1, 1, 128, BF), (6, 2200, 2, 1, 1, 128, BF), (2300, 4, 1, 1, 1, 64, F32)])
def test_fork(pkv, rows, prompt, new, layers, hkv, d, dtype):
    rng, tables, lens, refs = fork_case(rows, rows, prompt, [3, 16, 21, 0, 32, 15, 1], slack=rows * 5 + 20)
    for parents in (np.arange(rows), rng.integers(0, rows, rows), np.zeros(rows, int),
                    np.where(rng.random(rows) < 0.4, -1, rng.integers(0, rows, rows)), np.full(rows, -1)):
        (t, n), rg, want, (kg, vg, k, v) = run_fork(pkv, tables, lens, parents, refs, new, layers, hkv, d, dtype)
        assert pkv.pkv_get_last_error() == 0
        assert np.array_equal(t.cpu().numpy(), want[0]) and np.array_equal(n.cpu().numpy(), want[1])
        assert np.array_equal(rg.cpu().numpy(), want[2])
        assert torch.equal(kg.cpu(), k) and torch.equal(vg.cpu(), v)


def test_fork_other_holders_and_reserved_blocks(pkv):
    rng, tables, lens, refs = fork_case(3, 6, 40, [5, 5, 5, 9, 9, 30], holders=2)
    refs[tables[0, (lens[0] - 1) // 16]] += 1             # a prefix cache holds row 0's last block too
    for b in (1, 3):                                      # rows that reserved a block ahead
        free = int(np.flatnonzero(refs == 0)[-1 - b])
        tables[b, (lens[b] + 15) // 16] = free
        refs[free] = 1
    for parents in ([0, 0, 1, 1, 3, 5], [5, 4, 3, 2, 1, 0], [1, 1, 1, 1, 1, 1]):
        for new in (0, 1, 17):
            (t, n), rg, want, _ = run_fork(pkv, tables, lens, parents, refs, new)
            assert np.array_equal(t.cpu().numpy(), want[0]) and np.array_equal(rg.cpu().numpy(), want[2])


def test_fork_a_large_pool_and_tables_alone(pkv):
    rng, tables, lens, refs = fork_case(4, 64, 160, [7, 20, 33], blocks=150000)
    refs[:140000] = np.maximum(refs[:140000], 1)           # nearly everything is in use
    parents = rng.integers(0, 64, 64)
    (t, n), rg, want, _ = run_fork(pkv, tables, lens, parents, refs, 40, caches=False)
    assert np.array_equal(t.cpu().numpy(), want[0]) and np.array_equal(rg.cpu().numpy(), want[2])


@pytest.mark.parametrize("rows", [6, 40])
def test_fork_errors_change_nothing(pkv, rows):
    rng, tables, lens, refs = fork_case(5, rows, 40, [5, 9, 30], slack=3)
    bad_table, bad_len, long_len = tables.copy(), lens.copy(), lens.copy()
    bad_table[2, 1] = -1
    big_table = tables.copy()
    big_table[4, 0] = len(refs)
    bad_len[1] = -1
    long_len[0] = tables.shape[1] * 16 + 1
    rest = list(range(6, rows))
    ok = np.array([0, 0, 1, 3, 3, 5] + rest)
    for what, (tb, ln, par, new, status) in {
            "pool": (tables, lens, ok, 40, pkv.PKV_ERR_NO_MEMORY),
            "parent": (tables, lens, np.array([0, 0, rows, 3, 3, 5] + rest), 1, pkv.PKV_ERR_INDEX),
            "parent below": (tables, lens, np.array([0, -2, 1, 3, 3, 5] + rest), 1, pkv.PKV_ERR_INDEX),
            "hole": (bad_table, lens, ok, 1, pkv.PKV_ERR_INDEX), "id": (big_table, lens, ok, 1, pkv.PKV_ERR_INDEX),
            "length": (tables, bad_len, ok, 1, pkv.PKV_ERR_INDEX), "too long": (tables, long_len, ok, 1, pkv.PKV_ERR_INDEX),
            "no room in the row": (tables, lens, ok, 1000, pkv.PKV_ERR_INDEX)}.items():
        k = torch.randn(len(refs), 2, 16, 128).to(BF)
        kg, vg, rg = k.cuda(), k.cuda(), dev(refs)
        t, n = pkv.pkv_fork_tables(dev(tb), dev(ln), dev(par.astype(np.int32)), rg, kg, vg, new_tokens=new)
        assert pkv.pkv_get_last_error() == status, what
        assert np.array_equal(t.cpu().numpy(), tb) and np.array_equal(n.cpu().numpy(), ln), what
        assert np.array_equal(rg.cpu().numpy(), refs) and torch.equal(kg.cpu(), k) and torch.equal(vg.cpu(), k), what


def test_fork_replays_from_a_graph(pkv):
    rng, tables, lens, refs = fork_case(6, 8, 40, [5, 9, 30])
    parents = np.array([0, 0, 1, 3, 3, 5, 7, 7], np.int32)
    k = torch.randn(len(refs), 2, 16, 128).to(BF).cuda()
    t0, l0, par, r0 = dev(tables), dev(lens), dev(parents), dev(refs)
    r1, k1 = r0.clone(), k.clone()
    want = pkv.pkv_fork_tables(t0, l0, par, r1, k1, k1.clone())
    r2, k2, v2 = r0.clone(), k.clone(), k.clone()
    out = (torch.empty_like(t0), torch.empty_like(l0))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkv.pkv_fork_tables(t0, l0, par, r2, k2, v2, out=out)
    assert torch.equal(r2, r0)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1]) and torch.equal(r2, r1) and torch.equal(k2, k1)


# ----------------------------------------------------------------------------- runs of them together
def test_draft_verify_and_go_on(pkv):
    """Three steps of drafting: masks from the parents, the draft's K/V written, attention over the
    tree, a path kept, the cache compacted, and plain attention over what is left, against the
    kept tokens alone in a cache that never saw a draft."""
    rng = np.random.default_rng(0)
    S, hq, hkv, d = 5, 8, 2, 128
    n = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).to(BF)  # noqa: E731
    lens = rng.integers(3, 90, S).astype(np.int32)
    tables, pool = ref.tables_for(rng, lens + 80)
    k, v = n(pool, hkv, 16, d), n(pool, hkv, 16, d)
    kg, vg, tg = k.cuda(), v.cuda(), dev(tables)
    for step in range(3):
        nodes = rng.integers(1, 14, S)
        qsl = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
        parents = np.concatenate([ref.random_parents(rng, m) for m in nodes])
        q, kn, vn = n(qsl[-1], hq, d), n(qsl[-1], hkv, d), n(qsl[-1], hkv, d)
        full = (lens + nodes).astype(np.int32)
        lg, qg = dev(full), dev(qsl)
        mask = pkv.pkv_tree_mask(dev(parents), qg, int(nodes.max()))
        slots = pkv.pkv_slot_mapping(tg, lg, qg, int(qsl[-1]))
        pkv.pkv_write(kn.cuda(), vn.cuda(), slots, kg, vg)
        got = pkv.paged_attention_tree(q.cuda(), kg, vg, tg, lg, qg, mask, 0.1, int(nodes.max()), int(full.max()))
        for i in range(S):  # the same on the host
            for j in range(nodes[i]):
                p = lens[i] + j
                k[tables[i, p // 16], :, p % 16] = kn[qsl[i] + j]
                v[tables[i, p // 16], :, p % 16] = vn[qsl[i] + j]
        hm, _ = ref.tree_mask(parents, qsl, mask.shape[1])
        check(got, *ref.tree_attention(q, k, v, tables, full, qsl, hm, 0.1), what=f"step {step}")
        path = np.full((S, int(nodes.max())), -1, np.int32)
        path_lens = np.zeros(S, np.int32)
        for i in range(S):  # a random node and its ancestors are kept
            u, chain = int(rng.integers(nodes[i])), []
            while u >= 0:
                chain.append(u)
                u = parents[qsl[i] + u]
            path_lens[i] = len(chain)
            path[i, :len(chain)] = chain[::-1]
        new = pkv.pkv_compact_path(dev(path), dev(path_lens), tg, lg, qg, kg, vg)
        kk, vv, after = ref.compact(path, path_lens, tables, full, qsl, k[None], v[None])
        k, v, lens = kk[0], vv[0], after
        assert new.cpu().numpy().tolist() == lens.tolist()
        q1 = n(S, hq, d)
        one = np.arange(S + 1).astype(np.int32)
        got = pkv.paged_attention(q1.cuda(), kg, vg, tg, new, dev(one), 0.1, 1, int(lens.max()))
        ones = np.ones((S, 1), np.uint64)
        check(got, *ref.tree_attention(q1, k, v, tables, lens, one, ones, 0.1), what=f"after step {step}")
    assert pkv.pkv_get_last_error() == 0


def test_beam_search_over_the_paged_cache(pkv):
    """Beam search of a small recurrent-free model (its logits are its attention output times a
    matrix, its K, V and q rows of a table) through selection, fork and the fused step, against
    the same search on whole sequences in 64 bits."""
    rng = np.random.default_rng(2)
    N, W, V, hq, hkv, d, steps = 3, 4, 211, 4, 2, 128, 20
    R = N * W
    n = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32))  # noqa: E731
    qt, kt, vt = n(V, hq, d) * 0.6, n(V, hkv, d), n(V, hkv, d)
    head = n(hq * d, V) * 0.4
    prompts = [list(rng.integers(0, V, m)) for m in (21, 16, 5)]
    pool = 200
    kc, vc = torch.zeros(pool, hkv, 16, d, device="cuda"), torch.zeros(pool, hkv, 16, d, device="cuda")
    qg, kg, vg, hg = qt.cuda(), kt.cuda(), vt.cuda(), head.cuda()

    def attend(seq):  # the last token's output over its sequence, in 64 bits
        q, k, v = qt[seq[-1]].double(), kt[seq].double(), vt[seq].double()
        o = []
        for h in range(hq):
            g = h * hkv // hq
            o.append(torch.softmax(k[:, g] @ q[h] * 0.1, 0) @ v[:, g])
        return torch.cat(o) @ head.double()

    # the prompts once, in blocks that the beams of a request share
    tables = np.full((R, 6), -1, np.int32)
    refs = np.zeros(pool, np.int32)
    at = 0
    for i, p in enumerate(prompts):
        blocks = (len(p) + 15) // 16
        for w in range(W):
            tables[i * W + w, :blocks] = np.arange(at, at + blocks)
        refs[at:at + blocks] += W
        at += blocks
    lens = np.array([len(prompts[i // W]) for i in range(R)], np.int32)
    toks = np.concatenate(prompts)
    qsl = np.concatenate([[0], np.cumsum([len(p) for p in prompts])]).astype(np.int32)
    tg = dev(tables)
    slots = pkv.pkv_slot_mapping(tg[::W].contiguous(), dev(lens[::W].copy()), dev(qsl), len(toks))
    pkv.pkv_write(kg[toks], vg[toks], slots, kc, vc)
    lg, rg = dev(lens), dev(refs)
    logits = torch.stack([attend(p) for p in prompts]).float().cuda()[:, None].expand(N, W, V).contiguous()
    cum = torch.full((N, W), -float("inf"), device="cuda")
    cum[:, 0] = 0
    one = dev(np.arange(R + 1).astype(np.int32))
    base = torch.arange(N, device="cuda", dtype=torch.int32)[:, None] * W
    # the same search on whole sequences
    want = [[(0.0, p)] for p in prompts]
    seqs = [[list(p) for _ in range(W)] for p in prompts]
    for step in range(steps):
        cum, par, tok = pkv.pkv_beam_select(logits, cum, W)
        tg, lg = pkv.pkv_fork_tables(tg, lg, (base + par).view(-1), rg, kc, vc)
        t = tok.view(-1).long()
        lg = lg + 1
        out = pkv.paged_attention_step(qg[t], kg[t], vg[t], kc, vc, tg, lg, one, 0.1, 1, 96)
        logits = (out.view(R, hq * d) @ hg).view(N, W, V)
        pn, tn = par.cpu().numpy(), tok.cpu().numpy()
        for i in range(N):
            grown = []
            for s, seq in want[i]:
                lp = torch.log_softmax(attend(seq), 0)
                grown += [(s + float(lp[x]), seq + [x]) for x in range(V)]
            grown.sort(key=lambda c: -c[0])
            want[i] = grown[:W]
            seqs[i] = [seqs[i][pn[i, w]] + [int(tn[i, w])] for w in range(W)]
    assert pkv.pkv_get_last_error() == 0
    for i in range(N):
        assert [list(map(int, s)) for _, s in want[i]] == [list(map(int, s)) for s in seqs[i]], i
        # scores of 20 steps, each off by the fp32 logits: 512 products of size up to 20 in 32 bits
        assert np.allclose([s for s, _ in want[i]], cum[i].cpu().numpy(), atol=steps * 512 * 2.0**-24 * 20)
    # every block is held by as many rows as name it
    t = tg.cpu().numpy()
    assert np.array_equal(np.bincount(t[t >= 0], minlength=pool), rg.cpu().numpy())


def test_results_are_handed_out_once_and_scratch_is_per_stream(pkv):
    """Small results come from a store of ready parts and scratch is kept per stream: results of many
    calls stay distinct, and calls on several streams at once do not disturb one another."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    xs = [torch.randn((2, 3, 5000), generator=gen, device="cuda") for _ in range(4)]
    cum = torch.randn((2, 3), generator=gen, device="cuda")
    want = [pkv.pkv_beam_select(x, cum, 6) for x in xs]
    flat = [t for w in want for t in w]
    spans = sorted((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in flat)
    assert all(a[1] <= b[0] for a, b in zip(spans, spans[1:]))
    many = [pkv.pkv_beam_select(xs[i % 4], cum, 6) for i in range(100)]
    assert len({t.data_ptr() for m in many for t in m}) == 300
    for i, m in enumerate(many):
        assert all(torch.equal(a, b) for a, b in zip(m, want[i % 4]))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [[] for _ in xs]
    for _ in range(50):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(pkv.pkv_beam_select(xs[i], cum, 6))
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(torch.equal(a, b) for m in g for a, b in zip(m, w))
    # a graph keeps its own memory: replays after other calls, and the other way round
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = pkv.pkv_beam_select(xs[0], cum, 6)
    for _ in range(3):
        others = [pkv.pkv_beam_select(xs[1], cum, 6) for _ in range(40)]
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want[0]))
        assert all(torch.equal(a, b) for m in others for a, b in zip(m, want[1]))


def test_small_results_are_tensors_of_their_own(pkv):
    """Results are made many at a time, but share neither memory nor versions (a change in place of one must not
    spoil what another was saved for) nor inference mode."""
    x, cum = torch.randn(2, 3, 500, device="cuda"), torch.zeros(2, 3, device="cuda")
    with torch.inference_mode():
        pkv.pkv_beam_select(x, cum, 5)
    w = torch.ones(2, 5, device="cuda", requires_grad=True)
    a = pkv.pkv_beam_select(x, cum, 5)
    b = pkv.pkv_beam_select(x, cum, 5)
    assert not a[0].is_inference()
    loss = (a[0] * w).sum() + torch.gather(w, 1, (a[2] % 5).long()).sum()
    want = a[0].clone()
    for t in b:
        t.add_(1)
    loss.backward()
    assert torch.equal(w.grad, want + torch.zeros_like(w).scatter_add_(1, (a[2] % 5).long(), torch.ones_like(w)))
    a[0].add_(w)  # and may be changed like any other
    assert a[0].requires_grad


def test_calls_from_several_threads(pkv):
    import threading
    x = torch.randn(2, 3, 5000, device="cuda")
    cum = torch.randn(2, 3, device="cuda")
    want = pkv.pkv_beam_select(x, cum, 6)
    bad = []

    def work():
        for _ in range(200):  # all on one stream
            got = pkv.pkv_beam_select(x, cum, 6)
            if not all(torch.equal(a, b) for a, b in zip(got, want)):
                bad.append(1)
    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
