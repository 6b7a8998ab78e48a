"""Candidate continuations on the host: the references against independent forms, and every
refusal of the C entries and the binding that needs no GPU."""
import ctypes

import numpy as np
import pytest
import torch

import candidates_ref as ref

P = ctypes.c_void_p
F = P(0x1000)  # never dereferenced: every call below fails its host checks first
G = P(0x200000)
B = ctypes.byref


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_248_gb300 import _build
    _build.build()
    import paged_kv_cache_248_gb300 as m
    m.lib()
    return m


# ----------------------------------------------------------------------------- references
def test_tree_reference_of_a_chain_is_causal_attention():
    rng = np.random.default_rng(0)
    lens, m = np.array([37], np.int32), 5
    qsl = np.array([0, m], np.int32)
    tables, pool = ref.tables_for(rng, lens)
    k, v = (torch.from_numpy(rng.standard_normal((pool, 2, 16, 64)).astype(np.float32)) for _ in "kv")
    q = torch.from_numpy(rng.standard_normal((m, 4, 64)).astype(np.float32))
    mask, depths = ref.tree_mask(np.arange(-1, m - 1), qsl, 1)
    assert depths.tolist() == list(range(m))
    out, _ = ref.tree_attention(q, k, v, tables, lens, qsl, mask, 0.125)
    ids = torch.from_numpy(tables[0, :3].astype(np.int64))
    kd = k[ids].transpose(0, 1).reshape(2, -1, 64)[:, :37].double().repeat_interleave(2, 0)
    vd = v[ids].transpose(0, 1).reshape(2, -1, 64)[:, :37].double().repeat_interleave(2, 0)
    bias = torch.ones(m, 37, dtype=torch.bool).tril(32)
    want = torch.nn.functional.scaled_dot_product_attention(q.double().transpose(0, 1), kd, vd, attn_mask=bias, scale=0.125)
    assert (out - want.transpose(0, 1)).abs().max() < 1e-12


def test_beam_reference_against_log_softmax():
    rng = np.random.default_rng(1)
    x = torch.from_numpy(rng.standard_normal((2, 3, 50)))
    cum = rng.standard_normal((2, 3)).astype(np.float32)
    s, p, t = ref.beam_select(x, cum, 7)
    full = torch.log_softmax(x, -1) + torch.from_numpy(cum).double()[:, :, None]
    top = full.reshape(2, -1).topk(7)
    assert np.allclose(s, top.values.numpy(), atol=1e-12)
    assert np.array_equal(p * 50 + t, top.indices.numpy())


def test_fork_reference_keeps_the_counts():
    tables = np.array([[4, 7, 1, -1], [4, 7, 2, -1], [4, 7, 3, -1]], np.int32)
    refs = np.array([0, 1, 1, 1, 4, 0, 0, 3], np.int32)  # block 4 has one more user
    out, n, after = ref.fork(tables, [40, 40, 40], [1, 1, 0], refs, 1)
    # rows 0 and 1 continue row 1: the first keeps block 2, the second copies it to the lowest free block
    assert out.tolist() == [[4, 7, 2, -1], [4, 7, 0, -1], [4, 7, 1, -1]] and n.tolist() == [40, 40, 40]
    assert after.tolist() == [1, 1, 1, 0, 4, 0, 0, 3]
    assert ref.fork(tables, [48, 48, 48], [0, 0, 0], np.array([1] * 8), 17) is None


# ----------------------------------------------------------------------------- refusals of the C entries
def _desc(pkv, nb=4, bs=16, hkv=2, d=128, dt=1):
    return pkv._CacheDesc(nb, bs, hkv, d, dt)


def test_tree_mask_refusals(pkv):
    L = pkv.lib()
    ok = [F, F, 1, 4, F, 1, None, None]
    for at, bad in ((0, None), (1, None), (2, -1), (2, 0), (3, -1), (4, None), (4, P(0x1004)), (5, 0)):
        args = list(ok)
        args[at] = bad
        assert L.pkv_tree_mask(*args) == pkv.PKV_ERR_INVALID_ARG, (at, bad)
    assert L.pkv_tree_mask(None, None, 0, 0, None, 1, None, None) == pkv.PKV_OK


def test_tree_attention_refusals(pkv):
    L = pkv.lib()
    d = _desc(pkv)
    names = "q k v cache bt max_blocks lens qsl mask words seqs hq tokens max_q max_len scale out ws bytes stream".split()
    ok = dict(zip(names, [F, F, F, B(d), F, 4, F, F, F, 1, 1, 4, 8, 8, 64, 1.0, F, F, 1 << 30, None]))

    def call(**kw):
        a = {**ok, **kw}
        return L.paged_attention_tree(*[a[n] for n in names])

    for kw in (dict(q=None), dict(k=None), dict(v=None), dict(bt=None), dict(lens=None), dict(qsl=None), dict(mask=None),
               dict(out=None), dict(q=P(0x1008)), dict(k=P(0x1008)), dict(v=P(0x1008)), dict(out=P(0x1008)),
               dict(mask=P(0x1004)), dict(max_blocks=0), dict(words=0), dict(words=1, max_q=65), dict(seqs=0),
               dict(seqs=-1), dict(hq=0), dict(hq=3), dict(tokens=-1), dict(max_q=0), dict(max_len=0),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(cache=None), dict(cache=B(_desc(pkv, bs=8)))):
        assert call(**kw) == pkv.PKV_ERR_INVALID_ARG, kw
    for kw in (dict(cache=B(_desc(pkv, d=64))), dict(cache=B(_desc(pkv, d=96, dt=0))), dict(hq=34), dict(tokens=1 << 31),
               dict(seqs=1 << 30)):
        assert call(**kw) == pkv.PKV_ERR_UNSUPPORTED, kw
    assert call(tokens=0) == pkv.PKV_OK


def test_compact_refusals(pkv):
    L = pkv.lib()
    names = "path max_path path_lens bt max_blocks lens qsl seqs k v cache layers new stream".split()
    ok = dict(zip(names, [F, 4, F, F, 4, F, F, 2, F, F, B(_desc(pkv)), 1, G, None]))

    def call(**kw):
        a = {**ok, **kw}
        return L.pkv_compact_path(*[a[n] for n in names])

    for kw in (dict(path=None), dict(max_path=-1), dict(path_lens=None), dict(bt=None), dict(max_blocks=0), dict(lens=None),
               dict(qsl=None), dict(seqs=-1), dict(k=None), dict(v=None), dict(k=P(0x1008)), dict(layers=0), dict(new=None),
               dict(new=F), dict(new=P(0x1004)), dict(layers=65536),
               dict(lens=P(0x500000), path_lens=P(0x600000), new=F)):
        assert call(**kw) == pkv.PKV_ERR_INVALID_ARG, kw
    assert call(cache=B(_desc(pkv, d=64))) == pkv.PKV_ERR_UNSUPPORTED
    assert call(seqs=0) == pkv.PKV_OK


def test_beam_refusals(pkv):
    L = pkv.lib()
    names = "x dtype stride cum fin eos seqs beams vocab select s p t ws bytes stream".split()
    ok = dict(zip(names, [F, 1, 100, F, None, 0, 2, 4, 100, 8, F, F, F, F, 1 << 30, None]))

    def call(**kw):
        a = {**ok, **kw}
        return L.pkv_beam_select(*[a[n] for n in names])

    for kw in (dict(x=None), dict(cum=None), dict(s=None), dict(p=None), dict(t=None), dict(stride=99), dict(seqs=-1),
               dict(beams=0), dict(vocab=0), dict(select=0), dict(fin=F, eos=-1), dict(fin=F, eos=100), dict(x=P(0x1001)),
               dict(x=P(0x1002), dtype=0)):
        assert call(**kw) == pkv.PKV_ERR_INVALID_ARG, kw
    for kw in (dict(dtype=2), dict(beams=65), dict(select=65), dict(beams=64, vocab=1 << 25, stride=1 << 25)):
        assert call(**kw) == pkv.PKV_ERR_UNSUPPORTED, kw
    assert call(seqs=0) == pkv.PKV_OK
    n = ctypes.c_int64(-1)
    assert L.pkv_beam_workspace(0, 4, 100, 8, B(n)) == pkv.PKV_OK and n.value == 0
    assert L.pkv_beam_workspace(2, 4, 100, 8, None) == pkv.PKV_ERR_INVALID_ARG


def test_fork_refusals(pkv):
    L = pkv.lib()
    names = "bt lens rows max_blocks parents new refs out_bt out_lens k v cache layers ws bytes stream".split()
    ok = dict(zip(names, [F, P(0x40000), 4, 8, P(0x50000), 1, P(0x60000), G, P(0x70000), P(0x80000), P(0x90000),
                          B(_desc(pkv)), 1, P(0xa0000), 1 << 20, None]))

    def call(**kw):
        a = {**ok, **kw}
        return L.pkv_fork_tables(*[a[n] for n in names])

    for kw in (dict(bt=None), dict(lens=None), dict(rows=-1), dict(max_blocks=0), dict(parents=None), dict(new=-1),
               dict(refs=None), dict(out_bt=None), dict(out_lens=None), dict(k=None), dict(v=None), dict(layers=0),
               dict(out_bt=F), dict(out_bt=P(0x1010)), dict(out_lens=P(0x40000)), dict(out_lens=P(0x50004)),
               dict(k=P(0x80008))):
        assert call(**kw) == pkv.PKV_ERR_INVALID_ARG, kw
    for kw in (dict(rows=4097), dict(new=65537), dict(cache=B(_desc(pkv, d=64)))):
        assert call(**kw) == pkv.PKV_ERR_UNSUPPORTED, kw
    assert call(rows=0) == pkv.PKV_OK
    n = ctypes.c_int64(0)
    assert L.pkv_fork_workspace(4, B(n)) == pkv.PKV_OK and n.value >= 4 * 13 and n.value % 256 == 0
    assert L.pkv_fork_workspace(-1, B(n)) == pkv.PKV_ERR_INVALID_ARG
    assert L.pkv_fork_workspace(4097, B(n)) == pkv.PKV_ERR_UNSUPPORTED


# ----------------------------------------------------------------------------- refusals of the binding
def test_binding_refuses_shapes_before_any_cuda_call(pkv):
    z = torch.zeros
    i32 = lambda *s: z(s, dtype=torch.int32)  # noqa: E731
    k = z(4, 2, 16, 128, dtype=torch.bfloat16)
    q = z(3, 4, 128, dtype=torch.bfloat16)
    mask = z(3, 1, dtype=torch.int64)
    with pytest.raises(ValueError, match="tree_mask"):
        pkv.paged_attention_tree(q, k, k, i32(1, 4), i32(1), i32(2), mask[:2], 1.0, 3, 8)
    with pytest.raises(ValueError, match="number of requests"):
        pkv.paged_attention_tree(q, k, k, i32(1, 4), i32(1), i32(3), mask, 1.0, 3, 8)
    with pytest.raises(ValueError, match="head_dim"):
        pkv.paged_attention_tree(q[:, :, :64], k, k, i32(1, 4), i32(1), i32(2), mask, 1.0, 3, 8)
    with pytest.raises(ValueError, match="path"):
        pkv.pkv_compact_path(i32(2, 3), i32(1), i32(1, 4), i32(1), i32(2), k, k)
    with pytest.raises(ValueError, match="both be"):
        pkv.pkv_compact_path(i32(1, 3), i32(1), i32(1, 4), i32(1), i32(2), k[None], k)
    x = z(2, 4, 100)
    with pytest.raises(ValueError, match="num_beams"):
        pkv.pkv_beam_select(x[0], z(2, 4), 8)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        pkv.pkv_beam_select(x.half(), z(2, 4), 8)
    with pytest.raises(ValueError, match="contiguous rows"):
        pkv.pkv_beam_select(x.transpose(0, 1), z(4, 2), 8)
    with pytest.raises(ValueError, match="contiguous rows"):
        pkv.pkv_beam_select(x[:, :, ::2], z(2, 4), 8)
    with pytest.raises(ValueError, match="contiguous rows"):
        pkv.pkv_beam_select(x[:, :1].expand(2, 4, 100), z(2, 4), 8)
    for big in ((1, 1, 1 << 31), (1, 1 << 31, 4), (1 << 31, 1, 4)):  # a size must not wrap round to a small one
        with pytest.raises(ValueError, match="32 bits"):
            pkv.pkv_beam_select(z(1).expand(big), z(1, 1), 1)
    wide = torch.zeros(1, 1, dtype=torch.int32).expand(1, (1 << 32) + 4)
    with pytest.raises(ValueError, match="32 bits"):
        pkv.pkv_fork_tables(wide, i32(1), i32(1), i32(4), k, k)
    with pytest.raises(ValueError, match="32 bits"):
        pkv.pkv_compact_path(wide, i32(1), i32(1, 4), i32(1), i32(2), k, k)
    with pytest.raises(ValueError, match="32 bits"):
        pkv.paged_attention_tree(q, k, k, wide, i32(1), i32(2), mask, 1.0, 3, 8)
    with pytest.raises(ValueError, match="cum_scores"):
        pkv.pkv_beam_select(x, z(2, 3), 8)
    with pytest.raises(ValueError, match="finished"):
        pkv.pkv_beam_select(x, z(2, 4), 8, finished=z(2, 3, dtype=torch.bool))
    with pytest.raises(ValueError, match="together"):
        pkv.pkv_fork_tables(i32(2, 4), i32(2), i32(2), i32(4), k, None)
    with pytest.raises(ValueError, match="ref_counts"):
        pkv.pkv_fork_tables(i32(2, 4), i32(2), i32(2), i32(5), k, k)
    with pytest.raises(ValueError, match="parents"):
        pkv.pkv_fork_tables(i32(2, 4), i32(2), i32(3), i32(4), k, k)
