"""Calls on a named stream beside unrelated work of the current one, which still reads memory that the allocator
has back already: neither may find the other's values."""
import numpy as np
import pytest
import torch

import candidates_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    import paged_kv_cache_248_gb300 as m
    m.lib()
    assert m.pkv_get_last_error() == 0
    return m


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def calls(pkv):
    """{name: (call, bytes of the scratch that it asks for)}; every call returns tensors."""
    import ctypes
    rng = np.random.default_rng(0)
    lens = np.array([3000, 40, 700], np.int32)
    qsl = np.array([0, 16, 20, 60], np.int32)
    tables, pool = ref.tables_for(rng, lens)
    parents = np.concatenate([ref.random_parents(rng, m) for m in (16, 4, 40)])
    q = torch.randn(60, 16, 128, device="cuda").bfloat16()
    k, v = (torch.randn(pool, 4, 16, 128, device="cuda").bfloat16() for _ in "kv")
    bt, ln, qs, par = dev(tables), dev(lens), dev(qsl), dev(parents)
    mask = pkv.pkv_tree_mask(par, qs, 40)
    x, cum = torch.randn(4, 8, 100000, device="cuda"), torch.randn(4, 8, device="cuda")
    rows = 512
    ft = np.arange(rows * 8, dtype=np.int32).reshape(rows, 8)
    fl, fp = np.full(rows, 120, np.int32), np.repeat(np.arange(rows // 2, dtype=np.int32), 2)
    refs0 = np.concatenate([np.ones(rows * 8, np.int32), np.zeros(rows, np.int32)])
    ftd, fld, fpd, r0 = dev(ft), dev(fl), dev(fp), dev(refs0)

    def fork(stream=None, refs=None):
        assert stream is None or refs is not None  # (a count made here would be the current stream's)
        return pkv.pkv_fork_tables(ftd, fld, fpd, refs if refs is not None else r0.clone(), None, None, stream=stream)

    n = ctypes.c_int64(0)
    desc = pkv._cache_desc(k, v)
    assert pkv.lib().pkv_tree_workspace(ctypes.byref(desc), 16, 40, ctypes.byref(n)) == 0
    tree_bytes = n.value
    assert pkv.lib().pkv_beam_workspace(4, 8, 100000, 8, ctypes.byref(n)) == 0
    return {"tree": (lambda **kw: (pkv.paged_attention_tree(q, k, v, bt, ln, qs, mask, 0.1, 40, 3000, **kw),), tree_bytes),
            "mask": (lambda **kw: (pkv.pkv_tree_mask(par, qs, 40, **kw),), 512),
            "beam": (lambda **kw: pkv.pkv_beam_select(x, cum, 8, **kw), n.value),
            "fork": (fork, rows * 12 + 4),
            "attention": (lambda **kw: (pkv.paged_attention(q, k, v, bt, ln, qs, 0.1, 40, 3000, **kw),), q.numel() * 2)}


def test_named_streams_beside_work_of_the_current_one(pkv):
    table = calls(pkv)
    for name, (call, scratch) in table.items():
        want = call()
        torch.cuda.synchronize()
        for size in {scratch, *(t.numel() * t.element_size() for t in want)}:
            side = torch.cuda.Stream()
            extra = {"refs": torch.cat([torch.ones(4096), torch.zeros(512)]).int().cuda()} if name == "fork" else {}
            side.wait_stream(torch.cuda.current_stream())
            temporary = torch.full((max(1, size // 4),), 3.0, device="cuda")
            torch.cuda._sleep(10_000_000)  # a few milliseconds: what follows runs after the call on the other stream
            doubled = temporary * 2
            lo, hi = temporary.data_ptr(), temporary.data_ptr() + temporary.numel() * 4
            del temporary
            got = call(stream=side, **extra)
            assert not any(lo <= t.data_ptr() < hi for t in got), name
            torch.cuda.synchronize()
            assert (doubled == 6).all(), name
            assert all(torch.equal(a, b) for a, b in zip(got, want)), name
    assert pkv.pkv_get_last_error() == 0


def test_results_of_a_named_stream_outlive_their_use_on_the_current_one(pkv):
    """A result is dropped while the current stream still has to read it: later calls on its stream leave it alone."""
    table = calls(pkv)
    call, _ = table["tree"]
    want = call()[0].float().sum(0)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = call(stream=side)[0]
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(10_000_000)
    total = got.float().sum(0)
    del got
    for _ in range(4):
        other = torch.empty(0)
        with torch.cuda.stream(side):
            other = torch.full((60, 16, 128), 9.0, dtype=torch.bfloat16, device="cuda")
        del other
    torch.cuda.synchronize()
    assert torch.equal(total, want)


def test_streams_of_another_library(pkv):
    """Anything that tells a stream's handle names it."""
    import types
    side = torch.cuda.Stream()
    for name, (call, _) in calls(pkv).items():
        want = call()
        torch.cuda.synchronize()
        extra = {"refs": torch.cat([torch.ones(4096), torch.zeros(512)]).int().cuda()} if name == "fork" else {}
        torch.cuda.synchronize()
        got = call(stream=types.SimpleNamespace(cuda_stream=side.cuda_stream), **extra)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), name
    assert pkv.pkv_get_last_error() == 0


@pytest.mark.parametrize("name", ["tree", "mask", "beam", "fork"])
def test_named_streams_within_a_captured_graph(pkv, name):
    """A captured call on a side stream keeps memory of the graph's: replays after other work give the same again."""
    call, _ = calls(pkv)[name]
    want = call()
    refs = torch.cat([torch.ones(4096), torch.zeros(512)]).int().cuda()
    first = refs.clone()
    extra = {"refs": refs} if name == "fork" else {}
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        refs.copy_(first)
        side.wait_stream(torch.cuda.current_stream())
        got = call(stream=side, **extra)
        other = torch.full((1 << 24,), 5.0, device="cuda") * 2  # work of the capturing stream meanwhile
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(3):
        junk = [torch.full((1 << 22,), 9.0, device="cuda") for _ in range(4)]
        own = {"refs": first.clone()} if name == "fork" else {}
        side.wait_stream(torch.cuda.current_stream())
        g.replay()
        again = call(stream=side, **own)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and (other == 10).all()
        assert all(torch.equal(a, b) for a, b in zip(again, want))
        del junk
    assert pkv.pkv_get_last_error() == 0
