"""Where the binding takes results and scratch from, and what it does with the tensors it is given.  No GPU: torch's
device, streams and allocator are stood in for, and every call is one that libpkv has nothing to do for."""
import contextlib
import types
import weakref

import pytest
import torch

HOST = -1  # what a CPU tensor's get_device() says, and so the "current device" here


class Kept(torch.Tensor):
    """A CPU tensor that notes who records a use of it."""

    def record_stream(self, stream):
        LOG.append(("record", stream))


class Stream:
    def __init__(self, cuda_stream, name):
        self.cuda_stream, self.name = cuda_stream, name


LOG = []
MADE = []


@pytest.fixture
def pkv(monkeypatch):
    from paged_kv_cache_248_gb300 import _build
    _build.build()
    import paged_kv_cache_248_gb300 as m
    m.lib()
    LOG.clear()
    MADE.clear()
    main = Stream(0, "main")
    here = [main]
    real = torch.empty

    def empty(shape, dtype=None, device=None):
        LOG.append(("empty", here[-1]))
        t = real(shape, dtype=dtype).as_subclass(Kept)
        MADE.append(weakref.ref(t))
        return t

    @contextlib.contextmanager
    def on(stream):
        here.append(stream)
        yield
        here.pop()

    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: Stream(handle, "foreign"))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: here[-1])
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: HOST, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: here[-1].cuda_stream, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_isCurrentStreamCapturing", lambda: False, raising=False)
    monkeypatch.setattr(m, "_dev", lambda t, name, dtype=None, here=None: None)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: HOST)
    monkeypatch.setattr(m, "_nat", None)  # set up anew with the stand-ins, and again with torch's own after the test
    m.main_stream = main
    yield m
    m._nat = None


def i32(*s):
    return torch.zeros(s, dtype=torch.int32)


K = torch.zeros(4, 2, 16, 128, dtype=torch.bfloat16)
Q = torch.zeros(0, 4, 128, dtype=torch.bfloat16)
def _refused(m, call, *args, **kw):
    """A call without tokens that is refused, after it has asked for its result."""
    with pytest.raises(m.PkvError):
        call(*args, **kw)


CALLS = {  # nothing to do: no tokens, no requests, no rows
    "tree": lambda m, **kw: m.paged_attention_tree(Q, K, K, i32(1, 4), i32(1), i32(2), torch.zeros(0, 1, dtype=torch.int64),
                                                   1.0, 1, 8, **kw),
    "tree_mask": lambda m, **kw: m.pkv_tree_mask(i32(0), i32(2), 8, **kw),
    "compact": lambda m, **kw: m.pkv_compact_path(i32(0, 3), i32(0), i32(0, 4), i32(0), i32(1), K, K, **kw),
    "beam": lambda m, **kw: m.pkv_beam_select(torch.zeros(0, 4, 100), torch.zeros(0, 4), 8, **kw),
    "fork": lambda m, **kw: m.pkv_fork_tables(i32(0, 4), i32(0), i32(0), i32(4), K, K, **kw),
    "slots": lambda m, **kw: m.pkv_slot_mapping(i32(1, 4), i32(1), i32(2), 0, **kw),
    "attention": lambda m, **kw: m.paged_attention(Q, K, K, i32(1, 4), i32(1), i32(2), 1.0, 1, 8, **kw),
    "cascade": lambda m, **kw: m.paged_attention_cascade(Q, K, K, i32(1, 4), i32(1), i32(2), 1.0, 1, 8, i32(0, 1), i32(0),
                                                         i32(1), i32(0), **kw),
    "step": lambda m, **kw: _refused(m, m.paged_attention_step, Q, Q[:, :2], Q[:, :2], K, K, i32(1, 4), i32(1), i32(2), 1.0,
                                     1, 8, **kw),
}


@pytest.mark.parametrize("call", CALLS)
def test_a_named_stream_works_in_memory_of_its_own(pkv, call):
    """The allocator may hand out memory whose last user still runs on the stream that it is asked on.  So whatever a call
    on a named stream writes is asked for on that stream; and what it returns, which the caller's stream reads later, is
    recorded there."""
    side = Stream(7, "side")
    got = CALLS[call](pkv, stream=side)
    results = got if isinstance(got, tuple) else (got,)
    asked = [s for what, s in LOG if what == "empty"]
    assert len(asked) >= len(results) and all(s is side for s in asked), [s.name for s in asked]
    recorded = [s for what, s in LOG if what == "record"]
    assert len(recorded) >= len(results) and all(s is pkv.main_stream for s in recorded), [s.name for s in recorded]


@pytest.mark.parametrize("call", CALLS)
def test_a_stream_that_is_not_torchs_needs_its_handle_only(pkv, call):
    CALLS[call](pkv, stream=types.SimpleNamespace(cuda_stream=9))
    asked = [(s.cuda_stream, s.name) for what, s in LOG if what == "empty"]
    assert asked and all(s == (9, "foreign") for s in asked)


@pytest.mark.parametrize("call", CALLS)
def test_the_current_stream_needs_no_record(pkv, call):
    CALLS[call](pkv)
    assert [s for what, s in LOG if what == "record"] == []
    assert all(s is pkv.main_stream for what, s in LOG if what == "empty")


@pytest.mark.parametrize("call", ["beam", "fork"])
def test_a_workspace_has_a_length(pkv, call):
    """The bytes that a call may use are its workspace's, whatever its shape; a tensor of no dimension has none to tell."""
    with pytest.raises(ValueError, match="workspace"):
        CALLS[call](pkv, workspace=torch.zeros((), dtype=torch.uint8))
    for shape in ((1 << 20,), (4, 1 << 18), (1 << 20, 1), (0,), (0, 4), (1,) * 5):
        CALLS[call](pkv, workspace=torch.zeros(shape, dtype=torch.uint8))
    with pytest.raises(ValueError, match="workspace"):
        CALLS[call](pkv, workspace=torch.zeros((1,) * 6, dtype=torch.uint8))


def test_a_shape_that_is_none_is_an_error_of_its_own(pkv):
    """Numbers that a tensor-like object gives for its shape or strides are looked at when they are read."""
    odd = types.SimpleNamespace(shape=("x", 4, 100))
    with pytest.raises(TypeError):
        pkv.pkv_beam_select(odd, torch.zeros(0, 4), 8)
    with pytest.raises(TypeError):
        pkv.pkv_beam_select(torch.zeros(0, 4, 100), types.SimpleNamespace(shape=(0, None)), 8)
    with pytest.raises(OverflowError):
        pkv.pkv_beam_select(types.SimpleNamespace(shape=(1 << 70, 4, 100)), torch.zeros(0, 4), 8)
    strided = types.SimpleNamespace(shape=(2, 4, 100), dtype=torch.float32, is_contiguous=lambda: False,
                                    stride=lambda: (400, "x", 1))
    with pytest.raises(TypeError):
        pkv.pkv_beam_select(strided, torch.zeros(2, 4), 8)


def test_shutdown_gives_back_what_the_binding_keeps(pkv):
    """Scratch stays for the next call on its stream, and ready results for the next of their shape, until pkv_shutdown."""
    for _ in range(3):
        CALLS["beam"](pkv)
        CALLS["fork"](pkv)
        pkv.pkv_fork_tables(i32(0, 4), i32(0), i32(0), i32(4), None, None)
    assert any(t() is not None for t in MADE)
    pkv.pkv_shutdown()
    assert all(t() is None for t in MADE)
    CALLS["beam"](pkv)  # and calls go on as before
    assert any(t() is not None for t in MADE)
    pkv.pkv_shutdown()
    pkv.pkv_shutdown()
    assert all(t() is None for t in MADE)


class Elsewhere(torch.Tensor):
    """A CPU tensor that says it lies on another CUDA device than the current one."""
    is_cuda = True

    def get_device(self):
        return 1


@pytest.mark.parametrize("which", ["parents", "query_start_loc", "out", "depths"])
def test_tree_masks_are_refused_on_another_device(pkv, monkeypatch, which):
    """The kernel runs on the current device, and what lies on another cannot be read there."""
    monkeypatch.undo()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: types.SimpleNamespace(cuda_stream=0))

    class Here(Elsewhere):
        def get_device(self):
            return 0

    given = {"parents": i32(0), "query_start_loc": i32(2), "out": torch.zeros(0, 1, dtype=torch.int64), "depths": i32(0)}
    given = {n: t.as_subclass(Elsewhere if n == which else Here) for n, t in given.items()}
    with pytest.raises(ValueError, match=f"{which} must be a tensor on the current CUDA device"):
        pkv.pkv_tree_mask(given["parents"], given["query_start_loc"], 8, out=given["out"], depths=given["depths"])
    given[which] = given[which].as_subclass(Here)
    pkv.pkv_tree_mask(given["parents"], given["query_start_loc"], 8, out=given["out"], depths=given["depths"])
