"""A decoding step over a cache in 8 bits, without a GPU: the plain implementations, the host checks, the binding's refusals."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import step8_ref as ref


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_248_gb300 import _build
    _build.build()
    import paged_kv_cache_248_gb300 as m
    m.lib()
    return m


def test_every_code_is_read_and_written_as_torch_does():
    codes = np.arange(256, dtype=np.uint8)
    values = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(ref.decode8(codes), values)
    numbers = (codes & 127) != 127
    np.testing.assert_array_equal(ref.encode8(values[numbers]), codes[numbers])
    x = np.random.default_rng(0).standard_normal(20000).astype(np.float32) * np.exp2(
        np.random.default_rng(1).integers(-12, 9, 20000)).astype(np.float32)
    want = torch.from_numpy(x).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(ref.encode8(x), want)
    np.testing.assert_array_equal(ref.encode8([np.inf, -1e9, np.nan]), [0x7e, 0xfe, 0x7f])


def test_scales_are_the_least_power_of_two():
    for amax in (448.0, 448.0001, 1.0, 1.75, 1.7500001, 3.4e38, 1e-30, 0.0):
        s = ref.scale_for(amax)
        assert amax <= 448 * s and (s == 2.0 ** -80 or amax > 448 * s / 2) and np.log2(s) % 1 == 0


def test_turning_keeps_lengths_and_angles_between_positions():
    cs = ref.angles(50, 32)
    x, y = np.random.default_rng(3).standard_normal((2, 48)).astype(np.float32)
    for inter in (False, True):
        a, b = ref.rotated(x, cs[40], inter), ref.rotated(y, cs[17], inter)
        c, d = ref.rotated(x, cs[23], inter), ref.rotated(y, cs[0], inter)
        assert abs(a @ b - c @ d) < 1e-4  # of the difference of positions only
        np.testing.assert_array_equal(a[32:], x[32:])


def test_sampling_by_counting():
    # three candidates of weights 1/2, 1/4, 1/4 by hand
    x = np.log(np.array([[0.25, 0.5, 0.25]], np.float32))
    for u, token in ((0.0, 1), (0.49, 1), (0.51, 0), (0.76, 2), (0.9999, 2)):
        assert ref.sample(x, [u])[0][0] == token
    assert ref.sample(x, [0.99], top_k=[1])[0][0] == 1
    assert ref.sample(x, [0.99], top_p=[0.6])[0][0] == 0
    assert ref.sample(x, [0.99], min_p=[0.9])[0][0] == 1
    assert ref.sample(np.full((1, 3), np.nan, np.float32), [0.5])[0][0] == -1


def source(name):
    """A kernel's source without its comments."""
    import paged_kv_cache_248_gb300 as m
    with open(os.path.join(os.path.dirname(m.__file__), "csrc", name)) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


def test_weights_are_waited_for_before_they_are_read_again():
    # stores to tensor memory are asynchronous, and a load waits for loads only: an order that no result shows
    s = source("k_q8_chunk.cu")
    body = s[s.index("void row_weights("):s.index("void softmax_warps(")]
    move = body[body.index("most > kTop + kMost"):]
    assert 0 < move.find("tmem_st_wait()") < min(move.index("scale_o("), move.index("scale_p("))


def test_a_clusters_shared_memory_is_touched_once_all_of_it_runs():
    # a CTA may begin long after its cluster's others, and has no shared memory before
    s = source("k_sample.cu")
    body = s[s.index("sample_kernel(const Params P)"):]
    first = body.index("map_shared_rank(")
    assert 0 < body.find("cluster.barrier_arrive()") < body.find("grid_dep_wait()")
    assert 0 < body.find("cluster.barrier_wait()") < first < body.index("cluster.sync()")


P = ctypes.c_void_p
FAKE = P(0x10000)  # never dereferenced: every call below fails its host checks first


def _append(pkv, **over):
    d = over.pop("desc", None) or pkv._CacheDesc(8, 16, 2, 128, pkv.PKV_E4M3)
    a = dict(q=FAKE, k=FAKE, v=FAKE, dtype=pkv.PKV_BF16, qs=512, ks=256, vs=256, hq=4, cs=FAKE, rot=128, inter=0, na=10,
             pos=None, kc=FAKE, vc=FAKE, sc=FAKE, desc=ctypes.byref(d), bt=FAKE, mb=4, sl=FAKE, qsl=FAKE, n=1, t=2, mq=2,
             qo=P(0x900000), qos=512, stream=None)
    a.update(over)
    return pkv.lib().pkv_rope_append(*a.values())


@pytest.mark.parametrize("over,status", [
    (dict(t=0), 0), (dict(t=-1), 1), (dict(n=0), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(sc=None), 1),
    (dict(cs=None), 1), (dict(rot=-16), 1), (dict(rot=144), 1), (dict(rot=24), 2), (dict(mq=0), 1), (dict(mb=0), 1),
    (dict(dtype=0), 2), (dict(qo=None), 1), (dict(q=None), 1), (dict(hq=0), 1), (dict(ks=128), 1), (dict(vs=257), 1),
    (dict(qs=1 << 40), 2), (dict(k=P(0x10008)), 1), (dict(cs=P(0x10004)), 1), (dict(sc=P(0x10004)), 1), (dict(na=-1), 1),
    (dict(qo=P(0x10010)), 1),                    # overlaps q, not the same
    (dict(qo=FAKE, qos=1024), 1),                # q itself, otherwise spaced
])
def test_append_host_checks(pkv, over, status):
    assert _append(pkv, **over) == status


@pytest.mark.parametrize("k,v,stride,status", [
    (0x10000, 0x800000, 256, 1),            # k is q, which is written
    (0x800000, 0x10000 + 512, 256, 1),      # v begins within q's first token
    (0x10000 + 1024, 0x800000, 1024, 1),    # columns behind q's, of rows otherwise spaced
    (0x10000 + 512, 0x10000 + 1536, 1024, 1),   # k's columns begin within q's
    (0x10000 + 1024, 0x10000 - 256, 768, 1),    # v's columns end within the next token's q
])
def test_append_refuses_queries_in_place_over_keys_or_values(pkv, k, v, stride, status):
    assert _append(pkv, qo=FAKE, qs=768, qos=768, k=P(k), v=P(v), ks=stride, vs=stride) == status


def test_append_checks_the_cache(pkv):
    desc = pkv._CacheDesc
    assert _append(pkv, desc=desc(8, 16, 2, 64, pkv.PKV_E4M3)) == pkv.PKV_ERR_UNSUPPORTED
    assert _append(pkv, desc=desc(8, 15, 2, 128, pkv.PKV_E4M3)) == pkv.PKV_ERR_INVALID_ARG
    assert _append(pkv, desc=desc(8, 16, 2, 128, 7)) == pkv.PKV_ERR_UNSUPPORTED
    assert _append(pkv, desc=desc(8, 16, 2, 128, pkv.PKV_BF16)) == pkv.PKV_ERR_INVALID_ARG  # scales of a 16-bit cache
    assert _append(pkv, desc=desc(8, 16, 2, 128, pkv.PKV_F32), sc=None) == pkv.PKV_ERR_UNSUPPORTED  # bf16 inputs


def _q8(pkv, **over):
    d = over.pop("desc", None) or pkv._CacheDesc(8, 16, 2, 128, pkv.PKV_E4M3)
    a = dict(q=FAKE, k=FAKE, v=FAKE, sc=FAKE, desc=ctypes.byref(d), bt=FAKE, mb=4, sl=FAKE, qsl=FAKE, n=1, hq=4, t=2,
             mq=2, ml=30, scale=ctypes.c_float(0.1), out=FAKE, ws=FAKE, wb=1 << 30, stream=None)
    a.update(over)
    return pkv.lib().paged_attention_q8(*a.values())


@pytest.mark.parametrize("over,status", [
    (dict(t=0), 0), (dict(t=-1), 1), (dict(n=0), 1), (dict(q=None), 1), (dict(sc=None), 1), (dict(out=None), 1),
    (dict(hq=3), 1), (dict(hq=34), 2), (dict(mq=0), 1), (dict(ml=0), 1), (dict(mb=0), 1),
    (dict(scale=ctypes.c_float(float("nan"))), 1), (dict(q=P(0x10008)), 1), (dict(sc=P(0x10004)), 1),
    (dict(t=1 << 31), 2), (dict(n=1 << 30), 2)])
def test_attention_host_checks(pkv, over, status):
    assert _q8(pkv, **over) == status


def test_other_calls_refuse_a_cache_in_8_bits(pkv):
    d = pkv._CacheDesc(8, 16, 2, 128, pkv.PKV_E4M3)
    L, r = pkv.lib(), ctypes.byref(d)
    assert L.pkv_write(FAKE, FAKE, FAKE, 1, FAKE, FAKE, r, None) == pkv.PKV_ERR_UNSUPPORTED
    assert L.paged_attention(FAKE, FAKE, FAKE, r, FAKE, 1, FAKE, FAKE, 1, 2, 1, 1, 1, ctypes.c_float(1.0), FAKE,
                             None) == pkv.PKV_ERR_UNSUPPORTED
    for dt in (pkv.PKV_BF16, pkv.PKV_F32):
        assert _q8(pkv, desc=pkv._CacheDesc(8, 16, 2, 128, dt)) == pkv.PKV_ERR_UNSUPPORTED


def _sample(pkv, **over):
    a = dict(x=FAKE, dt=1, stride=100, temp=None, k=None, p=None, m=None, u=FAKE, n=2, v=100, out=FAKE, lp=None, stream=None)
    a.update(over)
    return pkv.lib().pkv_sample(*a.values())


@pytest.mark.parametrize("over,status", [
    (dict(n=0), 0), (dict(n=-1), 1), (dict(v=0), 1), (dict(v=(1 << 20) + 1, stride=1 << 21), 2), (dict(dt=2), 2),
    (dict(x=None), 1), (dict(u=None), 1), (dict(out=None), 1), (dict(stride=99), 1), (dict(x=P(0x10001)), 1),
    (dict(x=P(0x10002), dt=0), 1)])
def test_sample_host_checks(pkv, over, status):
    assert _sample(pkv, **over) == status


def test_binding_refuses_what_does_not_fit(pkv):
    z = torch.zeros
    kc, sc = z(4, 2, 16, 128, dtype=torch.uint8), z(4, 2, 2)
    bt, sl, qsl = z(1, 4, dtype=torch.int32), z(1, dtype=torch.int32), z(2, dtype=torch.int32)
    k, q = z(3, 2, 128, dtype=torch.bfloat16), z(3, 4, 128, dtype=torch.bfloat16)
    cs = z(8, 128)
    ok = dict(k=k, v=k, cos_sin=cs, k_cache=kc, v_cache=kc, block_tables=bt, seq_lens=sl, query_start_loc=qsl,
              max_query_len=3, q=q, scales=sc)
    for over, what in ((dict(k=k[:, :1]), "k and v"), (dict(q=q[:2]), "q must"), (dict(scales=None), "scales belong"),
                       (dict(scales=sc[:3]), "scales must"), (dict(cos_sin=cs[0]), "cos_sin must"),
                       (dict(q=None, q_out=q), "q_out without q"), (dict(q_out=q[:, :2]), "q_out must"),
                       (dict(k_cache=kc.to(torch.int8), v_cache=kc.to(torch.int8)), "unsupported cache dtype"),
                       (dict(positions=bt[0]), "positions must"), (dict(seq_lens=z(2, dtype=torch.int32)), "disagree")):
        with pytest.raises(ValueError, match=what):
            pkv.pkv_rope_append(**{**ok, **over})
    ok = dict(q=q, k_cache=kc, v_cache=kc, scales=sc, block_tables=bt, seq_lens=sl, query_start_loc=qsl, scale=0.1,
              max_query_len=3, max_seq_len=9)
    for over, what in ((dict(k_cache=kc.bfloat16(), v_cache=kc.bfloat16()), "8 bits"), (dict(q=q[..., :64]), "q must"),
                       (dict(scales=sc[..., :1]), "scales must"), (dict(out=q[:2]), "out must")):
        with pytest.raises(ValueError, match=what):
            pkv.paged_attention_q8(**{**ok, **over})
    x, u = z(2, 10), z(2)
    for args, what in (((x[0], u), "logits must"), ((x.double(), u), "logits must"), ((x.T, z(10)), "contiguous rows"),
                       ((x, z(3)), "uniform must"), ((x, u, z(3)), "temperature must")):
        with pytest.raises(ValueError, match=what):
            pkv.pkv_sample(*args)
    with pytest.raises(ValueError, match="out must be"):
        pkv.pkv_sample(x, u, out=x)
