"""A decoding step over a cache in 8 bits on the GPU, against plain implementations in 64 bits.

Tolerances.  Rotations and codes: the definition rounds to fp32 after each operation, so results are equal
bit by bit.  Attention: |out - exact| <= 2^-8 |exact| (the result's rounding to bf16, half a step of 2^-7) + 2^-9 sum w |v|: a
weight is off by the rounding of its score (fp32, |score| below 2^8 here: 2^-12 at most with the products' sums), the
exponential (2^-22) and its representation (2^-11), 2^-10 together, and as much again of the row's sum of weights.
Sampling: tokens equal, logprobs within 2^-22 of themselves and of 1.
"""
import numpy as np
import pytest
import torch

import step8_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    import paged_kv_cache_248_gb300 as m
    m.lib()
    return m


@pytest.fixture(autouse=True)
def no_error_left(pkv):
    yield
    assert pkv.pkv_get_last_error() == 0


def gpu(*a):
    out = tuple(torch.from_numpy(np.ascontiguousarray(x)).cuda() for x in a)
    return out[0] if len(out) == 1 else out


def bf16(shape, seed, scale=1.0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).mul(scale).bfloat16()


# ----------------------------------------------------------------------------- append
def append_case(ctx, new, hq, hkv, d, rot, kind, seed, table=None):
    tables, lens, qsl, pool = ref.requests(ctx, new, seed)
    t = int(qsl[-1])
    dtype = torch.float32 if kind == "f32" else torch.bfloat16
    gen = torch.Generator().manual_seed(seed)
    qkv = torch.randn((t, (hq + 2 * hkv) * d), generator=gen).to(dtype)
    if kind == "e4m3":  # tokens of very different size, so that scales have to grow
        qkv *= torch.exp2(torch.randint(-6, 7, (t, 1), generator=gen)).to(dtype)
    cs = ref.angles(int(lens.max()) + 3, rot, seed) if rot else None
    return tables, lens, qsl, pool, qkv, cs


def split(qkv, hq, hkv, d):
    return (qkv[:, :hq * d].unflatten(1, (hq, d)), qkv[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d)),
            qkv[:, (hq + hkv) * d:].unflatten(1, (hkv, d)))


def run_append(pkv, ctx, new, hq, hkv, d, rot, kind, inter=False, seed=0, positions=False, in_place=False):
    tables, lens, qsl, pool, qkv, cs = append_case(ctx, new, hq, hkv, d, rot, kind, seed)
    q, k, v = split(qkv, hq, hkv, d)
    pos = np.random.default_rng(seed).integers(0, len(cs), len(qkv)).astype(np.int32) if positions else None
    if kind == "e4m3":
        cache, scales = ref.pool8(pool, hkv, seed)
        want_c, want_s = cache.copy(), scales.copy()
        gc, gs = gpu(cache, scales)
    else:
        cache = torch.randn((2, pool, hkv, 16, d), generator=torch.Generator().manual_seed(seed)).to(qkv.dtype)
        want_c, want_s, gc, gs = cache.float().numpy().copy(), None, cache.cuda(), None
    f = lambda x: x.float().numpy()  # noqa: E731
    want_q = ref.append(f(q), f(k), f(v), cs, want_c[0], want_c[1], tables, lens, qsl, want_s, pos, inter)
    gqkv = qkv.cuda()
    gq, gk, gv = split(gqkv, hq, hkv, d)
    out = pkv.pkv_rope_append(gk, gv, None if cs is None else gpu(cs), gc[0], gc[1], *gpu(tables, lens, qsl), max(1, int(max(new))),
                              q=gq, scales=gs, positions=None if pos is None else gpu(pos), interleaved=inter,
                              q_out=gq if in_place else None)
    assert pkv.pkv_get_last_error() == 0
    torch.testing.assert_close(out.cpu(), torch.from_numpy(want_q).to(qkv.dtype), rtol=0, atol=0)
    if in_place:
        assert out is gq
        torch.testing.assert_close(gqkv[:, hq * d:].cpu(), qkv[:, hq * d:], rtol=0, atol=0)
    if kind == "e4m3":
        np.testing.assert_array_equal(gs.cpu().numpy(), want_s)
        np.testing.assert_array_equal(gc.cpu().numpy(), want_c)
    else:
        torch.testing.assert_close(gc.cpu(), torch.from_numpy(want_c).to(qkv.dtype), rtol=0, atol=0)


@pytest.mark.parametrize("kind,hq,hkv,d,rot,inter", [
    ("bf16", 8, 2, 128, 128, False), ("bf16", 3, 1, 128, 64, True), ("bf16", 7, 7, 128, 0, False), ("bf16", 4, 2, 128, 16, False),
    ("f32", 4, 2, 64, 64, False), ("f32", 5, 1, 64, 32, True), ("f32", 6, 3, 128, 128, True), ("f32", 2, 2, 128, 48, False),
    ("e4m3", 8, 2, 128, 128, False), ("e4m3", 6, 3, 128, 96, True), ("e4m3", 3, 1, 128, 0, False), ("e4m3", 16, 8, 128, 32, False)])
@pytest.mark.parametrize("ctx,new", [([0], [1]), ([15, 16, 17, 5], [1, 1, 1, 1]), ([0, 31, 7, 100], [40, 1, 25, 16]),
                                     ([3, 0, 12], [13, 16, 20])])
def test_append(pkv, kind, hq, hkv, d, rot, inter, ctx, new):
    run_append(pkv, ctx, new, hq, hkv, d, rot, kind, inter, seed=len(ctx) + hq)


@pytest.mark.parametrize("kind", ["bf16", "f32", "e4m3"])
def test_append_positions_in_place_and_empty_requests(pkv, kind):
    run_append(pkv, [10, 0, 33, 4, 0], [5, 0, 1, 0, 18], 4, 2, 128, 64, kind, seed=5, positions=True, in_place=True)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_append_many_requests(pkv, kind):
    rng = np.random.default_rng(2)
    n = 150
    run_append(pkv, rng.integers(0, 60, n), rng.integers(0, 9, n), 2, 1, 128, 128, kind, seed=7)
    run_append(pkv, rng.integers(0, 60, n), np.ones(n, int), 2, 1, 128, 128, kind, seed=8)


@pytest.mark.parametrize("ctx,new", [([15], [2]), ([40, 31], [3, 2]), ([15, 15, 15], [2, 2, 2]), ([0, 14, 15], [13, 18, 17]), ([3, 15], [16, 18])])
def test_append_requests_that_touch_as_many_blocks_as_they_can(pkv, ctx, new):
    run_append(pkv, ctx, new, 4, 2, 128, 128, "e4m3", seed=sum(new))


@pytest.mark.parametrize("hq,hkv,rot,inter", [(3, 3, 64, True), (8, 8, 128, False), (20, 20, 32, False), (40, 5, 0, False)])
def test_append_single_tokens_of_any_number_of_heads(pkv, hq, hkv, rot, inter):
    rng = np.random.default_rng(hkv)
    run_append(pkv, rng.integers(0, 60, 70), np.ones(70, int), hq, hkv, 128, rot, "e4m3", inter=inter, seed=hkv)
    run_append(pkv, rng.integers(0, 60, 9), rng.integers(0, 2, 9), hq, hkv, 128, rot, "e4m3", inter=inter, seed=hkv, in_place=True)


def test_append_single_tokens_that_are_infinite_or_fit_nowhere(pkv):
    tables, lens, qsl, pool, qkv, cs = append_case([20, 5, 40, 9, 30], [1] * 5, 4, 2, 128, 128, "e4m3", 3)
    qkv[3, 4 * 128:4 * 128 + 4] = torch.tensor([float("inf"), -float("inf"), float("nan"), 3.0]).bfloat16()
    tables[1, 0] = pool + 7              # a bad block
    lens[2] = 16 * tables.shape[1] + 5   # past the table's row
    cs = cs[:30]                         # request 4: its position (30) has no row
    q, k, v = split(qkv, 4, 2, 128)
    cache, scales = ref.pool8(pool, 2, 3)
    want_c, want_s = cache.copy(), scales.copy()
    good = [0, 3]
    f = lambda x: x[good].float().numpy()  # noqa: E731
    ref.append(None, f(k), f(v), cs, want_c[0], want_c[1], tables[good], lens[good], np.array([0, 1, 2]), want_s)
    gc, gs = gpu(cache, scales)
    out = pkv.pkv_rope_append(k.cuda(), v.cuda(), gpu(cs), gc[0], gc[1], *gpu(tables, lens, qsl), 1, q=q.cuda(), scales=gs).cpu()
    assert pkv.pkv_peek_error_bits() == 1 + 4 and pkv.pkv_get_last_error() == pkv.PKV_ERR_INDEX
    assert not out[2].any() and not out[4].any()
    for t, p in ((0, 20), (1, 5), (3, 9)):
        torch.testing.assert_close(out[t], torch.from_numpy(ref.rotated(q[t].float().numpy(), cs[p], False)).bfloat16(), rtol=0, atol=0)
    np.testing.assert_array_equal(gs.cpu().numpy(), want_s)
    np.testing.assert_array_equal(gc.cpu().numpy() & 127, want_c & 127)  # (a NaN has either sign)


def test_append_grows_a_block_token_by_token(pkv):
    # one block filled token by token, sizes doubling: each token's codes come out as if written once in the last units,
    # since the codes stay in the normal range
    hkv, n = 2, 16
    cache, scales = torch.zeros((2, 1, hkv, 16, 128), dtype=torch.uint8, device="cuda"), torch.full((1, hkv, 2), 9e9, device="cuda")
    x = (1.0 + torch.rand((n, hkv, 128), generator=torch.Generator().manual_seed(0))) * torch.exp2(torch.arange(n) // 4)[:, None, None]
    x = x.bfloat16().cuda()
    tables = gpu(np.zeros((1, 1), np.int32))
    for j in range(n):
        pkv.pkv_rope_append(x[j:j + 1], x[j:j + 1], None, cache[0], cache[1], tables, gpu(np.array([j + 1], np.int32)),
                            gpu(np.array([0, 1], np.int32)), 1, scales=scales)
    s = ref.scale_for(float(x[:, 0].max()))
    assert float(scales[0, 0, 0]) == s
    np.testing.assert_array_equal(cache[1, 0, 0].cpu().numpy(), ref.encode8(x[:, 0].float().cpu().numpy() / s))
    # again with the last token alone: nothing changes
    before = cache.clone()
    pkv.pkv_rope_append(x[-1:], x[-1:], None, cache[0], cache[1], tables, gpu(np.array([16], np.int32)),
                        gpu(np.array([0, 1], np.int32)), 1, scales=scales)
    assert torch.equal(before, cache)


def test_append_infinities_and_nan(pkv):
    x = torch.ones((2, 1, 128))
    x[0, 0, :4] = torch.tensor([float("inf"), -float("inf"), float("nan"), 3.0])
    x[1, 0, :2] = torch.tensor([3e38, 1e-38])
    x = x.bfloat16()
    for rows in (x[:1], x):
        want_c, want_s = np.zeros((2, 1, 1, 16, 128), np.uint8), np.zeros((1, 1, 2), np.float32)
        f = rows.float().numpy()
        tables, lens, qsl = np.zeros((1, 1), np.int32), np.array([len(rows)], np.int32), np.array([0, len(rows)], np.int32)
        ref.append(None, f, f, None, want_c[0], want_c[1], tables, lens, qsl, want_s)
        gc, gs = torch.zeros((2, 1, 1, 16, 128), dtype=torch.uint8, device="cuda"), torch.zeros((1, 1, 2), device="cuda")
        assert pkv.pkv_rope_append(rows.cuda(), rows.cuda(), None, gc[0], gc[1], *gpu(tables, lens, qsl), 2, scales=gs) is None
        np.testing.assert_array_equal(gs.cpu().numpy(), want_s)
        np.testing.assert_array_equal(gc.cpu().numpy() & 127, want_c & 127)  # (a NaN has either sign)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_append_bad_data_is_flagged_and_skipped(pkv, kind):
    tables, lens, qsl, pool, qkv, cs = append_case([20, 5, 40, 0, 9], [3, 2, 1, 4, 3], 4, 2, 128, 128, kind, 3)
    tables[1, 0] = pool + 7           # a bad block
    lens[2] = 16 * tables.shape[1] + 5  # past the table's row
    cs = cs[:22]                      # request 0: its last position (22) has no row
    q, k, v = split(qkv, 4, 2, 128)
    if kind == "e4m3":
        cache, scales = ref.pool8(pool, 2, 3)
        gc, gs = gpu(cache, scales)
    else:
        gc, gs = torch.zeros((2, pool, 2, 16, 128), dtype=torch.bfloat16, device="cuda"), None
    before = gc.clone()
    out = pkv.pkv_rope_append(k.cuda(), v.cuda(), gpu(cs), gc[0], gc[1], *gpu(tables, lens, qsl), 4, q=q.cuda(), scales=gs)
    assert pkv.pkv_get_last_error() == pkv.PKV_ERR_INDEX
    out = out.cpu()
    want = torch.from_numpy(np.stack([ref.rotated(q[t].float().numpy(), cs[p], False) for t, p in
                                      ((0, 20), (1, 21), (3, 5), (4, 6), (6, 0), (7, 1), (8, 2), (9, 3))])).bfloat16()
    torch.testing.assert_close(out[[0, 1, 3, 4, 6, 7, 8, 9]], want, rtol=0, atol=0)
    assert not out[2].any() and not out[5].any()
    b, s = tables[0][1], 22 % 16
    assert torch.equal(gc[:, b, :, s], before[:, b, :, s])
    touched = set(tables[0][1:2]) | set(tables[3][:1]) | set(tables[4][:1])
    for b in range(pool):
        assert torch.equal(gc[:, b], before[:, b]) == (b not in touched)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("new", [[1, 1], [3, 20]])
def test_append_the_lengths_of_empty_requests_are_not_looked_at(pkv, kind, new):
    # a padded batch: places of requests that are not there, with lengths of any kind
    tables, lens, qsl, pool, qkv, cs = append_case([4, 30], new, 4, 2, 128, 128, kind, 3)
    q, k, v = split(qkv.cuda(), 4, 2, 128)
    cache, scales = ref.pool8(pool, 2, 3)
    got = []
    for pad in (0, 5):
        gc, gs = gpu(cache, scales) if kind == "e4m3" else (torch.zeros((2, pool, 2, 16, 128), dtype=torch.bfloat16, device="cuda"), None)
        more = np.array([-7, 10 ** 6, 0, 2 ** 31 - 1, -2 ** 31])[:pad].astype(np.int32)
        t = np.concatenate([tables, np.full((pad, tables.shape[1]), -1, np.int32)])
        out = pkv.pkv_rope_append(k, v, gpu(cs), gc[0], gc[1], *gpu(t, np.concatenate([lens, more]), np.pad(qsl, (0, pad), mode="edge")),
                                  max(new), q=q, scales=gs)
        assert pkv.pkv_get_last_error() == 0
        got.append((out, gc))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


def test_append_leaves_rows_behind_the_last_request(pkv):
    for kind in ("bf16", "e4m3"):
        tables, lens, qsl, pool, qkv, cs = append_case([4, 9], [2, 1], 4, 2, 128, 128, kind, 3)
        qkv = torch.cat([qkv, qkv])  # three tokens more than the requests have
        q, k, v = split(qkv.cuda(), 4, 2, 128)
        cache, scales = ref.pool8(pool, 2, 3)
        gc, gs = gpu(cache, scales) if kind == "e4m3" else (torch.zeros((2, pool, 2, 16, 128), dtype=torch.bfloat16, device="cuda"), None)
        out = torch.full_like(q, 7.0, memory_format=torch.contiguous_format)
        pkv.pkv_rope_append(k, v, gpu(cs), gc[0], gc[1], *gpu(tables, lens, qsl), 2, q=q, scales=gs, q_out=out)
        assert (out[3:] == 7).all() and not (out[:3] == 7).all()


# ----------------------------------------------------------------------------- attention
def check_attention(pkv, ctx, new, hq, hkv, seed=0, q_scale=1.0, max_q=None, bad=(), change=None):
    tables, lens, qsl, pool = ref.requests(ctx, new, seed)
    cache, scales = ref.pool8(pool, hkv, seed)
    if change:
        change(cache, scales, tables, lens, qsl)
    q = bf16((int(qsl[-1]), hq, 128), seed, q_scale)
    scale = 128 ** -0.5
    out = pkv.paged_attention_q8(q.cuda(), *gpu(cache[0], cache[1], scales, tables, lens, qsl), scale,
                                 max_q or max(1, int(max(new))), int(lens.max()))
    assert pkv.pkv_get_last_error() == (pkv.PKV_ERR_INDEX if bad else 0)
    for i in bad:
        assert not out[qsl[i]:qsl[i + 1]].any()
        cut = slice(qsl[i], qsl[i + 1])
        lens = lens.copy()
    good = [i for i in range(len(lens)) if i not in bad]
    sub = np.concatenate([np.arange(qsl[i], qsl[i + 1]) for i in good]).astype(int)
    starts = np.concatenate([[0], np.cumsum([qsl[i + 1] - qsl[i] for i in good])])
    want, size = ref.attention(q.double().numpy()[sub], cache[0], cache[1], scales, tables[good], lens[good], starts, scale)
    got = out.double().cpu().numpy()[sub]
    assert np.isfinite(got).all()
    over = np.abs(got - want) - (2.0 ** -8 * np.abs(want) + 2.0 ** -9 * size)
    assert over.max() <= 0, (over.max(), np.unravel_index(over.argmax(), over.shape))


@pytest.mark.parametrize("hq,hkv", [(4, 1), (2, 2), (8, 1), (16, 1), (6, 2), (14, 2), (10, 2), (5, 5)])
def test_attention_single_tokens(pkv, hq, hkv):
    check_attention(pkv, [0, 14, 15, 16, 126, 127, 128, 300, 1000], [1] * 9, hq, hkv, seed=hq)


@pytest.mark.parametrize("hq,hkv", [(4, 1), (2, 2), (16, 1), (6, 2), (12, 4)])
@pytest.mark.parametrize("ctx,new", [([0], [2]), ([0, 127, 5, 260], [7, 1, 130, 3]), ([100, 0, 30], [33, 64, 1]),
                                     ([0, 500, 0, 20], [1, 0, 150, 17])])
def test_attention_chunks(pkv, hq, hkv, ctx, new):
    check_attention(pkv, ctx, new, hq, hkv, seed=hq + len(ctx))


@pytest.mark.parametrize("ctx,new", [([9000], [1]), ([5000, 100, 4097], [1, 1, 1]), ([3000], [20]), ([2500, 2500], [5, 5])])
def test_attention_long(pkv, ctx, new):
    check_attention(pkv, ctx, new, 8, 2, seed=1)


def test_attention_many_requests(pkv):
    rng = np.random.default_rng(4)
    check_attention(pkv, rng.integers(0, 90, 300), np.ones(300, int), 4, 1, seed=2)
    check_attention(pkv, rng.integers(0, 90, 200), rng.integers(0, 4, 200), 4, 1, seed=3)


@pytest.mark.parametrize("hq,hkv", [(4, 1), (2, 2), (16, 1), (6, 2)])
@pytest.mark.parametrize("ctx,new", [([500, 0, 127, 128, 40, 3000, 7, 16, 90, 15, 200, 33], [1, 1, 1, 1, 200, 1, 1, 0, 1, 1, 0, 1]),
                                     ([0] * 20 + [70], [1] * 20 + [3]), ([9, 300, 2], [1, 2, 1]), ([10] * 9, [0] * 7 + [50, 1])])
def test_attention_single_tokens_beside_chunks(pkv, hq, hkv, ctx, new):
    check_attention(pkv, ctx, new, hq, hkv, seed=hq)


def test_attention_single_tokens_beside_chunks_with_bad_pages_and_lengths(pkv):
    ctx, new = [300, 40, 5, 77, 600, 9, 30, 20], [1, 1, 90, 1, 1, 1, 1, 1]

    def change(cache, scales, tables, lens, qsl):
        tables[0, 4] = len(scales) + 5       # a single token's page
        lens[3] = 16 * tables.shape[1] + 1   # longer than its table
        lens[5] = 0                          # less than its tokens
    check_attention(pkv, ctx, new, 4, 2, seed=3, bad=(0, 3, 5), change=change)

    def change_chunk(cache, scales, tables, lens, qsl):
        tables[2, 1] = -1
    check_attention(pkv, ctx, new, 4, 2, seed=3, bad=(2,), change=change_chunk)


def test_attention_sharp_scores(pkv):
    check_attention(pkv, [700, 90], [1, 40], 8, 2, seed=4, q_scale=12.0)


def test_attention_scales_far_apart(pkv):
    # V's scales of 2^-20 .. 2^20, a zero scale (its values are 0, its keys still count), K's as they are
    def change(cache, scales, tables, lens, qsl):
        scales[..., 1] = np.exp2(np.random.default_rng(0).integers(-20, 21, scales.shape[:2]))
        scales[tables[0][3], :, 1] = 0.0
    check_attention(pkv, [200, 1000], [1, 9], 4, 2, seed=5, change=change)


def test_attention_scales_of_any_value(pkv):
    def change(cache, scales, tables, lens, qsl):
        scales *= np.random.default_rng(0).uniform(0.5, 1.0, scales.shape).astype(np.float32)
    check_attention(pkv, [200, 1000], [1, 9], 4, 2, seed=6, change=change)


@pytest.mark.parametrize("new", [1, 30])
def test_attention_one_key_above_a_long_flat_rest(pkv, new):
    # the weights of the rest are small and all the same, and together as large as the first key's
    n = 4096

    def change(cache, scales, tables, lens, qsl):
        cache[:] = ref.encode8(np.zeros(1))[0]
        scales[:] = 1.0
        cache[1, :, :] = ref.encode8(np.full(1, 1.0))[0]
        first = tables[0][0]
        cache[0, first, :, 0, 0] = ref.encode8(np.full(1, 12.0))[0]
        cache[1, first, :, 0] = ref.encode8(np.full(1, -1.0))[0]
    tables, lens, qsl, pool = ref.requests([n], [new], 0)
    cache, scales = ref.pool8(pool, 1, 0)
    change(cache, scales, tables, lens, qsl)
    scale = 128 ** -0.5
    for gap in (4.0, 8.0, 8.7, 10.0):
        q = torch.zeros((new, 2, 128)).bfloat16()
        q[..., 0] = gap / (12.0 * scale)
        out = pkv.paged_attention_q8(q.cuda(), *gpu(cache[0], cache[1], scales, tables, lens, qsl), scale, new, n + new)
        want, size = ref.attention(q.double().numpy(), cache[0], cache[1], scales, tables, lens, qsl, scale)
        assert (np.abs(out.double().cpu().numpy() - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -9 * size).all()


@pytest.mark.parametrize("new,hq", [(1, 4), (1, 16), (1, 11), (30, 4)])
def test_attention_small_weights_beside_a_large_one(pkv, new, hq):
    # so many requests that a CTA does all of one: its reference is the first key's weight, whose V is 0, and what comes
    # out are the others' weights alone, 2^-14 to 2^-35 of it.  A single token's are held to 2^-11 of themselves down to 2^-29 of
    # the largest, and to 2^-40 of it below; a chunk's to 2^-21 and 2^-32 (V is 2 at most).
    n, requests, scale, least = 4000, 320 // new + 150, 128 ** -0.5, 2.0 ** (-40 if new == 1 else -32)
    gaps = np.array([10.0, 13.0, 14.0, 15.0, 15.6, 16.0, 16.3, 17.0, 17.5, 18.0, 20.0, 22.0, 24.0])
    tables, lens, qsl, pool = ref.requests([n], [new], 0)
    cache, scales = np.zeros((2, pool, 1, 16, 128), np.uint8), np.ones((pool, 1, 2), np.float32)
    cache[1] = ref.encode8(np.linspace(0.5, 2.0, 128))
    first = tables[0][0]
    cache[0, first, 0, 0, 0] = ref.encode8(np.full(1, 12.0))[0]
    cache[1, first, 0, 0] = 0
    q = torch.zeros((len(gaps), new, hq, 128)).bfloat16()
    q[..., 0] = torch.from_numpy(gaps / (12.0 * scale))[:, None, None]
    at = np.arange(requests) % len(gaps)
    out = pkv.paged_attention_q8(q[at].flatten(0, 1).cuda(), *gpu(cache[0], cache[1], scales, tables.repeat(requests, 0), lens.repeat(requests),
                                                                  (np.arange(requests + 1) * new).astype(np.int32)), scale, new, n + new)
    one = q[:, :, :1].flatten(0, 1).double().numpy()  # (all heads are alike)
    want, size = ref.attention(one, cache[0], cache[1], scales, tables.repeat(len(gaps), 0), lens.repeat(len(gaps)),
                               np.arange(len(gaps) + 1) * new, scale)
    pick = lambda x: x.reshape(len(gaps), new, 1, 128)[at]  # noqa: E731
    off = np.abs(out.double().cpu().numpy().reshape(requests, new, hq, 128) - pick(want))
    assert (off <= 2.0 ** -8 * np.abs(pick(want)) + 2.0 ** -9 * pick(size) + least * (n + new) * 2.0).all()


def test_attention_outliers_of_a_query(pkv):
    # one element a thousand times the others: they keep their share of the scores
    tables, lens, qsl, pool = ref.requests([300], [1], 0)
    cache, scales = ref.pool8(pool, 1, 0)
    cache[0, :, :, :, 5] = 0
    q = bf16((1, 4, 128), 0)
    q[..., 5] = 2000.0
    out = pkv.paged_attention_q8(q.cuda(), *gpu(cache[0], cache[1], scales, tables, lens, qsl), 0.3, 1, 301)
    want, size = ref.attention(q.double().numpy(), cache[0], cache[1], scales, tables, lens, qsl, 0.3)
    assert (np.abs(out.double().cpu().numpy() - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -9 * size).all()


@pytest.mark.parametrize("ctx,new", [([37, 130], [1, 1]), ([37, 130], [9, 40]), ([0, 120], [100, 3])])
def test_attention_nan_codes_that_no_one_sees(pkv, ctx, new):
    # behind the context, in other requests' blocks, and in the chunk's own later tokens (of K and V)
    tables, lens, qsl, pool = ref.requests(ctx, new, 2)
    cache, scales = ref.pool8(pool, 2, 2)
    plain = cache.copy()
    nan = np.ones((pool, 16), bool)
    for i, n in enumerate(lens):
        for p in range(int(n)):
            nan[tables[i][p // 16], p % 16] = False
    last = lens - 1  # each request's last token: seen by its own row alone
    for i in range(len(lens)):
        nan[tables[i][last[i] // 16], last[i] % 16] = True
    for c in range(2):
        cache[c][np.broadcast_to(nan[:, None, :], cache[c].shape[:3])] = 0x7f
    scales[~np.isin(np.arange(pool), tables)] = np.nan
    q = bf16((int(qsl[-1]), 4, 128), 1)
    out = pkv.paged_attention_q8(q.cuda(), *gpu(cache[0], cache[1], scales, tables, lens, qsl), 0.1, int(max(new)), int(lens.max()))
    got = out.double().cpu().numpy()
    want, size = ref.attention(q.double().numpy(), plain[0], plain[1], np.nan_to_num(scales), tables, lens, qsl, 0.1)
    ends = qsl[1:] - 1
    others = np.setdiff1d(np.arange(len(got)), ends)
    assert np.isnan(got[ends]).all()
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -9 * size)[others].all()


def test_attention_a_query_that_is_not_finite_spoils_its_row_alone(pkv):
    tables, lens, qsl, pool = ref.requests([50, 20], [6, 1], 2)
    cache, scales = ref.pool8(pool, 2, 2)
    q = bf16((7, 4, 128), 1)
    clean = q.clone()
    q[2, 1, 7], q[6, 3, 0] = float("inf"), float("nan")
    args = gpu(cache[0], cache[1], scales, tables, lens, qsl)
    a = pkv.paged_attention_q8(q.cuda(), *args, 0.1, 6, 56).float().cpu()
    b = pkv.paged_attention_q8(clean.cuda(), *args, 0.1, 6, 56).float().cpu()
    spoilt = torch.zeros((7, 4), dtype=torch.bool)
    spoilt[2, 1] = spoilt[6, 3] = True
    assert a[spoilt].isnan().all()
    want, size = ref.attention(clean.double().numpy(), cache[0], cache[1], scales, tables, lens, qsl, 0.1)
    near = np.abs(a.double().numpy() - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -9 * size
    assert near[~spoilt.numpy()].all() and torch.isfinite(b).all()


def test_attention_bad_pages_and_lengths(pkv):
    def change(cache, scales, tables, lens, qsl):
        tables[1, 2] = 10 ** 6
        tables[3, 0] = -1
    check_attention(pkv, [30, 60, 200, 5, 0], [1, 1, 1, 1, 1], 4, 2, seed=1, bad=(1, 3), change=change)
    check_attention(pkv, [30, 60, 200, 5, 0], [4, 70, 1, 9, 3], 4, 2, seed=1, bad=(1, 3), change=change)

    def shorter(cache, scales, tables, lens, qsl):
        lens[1] = 3  # fewer keys than tokens
    check_attention(pkv, [30, 60, 200], [4, 5, 1], 4, 2, seed=1, bad=(1,), change=shorter)
    check_attention(pkv, [30, 60, 200], [4, 5, 1], 4, 2, seed=1, max_q=4, bad=(1,))  # more tokens than said


def test_attention_leaves_rows_behind_the_last_request(pkv):
    tables, lens, qsl, pool = ref.requests([40, 3], [2, 1], 2)
    cache, scales = ref.pool8(pool, 2, 2)
    q = bf16((6, 4, 128), 1).cuda()
    out = torch.full_like(q, 7.0)
    assert pkv.paged_attention_q8(q, *gpu(cache[0], cache[1], scales, tables, lens, qsl), 0.1, 2, 42, out=out) is out
    assert (out[3:] == 7).all() and not (out[:3] == 7).any()


def test_attention_offsets_past_32_bits(pkv):
    # a pool of more than 4 GB, the request's blocks at its end
    hkv, pool = 8, 270000
    kc = torch.zeros((pool, hkv, 16, 128), dtype=torch.uint8, device="cuda")
    vc = torch.zeros_like(kc)
    sc = torch.ones((pool, hkv, 2), device="cuda")
    small, scales = ref.pool8(4, hkv, 1)
    ids = np.array([pool - 1, 7, pool - 3, pool - 2])
    at = torch.from_numpy(ids).cuda()
    kc[at], vc[at], sc[at] = gpu(small[0], small[1], scales)
    tables = ids[None].astype(np.int32)
    lens, qsl = np.array([60], np.int32), np.array([0, 1], np.int32)
    q = bf16((1, 8, 128), 1)
    out = pkv.paged_attention_q8(q.cuda(), kc, vc, sc, *gpu(tables, lens, qsl), 0.1, 1, 60)
    want, size = ref.attention(q.double().numpy(), small[0], small[1], scales, np.arange(4)[None], lens, qsl, 0.1)
    assert (np.abs(out.double().cpu().numpy() - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -9 * size).all()
    x = bf16((1, hkv, 128), 2).cuda()
    pkv.pkv_rope_append(x, x, None, kc, vc, *gpu(tables, np.array([61], np.int32), qsl), 1, scales=sc)
    assert kc[pool - 2, :, 12].any() and not kc[pool - 2 - (1 << 32) // (hkv * 2048), :, 12].any()


def test_attention_is_the_same_for_both_types_of_codes(pkv):
    tables, lens, qsl, pool = ref.requests([40, 3], [2, 1], 2)
    cache, scales = ref.pool8(pool, 2, 2)
    q = bf16((3, 4, 128), 1).cuda()
    kc, vc, *rest = gpu(cache[0], cache[1], scales, tables, lens, qsl)
    a = pkv.paged_attention_q8(q, kc, vc, *rest, 0.1, 2, 42)
    b = pkv.paged_attention_q8(q, kc.view(torch.float8_e4m3fn), vc.view(torch.float8_e4m3fn), *rest, 0.1, 2, 42)
    assert torch.equal(a, b)


@pytest.mark.parametrize("ctx,new", [([3000], [1]), ([700], [40]), ([0], [300]), ([130, 20], [3, 130])])
def test_attention_scores_that_grow_with_the_context(pkv, ctx, new):
    # every row's largest score lies near its end: references move again and again, within a tile too
    def change(cache, scales, tables, lens, qsl):
        for row, n in zip(tables, lens):
            blocks = row[:(n + 15) // 16]
            at = np.arange(len(blocks) * 16)
            for s in range(len(at)):
                cache[0, blocks[s // 16], :, s % 16, 0] = ref.encode8(np.full(1, 16.0))[0]
            scales[blocks, :, 0] = np.float32(2.0 ** -10) * (1 + np.arange(len(blocks)))[:, None]
    tables, lens, qsl, pool = ref.requests(ctx, new, 7)
    cache, scales = ref.pool8(pool, 2, 7)
    change(cache, scales, tables, lens, qsl)
    for size in (3.0, 300.0):
        q = bf16((int(qsl[-1]), 8, 128), 7, 0.1)
        q[..., 0] = size
        out = pkv.paged_attention_q8(q.cuda(), *gpu(cache[0], cache[1], scales, tables, lens, qsl), 0.5, max(new), int(lens.max()))
        want, of = ref.attention(q.double().numpy(), cache[0], cache[1], scales, tables, lens, qsl, 0.5)
        # a query's elements are held to 2^-22 of its largest one, half of that off at most: a score is off by g = 2^-23 max |q|
        # sum |K| scale, a weight's share by e^(2 g) (here, with one element 300 times the others, that is more than all else)
        grain = 2.0 ** -23 * size * 0.5 * (np.abs(ref.decode8(cache[0])).sum(-1).max(-1) * scales[..., 0]).max()
        assert grain < 0.2
        assert (np.abs(out.double().cpu().numpy() - want) <= 2.0 ** -8 * np.abs(want) + (2.0 ** -9 + np.expm1(2 * grain)) * of).all()


@pytest.mark.parametrize("new", [3, 40])
def test_attention_scores_that_grow_within_a_tile(pkv, new):
    # each 32 keys of a tile 2^20 above those before: a reference moves in every quarter of the tile, over weights that
    # have just been stored and sums that were rescaled a quarter before
    scale = 128 ** -0.5
    for ctx in (300, 450):
        tables, lens, qsl, pool = ref.requests([ctx], [new], 11)
        cache, scales = ref.pool8(pool, 2, 11)
        cache[0] = 0  # (scores come from one element alone)
        step = 20 * np.log(2.0)
        for p in range(int(lens[0])):
            cache[0, tables[0][p // 16], :, p % 16, 0] = ref.encode8(np.full(1, 2.0 * (p // 32)))[0]
        scales[..., 0] = 1.0
        q = torch.zeros((new, 4, 128)).bfloat16()
        q[..., 0] = step / (2.0 * scale)
        out = pkv.paged_attention_q8(q.cuda(), *gpu(cache[0], cache[1], scales, tables, lens, qsl), scale, new, int(lens[0]))
        want, of = ref.attention(q.double().numpy(), cache[0], cache[1], scales, tables, lens, qsl, scale)
        assert (np.abs(out.double().cpu().numpy() - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -9 * of).all()


@pytest.mark.parametrize("new", [1, 3, 40])
@pytest.mark.parametrize("far", [20, 25, 26, 30, 33, 38, 40])
def test_attention_a_key_far_above_others_of_its_tile(pkv, far, new):
    # a tile of small weights sets the references; of the next one the first 32 keys weigh 2^7.5 times as much, and a later one 2^far as
    # much, whose V is 0: what comes out are the 32, 2^(7.5 - far) of the largest, held to 2^-11 of themselves.  (So many requests, all
    # alike, that a CTA does all of one.)
    scale, ctx, requests = 128 ** -0.5, 256, 160
    tables, lens, qsl, pool = ref.requests([ctx], [new], 3)
    cache, scales = ref.pool8(pool, 2, 3)
    cache[0] = 0
    scales[:] = 1.0
    for p in range(int(lens[0])):
        at = cache[:, tables[0][p // 16], :, p % 16]
        at[0, :, 0] = ref.encode8(np.array([0.0 if p < 128 or p >= 160 else 4.0]))[0]
        at[0, :, 1] = ref.encode8(np.array([1.0 if p == 170 else 0.0]))[0]
        if p == 170:
            at[1] = 0
    q = torch.zeros((new, 8, 128)).bfloat16()
    q[..., 0], q[..., 1] = 7.5 * np.log(2.0) / (4.0 * scale), far * np.log(2.0) / scale
    out = pkv.paged_attention_q8(q.repeat(requests, 1, 1).cuda(), *gpu(cache[0], cache[1], scales, tables.repeat(requests, 0), lens.repeat(requests),
                                                                       (np.arange(requests + 1) * new).astype(np.int32)), scale, new, int(lens[0]))
    want, of = ref.attention(q.double().numpy(), cache[0], cache[1], scales, tables, lens, qsl, scale)
    off = np.abs(out.double().cpu().numpy().reshape(requests, *want.shape) - want)
    assert (off <= 2.0 ** -8 * np.abs(want) + 2.0 ** -9 * of + 2.0 ** -32 * int(lens[0]) * 448.0).all()


@pytest.mark.parametrize("scale", [-0.2, 0.0, 1e-30])
@pytest.mark.parametrize("new", [[1, 1], [1, 40]])
def test_attention_scales_of_the_scores(pkv, scale, new):
    tables, lens, qsl, pool = ref.requests([200, 77], new, 3)
    cache, scales = ref.pool8(pool, 2, 3)
    q = bf16((int(qsl[-1]), 6, 128), 3)
    out = pkv.paged_attention_q8(q.cuda(), *gpu(cache[0], cache[1], scales, tables, lens, qsl), scale, max(new), int(lens.max()))
    want, of = ref.attention(q.double().numpy(), cache[0], cache[1], scales, tables, lens, qsl, scale)
    assert (np.abs(out.double().cpu().numpy() - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -9 * of).all()


def test_attention_units_of_256_tokens(pkv):
    check_attention(pkv, [10, 0, 300], [700, 256, 257], 1, 1, seed=9)


@pytest.mark.parametrize("new", [[1, 1, 1], [1, 30, 5]])
def test_attention_into_rows_that_are_16_byte_aligned(pkv, new):
    tables, lens, qsl, pool = ref.requests([20, 0, 140], new, 5)
    cache, scales = ref.pool8(pool, 2, 5)
    q = bf16((int(qsl[-1]), 4, 128), 5).cuda()
    args = gpu(cache[0], cache[1], scales, tables, lens, qsl)
    want = pkv.paged_attention_q8(q, *args, 0.1, max(new), int(lens.max()))
    out = torch.full((q.numel() + 16,), 3.0, device="cuda").bfloat16()
    pkv.paged_attention_q8(q, *args, 0.1, max(new), int(lens.max()), out=out[8:-8].view(q.shape))
    assert torch.equal(out[8:-8].view(q.shape), want) and (out[:8] == 3).all() and (out[-8:] == 3).all()


# ----------------------------------------------------------------------------- sampling
def check_sample(pkv, x, u, **settings):
    """x fp32 or bf16 [N, V] (CPU), settings as numpy arrays."""
    given = {k: gpu(v) for k, v in settings.items() if v is not None}
    tokens, logprobs = pkv.pkv_sample(x if x.is_cuda else x.cuda(), gpu(np.asarray(u, np.float32)), **given)
    want, logs = ref.sample(x.float().cpu().numpy(), np.asarray(u, np.float32), **settings)
    np.testing.assert_array_equal(tokens.cpu().numpy(), want)
    got = logprobs.double().cpu().numpy()
    none = want < 0
    assert (got[none] == -np.inf).all()
    assert (np.abs(got[~none] - logs[~none]) <= 2.0 ** -22 * (1 + np.abs(logs[~none]))).all()


def peaked(n, v, seed, sigma=2.5, spikes=12):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((n, v)) * sigma
    return torch.from_numpy(x + (6 + 4 * rng.random((n, v))) * (rng.random((n, v)) < spikes / v)).float()


SETTINGS = [dict(), dict(top_k=50), dict(top_p=0.9), dict(min_p=0.02), dict(top_k=1000, top_p=0.95), dict(top_k=20, min_p=0.01, top_p=0.8),
            dict(min_p=1.0), dict(top_p=0.0), dict(top_k=1), dict(top_p=0.999999), dict(min_p=1e-9), dict(top_k=10 ** 9, top_p=1.0)]


@pytest.mark.parametrize("settings", SETTINGS)
@pytest.mark.parametrize("v,dtype", [(1, "f32"), (7, "bf16"), (1000, "f32"), (32000, "bf16"), (50257, "f32"), (128256, "bf16")])
def test_sample(pkv, settings, v, dtype):
    n = 6
    rng = np.random.default_rng(v)
    x = peaked(n, v, v).to(torch.float32 if dtype == "f32" else torch.bfloat16)
    s = {k: np.full(n, a, np.int32 if k == "top_k" else np.float32) for k, a in settings.items()}
    check_sample(pkv, x, rng.random(n, dtype=np.float32), temperature=(0.3 + 1.2 * rng.random(n)).astype(np.float32), **s)


@pytest.mark.parametrize("n,v", [(1, 300), (3, 9000), (40, 4097), (160, 2000), (400, 700)])
def test_sample_mixed_settings(pkv, n, v):
    rng = np.random.default_rng(n)
    pick = lambda of, t: rng.choice(of, n).astype(t)  # noqa: E731
    for dtype in (torch.float32, torch.bfloat16):
        check_sample(pkv, peaked(n, v, n).to(dtype), rng.random(n, dtype=np.float32), temperature=pick([0, 0.5, 1, 3], np.float32),
                     top_k=pick([0, -1, 5, 100], np.int32), top_p=pick([1, 0.5, 0.9, 2], np.float32), min_p=pick([0, -1, 0.1], np.float32))


@pytest.mark.parametrize("v", [5, 4096, 30000])
def test_sample_ties(pkv, v):
    # all logits the same: the mass of the first m is m, and borders are met exactly
    n = 8
    x = torch.zeros((n, v)).bfloat16()
    u = np.array([0, 0.25, 0.5, 0.75, 1 - 2.0 ** -24, 2.0 ** -30, 1e-38, 0.3], np.float32)
    check_sample(pkv, x, u)
    check_sample(pkv, x, u, top_k=np.full(n, 3, np.int32))
    check_sample(pkv, x, u, top_p=np.full(n, 0.5, np.float32))
    check_sample(pkv, x, u, top_p=np.full(n, 0.25, np.float32), top_k=np.full(n, v - 1, np.int32), min_p=np.ones(n, np.float32))
    two = x.clone()
    two[:, ::3] = 2.0  # two values
    check_sample(pkv, two, u)
    check_sample(pkv, two, u, top_k=np.full(n, v // 2, np.int32))
    few = torch.from_numpy(np.random.default_rng(v).integers(-3, 4, (n, v))).float()
    check_sample(pkv, few, u + np.float32(0), top_p=np.full(n, 0.8, np.float32))


@pytest.mark.parametrize("sigma", [1e-4, 0.1, 1.0, 30.0])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_sample_flat_and_sharp(pkv, sigma, dtype):
    n, v = 12, 40000
    rng = np.random.default_rng(3)
    x = torch.from_numpy(rng.standard_normal((n, v)) * sigma).to(dtype)
    u = rng.random(n, dtype=np.float32)
    check_sample(pkv, x, u)
    check_sample(pkv, x, u, top_p=np.full(n, 0.9, np.float32))
    check_sample(pkv, x, u, top_p=np.full(n, 0.3, np.float32), top_k=np.full(n, 30000, np.int32))
    check_sample(pkv, x + 100, u, min_p=np.full(n, 0.5, np.float32))


def test_sample_what_is_not_finite_is_no_candidate(pkv):
    x = peaked(5, 500, 1)
    x[0, ::2] = float("inf")
    x[1, :499] = -float("inf")
    x[2] = float("nan")
    x[3, 100:] = -float("inf")
    x[4, 3], x[4, 7] = float("nan"), float("inf")
    for kw in ({}, dict(temperature=np.zeros(5, np.float32)), dict(top_k=np.full(5, 1000, np.int32)), dict(top_p=np.full(5, 0.9, np.float32))):
        check_sample(pkv, x, np.full(5, 0.7), **kw)
    lowest = torch.full((1, 300), torch.finfo(torch.bfloat16).min).bfloat16()  # masked by the type's lowest value
    lowest[0, 200] = 1.0
    check_sample(pkv, lowest, [0.9])
    check_sample(pkv, torch.full((1, 300), -3.0e38), [0.5])


def test_sample_temperatures_at_the_ends(pkv):
    x = peaked(6, 3000, 2)
    check_sample(pkv, x, np.full(6, 0.9), temperature=np.array([1e-38, 1e-20, 1e-3, 100, 1e10, 3e38], np.float32))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("k", [20, 50, 1000, 9000, 10 ** 6])
def test_sample_top_k_that_ends_far_below_the_largest(pkv, dtype, k):
    # fewer than k logits within 2^-32 of the largest weight: which ones are kept matters to no sum
    n, v = 12, 9000
    x, u = peaked(n, v, k).to(dtype), np.random.default_rng(k).random(n, dtype=np.float32)
    u[:3] = 0.0, 1 - 2.0 ** -24, 1e-30
    s = dict(temperature=np.array([0.05, 0.1, 0.2, 0.3, 0.5, 1.0] * 2, np.float32), top_k=np.full(n, k, np.int32))
    check_sample(pkv, x, u, **s)
    check_sample(pkv, x, u, top_p=np.full(n, 0.95, np.float32), **s)
    check_sample(pkv, x, u, min_p=np.full(n, 1e-12, np.float32), **s)
    few = torch.full_like(x, torch.finfo(dtype).min)  # words that are not allowed have the type's lowest value
    few[:, 100:130] = x[:, 100:130]
    check_sample(pkv, few, u, **s)


def test_sample_settings_out_of_range_are_flagged(pkv):
    nan = float("nan")
    x = peaked(6, 100, 3)
    t = np.array([1, -1, nan, np.inf, 1, 1], np.float32)
    u = np.array([0.5, 0.5, 0.5, 0.5, 1.0, nan], np.float32)
    tokens, logs = pkv.pkv_sample(x.cuda(), gpu(u), temperature=gpu(t))
    assert pkv.pkv_peek_error_bits() == 32 and pkv.pkv_get_last_error() == pkv.PKV_ERR_INDEX
    assert int(tokens[0]) >= 0 and (tokens[1:] == -1).all() and (logs[1:] == -np.inf).all()
    for kw in (dict(top_p=nan), dict(top_p=-0.1), dict(min_p=nan), dict(min_p=1.5)):
        given = {k: torch.tensor([1.0 if k == "top_p" else 0.0, v], device="cuda") for k, v in kw.items()}
        tokens, _ = pkv.pkv_sample(x[:2].cuda(), gpu(u[:2]), **given)
        assert pkv.pkv_get_last_error() == pkv.PKV_ERR_INDEX and int(tokens[0]) >= 0 and int(tokens[1]) == -1


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_sample_padded_and_unaligned_rows(pkv, dtype):
    x = peaked(7, 1003, 4).to(dtype).cuda()
    for view in (x[:, :1000], x[:, 1:], x[:, 3:998], x[::2, 5:], x[:1, 1:2]):
        check_sample(pkv, view, np.linspace(0, 0.99, len(view)), top_p=np.full(len(view), 0.9, np.float32))


@pytest.mark.parametrize("v,sigma", [(5000, 1.0), (5000, 2.5), (128256, 1.0)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("border", ["uniform", "top_p"])
def test_sample_numbers_next_to_a_border(pkv, v, sigma, dtype, border):
    # a share of the weights up to a token, rounded to fp32: 2^-25 from the border at most, and sums have to tell on which side
    n, rng = 24, np.random.default_rng(v)
    x = torch.from_numpy(rng.standard_normal((n, v)) * sigma).to(dtype)
    share, kept = np.zeros(n, np.float32), np.zeros(n, bool)
    for i, row in enumerate(x.double().numpy()):
        w = np.cumsum(np.exp(np.sort(row)[::-1] - row.max()))
        at = w[int(np.searchsorted(w, rng.random() * w[-1]))] / w[-1]
        share[i] = min(at, 1 - 2.0 ** -20)
        kept[i] = abs(float(share[i]) - at) > 2.0 ** -29  # (closer ones are 64-bit sums' own rounding)
    x, share = x[torch.from_numpy(kept)], share[kept]
    assert len(x) > n // 2
    if border == "uniform":
        check_sample(pkv, x, share)
    else:
        check_sample(pkv, x, np.full(len(x), 1 - 2.0 ** -24), top_p=share)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("p", [1.0, 0.999, 0.99999, 1e-4])
def test_sample_numbers_next_to_0_and_1(pkv, dtype, p):
    u = np.array([0, 1e-30, 1e-7, 1e-4, 0.01, 0.99, 0.999, 0.9999, 0.99999, 1 - 2.0 ** -20, 1 - 2.0 ** -24] * 2, np.float32)
    x = torch.cat([peaked(11, 50257, 8), peaked(11, 50257, 9, sigma=1.0, spikes=0)]).to(dtype)
    for kw in ({}, dict(top_k=np.full(22, 20000, np.int32)), dict(min_p=np.full(22, 1e-4, np.float32)), dict(temperature=np.full(22, 1.5, np.float32))):
        check_sample(pkv, x, u, top_p=np.full(22, p, np.float32), **kw)


@pytest.mark.parametrize("n,v", [(100, 30000), (320, 40000)])
def test_sample_many_rows_of_a_large_vocabulary(pkv, n, v):
    rng = np.random.default_rng(n)
    u, p = rng.random(n, dtype=np.float32), np.full(n, 0.8, np.float32)
    check_sample(pkv, peaked(n, v, n, sigma=1.0).bfloat16(), u, top_p=p)
    x = torch.zeros((n, v))  # equal logits, two values, a few
    x[::3, ::2] = 1.0
    x[1::3] = torch.from_numpy(rng.integers(0, 5, (len(x[1::3]), v))).float()
    check_sample(pkv, x, u)
    check_sample(pkv, x.bfloat16(), u, top_p=p)


@pytest.mark.parametrize("n,v", [(70, 2048), (150, 2300), (40, 4096), (76, 5000), (3, 8192), (19, 9001)])
def test_sample_short_rows_of_several_ctas(pkv, n, v):
    # the shortest rows that 2, 4 and 8 CTAs share, beside a kernel that holds SMs, so that CTAs of a cluster begin apart
    x = peaked(n, v, v).bfloat16().cuda()
    u = np.random.default_rng(v).random(n, dtype=np.float32)
    gu, busy, side = gpu(u), torch.randn((2048, 2048), device="cuda"), torch.cuda.Stream()
    want, _ = ref.sample(x.float().cpu().numpy(), u)
    torch.cuda.synchronize()
    got = []
    for _ in range(30):
        with torch.cuda.stream(side):
            busy @ busy
        got.append(pkv.pkv_sample(x, gu)[0])
    for tokens in got:
        np.testing.assert_array_equal(tokens.cpu().numpy(), want)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("v,low", [(5000, -22.0), (40000, -24.0), (128256, -26.0), (1 << 20, -27.0)])
def test_sample_logprobs_of_words_far_down(pkv, v, low, dtype):
    # numbers next to 1 fall to the tail, whose words weigh 2^-32 to 2^-39 of the largest each: closer than sums are told apart, so
    # any word will do that is 2^-28 of the mass from the number's place, twice that with the number's own rounding of the target, and
    # V^2 2^-63 of the largest weight (whole weights are V 2^-63 off at most)
    n, rng = 8, np.random.default_rng(v)
    x = torch.from_numpy(low + 0.3 * rng.standard_normal((n, v)))
    x[:, 17] = 0.0
    t = rng.uniform(0.9, 1.0, n).astype(np.float32)
    x, u = x.to(dtype), 1 - 2.0 ** -23
    tokens, logprobs = pkv.pkv_sample(x.cuda(), gpu(np.full(n, u, np.float32)), temperature=gpu(t))
    near, far = 2.0 ** -27 + v * v * 2.0 ** -63, 0
    for row, temp, token, logprob in zip(x.double().numpy(), t.astype(np.float64), tokens.tolist(), logprobs.tolist()):
        order = np.argsort(-row, kind="stable")
        w = np.exp((row[order] - row.max()) / temp)
        upto = np.cumsum(w[::-1])[::-1]  # the mass from each word on: small ones first, so that 64 bits hold them
        at = int(np.nonzero(order == token)[0][0])
        want = np.log(w[at] / upto[0])
        assert abs(logprob - want) <= 2.0 ** -22 * (1 + abs(want))
        place = 1 - upto[at:at + 2] / upto[0]  # where the word begins, and the next one
        assert place[0] <= u + near and place[-1] >= u - near
        far += want < -20
    assert far > 0


def test_sample_largest_vocabulary(pkv):
    v = 1 << 20
    x = peaked(2, v, 5, sigma=1.0)
    check_sample(pkv, x, [0.3, 0.99999])
    check_sample(pkv, x.bfloat16(), [0.3, 0.99999], top_p=np.full(2, 0.9, np.float32))


def test_sample_repeats_bit_by_bit(pkv):
    x = peaked(20, 32000, 6, sigma=1.0).cuda()
    u = gpu(np.linspace(0, 0.999, 20).astype(np.float32))
    p = gpu(np.full(20, 0.9, np.float32))
    first = pkv.pkv_sample(x, u, top_p=p)
    first = [t.clone() for t in first]
    for _ in range(5):
        again = pkv.pkv_sample(x, u, top_p=p)
        assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])


# ----------------------------------------------------------------------------- together
def decode_loop(pkv, steps, graph=False):
    """A small model's loop: projections, append, attention, logits, sampling; returns the tokens and the state."""
    gen = torch.Generator(device="cuda").manual_seed(0)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    n, hq, hkv, d, vocab = 3, 4, 2, 128, 1000
    embed, proj, head = rnd(vocab, 64), rnd(64, (hq + 2 * hkv) * d) / 8, rnd(hq * d, vocab) / 10
    prompt = [20, 1, 40]
    most = max(prompt) + steps + 1
    cols = (most + 15) // 16
    tables = torch.randperm(n * cols, generator=gen, device="cuda").int().view(n, cols)
    kc, vc = (torch.zeros((n * cols, hkv, 16, d), dtype=torch.uint8, device="cuda") for _ in range(2))
    sc = torch.zeros((n * cols, hkv, 2), device="cuda")
    cs = gpu(ref.angles(most, 128))
    lens = gpu(np.array(prompt, np.int32))
    tokens = torch.randint(vocab, (sum(prompt),), generator=gen, device="cuda")
    u, temp, top_p = torch.rand((steps, n), generator=gen, device="cuda"), torch.full((n,), 0.8, device="cuda"), torch.full((n,), 0.9, device="cuda")
    record = []

    def step(tokens, lens, qsl, max_q, u):
        qkv = (embed[tokens] @ proj).bfloat16()
        q, k, v = split(qkv, hq, hkv, d)
        q = pkv.pkv_rope_append(k, v, cs, kc, vc, tables, lens, qsl, max_q, q=q, scales=sc)
        o = pkv.paged_attention_q8(q, kc, vc, sc, tables, lens, qsl, d ** -0.5, max_q, most)
        logits = o[(qsl[1:] - 1).long()].float().view(n, hq * d) @ head
        next_tokens, logprobs = pkv.pkv_sample(logits, u, temperature=temp, top_p=top_p)
        return q, o, logits, next_tokens, logprobs

    qsl = gpu(np.concatenate([[0], np.cumsum(prompt)]).astype(np.int32))
    state = step(tokens, lens, qsl, max(prompt), u[0])
    record.append([t.clone() for t in state])
    ones = torch.arange(n + 1, dtype=torch.int32, device="cuda")
    cur, uu = state[3].clone().long(), u[1].clone()
    if graph:
        lens2 = lens + 1
        held = [t.clone() for t in (kc, vc, sc)]
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            step(cur, lens2, ones, 1, uu)
        torch.cuda.synchronize()
        for t, h in zip((kc, vc, sc), held):
            t.copy_(h)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            state = step(cur, lens2, ones, 1, uu)
        for j in range(1, steps):
            lens2.copy_(lens + j)
            uu.copy_(u[j])
            g.replay()
            record.append([t.clone() for t in state])
            cur.copy_(state[3].long())
    else:
        for j in range(1, steps):
            state = step(cur, lens + j, ones, 1, u[j])
            record.append([t.clone() for t in state])
            cur = state[3].long()
    return record, (kc, vc, sc, tables, cs, lens)


def test_a_decoding_loop_against_its_parts_in_64_bits(pkv):
    steps = 12
    record, (kc, vc, sc, tables, cs, lens) = decode_loop(pkv, steps)
    # the cache as it is after the last step holds what every step saw, but for the codes of blocks whose scales grew since;
    # the last step's attention sees exactly it
    q, o, logits, tokens, _ = record[-1]
    n = len(lens)
    final = (lens + steps - 1).cpu().numpy()
    want, size = ref.attention(q.double().cpu().numpy(), kc.cpu().numpy(), vc.cpu().numpy(), sc.cpu().numpy(), tables.cpu().numpy(),
                               final, np.arange(n + 1), 128 ** -0.5)
    assert (np.abs(o.double().cpu().numpy() - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -9 * size).all()
    for _, _, logits, tokens, logprobs in record:
        share = torch.log_softmax(logits.double() / 0.8, 1).gather(1, tokens.long()[:, None])[:, 0]
        assert (logprobs > share - 1e-5).all() and (logprobs <= 0).all()  # of what top-p keeps it is more
    assert pkv.pkv_get_last_error() == 0


def test_a_decoding_loop_replayed_from_a_graph(pkv):
    a, state_a = decode_loop(pkv, 10)
    b, state_b = decode_loop(pkv, 10, graph=True)
    for j, (x, y) in enumerate(zip(a, b)):
        assert torch.equal(x[3], y[3]), j
        assert torch.equal(x[1], y[1]), j
    for x, y in zip(state_a[:3], state_b[:3]):
        assert torch.equal(x, y)


def test_calls_on_named_streams_and_two_at_once(pkv):
    tables, lens, qsl, pool = ref.requests([400, 900, 30], [1, 1, 1], 2)
    cache, scales = ref.pool8(pool, 2, 2)
    args = gpu(cache[0], cache[1], scales, tables, lens, qsl)
    x = peaked(30, 5000, 1).cuda()
    u = torch.rand(30, device="cuda")
    qs = [bf16((3, 4, 128), s).cuda() for s in range(8)]
    want = [pkv.paged_attention_q8(q, *args, 0.1, 1, 901).clone() for q in qs]
    drawn = pkv.pkv_sample(x, u)[0].clone()
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got, toks = [], []
    for i, q in enumerate(qs):
        got.append(pkv.paged_attention_q8(q, *args, 0.1, 1, 901, stream=streams[i % 2]))
        toks.append(pkv.pkv_sample(x, u, stream=streams[(i + 1) % 2])[0])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and all(torch.equal(t, drawn) for t in toks)


def test_two_graphs_of_the_attention_at_once(pkv):
    tables, lens, qsl, pool = ref.requests([3000, 900], [1, 1], 2)
    cache, scales = ref.pool8(pool, 2, 2)
    args = gpu(cache[0], cache[1], scales, tables, lens, qsl)
    qs = [bf16((2, 4, 128), s).cuda() for s in range(2)]
    want = [pkv.paged_attention_q8(q, *args, 0.1, 1, 3001).clone() for q in qs]
    graphs, outs = [], []
    for q in qs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(pkv.paged_attention_q8(q, *args, 0.1, 1, 3001))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_refusals_on_the_gpu(pkv):
    tables, lens, qsl, pool = ref.requests([40, 3], [1, 1], 2)
    cache, scales = ref.pool8(pool, 2, 2)
    kc, vc, sc, bt, sl, st = gpu(cache[0], cache[1], scales, tables, lens, qsl)
    q = bf16((2, 4, 128), 1).cuda()
    for kw in (dict(workspace=torch.empty(100, device="cuda")), dict(out=q.float())):
        with pytest.raises(ValueError):
            pkv.paged_attention_q8(q, kc, vc, sc, bt, sl, st, 0.1, 1, 41, **kw)
    with pytest.raises(ValueError):
        pkv.paged_attention_q8(q, kc, vc, sc.cpu(), bt, sl, st, 0.1, 1, 41)
    with pytest.raises(pkv.PkvError):
        pkv.paged_attention_q8(bf16((2, 34, 128), 1).cuda(), kc, vc, sc, bt, sl, st, 0.1, 1, 41)
    k = bf16((2, 2, 128), 1).cuda()
    both = torch.empty((3, 4, 128), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(pkv.PkvError):  # q_out overlaps q
        pkv.pkv_rope_append(k, k, None, kc, vc, bt, sl, st, 1, q=both[:2], q_out=both[1:], scales=sc)
    with pytest.raises(ValueError):
        pkv.pkv_rope_append(k.transpose(1, 2), k, None, kc, vc, bt, sl, st, 1, scales=sc)
    with pytest.raises(ValueError):
        pkv.pkv_rope_append(k.float(), k.float(), None, kc, vc, bt, sl, st, 1, scales=sc)
    with pytest.raises(pkv.PkvError):
        pkv.pkv_rope_append(k, k, torch.zeros((50, 24), device="cuda"), kc, vc, bt, sl, st, 1, scales=sc)
    with pytest.raises(ValueError):
        pkv.pkv_sample(torch.zeros((2, 10), device="cuda"), torch.zeros(2))
    torch.cuda.synchronize()
    assert torch.equal(kc.cpu(), torch.from_numpy(cache[0]))
