"""Plain implementations of a decoding step over a cache in 8 bits: numpy, 64 bits (32 where the definition rounds), one
request and one head at a time."""
import math

import numpy as np
import torch

BLOCK = 16
LARGEST = np.float32(448.0)


def rotated(x, row, interleaved):
    """A head's row x (fp32) turned by row (cosines, sines), each product and difference rounded to fp32."""
    y, half = x.copy(), row.shape[0] // 2
    c, s = row[:half], row[half:]
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def decode8(codes):
    """Values of e4m3 codes."""
    c = codes.astype(np.int64)
    e, m = c >> 3 & 15, (c & 7) / 8.0
    v = np.where(e == 0, m * 2.0 ** -6, (1 + m) * np.exp2(e - 7.0))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c >= 128, -v, v)


def encode8(x):
    """The e4m3 codes next to x, even ones of two, at most +-448; NaN is 0x7f."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(np.where(np.isnan(x), 0.0, x)), 448.0)
    e = np.floor(np.log2(np.maximum(a, 2.0 ** -6)))
    n = np.rint(a / np.exp2(e - 3)).astype(np.int64)  # 8 .. 16 in the binade e; below 8: subnormal
    code = np.where(e <= -6, n, ((e + 7).astype(np.int64) << 3) + n - 8)
    code = np.where((e <= -6) & (n >= 8), 8 + n - 8, code)
    return np.where(np.isnan(x), 0x7f, np.where(np.signbit(x), 128 + code, code)).astype(np.uint8)


def scale_for(amax):
    """The least power of two s, at least 2^-80, with amax <= 448 s."""
    if amax == 0:
        return 2.0 ** -80
    m, e = math.frexp(float(amax) / 448.0)
    return max(2.0 ** (e - 1 if m == 0.5 else e), 2.0 ** -80)


def append(q, k, v, cos_sin, k_cache, v_cache, tables, lens, qsl, scales=None, positions=None, interleaved=False):
    """q, k, v fp32 [T, H, d]; caches fp32 (or uint8 codes, with scales), changed in place.  Returns q rotated."""
    out = None if q is None else q.copy()
    for i, n in enumerate(lens):
        t0, t1 = int(qsl[i]), int(qsl[i + 1])
        ctx = int(n) - (t1 - t0)
        rows = {}
        for t in range(t0, t1):
            p = ctx + t - t0
            kt, vt = k[t], v[t]
            if cos_sin is not None:
                row = cos_sin[p if positions is None else positions[t]]
                kt = rotated(kt, row, interleaved)
                if q is not None:
                    out[t] = rotated(q[t], row, interleaved)
            b, s = int(tables[i][p // BLOCK]), p % BLOCK
            if scales is None:
                k_cache[b, :, s], v_cache[b, :, s] = kt, vt
            else:
                rows.setdefault((p // BLOCK, b), []).append((s, kt, vt))
        for (j, b), new in rows.items():
            held = new[0][0]
            for c, cache in ((0, k_cache), (1, v_cache)):
                for h in range(k.shape[1]):
                    x = np.stack([r[1 + c][h] for r in new]).astype(np.float64)
                    old = float(scales[b, h, c]) if held else 0.0
                    now = max(old, scale_for(np.abs(x[np.isfinite(x)]).max(initial=0.0)))
                    if held and now != old:
                        cache[b, h, :held] = encode8(decode8(cache[b, h, :held]) * (old / now))
                    for r, (s, _, _) in enumerate(new):
                        cache[b, h, s] = encode8(x[r] / now)
                    scales[b, h, c] = now
    return out


def attention(q, k_cache, v_cache, scales, tables, lens, qsl, scale):
    """(out, mean of |V| under the weights), fp64 [T, Hq, 128]."""
    hq, hkv = q.shape[1], k_cache.shape[1]
    out, size = np.zeros(q.shape), np.zeros(q.shape)
    for i, n in enumerate(lens):
        t0, t1 = int(qsl[i]), int(qsl[i + 1])
        ids = np.asarray(tables[i][:(int(n) + BLOCK - 1) // BLOCK], np.int64)
        for g in range(hkv):
            k = (decode8(k_cache[ids, g]) * scales[ids, g, 0].astype(np.float64)[:, None, None]).reshape(-1, 128)
            v = (decode8(v_cache[ids, g]) * scales[ids, g, 1].astype(np.float64)[:, None, None]).reshape(-1, 128)
            for h in range(g * hq // hkv, (g + 1) * hq // hkv):
                for t in range(t0, t1):
                    seen = int(n) - (t1 - t0) + t - t0 + 1
                    s = k[:seen] @ q[t, h] * scale
                    w = np.exp(s - s.max())
                    w /= w.sum()
                    out[t, h], size[t, h] = w @ v[:seen], w @ np.abs(v[:seen])
    return out, size


def sample(logits, u, temperature=None, top_k=None, top_p=None, min_p=None):
    """(tokens, logprobs) of fp32 rows, in 64 bits."""
    n = logits.shape[0]
    token, logprob = np.full(n, -1, np.int32), np.full(n, -np.inf)
    for r in range(n):
        t = 1.0 if temperature is None else float(temperature[r])
        x = logits[r].astype(np.float64)
        order = np.argsort(-np.where(np.isfinite(x), x, -np.inf), kind="stable")[:int(np.isfinite(x).sum())]
        if len(order) == 0:
            continue
        if t == 0:
            token[r], logprob[r] = order[0], 0.0
            continue
        if top_k is not None and top_k[r] > 0:
            order = order[:int(top_k[r])]
        w = np.exp((x[order] - x[order[0]]) / t)
        if min_p is not None and min_p[r] > 0:
            w = w[w >= float(min_p[r])]
        if top_p is not None and top_p[r] < 1:
            upto = np.cumsum(w)
            w = w[:max(1, int(np.searchsorted(upto, float(top_p[r]) * math.fsum(w), side="left")) + 1)]
        upto = np.cumsum(w)
        at = min(int(np.searchsorted(upto, float(u[r]) * upto[-1], side="right")), len(w) - 1)
        token[r], logprob[r] = order[at], math.log(w[at] / upto[-1])
    return token, logprob


def requests(ctx, new, seed=0, slack=3, extra=2):
    """Tables, lengths and starts of requests (numpy), and the pool's number of blocks."""
    rng = np.random.default_rng(seed)
    ctx, new = np.asarray(ctx), np.asarray(new)
    lens = (ctx + new).astype(np.int32)
    held = (lens + BLOCK - 1) // BLOCK
    pool = int(held.sum()) + slack
    ids = rng.permutation(pool).astype(np.int32)
    tables = np.full((len(lens), int(held.max()) + extra), -1, np.int32)
    ends = np.cumsum(held)
    for i, n in enumerate(held):
        tables[i, :n] = ids[ends[i] - n:ends[i]]
    return tables, lens, np.concatenate([[0], np.cumsum(new)]).astype(np.int32), pool


def pool8(pool, hkv, seed=0):
    """Codes [2, pool, hkv, 16, 128] and scales [pool, hkv, 2] of values whose size differs from block to block."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((2, pool, hkv, BLOCK, 128)).astype(np.float32)
    scales = np.exp2(rng.integers(-9, -5, (pool, hkv, 2))).astype(np.float32)
    codes = torch.from_numpy(x / scales.transpose(2, 0, 1)[..., None, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return codes.view(torch.uint8).numpy(), scales


def angles(n, rot, seed=0, base=10000.0):
    a = np.arange(n)[:, None] * base ** (-np.arange(0, rot, 2) / max(rot, 1))
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)
