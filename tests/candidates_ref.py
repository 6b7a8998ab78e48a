"""Plain 64-bit references for requests with several candidate continuations: attention of
drafted trees, the accepted path, beam selection and forked tables.  Host only, loops over
requests, no code shared with the package."""
from __future__ import annotations

import math

import numpy as np
import torch

BLOCK = 16


def tree_mask(parents, qsl, words):
    """(mask uint64 [T, words], depths int32 [T]) from each node's parent."""
    T = len(parents)
    mask, depths = np.zeros((T, words), np.uint64), np.zeros(T, np.int32)
    for i in range(len(qsl) - 1):
        for j in range(qsl[i + 1] - qsl[i]):
            u, d = j, -1
            while u >= 0:
                mask[qsl[i] + j, u // 64] |= np.uint64(1 << (u % 64))
                u, d = int(parents[qsl[i] + u]), d + 1
            depths[qsl[i] + j] = d
    return mask, depths


def random_parents(rng, n, chain=0.5):
    return np.array([j - 1 if j == 0 or rng.random() < chain else int(rng.integers(-1, j)) for j in range(n)], np.int32)


def tables_for(rng, lens, num_blocks=None, pad=2, junk=-1):
    """Distinct random blocks for requests of these lengths; entries behind them are `junk`."""
    held = [(int(n) + BLOCK - 1) // BLOCK for n in lens]
    pool = num_blocks or sum(held) + 3
    ids = rng.permutation(pool)[:sum(held)].astype(np.int32)
    tables = np.full((len(held), max(max(held), 1) + pad), junk, np.int32)
    at = 0
    for i, n in enumerate(held):
        tables[i, :n] = ids[at:at + n]
        at += n
    return tables, pool


def tree_attention(q, k_cache, v_cache, tables, lens, qsl, mask, scale):
    """(out, tol) in 64 bits [T, Hq, d]: the definition over the seen keys alone, and how far a
    right kernel may be off.

    The bound counts, per output, with A = sum p |v| (p the normalised weights):
      * each score: d products and sums in 32 bits, the scale and the subtraction of the maximum,
        at most (d + 8) 2^-24 sum |q k| |scale| of absolute error, which is e^that - 1 on p and
        the same on the normaliser (the largest of the row's keys is taken);
      * the sums over n keys in 32 bits: n 2^-24 each, twice, and 64 2^-24 for the exponents and joins;
      * bf16: one rounding of each weight, half a step (2^-8) of it;
      * one rounding of the result: half a step of the output's type."""
    T, hq, d = q.shape
    hkv = k_cache.shape[1]
    bf16 = q.dtype == torch.bfloat16
    out, tol = torch.zeros(T, hq, d, dtype=torch.float64), torch.zeros(T, hq, d, dtype=torch.float64)
    for i in range(len(lens)):
        n, m = int(lens[i]), int(qsl[i + 1] - qsl[i])
        ctx = n - m
        ids = torch.from_numpy(tables[i, :(n + BLOCK - 1) // BLOCK].astype(np.int64))
        k = k_cache[ids].double().transpose(0, 1).reshape(hkv, -1, d)[:, :n]
        v = v_cache[ids].double().transpose(0, 1).reshape(hkv, -1, d)[:, :n]
        for j in range(m):
            t = int(qsl[i]) + j
            seen = torch.tensor([u < ctx or bool(int(mask[t, (u - ctx) // 64]) >> ((u - ctx) % 64) & 1) for u in range(n)],
                                dtype=torch.bool)
            if not seen.any():
                continue
            for h in range(hq):
                ks, vs = k[h * hkv // hq][seen], v[h * hkv // hq][seen]
                s = ks @ q[t, h].double() * scale
                p = torch.softmax(s, 0)
                out[t, h] = p @ vs
                off = (d + 8) * 2.0**-24 * float((ks.abs() @ q[t, h].double().abs()).max()) * abs(scale)
                rel = 2 * math.expm1(off) + (2 * n + 64) * 2.0**-24 + (2.0**-8 if bf16 else 0.0)
                half = torch.finfo(q.dtype).eps / 2
                tol[t, h] = rel * (p @ vs.abs()) * (1 + half) + half * out[t, h].abs()
    return out, tol


def compact(path, path_lens, tables, lens, qsl, k_cache, v_cache):
    """New caches ([layers, blocks, Hkv, 16, d]) and lengths."""
    k, v, after = k_cache.clone(), v_cache.clone(), []
    for i in range(len(lens)):
        base = int(lens[i]) - int(qsl[i + 1] - qsl[i])
        for a in range(int(path_lens[i])):
            s, t = base + int(path[i, a]), base + a
            for new, old in ((k, k_cache), (v, v_cache)):
                new[:, tables[i, t // BLOCK], :, t % BLOCK] = old[:, tables[i, s // BLOCK], :, s % BLOCK]
        after.append(base + int(path_lens[i]))
    return k, v, np.array(after, np.int32)


def beam_select(logits, cum, select, finished=None, eos=0):
    """(scores float64, parents, tokens): all candidates sorted by score, then beam, then token."""
    N, W, V = logits.shape
    score, par, tok = np.full((N, select), -np.inf), np.full((N, select), -1, np.int32), np.full((N, select), -1, np.int32)
    x = logits.double().numpy()
    for n in range(N):
        s = np.full((W, V), -np.inf)
        for w in range(W):
            c = float(cum[n, w])
            if finished is not None and finished[n, w]:
                s[w, eos] = c
                continue
            with np.errstate(all="ignore"):
                top = x[n, w].max()
                lse = top + np.log(np.sum(np.exp(x[n, w] - top)))
                s[w] = c + (x[n, w] - lse)
        s = np.where(np.isfinite(s), s, -np.inf).reshape(-1)
        order = np.argsort(-s, kind="stable")[:select]
        live = [o for o in order if s[o] > -np.inf]
        for r, o in enumerate(live):
            score[n, r], par[n, r], tok[n, r] = s[o], o // V, o % V
    return score, par, tok


def fork(tables, lens, parents, refs, new, copy_block=lambda dst, src: None):
    """(new tables, new lengths, new counts), or None where the pool is too small."""
    refs = [int(c) for c in refs]
    n = [int(lens[p]) if p >= 0 else 0 for p in parents]
    rows = [[int(x) for x in tables[p][:(n[b] + BLOCK - 1) // BLOCK]] if p >= 0 else [] for b, p in enumerate(parents)]
    for r in tables:
        for x in r:
            if x >= 0:
                refs[x] -= 1
    for r in rows:
        for x in r:
            refs[x] += 1
    enders = {}
    for b, r in enumerate(rows):
        if new > 0 and n[b] % BLOCK:
            enders.setdefault(r[-1], []).append(b)
    copies = {}
    for x, bs in enders.items():
        for b in (bs[1:] if refs[x] == len(bs) else bs):
            copies[b] = x
    for x in copies.values():
        refs[x] -= 1
    free = [x for x, c in enumerate(refs) if c == 0]
    for b, r in enumerate(rows):
        want = ([copies[b]] if b in copies else [])
        fresh = (n[b] + new + BLOCK - 1) // BLOCK - len(r) if parents[b] >= 0 else 0
        if len(want) + fresh > len(free):
            return None
        if want:
            r[-1] = free.pop(0)
            refs[r[-1]] += 1
            copy_block(r[-1], want[0])
        for _ in range(fresh):
            r.append(free.pop(0))
            refs[r[-1]] += 1
    out = np.full(np.shape(tables), -1, np.int32)
    for b, r in enumerate(rows):
        out[b, :len(r)] = r
    return out, np.array(n, np.int32), np.array(refs, np.int32)
