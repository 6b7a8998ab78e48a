"""The operators of a decoding step over a cache in 8 bits, as cases to measure.

Three operators:

* ``append``  a projection's new queries, keys and values: queries and keys rotated by their positions, keys
              and values put into the paged cache (bf16 or fp32, or 8 bits with a scale for each block and head);
* ``q8``      attention over a paged cache in 8 bits (e4m3) with a scale for each block and head;
* ``sample``  tokens drawn from logits, with temperature, top-k, min-p and top-p, from given random numbers.

``run`` computes a pass either in its plain form (elementary torch operations) or, where ``own`` is
true, through the calls of the package.  ``exact`` computes the same in 64 bits.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 16
LARGEST = 448.0  # of e4m3
LEAST_SCALE = 2.0 ** -80


# ----------------------------------------------------------------------------- cases
def listed():
    return [
        # one user's next token in one layer, a bf16 cache
        {"name": "append_one_user", "op": "append", "cache": "bf16", "seqs": 1, "lo": 500, "hi": 500, "new_lo": 1,
         "new_hi": 1, "hq": 32, "hkv": 8, "d": 128, "rot": 128, "interleaved": False},
        # a serving batch's next tokens, an 8-bit cache: the blocks' scales may have to grow
        {"name": "append_decode_q8", "op": "append", "cache": "e4m3", "seqs": 64, "lo": 128, "hi": 4096, "new_lo": 1,
         "new_hi": 1, "hq": 32, "hkv": 8, "d": 128, "rot": 128, "interleaved": False},
        # prompts, in chunks of up to 1024 tokens that begin anywhere in a block
        {"name": "append_prompts_q8", "op": "append", "cache": "e4m3", "seqs": 8, "lo": 0, "hi": 2000, "new_lo": 300,
         "new_hi": 1024, "hq": 32, "hkv": 8, "d": 128, "rot": 128, "interleaved": False},
        # an fp32 cache, small heads that are rotated in part, neighbours as pairs
        {"name": "append_f32", "op": "append", "cache": "f32", "seqs": 5, "lo": 100, "hi": 700, "new_lo": 3,
         "new_hi": 13, "hq": 8, "hkv": 2, "d": 64, "rot": 32, "interleaved": True},
        # one user's next token after a short context
        {"name": "q8_one_user", "op": "q8", "seqs": 1, "lo": 500, "hi": 500, "new_lo": 1, "new_hi": 1, "hq": 32,
         "hkv": 8},
        # an ordinary serving batch
        {"name": "q8_decode", "op": "q8", "seqs": 64, "lo": 128, "hi": 4096, "new_lo": 1, "new_hi": 1, "hq": 32,
         "hkv": 8},
        # long documents, eight query heads a kv head
        {"name": "q8_long", "op": "q8", "seqs": 32, "lo": 32768, "hi": 32768, "new_lo": 1, "new_hi": 1, "hq": 64,
         "hkv": 8},
        # prompts in chunks of 512 tokens
        {"name": "q8_chunks", "op": "q8", "seqs": 8, "lo": 0, "hi": 2048, "new_lo": 512, "new_hi": 512, "hq": 32,
         "hkv": 8},
        # ragged: fresh requests beside old ones, single tokens beside chunks, three query heads a kv head
        {"name": "q8_ragged", "op": "q8", "seqs": 33, "lo": 0, "hi": 1500, "new_lo": 1, "new_hi": 61, "hq": 12,
         "hkv": 4},
        # one user, a small vocabulary, the usual settings
        {"name": "sample_one_user", "op": "sample", "dtype": "bf16", "seqs": 1, "vocab": 32000, "pad": 0,
         "filters": "all"},
        # a batch over a large vocabulary, each request with settings of its own
        {"name": "sample_batch", "op": "sample", "dtype": "bf16", "seqs": 64, "vocab": 128256, "pad": 0,
         "filters": "mixed"},
        # fp32 logits of an odd vocabulary in padded rows, top-p alone: all of the mass counts
        {"name": "sample_top_p", "op": "sample", "dtype": "f32", "seqs": 33, "vocab": 50257, "pad": 47,
         "filters": "top_p"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


HEADS = ((32, 8), (64, 8), (8, 8), (12, 4), (16, 1), (14, 2), (10, 2), (28, 4))


def draw(rng):
    op = rng.choice(("append", "q8", "q8", "sample"))
    if op == "append":
        cache = rng.choice(("bf16", "e4m3", "e4m3", "f32"))
        hq, hkv = rng.choice(HEADS)
        d = rng.choice((64, 128)) if cache == "f32" else 128
        new = _log_int(rng, 1, 1024)
        return {"op": op, "cache": cache, "seqs": min(_log_int(rng, 1, 128), max(1, 4096 // new)),
                "lo": rng.randint(0, 100), "hi": _log_int(rng, 100, 4000), "new_lo": rng.randint(1, new),
                "new_hi": new, "hq": hq, "hkv": hkv, "d": d, "rot": rng.choice((d, d, d // 2, 16, 0)),
                "interleaved": rng.random() < 0.3}
    if op == "q8":
        hq, hkv = rng.choice(HEADS)
        new = 1 if rng.random() < 0.5 else _log_int(rng, 2, 512)
        hi = _log_int(rng, 16, 32768 if new == 1 else 4000)
        most = 32 * 32768 // hi if new == 1 else 8 * 512 * 2048 // (new * max(hi, 512))
        return {"op": op, "seqs": max(1, min(_log_int(rng, 1, 128), most)), "lo": rng.randint(0, hi), "hi": hi,
                "new_lo": rng.randint(1, new), "new_hi": new, "hq": hq, "hkv": hkv}
    vocab = _log_int(rng, 300, 130000)
    f32 = rng.random() < 0.5
    return {"op": op, "dtype": "f32" if f32 else "bf16", "vocab": vocab, "pad": rng.choice((0, 0, 1, 8, 37)),
            "seqs": min(_log_int(rng, 1, 256), max(1, 64 * 128256 // (vocab * (2 if f32 else 1)))),
            "filters": rng.choice(("all", "mixed", "mixed", "top_p", "none"))}


# ----------------------------------------------------------------------------- inputs
def _spread(lo, hi, n):
    """n whole numbers spread evenly over lo .. hi: the same ones for every seed, in another order."""
    return np.linspace(hi, lo, n).round().astype(np.int64) if n > 1 else np.array([hi])


def _tables(lens, rng, longest, slack=1.1):
    """Block tables of requests of these lengths, their blocks spread over the pool by chance."""
    held = (lens + BLOCK - 1) // BLOCK
    pool = int(math.ceil(slack * (int(lens.sum()) / BLOCK + len(held))))
    ids = rng.permutation(pool).astype(np.int32)
    tables = np.full((len(held), longest // BLOCK + 3), -1, np.int32)
    ends = np.cumsum(held)
    for i, n in enumerate(held):
        tables[i, :n] = ids[ends[i] - n:ends[i]]
    return tables, pool


def _sizes(case):
    """Each request's context before the call and its new tokens."""
    ctx = np.random.default_rng(1).permutation(_spread(case["lo"], case["hi"], case["seqs"]))
    return ctx, _spread(case["new_lo"], case["new_hi"], case["seqs"])


def _requests(case, rng):
    ctx, new = _sizes(case)
    order = rng.permutation(case["seqs"])
    new, lens = new[order], (ctx + new)[order].astype(np.int32)
    tables, pool = _tables(lens, rng, case["hi"] + case["new_hi"])
    qsl = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    return {"tables": dev(tables), "lens": dev(lens), "qsl": dev(qsl), "max_q": int(new.max()),
            "max_len": int(lens.max())}, lens, new, tables, qsl, pool


def _cache8(pool, hkv, d, gen):
    """A pool of keys and values in 8 bits, [2, pool, hkv, 16, d], and its scales [pool, hkv, 2]: what blocks hold that
    were filled with values whose size differs from block to block."""
    cache = torch.empty((2, pool, hkv, BLOCK, d), dtype=torch.uint8, device="cuda")
    scales = torch.empty((pool, hkv, 2), dtype=torch.float32, device="cuda")
    step = max(1, (1 << 27) // (hkv * BLOCK * d))
    for c in range(2):
        for a in range(0, pool, step):
            n = min(step, pool - a)
            size = torch.exp2(torch.rand((n, hkv, 1, 1), generator=gen, device="cuda") * 2 - 1)
            x = torch.randn((n, hkv, BLOCK, d), generator=gen, device="cuda") * size
            s = _scale_of(x.abs().amax((2, 3)))
            scales[a:a + n, :, c] = s
            cache[c, a:a + n] = (x / s[:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    return cache, scales


def _scale_of(amax):
    """The least power of two s with amax <= 448 s."""
    m, e = torch.frexp(amax.double() / LARGEST)
    return torch.ldexp(torch.ones_like(m), torch.where(m == 0.5, e - 1, e)).clamp(min=LEAST_SCALE).float()


def prepare(case, seed):
    return {"append": _prepare_append, "q8": _prepare_q8, "sample": _prepare_sample}[case["op"]](case, seed)


def _prepare_append(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    hq, hkv, d, rot = case["hq"], case["hkv"], case["d"], case["rot"]
    s, lens, new, tables, qsl, pool = _requests(case, rng)
    dtype = torch.float32 if case["cache"] == "f32" else torch.bfloat16
    # one projection makes queries, keys and values side by side
    qkv = torch.randn((int(qsl[-1]), (hq + 2 * hkv) * d), generator=gen, device="cuda").to(dtype)
    s["q"] = qkv[:, :hq * d].unflatten(1, (hq, d))
    s["k"] = qkv[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
    s["v"] = qkv[:, (hq + hkv) * d:].unflatten(1, (hkv, d))
    s["cos_sin"] = None
    if rot:
        angle = torch.arange(s["max_len"], dtype=torch.float64, device="cuda")[:, None] * torch.pow(
            500000.0, -torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
    if case["cache"] == "e4m3":
        s["cache"], s["scales"] = _cache8(pool, hkv, d, gen)
        touched = [tables[i, (lens[i] - new[i]) // BLOCK:(lens[i] - 1) // BLOCK + 1] for i in range(case["seqs"])]
        s["touched"] = torch.from_numpy(np.concatenate(touched).astype(np.int64)).cuda()
    else:
        s["cache"] = torch.randn((2, pool, hkv, BLOCK, d), generator=gen, device="cuda").to(dtype)
        s["scales"] = None
    return {**s, "op": "append", "interleaved": case["interleaved"]}


def _prepare_q8(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s, _, _, _, qsl, pool = _requests(case, rng)
    s["cache"], s["scales"] = _cache8(pool, case["hkv"], 128, gen)
    s["q"] = torch.randn((int(qsl[-1]), case["hq"], 128), generator=gen, device="cuda", dtype=torch.bfloat16)
    return {**s, "op": "q8", "scale": 1.0 / math.sqrt(128.0)}


def _prepare_sample(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    n, v = case["seqs"], case["vocab"]
    unit = lambda: torch.rand((n,), generator=gen, device="cuda")  # noqa: E731
    pick = lambda *of: torch.tensor(of, device="cuda")[torch.randint(len(of), (n,), generator=gen, device="cuda")]  # noqa: E731
    logits = torch.randn((n, v + case["pad"]), generator=gen, device="cuda") * 2.5
    # a few words of each row stand out, as in a model's answers
    logits += (6.0 + 4.0 * torch.rand(logits.shape, generator=gen, device="cuda")) * (
        torch.rand(logits.shape, generator=gen, device="cuda") < 12.0 / v)
    s = {"op": "sample", "logits": logits.to(torch.float32 if case["dtype"] == "f32" else torch.bfloat16)[:, :v],
         "uniform": unit(), "temperature": 0.5 + unit(), "top_k": None, "top_p": None, "min_p": None}
    if case["filters"] == "all":
        s["top_k"], s["top_p"], s["min_p"] = pick(20, 50, 100).int(), pick(0.8, 0.9, 0.95), pick(0.01, 0.05)
    if case["filters"] == "mixed":  # some greedy, some without a filter
        s["temperature"] = torch.where(unit() < 0.15, 0.0, s["temperature"])
        s["top_k"], s["top_p"], s["min_p"] = pick(0, 0, 40, 1000).int(), pick(1.0, 0.7, 0.9), pick(0.0, 0.0, 0.02)
    if case["filters"] == "top_p":
        s["top_p"] = 0.7 + 0.29 * unit()
    return s


# ----------------------------------------------------------------------------- one pass
def run(state):
    if own:
        import paged_kv_cache_248_gb300 as pkv
        return {"append": _own_append, "q8": _own_q8, "sample": _own_sample}[state["op"]](pkv, state)
    return {"append": _plain_append, "q8": _plain_q8, "sample": _plain_sample}[state["op"]](state)


def _held(s):
    """What the cache holds after an append: the cache itself, of one in 8 bits the values of the touched blocks."""
    if s["scales"] is None:
        return (s["cache"],)
    scales = s["scales"][s["touched"]]
    values = s["cache"][:, s["touched"]].view(torch.float8_e4m3fn).to(torch.bfloat16)
    return values * scales.bfloat16().permute(2, 0, 1)[:, :, :, None, None], scales


def _own_append(pkv, s):
    q = pkv.pkv_rope_append(s["k"], s["v"], s["cos_sin"], s["cache"][0], s["cache"][1], s["tables"], s["lens"], s["qsl"],
                            s["max_q"], q=s["q"], scales=s["scales"], interleaved=s["interleaved"])
    return q, *_held(s)


def _own_q8(pkv, s):
    return pkv.paged_attention_q8(s["q"], s["cache"][0], s["cache"][1], s["scales"], s["tables"], s["lens"], s["qsl"],
                                  s["scale"], s["max_q"], s["max_len"])


def _own_sample(pkv, s):
    return pkv.pkv_sample(s["logits"], s["uniform"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                          min_p=s["min_p"])


def _owner(qsl, n):
    """The request of each of n tokens, and the token's number in it."""
    t = torch.arange(n, device=qsl.device)
    i = torch.searchsorted(qsl, t, right=True) - 1
    return i, t - qsl[i]


def _rotated(x, row, interleaved):
    """Token t's heads x[t] rotated by the angles whose cosines and sines row[t] holds, in 32 bits."""
    rot = row.shape[1]
    cos, sin = row[:, None, :rot // 2], row[:, None, rot // 2:]
    x = x.float()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _plain_append(s):
    tables, lens, qsl = s["tables"].long(), s["lens"].long(), s["qsl"].long()
    i, j = _owner(qsl, s["k"].shape[0])
    ctx = lens - (qsl[1:] - qsl[:-1])
    p = ctx[i] + j
    block, at = tables[i, p // BLOCK], p % BLOCK
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    if s["cos_sin"] is not None:
        row = s["cos_sin"][p]
        q, k = _rotated(s["q"], row, s["interleaved"]), _rotated(s["k"], row, s["interleaved"])
    new = torch.stack([k, v])  # [2, T, hkv, d]
    cache = s["cache"]
    if s["scales"] is None:
        cache[:, block, :, at] = new.to(cache.dtype).transpose(0, 1)
        return q.to(s["q"].dtype), *_held(s)
    pool, hkv = cache.shape[1:3]
    # tokens of the request that a touched block has held so far; of any other block: all
    before = torch.full((pool,), BLOCK, dtype=torch.long, device=p.device)
    before[block] = (ctx[i] - p // BLOCK * BLOCK).clamp(min=0)
    least = torch.zeros((pool, hkv, 2), device=p.device).index_reduce_(0, block, new.abs().amax(-1).permute(1, 2, 0), "amax")
    touched = s["touched"]
    old = s["scales"][touched]
    scale = torch.maximum(torch.where(before[touched][:, None, None] > 0, old, 0.0), _scale_of(least[touched]))
    values = cache[:, touched].view(torch.float8_e4m3fn).float() * (old / scale).permute(2, 0, 1)[:, :, :, None, None]
    values = values.clamp(-LARGEST, LARGEST).to(torch.float8_e4m3fn).view(torch.uint8)
    keeps = torch.arange(BLOCK, device=p.device)[:, None] < before[touched][:, None, None, None]
    cache[:, touched] = torch.where(keeps, values, cache[:, touched])
    s["scales"][touched] = scale
    new = (new / s["scales"][block].permute(2, 0, 1)[..., None]).clamp(-LARGEST, LARGEST)
    cache[:, block, :, at] = new.to(torch.float8_e4m3fn).view(torch.uint8).transpose(0, 1)
    return q.to(s["q"].dtype), *_held(s)


def _plain_q8(s):
    q, tables, lens, qsl, cache = s["q"], s["tables"].long(), s["lens"].long(), s["qsl"].long(), s["cache"]
    n, hq, d = q.shape
    hkv = cache.shape[2]
    group, seqs, max_q = hq // hkv, lens.shape[0], s["max_q"]
    q_len = qsl[1:] - qsl[:-1]
    held = tables[:, :(s["max_len"] + BLOCK - 1) // BLOCK].clamp(min=0)
    most = held.shape[1] * BLOCK
    scales = s["scales"][held].permute(3, 0, 2, 1)[..., None, None]  # [2, seqs, hkv, blocks, 1, 1]
    kv = lambda c: (cache[c][held].view(torch.float8_e4m3fn).transpose(1, 2).float() * scales[c]).reshape(  # noqa: E731
        seqs, hkv, most, d)
    u = torch.arange(most, device=q.device)
    # queries in rows of their request, [seqs, max_q]
    j = torch.arange(max_q, device=q.device)
    t = torch.where(j < q_len[:, None], qsl[:-1, None] + j, 0)
    rows = q[t].float().view(seqs, max_q, hkv, group, d).permute(0, 2, 1, 3, 4).reshape(seqs, hkv, max_q * group, d)
    seen = u <= ((lens - q_len)[:, None] + j)[:, :, None]  # [seqs, max_q, most]
    score = torch.matmul(rows, kv(0).transpose(2, 3)).view(seqs, hkv, max_q, group, most) * s["scale"]
    score = torch.where(seen[:, None, :, None, :], score, -math.inf)
    p = torch.exp(score - score.amax(-1, keepdim=True))
    v = torch.where((u < lens[:, None])[:, None, :, None], kv(1), 0.0)
    o = torch.matmul(p.view(seqs, hkv, max_q * group, most), v).view(seqs, hkv, max_q, group, d)
    o = (o / p.sum(-1, keepdim=True)).permute(0, 2, 1, 3, 4).reshape(seqs, max_q, hq, d)
    i, at = _owner(qsl, n)
    return o[i, at].to(q.dtype)


def _plain_sample(s):
    # (in 64 bits: sums that decide between two words may lie closer together than 32 bits tell)
    x, dev = s["logits"].double(), s["logits"].device
    n, v = x.shape
    setting = lambda name, off: torch.full((n,), off, dtype=torch.float64, device=dev) if s[name] is None else s[name].double()  # noqa: E731
    top_k, top_p, min_p = setting("top_k", 0.0), setting("top_p", 1.0)[:, None], setting("min_p", 0.0)[:, None]
    temperature = s["temperature"].double()[:, None]
    greedy = temperature == 0
    x, at = torch.sort(x, dim=1, descending=True, stable=True)
    w = torch.exp((x - x[:, :1]) / torch.where(greedy, 1.0, temperature))
    most = torch.where(greedy[:, 0], 1.0, torch.where(top_k > 0, top_k, float(v)))[:, None]
    kept = (torch.arange(v, device=dev) < most) & (w >= min_p)
    w = torch.where(kept, w, 0.0)
    upto = torch.cumsum(w, 1)
    kept &= (upto - w < top_p * upto[:, -1:]) | (top_p >= 1.0)
    kept[:, 0] = True
    w = torch.where(kept, w, 0.0)
    upto = torch.cumsum(w, 1)
    mass = upto.gather(1, kept.sum(1, keepdim=True) - 1)
    place = (upto <= s["uniform"].double()[:, None] * mass).sum(1, keepdim=True)
    place = torch.minimum(place, kept.sum(1, keepdim=True) - 1)
    return at.gather(1, place)[:, 0].int(), torch.log(w.gather(1, place) / mass)[:, 0].float()


# ----------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    if case["op"] == "sample":
        n = case["seqs"] * case["vocab"]
        return {"bytes": n * (4 if case["dtype"] == "f32" else 2) + 28 * case["seqs"], "flops": 4.0 * n}
    ctx, new = _sizes(case)
    tokens = int(new.sum())
    if case["op"] == "append":
        size = 4 if case["cache"] == "f32" else 2
        held = 1 if case["cache"] == "e4m3" else size
        return {"bytes": tokens * case["d"] * (2 * case["hq"] * size + 2 * case["hkv"] * (size + held))
                + tokens * 4 * case["rot"] + 8 * case["seqs"],
                "flops": 3.0 * tokens * (case["hq"] + case["hkv"]) * case["rot"]}
    keys = int(ctx.sum()) + tokens
    seen = float((new * ctx + new * (new + 1) / 2).sum())
    return {"bytes": keys * (2 * case["hkv"] * (128 + 4 / BLOCK) + 4 / BLOCK) + tokens * 2 * case["hq"] * 128 * 2,
            "flops": 4.0 * seen * case["hq"] * 128}


# ----------------------------------------------------------------------------- the definition, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "q8": _exact_q8, "sample": _exact_sample}[case["op"]](s)


def _decode8(x):
    """The values of e4m3 bytes: sign, four bits of exponent (bias 7), three of mantissa."""
    x = x.long()
    e, m = x >> 3 & 15, (x & 7).double()
    value = torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * torch.exp2(e.double() - 7))
    return torch.where(x >= 128, -value, value)


def _round8(x):
    """The e4m3 value next to x, the even one of two; at most 448."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(x / step) * step).clamp(-LARGEST, LARGEST)


def _exact_append(s):
    tables, lens, qsl = s["tables"].cpu().numpy(), s["lens"].tolist(), s["qsl"].tolist()
    i_of = np.repeat(np.arange(len(lens)), np.diff(qsl))
    pos = np.concatenate([np.arange(n - (qsl[i + 1] - qsl[i]), n) for i, n in enumerate(lens)])
    q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
    if s["cos_sin"] is not None:
        row = s["cos_sin"].double()[torch.from_numpy(pos).cuda()]
        half = row.shape[1] // 2
        turn = torch.complex(row[:, :half], row[:, half:])[:, None]
        for x in (q, k):
            first, second = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if s["interleaved"] else (
                slice(0, half), slice(half, 2 * half))
            z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * turn
            x[..., first], x[..., second] = z.real, z.imag
    if s["scales"] is None:
        cache = s["cache"].double()
        block, at = torch.from_numpy(tables[i_of, pos // BLOCK]).long().cuda(), torch.from_numpy(pos % BLOCK).cuda()
        cache[0][block, :, at] = k
        cache[1][block, :, at] = v
        return q, cache
    found, scales = [], []
    for i, n in enumerate(lens):
        ctx = n - (qsl[i + 1] - qsl[i])
        for b in range(ctx // BLOCK, (n - 1) // BLOCK + 1):
            id_, a, e = int(tables[i, b]), max(ctx, b * BLOCK), min(n, (b + 1) * BLOCK)
            rows = slice(qsl[i] + a - ctx, qsl[i] + e - ctx)
            new = torch.stack([k[rows], v[rows]]).transpose(1, 2)  # [2, hkv, tokens, d]
            old = s["scales"][id_].double().T  # [2, hkv]
            need = torch.exp2(torch.ceil(torch.log2(new.abs().amax((2, 3)) / LARGEST))).clamp(min=LEAST_SCALE)
            scale = torch.maximum(old, need) if a > b * BLOCK else need
            code = _decode8(s["cache"][:, id_])
            kept = a - b * BLOCK
            code[:, :, :kept] = _round8(code[:, :, :kept] * (old / scale)[..., None, None])
            code[:, :, kept:kept + e - a] = _round8(new / scale[..., None, None])
            found.append(code * scale[..., None, None])
            scales.append(scale.T)
    return q, torch.stack(found, 1), torch.stack(scales)


def _exact_q8(s):
    tables, lens, qsl = s["tables"].tolist(), s["lens"].tolist(), s["qsl"].tolist()
    n, hq, d = s["q"].shape
    hkv = s["cache"].shape[2]
    out = torch.zeros((n, hq, d), dtype=torch.float64, device=s["q"].device)
    for i, length in enumerate(lens):
        t0, t1 = qsl[i], qsl[i + 1]
        ids = torch.tensor(tables[i][:(length + BLOCK - 1) // BLOCK], device=out.device)
        value = _decode8(s["cache"][:, ids]) * s["scales"][ids].double().permute(2, 0, 1)[..., None, None]
        k, v = value.transpose(1, 2).reshape(2, hkv, -1, d)[:, :, :length]
        last = torch.arange(length - (t1 - t0), length, device=out.device)[:, None]
        hidden = torch.arange(length, device=out.device) > last
        for h in range(hq):
            z = s["q"][t0:t1, h].double() @ k[h * hkv // hq].T * s["scale"]
            w = torch.softmax(z.masked_fill(hidden, -math.inf), 1)
            out[t0:t1, h] = w @ v[h * hkv // hq]
    return out


def _exact_sample(s):
    n, v = s["logits"].shape
    rows, u = s["logits"].double().cpu().numpy(), s["uniform"].double().cpu().numpy()
    setting = lambda name, off: np.full(n, off) if s[name] is None else s[name].double().cpu().numpy()  # noqa: E731
    top_k, top_p, min_p = setting("top_k", 0), setting("top_p", 1.0), setting("min_p", 0.0)
    temperature = s["temperature"].double().cpu().numpy()
    token, logprob = np.zeros(n, np.int32), np.zeros(n)
    for r in range(n):
        order = np.argsort(-rows[r], kind="stable")
        if temperature[r] == 0:
            token[r] = order[0]
            continue
        if top_k[r] > 0:
            order = order[:int(top_k[r])]
        w = np.exp((rows[r][order] - rows[r][order[0]]) / temperature[r])
        w = w[w >= min_p[r]]
        if top_p[r] < 1:
            w = w[:1 + int(np.searchsorted(np.cumsum(w), top_p[r] * math.fsum(w), side="left"))]
        mass = np.cumsum(w)
        at = min(int(np.searchsorted(mass, u[r] * mass[-1], side="right")), len(w) - 1)
        token[r], logprob[r] = order[at], math.log(w[at] / mass[-1])
    return torch.from_numpy(token), torch.from_numpy(logprob)
