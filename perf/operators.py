"""The operators for several candidate continuations of a request over the paged cache, as cases to measure.

Four operators:

* ``tree``     attention of drafted tokens, which form a tree, over the paged cache;
* ``compact``  the accepted path of such a tree moved together in the cache, in every layer;
* ``beam``     the best continuations of a group of beams out of their logits;
* ``fork``     block tables reordered after the beams they continue: reference counts, freed blocks,
               private copies of shared last blocks, fresh blocks for the tokens to come.

``run`` computes a pass either in its plain form (elementary torch operations) or, where ``own`` is
true, through the calls of the package.  ``exact`` computes the same in 64 bits, request by request.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 16


# ----------------------------------------------------------------------------- cases
def listed():
    return [
        # one user waiting for an answer: a handful of drafted tokens after a short context
        {"name": "tree_one_user", "op": "tree", "dtype": "bf16", "seqs": 1, "lo": 500, "hi": 500, "nodes_lo": 7,
         "nodes_hi": 7, "hq": 32, "hkv": 8, "d": 128},
        # an ordinary serving batch, a small tree for each request
        {"name": "tree_batch", "op": "tree", "dtype": "bf16", "seqs": 64, "lo": 128, "hi": 4096, "nodes_lo": 16,
         "nodes_hi": 16, "hq": 32, "hkv": 8, "d": 128},
        # long documents with wide trees: 64 drafted tokens of 8 query heads a kv head are 512 rows
        {"name": "tree_long", "op": "tree", "dtype": "bf16", "seqs": 8, "lo": 32768, "hi": 32768, "nodes_lo": 64,
         "nodes_hi": 64, "hq": 64, "hkv": 8, "d": 128},
        # ragged: fresh requests beside old ones, single tokens beside large trees, three query heads a kv head
        {"name": "tree_ragged", "op": "tree", "dtype": "bf16", "seqs": 33, "lo": 0, "hi": 1500, "nodes_lo": 1,
         "nodes_hi": 61, "hq": 12, "hkv": 4, "d": 128},
        # an fp32 cache, small heads
        {"name": "tree_f32", "op": "tree", "dtype": "f32", "seqs": 5, "lo": 100, "hi": 700, "nodes_lo": 3,
         "nodes_hi": 13, "hq": 8, "hkv": 2, "d": 64},
        # after a verification step: one layer's cache at a time
        {"name": "compact_layer", "op": "compact", "dtype": "bf16", "layers": 1, "seqs": 33, "ctx": 300, "nodes": 16,
         "accept": 5, "hkv": 8, "d": 128},
        # the same for a whole model's cache in one call
        {"name": "compact_model", "op": "compact", "dtype": "bf16", "layers": 32, "seqs": 64, "ctx": 250, "nodes": 64,
         "accept": 12, "hkv": 8, "d": 128},
        # one request, four beams, a small vocabulary
        {"name": "beam_one_user", "op": "beam", "dtype": "bf16", "seqs": 1, "beams": 4, "vocab": 32000, "select": 8,
         "finished": False},
        # a batch of requests over a large vocabulary
        {"name": "beam_batch", "op": "beam", "dtype": "bf16", "seqs": 64, "beams": 4, "vocab": 128256, "select": 8,
         "finished": False},
        # wide beams, fp32 logits, an odd vocabulary, some beams at their end
        {"name": "beam_wide", "op": "beam", "dtype": "f32", "seqs": 9, "beams": 16, "vocab": 50257, "select": 32,
         "finished": True},
        # one request's beams after a step
        {"name": "fork_one_user", "op": "fork", "dtype": "bf16", "layers": 1, "seqs": 1, "beams": 5, "prompt": 200,
         "done": 75, "hkv": 8, "d": 128},
        # a batch's beams after a step, with the last blocks of all layers copied
        {"name": "fork_batch", "op": "fork", "dtype": "bf16", "layers": 16, "seqs": 64, "beams": 8, "prompt": 1000,
         "done": 150, "hkv": 8, "d": 128},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("tree", "tree", "compact", "beam", "fork"))
    if op == "tree":
        f32 = rng.random() < 0.2
        hi = _log_int(rng, 16, 4000 if f32 else 32768)
        seqs = min(_log_int(rng, 1, 128), max(1, (16384 if f32 else 262144) // hi))
        nodes = _log_int(rng, 1, 24 if f32 else 64)
        hq, hkv = rng.choice(((32, 8), (64, 8), (8, 8), (12, 4), (16, 1), (14, 2), (10, 2)))
        return {"op": op, "dtype": "f32" if f32 else "bf16", "seqs": seqs, "lo": rng.randint(0, hi), "hi": hi,
                "nodes_lo": rng.randint(1, nodes), "nodes_hi": nodes, "hq": hq, "hkv": hkv,
                "d": rng.choice((64, 128)) if f32 else 128}
    if op == "compact":
        f32 = rng.random() < 0.25
        nodes = rng.randint(2, 64)
        return {"op": op, "dtype": "f32" if f32 else "bf16", "layers": _log_int(rng, 1, 16 if f32 else 32),
                "seqs": _log_int(rng, 1, 64), "ctx": rng.randint(0, 250), "nodes": nodes,
                "accept": rng.randint(1, min(nodes, 12)), "hkv": rng.choice((1, 2, 8)),
                "d": rng.choice((64, 128)) if f32 else 128}
    if op == "beam":
        beams = rng.choice((1, 2, 3, 4, 5, 8, 16))
        vocab = _log_int(rng, 300, 130000)
        f32 = rng.random() < 0.4
        seqs = min(_log_int(rng, 1, 64), max(1, 64 * 4 * 128256 // (beams * vocab * (2 if f32 else 1))))
        return {"op": op, "dtype": "f32" if f32 else "bf16", "seqs": seqs, "beams": beams, "vocab": vocab,
                "select": rng.randint(1, min(64, 2 * beams + 2)), "finished": rng.random() < 0.4}
    return {"op": op, "dtype": "bf16", "layers": _log_int(rng, 1, 16), "seqs": _log_int(rng, 1, 64),
            "beams": rng.randint(2, 8), "prompt": _log_int(rng, 20, 1000), "done": rng.randint(1, 150),
            "hkv": rng.choice((1, 2, 8)), "d": 128}


# ----------------------------------------------------------------------------- inputs
def _dtype(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def _spread(lo, hi, n):
    """n whole numbers spread evenly over lo .. hi: the same ones for every seed, in another order."""
    return np.linspace(hi, lo, n).round().astype(np.int64) if n > 1 else np.array([hi])


def _tables(lens, rng, total, longest, slack=1.1):
    """Block tables of requests of these lengths (`total` tokens in all, each at most `longest`), their
    blocks spread over the pool by chance."""
    held = [(int(n) + BLOCK - 1) // BLOCK for n in lens]
    pool = int(math.ceil(slack * (total / BLOCK + len(held))))
    ids = rng.permutation(pool).astype(np.int32)
    tables = np.full((len(held), longest // BLOCK + 3), -1, np.int32)
    at = 0
    for i, n in enumerate(held):
        tables[i, :n] = ids[at:at + n]
        at += n
    return tables, pool


def prepare(case, seed):
    return {"tree": _prepare_tree, "compact": _prepare_compact, "beam": _prepare_beam,
            "fork": _prepare_fork}[case["op"]](case, seed)


def _prepare_tree(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s, dtype = case["seqs"], _dtype(case)
    nodes = rng.permutation(_spread(case["nodes_lo"], case["nodes_hi"], s))
    ctx = rng.permutation(_spread(case["lo"], case["hi"], s))
    lens = (ctx + nodes).astype(np.int32)
    tables, pool = _tables(lens, rng, int(lens.sum()), case["hi"] + case["nodes_hi"])
    qsl = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
    words = (int(nodes.max()) + 63) // 64
    mask = np.zeros((int(qsl[-1]), words), np.uint64)
    for i in range(s):  # each drafted token continues an earlier one, or the context
        for j in range(int(nodes[i])):
            t = qsl[i] + j
            parent = int(rng.integers(-1, j)) if j and rng.random() < 0.5 else j - 1
            if parent >= 0:
                mask[t] = mask[qsl[i] + parent]
            mask[t, j // 64] |= np.uint64(1 << (j % 64))
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    draw_n = lambda *shape: torch.randn(shape, generator=gen, device="cuda", dtype=dtype)  # noqa: E731
    return {"op": "tree", "q": draw_n(int(qsl[-1]), case["hq"], case["d"]),
            "k_cache": draw_n(pool, case["hkv"], BLOCK, case["d"]),
            "v_cache": draw_n(pool, case["hkv"], BLOCK, case["d"]), "tables": dev(tables), "lens": dev(lens),
            "qsl": dev(qsl), "mask": dev(mask.view(np.int64)), "scale": 1.0 / math.sqrt(case["d"]),
            "max_q": int(nodes.max()), "max_len": int(lens.max())}


def _prepare_compact(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s, nodes, accept = case["seqs"], case["nodes"], case["accept"]
    ctx = rng.permutation(_spread(0, case["ctx"], s))
    lens = (ctx + nodes).astype(np.int32)
    tables, pool = _tables(lens, rng, int(lens.sum()), case["ctx"] + nodes)
    path = np.full((s, accept), -1, np.int32)
    path_lens = _path_lens(case)[rng.permutation(s)]
    for i in range(s):
        # the first drafted token is always kept, the later ones come from anywhere behind it
        rest = np.sort(rng.permutation(np.arange(2, max(2, nodes)))[:path_lens[i] - 1])
        path[i, :path_lens[i]] = np.concatenate([[0], rest])
    shape = (case["layers"], pool, case["hkv"], BLOCK, case["d"])
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    return {"op": "compact", "k_cache": torch.randn(shape, generator=gen, device="cuda", dtype=_dtype(case)),
            "v_cache": torch.randn(shape, generator=gen, device="cuda", dtype=_dtype(case)), "tables": dev(tables),
            "lens": dev(lens), "qsl": dev(np.arange(s + 1, dtype=np.int32) * nodes), "path": dev(path),
            "path_lens": dev(path_lens)}


def _path_lens(case):
    most = max(1, min(case["accept"], case["nodes"] - 1))
    return (np.arange(case["seqs"]) % most + 1).astype(np.int32)


def _prepare_beam(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s, w, v = case["seqs"], case["beams"], case["vocab"]
    logits = torch.randn((s, w, v), generator=gen, device="cuda") * 2.5
    # a few words of each beam stand out, as in a model's answers
    logits += 6.0 * (torch.rand((s, w, v), generator=gen, device="cuda") < 12.0 / v)
    cum = -3.0 * torch.rand((s, w), generator=gen, device="cuda") - 5.0
    state = {"op": "beam", "logits": logits.to(_dtype(case)), "cum": cum, "select": case["select"],
             "finished": None, "eos": 2}
    if case["finished"]:
        state["finished"] = torch.rand((s, w), generator=gen, device="cuda") < 0.3
        state["cum"] = torch.where(state["finished"], cum - 4.0, cum)
    return state


def _prepare_fork(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s, w = case["seqs"], case["beams"]
    shared = case["prompt"] // BLOCK  # a request's beams share the prompt's full blocks
    done = rng.permutation(_spread(case["done"] // 2, case["done"], s))
    lens = np.repeat(case["prompt"] + done, w).astype(np.int32)
    held = (lens + BLOCK - 1) // BLOCK
    need = s * shared + int((held - shared).sum())
    pool = int(1.2 * need) + 4 * s * w
    ids = rng.permutation(pool).astype(np.int32)
    tables = np.full((s * w, (case["prompt"] + case["done"]) // BLOCK + 3), -1, np.int32)
    at = 0
    for i in range(s):
        common, at = ids[at:at + shared], at + shared
        for b in range(i * w, (i + 1) * w):
            own_blocks = int(held[b]) - shared
            tables[b, :shared] = common
            tables[b, shared:held[b]] = ids[at:at + own_blocks]
            at += own_blocks
    refs = np.bincount(tables[tables >= 0], minlength=pool).astype(np.int32)
    kept = (w + 1) // 2  # half of the beams go on, each with one continuation or more
    parents = np.empty((s, w), np.int32)
    for i in range(s):
        alive = rng.permutation(w)[:kept]
        parents[i] = i * w + rng.permutation(np.concatenate([alive, rng.choice(alive, w - kept)]))
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    shape = (case["layers"], pool, case["hkv"], BLOCK, case["d"])
    return {"op": "fork", "tables": dev(tables), "lens": dev(lens), "parents": dev(parents.reshape(-1)),
            "refs": dev(refs), "k_cache": torch.randn(shape, generator=gen, device="cuda", dtype=_dtype(case)),
            "v_cache": torch.randn(shape, generator=gen, device="cuda", dtype=_dtype(case)), "new_tokens": 1}


# ----------------------------------------------------------------------------- one pass
def run(state):
    if own:
        import paged_kv_cache_248_gb300 as pkv
        return {"tree": _own_tree, "compact": _own_compact, "beam": _own_beam, "fork": _own_fork}[state["op"]](pkv, state)
    return {"tree": _plain_tree, "compact": _plain_compact, "beam": _plain_beam, "fork": _plain_fork}[state["op"]](state)


def _own_tree(pkv, s):
    return pkv.paged_attention_tree(s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lens"], s["qsl"], s["mask"],
                                    s["scale"], s["max_q"], s["max_len"])


def _own_compact(pkv, s):
    lens = pkv.pkv_compact_path(s["path"], s["path_lens"], s["tables"], s["lens"], s["qsl"], s["k_cache"],
                                s["v_cache"])
    return s["k_cache"], s["v_cache"], lens


def _own_beam(pkv, s):
    return pkv.pkv_beam_select(s["logits"], s["cum"], s["select"], finished=s["finished"], eos_token=s["eos"])


def _own_fork(pkv, s):
    tables, lens = pkv.pkv_fork_tables(s["tables"], s["lens"], s["parents"], s["refs"], s["k_cache"], s["v_cache"],
                                       new_tokens=s["new_tokens"])
    s["tables"], s["lens"] = tables, lens
    return tables, lens, s["refs"], s["k_cache"], s["v_cache"]


def _plain_tree(s):
    q, tables, lens, qsl = s["q"], s["tables"].long(), s["lens"].long(), s["qsl"].long()
    n, hq, d = q.shape
    hkv = s["k_cache"].shape[1]
    group = hq // hkv
    seqs, most = lens.shape[0], s["max_len"]
    q_len = qsl[1:] - qsl[:-1]
    u = torch.arange(most, device=q.device)
    block = tables[:, u // BLOCK].clamp(min=0)
    k = s["k_cache"][block, :, u % BLOCK].float()  # [seqs, most, hkv, d]
    v = s["v_cache"][block, :, u % BLOCK].float()
    # queries in rows of their request, [seqs, max_q]
    j = torch.arange(s["max_q"], device=q.device)
    real = j < q_len[:, None]
    t = torch.where(real, qsl[:-1, None] + j, 0)
    rows = q[t].float().view(seqs, s["max_q"], hkv, group, d)
    # key u of request i is seen by drafted token j: context, or a bit of j's mask
    node = u - (lens - q_len)[:, None]  # [seqs, most]
    bit = node.clamp(min=0)
    word = s["mask"][t].gather(2, (bit // 64).clamp(max=s["mask"].shape[1] - 1)[:, None, :].expand(-1, s["max_q"], -1))
    drafted = ((word >> (bit % 64)[:, None, :]) & 1).bool() & (node < q_len[:, None])[:, None, :]
    seen = torch.where((node < 0)[:, None, :], True, drafted)  # [seqs, max_q, most]
    live = u < lens[:, None]
    v = torch.where(live[:, :, None, None], v, 0.0)
    score = torch.matmul(rows.permute(0, 2, 1, 3, 4).reshape(seqs, hkv, s["max_q"] * group, d),
                         k.permute(0, 2, 3, 1)).view(seqs, hkv, s["max_q"], group, most) * s["scale"]
    score = torch.where(seen[:, None, :, None, :], score, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(torch.isinf(top), 0.0, top))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(seqs, hkv, s["max_q"] * group, most), v.permute(0, 2, 1, 3))
    o = o.view(seqs, hkv, s["max_q"], group, d) / torch.where(total > 0, total, 1.0)
    o = o.permute(0, 2, 1, 3, 4).reshape(seqs * s["max_q"], hq, d)
    # each token's row in the padded layout
    i = torch.searchsorted(qsl, torch.arange(n, device=q.device), right=True) - 1
    return o[i * s["max_q"] + torch.arange(n, device=q.device) - qsl[i]].to(q.dtype)


def _plain_compact(s):
    path, path_lens, tables, lens = s["path"].long(), s["path_lens"].long(), s["tables"].long(), s["lens"].long()
    base = lens - (s["qsl"][1:] - s["qsl"][:-1]).long()
    i, a = ((torch.arange(path.shape[1], device=path.device) < path_lens[:, None]) & (path >= 0)).nonzero(as_tuple=True)
    src, dst = base[i] + path[i, a], base[i] + a
    sb, so, db, do = tables[i, src // BLOCK], src % BLOCK, tables[i, dst // BLOCK], dst % BLOCK
    s["k_cache"][:, db, :, do] = s["k_cache"][:, sb, :, so]
    s["v_cache"][:, db, :, do] = s["v_cache"][:, sb, :, so]
    return s["k_cache"], s["v_cache"], (base + path_lens).int()


def _plain_beam(s):
    x = s["logits"].double()  # candidates of two beams may lie closer together than 32 bits tell
    n, w, v = x.shape
    top = x.amax(-1, keepdim=True)
    lse = top + torch.log(torch.exp(x - top).sum(-1, keepdim=True))
    score = s["cum"].double()[:, :, None] + (x - lse)
    if s["finished"] is not None:  # a finished beam stands for itself
        end = torch.where(torch.arange(v, device=x.device) == s["eos"], s["cum"].double()[:, :, None], -math.inf)
        score = torch.where(s["finished"][:, :, None], end, score)
    score = torch.where(torch.isfinite(score), score, -math.inf).view(n, w * v)
    best, at = torch.sort(score, dim=1, descending=True, stable=True)
    best, at = best[:, :s["select"]], at[:, :s["select"]]
    none = torch.isinf(best)
    return best.float(), torch.where(none, -1, at // v).int(), torch.where(none, -1, at % v).int()


def _plain_fork(s):
    tables, lens, parents, refs, new = s["tables"].long(), s["lens"].long(), s["parents"].long(), s["refs"], s["new_tokens"]
    rows, cols = tables.shape
    pool, dev = refs.shape[0], tables.device
    from_row = parents.clamp(min=0)
    kept = parents >= 0
    n = torch.where(kept, lens[from_row], 0)
    held = (n + BLOCK - 1) // BLOCK
    col = torch.arange(cols, device=dev)
    out = torch.where((col < held[:, None]) & kept[:, None], tables[from_row], -1)
    count = lambda t: torch.zeros(pool + 1, dtype=torch.int32, device=dev).index_add_(  # noqa: E731
        0, torch.where(t >= 0, t, pool).reshape(-1), torch.ones(t.numel(), dtype=torch.int32, device=dev))
    left = torch.zeros(pool + 1, dtype=torch.int32, device=dev)
    left[:pool] = refs
    left += count(out) - count(tables)
    left[pool] = 1
    # a shared last block with room in it: its first row goes on with it, the others get a copy
    partial = (n % BLOCK != 0) & kept & (new > 0)
    row = torch.arange(rows, device=dev)
    last = torch.where(partial, out.gather(1, (held - 1).clamp(min=0)[:, None])[:, 0], pool)
    sharers = count(torch.where(partial, last, -1))
    first = torch.full((pool + 1,), rows, dtype=torch.int64, device=dev).scatter_reduce_(0, last, row, "amin")
    copy = partial & ((left[last] > sharers[last]) | (first[last] != row))
    left -= count(torch.where(copy, last, -1))
    left[pool] = 1
    grow = torch.where(kept, (n + new + BLOCK - 1) // BLOCK - held, 0)
    need = copy.long() + grow
    start = torch.cumsum(need, 0) - need
    free = torch.argsort((left != 0).to(torch.int8), stable=True)  # free blocks first, in order of their ids
    where_copy = (col == (held - 1)[:, None]) & copy[:, None]
    where_grow = (col >= held[:, None]) & (col < (held + grow)[:, None])
    place = start[:, None] + torch.where(where_grow, copy.long()[:, None] + col - held[:, None], 0)
    fresh = where_copy | where_grow
    out = torch.where(fresh, free[torch.where(fresh, place, 0)], out)
    left += count(torch.where(fresh, out, -1))
    s["refs"].copy_(left[:pool])
    at = copy.nonzero()[:, 0]
    src, dst = last[at], out[at, held[at] - 1]
    s["k_cache"][:, dst] = s["k_cache"][:, src]
    s["v_cache"][:, dst] = s["v_cache"][:, src]
    s["tables"], s["lens"] = out.int(), n.int()
    return s["tables"], s["lens"], s["refs"], s["k_cache"], s["v_cache"]


# ----------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "tree":
        nodes = int(_spread(case["nodes_lo"], case["nodes_hi"], case["seqs"]).sum())
        ctx = int(_spread(case["lo"], case["hi"], case["seqs"]).sum())
        per_key = 2 * case["hkv"] * case["d"] * size + 4 / BLOCK
        seen = ctx / case["seqs"] + nodes / case["seqs"] / 4 + 1  # a node sees about a quarter of its tree
        return {"bytes": (ctx + nodes) * per_key + nodes * (2 * case["hq"] * case["d"] * size + 8),
                "flops": 4.0 * nodes * seen * case["hq"] * case["d"]}
    if case["op"] == "compact":
        moved = int((_path_lens(case) - 1).sum())
        return {"bytes": case["layers"] * moved * 4 * case["hkv"] * case["d"] * size + 8 * moved + 20 * case["seqs"],
                "flops": 0}
    if case["op"] == "beam":
        n = case["seqs"] * case["beams"] * case["vocab"]
        return {"bytes": n * size + 12 * case["seqs"] * case["select"], "flops": 4.0 * n}
    rows = case["seqs"] * case["beams"]
    lens = case["prompt"] + _spread(case["done"] // 2, case["done"], case["seqs"])
    # a beam without an heir of its own leaves its place to a second heir of another, which copies one block
    copies = int((lens % BLOCK != 0).sum()) * (case["beams"] // 2)
    blocks = int(((lens + BLOCK - 1) // BLOCK).sum()) * case["beams"]
    return {"bytes": case["layers"] * copies * 4 * BLOCK * case["hkv"] * case["d"] * size + 8 * blocks + 20 * rows,
            "flops": 0}


# ----------------------------------------------------------------------------- the definition, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"tree": _exact_tree, "compact": _exact_compact, "beam": _exact_beam, "fork": _exact_fork}[case["op"]](s)


def _exact_tree(s):
    tables, lens, qsl = s["tables"].tolist(), s["lens"].tolist(), s["qsl"].tolist()
    n, hq, d = s["q"].shape
    hkv = s["k_cache"].shape[1]
    out = torch.zeros((n, hq, d), dtype=torch.float64, device=s["q"].device)
    mask = s["mask"].cpu().numpy().view(np.uint64)
    for i, length in enumerate(lens):
        t0, t1 = qsl[i], qsl[i + 1]
        m = t1 - t0
        ids = torch.tensor(tables[i][:(length + BLOCK - 1) // BLOCK], device=out.device)
        k = s["k_cache"][ids].double().transpose(0, 1).reshape(hkv, -1, d)[:, :length]
        v = s["v_cache"][ids].double().transpose(0, 1).reshape(hkv, -1, d)[:, :length]
        seen = np.ones((m, length), bool)
        for j in range(m):
            seen[j, length - m:] = [bool(int(mask[t0 + j, b // 64]) >> (b % 64) & 1) for b in range(m)]
        seen = torch.from_numpy(seen).to(out.device)
        for h in range(hq):
            z = s["q"][t0:t1, h].double() @ k[h * hkv // hq].T * s["scale"]
            w = torch.where(seen, torch.exp(z - z.max()), 0.0)
            out[t0:t1, h] = (w @ v[h * hkv // hq]) / w.sum(1, keepdim=True)
    return out


def _exact_compact(s):
    tables, lens, qsl = s["tables"].tolist(), s["lens"].tolist(), s["qsl"].tolist()
    path, path_lens = s["path"].tolist(), s["path_lens"].tolist()
    after = []
    old_k, old_v = s["k_cache"].clone(), s["v_cache"].clone()
    for i, length in enumerate(lens):
        base = length - (qsl[i + 1] - qsl[i])
        for a in range(path_lens[i]):
            src, dst = base + path[i][a], base + a
            for new, old in ((s["k_cache"], old_k), (s["v_cache"], old_v)):
                new[:, tables[i][dst // BLOCK], :, dst % BLOCK] = old[:, tables[i][src // BLOCK], :, src % BLOCK]
        after.append(base + path_lens[i])
    return s["k_cache"], s["v_cache"], torch.tensor(after, dtype=torch.int32)


def _exact_beam(s):
    n, w, v = s["logits"].shape
    k = s["select"]
    cum = s["cum"].double().cpu().numpy()
    done = None if s["finished"] is None else s["finished"].cpu().numpy()
    best = np.full((n, k), -np.inf)
    parent, token = np.full((n, k), -1, np.int32), np.full((n, k), -1, np.int32)
    for i in range(n):
        found = []
        for b in range(w):
            if done is not None and done[i, b]:
                found.append((-cum[i, b], b, s["eos"]))
                continue
            x = s["logits"][i, b].float().cpu().numpy().astype(np.float64)
            lse = np.logaddexp.reduce(x)
            for t in np.argsort(-x, kind="stable")[:k]:
                found.append((-(cum[i, b] + (x[t] - lse)), b, int(t)))
        found.sort()
        for c, (score, b, t) in enumerate(found[:k]):
            best[i, c], parent[i, c], token[i, c] = -score, b, t
    return torch.from_numpy(best), torch.from_numpy(parent), torch.from_numpy(token)


def _exact_fork(s):
    tables, lens, parents, refs = s["tables"].tolist(), s["lens"].tolist(), s["parents"].tolist(), s["refs"].tolist()
    cols, new = len(tables[0]), s["new_tokens"]
    rows, n = [], []
    for p in parents:
        n.append(lens[p] if p >= 0 else 0)
        rows.append(tables[p][:(n[-1] + BLOCK - 1) // BLOCK] if p >= 0 else [])
    for r in tables:
        for x in r:
            if x >= 0:
                refs[x] -= 1
    for r in rows:
        for x in r:
            refs[x] += 1
    at_end = {}
    for b, r in enumerate(rows):
        if new > 0 and n[b] % BLOCK:
            at_end.setdefault(r[-1], []).append(b)
    copies = []
    for x, sharers in at_end.items():
        alone = refs[x] == len(sharers)
        copies += [(b, x) for b in (sharers[1:] if alone else sharers)]
    for _, x in copies:
        refs[x] -= 1
    free = iter([x for x, c in enumerate(refs) if c == 0])
    copy_of = dict(copies)
    for b, r in enumerate(rows):
        if b in copy_of:
            r[-1] = next(free)
            refs[r[-1]] += 1
            for cache in (s["k_cache"], s["v_cache"]):
                cache[:, r[-1]] = cache[:, copy_of[b]]
        if parents[b] >= 0:
            while len(r) * BLOCK < n[b] + new:
                r.append(next(free))
                refs[r[-1]] += 1
    out = [r + [-1] * (cols - len(r)) for r in rows]
    whole = lambda a: torch.tensor(a, dtype=torch.int32)  # noqa: E731
    return whole(out), whole(n), whole(refs), s["k_cache"], s["v_cache"]
