"""Cases of the operators of drafted trees and of windows with sinks, in their plain form and as calls of the library.

A tree step: the tree's tables (positions and ancestor masks from parent pointers), attention of the drafted nodes over
the paged cache, the accepted path, and the move of its keys and values into place; and the same attention for chains
under a sliding window whose first keys stay visible.  ``own`` False computes them from elementary torch operations;
``own`` True calls the library.
"""
import math
import random

import torch

own = False

MAX_SEQ = 1 << 20          # bound on a request's length that calls without a plan are told


# --------------------------------------------------------------------------- #
# Cases
# --------------------------------------------------------------------------- #
def _attn(name, tree, reqs, rows, ragged, ctx_lo, ctx_hi, hq, hkv, d, window=0, sinks=0, kv="bf16", page_size=16):
    """``rows``: query rows of the longest window (``tree``: drafted nodes, else a chain's tokens); contexts between
    ``ctx_lo`` and ``ctx_hi`` keys; ``window`` 0: the whole context."""
    return {"name": name, "op": "attn", "tree": tree, "reqs": reqs, "rows": rows, "ragged": ragged, "ctx_lo": ctx_lo,
            "ctx_hi": ctx_hi, "hq": hq, "hkv": hkv, "d": d, "window": window, "sinks": sinks, "kv": kv,
            "page_size": page_size}


def _trees(name, op, reqs, rows, ragged, levels, window=0, sinks=0):
    """``op`` "tables" or "accept"; trees of up to ``rows`` nodes and ``levels`` levels below the root."""
    return {"name": name, "op": op, "reqs": reqs, "rows": rows, "ragged": ragged, "levels": levels, "window": window,
            "sinks": sinks}


def _move(name, layers, reqs, rows, levels, hkv, d, kv="bf16", page_size=16):
    """The drafted rows of every layer are written to the cache, then the accepted paths are moved together."""
    return {"name": name, "op": "move", "layers": layers, "reqs": reqs, "rows": rows, "levels": levels, "hkv": hkv,
            "d": d, "kv": kv, "page_size": page_size}


def listed():
    return [
        # the verify step of a batch with drafted trees: the draft block's heads and contexts, up to 64 nodes a request
        _attn("tree verify 8x64", True, 8, 64, True, 1024, 1600, 32, 8, 128),
        # one request with a long context, the verify sweep's heads
        _attn("tree long 1x48", True, 1, 48, False, 65536, 65536, 24, 4, 256),
        # trees over a 4-bit cache
        _attn("tree nvfp4 4x32", True, 4, 32, False, 16384, 16384, 24, 4, 256, kv="nvfp4"),
        # one token of one streaming request: the smallest call
        _attn("sinks token 1x1", False, 1, 1, False, 3001, 3001, 8, 2, 64, 1024, 4),
        # plain decoding of a serving batch in a layer with a sliding window; the pages between are freed
        _attn("sinks decode 64x1", False, 64, 1, False, 300, 20000, 32, 8, 128, 4096, 4),
        # a chunk of a long prompt in such a layer
        _attn("sinks prompt 1x2049", False, 1, 2049, False, 6001, 6001, 32, 8, 128, 2048, 4),
        # the tables of a step's trees: a verify batch, a large serving batch
        _trees("tree tables 8x64", "tables", 8, 64, True, 7),
        _trees("tree tables 256x255", "tables", 256, 255, True, 12),
        # the accepted paths of the same
        _trees("accept 8x64", "accept", 8, 64, True, 7),
        _trees("accept 256x255", "accept", 256, 255, True, 12),
        # the accepted rows moved into place: a verify batch, a larger one over more layers
        _move("move 8x64", 1, 8, 64, 7, 8, 128),
        _move("move 32x61 8 layers", 8, 32, 61, 7, 4, 256),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("attn", "attn", "attn", "tables", "accept", "move"))
    hq, hkv, d = rng.choice(((24, 4, 256), (32, 8, 128), (4, 1, 64), (8, 2, 64), (12, 12, 64), (40, 8, 128),
                             (16, 1, 128), (16, 8, 256)))
    if op == "attn":
        tree = rng.random() < 0.5
        reqs, hi = _log(rng, 1, 64), _log(rng, 1, 65536)
        hi = max(1, min(hi, int(2.6e8 / (reqs * hkv * d))))             # pools within the largest listed case's
        window, sinks = (0, 0) if rng.random() < 0.4 else (_log(rng, 1, 8192), rng.randint(0, 70))
        # rows within the largest listed case's work, both of what a row sees and of the whole context (the plain form)
        seen = min(hi, window + sinks) if window else hi
        room = min(6.0e10 / (4.0 * hq * d * reqs * (seen + 64)), 5.0e8 / (reqs * hq * (hi + 64.0)))
        rows = _log(rng, 1, max(1, min(256 if tree else 2048, int(room))))
        c = _attn("", tree, reqs, rows, rng.random() < 0.5, rng.randint(1, hi), hi, hq, hkv, d, window, sinks,
                  rng.choice(("bf16", "bf16", "nvfp4")), rng.choice((16, 32, 64)))
    elif op in ("tables", "accept"):
        window, sinks = (0, 0) if op == "accept" or rng.random() < 0.7 else (rng.randint(1, 12), rng.randint(0, 70))
        c = _trees("", op, _log(rng, 1, 256), _log(rng, 1, 255), rng.random() < 0.5, rng.randint(1, 12), window, sinks)
    else:
        c = _move("", rng.randint(1, 8), _log(rng, 1, 32), _log(rng, 1, 61), rng.randint(1, 7), min(hkv, 8), d,
                  rng.choice(("bf16", "bf16", "nvfp4")), rng.choice((16, 32, 64)))
    del c["name"]
    return c


def _sizes(case):
    """(window rows, context lengths) of each request: fixed by the case, the first the longest."""
    rng = random.Random(case["rows"] * 131 + case["reqs"])
    n, P = case["rows"], case["reqs"]
    lo, hi = case.get("ctx_lo", 1), case.get("ctx_hi", 4000)
    rows = [n] + [rng.randint(max(1, n // 2), n) if case.get("ragged") else n for _ in range(P - 1)]
    return rows, [hi] + [rng.randint(lo, hi) for _ in range(P - 1)]


def _tree(rng, n, levels):
    """Parents of n nodes in level order: node 0 the root, each level's nodes under likelier nodes of the one before."""
    parents, prev = [-1], [0]
    while len(parents) < n:
        room = n - len(parents)
        size = min(room, rng.randint(1, max(1, 2 * (n - 1) // levels)))
        at = sorted(prev[int(len(prev) * rng.random() ** 2)] for _ in range(size))
        prev = list(range(len(parents), len(parents) + size))
        parents += at
    return parents


def _depths(parents):
    out = []
    for p in parents:
        out.append(0 if p < 0 else out[p] + 1)
    return out


# --------------------------------------------------------------------------- #
# Inputs
# --------------------------------------------------------------------------- #
def prepare(case, seed):
    return {"attn": _prepare_attn, "tables": _prepare_trees, "accept": _prepare_trees,
            "move": _prepare_move}[case["op"]](case, seed)


def _indptr(rows):
    out = [0]
    for w in rows:
        out.append(out[-1] + w)
    return out


def _pools(s, case, pages, g):
    """K and V pools: normal values, or 4-bit codes with their block scales."""
    hkv, ps, d = case["hkv"], case["page_size"], case["d"]
    for name in ("k", "v"):
        if case["kv"] == "bf16":
            s[name + "_pool"] = torch.randn(pages, hkv, ps, d, generator=g, device="cuda", dtype=torch.bfloat16)
        else:
            s[name + "_pool"] = torch.randint(0, 256, (pages, hkv, ps, d // 2), generator=g, device="cuda",
                                              dtype=torch.uint8)
            s[name + "_scales"] = torch.randint(0x30, 0x40, (pages, hkv, ps, d // 16), generator=g, device="cuda",
                                                dtype=torch.uint8)
    s["code_values"] = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0.0, -.5, -1, -1.5, -2, -3, -4, -6], device="cuda")


def _prepare_attn(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = random.Random(seed)
    rows, ctx = _sizes(case)
    indptr, ps, n, P = _indptr(rows), case["page_size"], case["window"], case["reqs"]
    seq = [c + w for c, w in zip(ctx, rows)]
    stride = -(-max(seq) // ps)
    i32 = dict(dtype=torch.int32, device="cuda")
    # pages a row can still see: the sinks' and those of the window and behind
    first = [max(0, c - n + 1) // ps if n else 0 for c in ctx]
    kept = -(-case["sinks"] // ps) if n else 0
    col = torch.arange(stride, device="cuda")
    ends = torch.tensor([-(-m // ps) for m in seq], device="cuda")
    live = (col < ends[:, None]) & ((col >= torch.tensor(first, device="cuda")[:, None]) | (col < kept))
    total = int(live.sum())
    pages = total + total // 10 + 1
    perm = torch.randperm(pages, generator=g, device="cuda", dtype=torch.int32)
    table = torch.full((P, stride), -1, **i32)
    table[live] = perm[:total]
    d, hq = case["d"], case["hq"]
    s = {"case": case, "q": torch.randn(indptr[-1], hq, d, generator=g, device="cuda", dtype=torch.bfloat16),
         "table": table, "seq": torch.tensor(seq, **i32), "indptr": torch.tensor(indptr, **i32), "rows": rows, "ctx": ctx,
         "o": torch.zeros(indptr[-1], hq, d, dtype=torch.bfloat16, device="cuda"),
         "lse": torch.zeros(indptr[-1], hq, device="cuda"), "gscale": 0.3, "mask": None, "pos": None}
    _pools(s, case, pages, g)
    if case["tree"]:
        words = -(-max(rows) // 32)
        bits, pos, s["parents"] = [], [], []
        for c, w in zip(ctx, rows):
            parents = _tree(rng, w, rng.randint(2, 9))
            s["parents"].append(parents)
            pos += [c + h for h in _depths(parents)]
            sets = []
            for i, p in enumerate(parents):
                sets.append((sets[p] if p >= 0 else 0) | 1 << i)
            bits += [[x >> 32 * k & 0xffffffff for k in range(words)] for x in sets]
        s["mask"] = torch.tensor(bits, dtype=torch.int64, device="cuda").to(torch.int32)
        s["pos"] = torch.tensor(pos, **i32)
    if own:
        import speculative_decode_verify_paged_gb300 as sa
        s["plan"] = sa.spec_attn_masked_plan_create(
            num_reqs=P, total_q_rows=indptr[-1], max_w=max(rows), num_q_heads=hq, num_kv_heads=case["hkv"], head_dim=d,
            num_pages=pages, block_table_stride=stride, max_seq_len=max(seq), kv_dtype=int(case["kv"] == "nvfp4"),
            page_size=ps, tree=int(case["tree"]), window_left=n, sink_keys=case["sinks"])
        s["ws"] = torch.zeros(s["plan"].workspace_bytes, dtype=torch.uint8, device="cuda")
    return s


def _prepare_trees(case, seed):
    rng = random.Random(seed)
    rows, _ = _sizes(case)
    ctx = [rng.randint(1, 16384) for _ in rows]
    trees = [_tree(rng, w, case["levels"]) for w in rows]
    indptr = _indptr(rows)
    i32 = dict(dtype=torch.int32, device="cuda")
    i64 = dict(dtype=torch.int64, device="cuda")
    s = {"case": case, "indptr": torch.tensor(indptr, **i32),
         "seq": torch.tensor([c + w for c, w in zip(ctx, rows)], **i32),
         "parents": torch.tensor([p for t in trees for p in t], **i32), "words": -(-case["rows"] // 32),
         "ws": torch.zeros(256, dtype=torch.uint8, device="cuda")}
    if case["op"] == "tables":
        s["pos"] = torch.zeros(indptr[-1], **i32)
        s["mask"] = torch.zeros(indptr[-1], s["words"], **i32)
        return s
    draft, target = [], []
    for t in trees:
        tokens = [rng.randrange(128256) for _ in t]
        children = {}
        for j, p in enumerate(t):
            children.setdefault(p, []).append(j)
        draft += tokens
        # the model agrees with one of a node's children three times in four
        target += [tokens[rng.choice(children[j])] if j in children and rng.random() < 0.75 else rng.randrange(128256)
                   for j in range(len(t))]
    s["draft"], s["target"] = torch.tensor(draft, **i64), torch.tensor(target, **i64)
    s["path"] = torch.zeros(case["reqs"], case["levels"] + 4, **i32)
    s["accepted"], s["ctx"] = torch.zeros(case["reqs"], **i32), torch.zeros(case["reqs"], **i32)
    s["next"] = torch.zeros(case["reqs"], **i64)
    return s


def _prepare_move(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = random.Random(seed)
    rows, ctx = _sizes(case)
    indptr, ps, P, hkv, d = _indptr(rows), case["page_size"], case["reqs"], case["hkv"], case["d"]
    seq = [c + w for c, w in zip(ctx, rows)]
    stride = -(-max(seq) // ps)
    # the windows' pages only: the others do not matter here
    table = torch.full((P, stride), -1, dtype=torch.int32)
    first, last = [c // ps for c in ctx], [-(-m // ps) for m in seq]
    pages = sum(last) - sum(first) + 1
    perm = torch.randperm(pages, generator=g, device="cuda", dtype=torch.int32).cpu()
    at, slots, paths, accepted = 0, [], [], []
    for r in range(P):
        n = last[r] - first[r]
        table[r, first[r]:last[r]] = perm[at:at + n]
        at += n
        slots += [int(table[r, (ctx[r] + i) // ps]) * ps + (ctx[r] + i) % ps for i in range(rows[r])]
        parents, path = _tree(rng, rows[r], case["levels"]), [0]
        while rng.random() < 0.8:
            below = [j for j, p in enumerate(parents) if p == path[-1]]
            if not below:
                break
            path.append(rng.choice(below))
        path = path[:16]
        accepted.append(len(path))
        paths.append(path + [-1] * (16 - len(path)))
    i32 = dict(dtype=torch.int32, device="cuda")
    s = {"case": case, "table": table.cuda(), "seq": torch.tensor(seq, **i32), "indptr": torch.tensor(indptr, **i32),
         "path": torch.tensor(paths, **i32), "accepted": torch.tensor(accepted, **i32),
         "slot": torch.tensor(slots, dtype=torch.int64, device="cuda"), "pools": [], "new": [],
         "q": torch.zeros(indptr[-1], 0, d, dtype=torch.bfloat16, device="cuda"),
         "pos": torch.zeros(1, indptr[-1], **i32), "gscale": 2.0 ** -8,
         "ws": torch.zeros(256, dtype=torch.uint8, device="cuda")}
    for _ in range(case["layers"]):
        pool = {}
        _pools(pool, case, pages, g)
        s["code_values"] = pool.pop("code_values")
        s["pools"].append(pool)
        s["new"].append([torch.randn(indptr[-1], hkv, d, generator=g, device="cuda", dtype=torch.bfloat16)
                         for _ in range(2)])
    if own:
        import speculative_decode_verify_paged_gb300 as sa
        s["plan"] = sa.spec_attn_norm_rope_plan_create(num_q_heads=0, num_kv_heads=hkv, head_dim=d, rot_dim=0, inv_freq=[],
                                                       page_size=ps, num_pages=pages, kv_dtype=int(case["kv"] == "nvfp4"),
                                                       q_row_stride=s["q"].stride(0), q_out_row_stride=s["q"].stride(0))
        s["lists"] = [[p.get(name) for p in s["pools"]] for name in ("k_pool", "v_pool", "k_scales", "v_scales")]
    return s


# --------------------------------------------------------------------------- #
# One pass
# --------------------------------------------------------------------------- #
def run(s):
    op = s["case"]["op"]
    if own:
        return {"attn": _own_attn, "tables": _own_tables, "accept": _own_accept, "move": _own_move}[op](s)
    return {"attn": _plain_attn, "tables": _plain_tables, "accept": _plain_accept, "move": _plain_move}[op](s)


def _own_attn(s):
    import speculative_decode_verify_paged_gb300 as sa
    sa.spec_attn_run_masked(s["plan"], s["q"], s["k_pool"], s["v_pool"], s["table"], s["seq"], s["indptr"], s["mask"],
                            s["pos"], s["o"], s["lse"], s["ws"], s.get("k_scales"), s.get("v_scales"), s["gscale"],
                            s["gscale"])
    return [s["o"], s["lse"]]


def _e4m3(byte):
    return byte.view(torch.float8_e4m3fn).float()


def _values(s, name):
    """A pool's pages in 32 bits."""
    pool = s[name + "_pool"]
    if s["case"]["kv"] == "bf16":
        return pool.float()
    v = torch.stack([s["code_values"][(pool & 15).long()], s["code_values"][(pool >> 4).long()]], -1).flatten(-2)
    return (v.unflatten(-1, (-1, 16)) * (_e4m3(s[name + "_scales"]) * s["gscale"])[..., None]).flatten(-2)


def _plain_attn(s):
    """Padded to [request, longest window] x [request, longest length], masked, in 32 bits."""
    c = s["case"]
    P, hq, hkv, d, n = c["reqs"], c["hq"], c["hkv"], c["d"], c["window"]
    indptr, total, G, W = s["indptr"].long(), s["q"].shape[0], c["hq"] // c["hkv"], max(s["rows"])
    i = torch.arange(W, device="cuda")
    at = (indptr[:-1, None] + i).clamp(max=total - 1)                       # [P, W]
    q = s["q"][at].float().unflatten(2, (hkv, G)).permute(0, 2, 3, 1, 4).reshape(P, hkv, G * W, d)
    pages = s["table"].clamp(min=0).long()
    k, v = (_values(s, t)[pages].permute(0, 2, 1, 3, 4).flatten(2, 3) for t in ("k", "v"))   # [P, Hkv, S, d]
    j = torch.arange(k.shape[2], device="cuda")
    seq = s["seq"].long()[:, None, None]
    ctx = seq - (indptr[1:] - indptr[:-1])[:, None, None]
    if c["tree"]:
        row_pos = s["pos"][at].long()[..., None]
        node = (j - ctx).clamp(min=0, max=32 * s["mask"].shape[1] - 1).expand(P, W, -1)
        bit = torch.gather(s["mask"][at], 2, node >> 5) >> (node & 31).int() & 1
        inside = (j >= ctx) & (bit != 0)
    else:
        row_pos = ctx + i[:, None]
        inside = (j >= ctx) & (j <= row_pos) & ((j > row_pos - n) | (j < c["sinks"]) if n else torch.ones_like(j > 0))
    before = j < ctx
    if n:
        before = before & ((j > row_pos - n) | (j < c["sinks"]))
    seen = (before | inside) & (j < seq)                                    # [P, W, S]
    x = torch.matmul(q, k.transpose(2, 3)).div_(math.sqrt(d))
    x.view(P, hkv, G, W, -1).masked_fill_(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    x.sub_(m).exp_()
    denominator = x.sum(-1, keepdim=True)
    o = torch.matmul(x, v) / denominator
    lse = (m + torch.log(denominator))[..., 0]
    row = torch.arange(total, device="cuda")
    req = torch.searchsorted(indptr, row, right=True) - 1
    w = row - indptr[req]
    o = o.reshape(P, hkv, G, W, d)[req, :, :, w].reshape(total, hq, d).to(torch.bfloat16)
    return [o, lse.reshape(P, hkv, G, W)[req, :, :, w].reshape(total, hq)]


def _own_tables(s):
    import speculative_decode_verify_paged_gb300 as sa
    c = s["case"]
    sa.spec_attn_build_tree(s["parents"], s["seq"], s["indptr"], s["pos"], s["mask"], s["ws"], max_w=c["rows"],
                            window_left=c["window"], sink_keys=c["sinks"])
    return [s["pos"], s["mask"]]


def _requests(s):
    """Of every row: its request, its place in the window, the window's first row, its context length."""
    indptr = s["indptr"].long()
    row = torch.arange(s["parents"].numel(), device="cuda")
    req = torch.searchsorted(indptr, row, right=True) - 1
    ctx = s["seq"].long() - (indptr[1:] - indptr[:-1])
    return req, row - indptr[req], indptr[req], ctx[req]


def _plain_tables(s):
    c = s["case"]
    _, i, first, ctx = _requests(s)
    row, n = torch.arange(i.numel(), device="cuda"), c["window"]
    parents = s["parents"].long()
    depth = torch.zeros_like(i)
    up = row
    chain = [row]
    for _ in range(c["levels"] * 8 + 8 if i.numel() else 0):      # as deep as any of these trees
        p = parents[up]
        depth += p >= 0
        up = torch.where(p >= 0, first + p, up)
        chain.append(up)
    chain = torch.stack(chain, 1)                                  # [row, steps]: the row and its ancestors
    far = depth[:, None] - depth[chain]
    seen = torch.ones_like(chain, dtype=torch.bool)
    if n:
        seen = (far < n) | (ctx[:, None] + depth[chain] < c["sinks"])
    node = chain - first[:, None]
    bits = torch.zeros(i.numel(), 32 * s["words"], dtype=torch.bool, device="cuda")
    bits[row[:, None].expand_as(node)[seen], node[seen]] = True
    weights = 1 << torch.arange(32, device="cuda")
    words = (bits.unflatten(1, (-1, 32)) * weights).sum(-1)
    return [(ctx + depth).to(torch.int32), words.to(torch.int32)]


def _own_accept(s):
    import speculative_decode_verify_paged_gb300 as sa
    sa.spec_attn_accept_tree(s["parents"], s["draft"], s["target"], s["seq"], s["indptr"], s["path"], s["accepted"],
                             s["next"], s["ctx"], s["ws"], max_w=s["case"]["rows"])
    return [s["path"], s["accepted"], s["next"], s["ctx"]]


def _plain_accept(s):
    req, i, first, _ = _requests(s)
    parents, total = s["parents"].long(), i.numel()
    ok = (parents >= 0) & (s["draft"] == s["target"][first + parents.clamp(min=0)])
    # lowest accepted child of every node
    child = torch.full((total + 1,), total, dtype=torch.int64, device="cuda")
    child.scatter_reduce_(0, torch.where(ok, first + parents, total), torch.arange(total, device="cuda"), "amin")
    indptr = s["indptr"].long()
    at, live = indptr[:-1], torch.ones(indptr.numel() - 1, dtype=torch.bool, device="cuda")
    path, accepted, last = [], torch.zeros_like(at), at
    for _ in range(s["path"].shape[1]):
        path.append(torch.where(live, at - indptr[:-1], -1))
        accepted += live
        last = torch.where(live, at, last)
        below = child[at]
        live = live & (below < total)
        at = torch.where(live, below, at)
    ctx = s["seq"].long() - (indptr[1:] - indptr[:-1]) + accepted
    return [torch.stack(path, 1).to(torch.int32), accepted.to(torch.int32), s["target"][last], ctx.to(torch.int32)]


def _moved(s):
    """The pools, or the values that the kept slots of 4-bit ones stand for."""
    out = []
    for pool in s["pools"]:
        for name in ("k", "v"):
            if s["case"]["kv"] == "bf16":
                out.append(pool[name + "_pool"])
                continue
            page, at = s["slot"] // s["case"]["page_size"], s["slot"] % s["case"]["page_size"]
            c = pool[name + "_pool"][page, :, at]
            v = torch.stack([s["code_values"][(c & 15).long()], s["code_values"][(c >> 4).long()]], -1).flatten(-2)
            scale = _e4m3(pool[name + "_scales"][page, :, at]) * s["gscale"]
            out.append((v.unflatten(-1, (-1, 16)) * scale[..., None]).flatten(-2))
    return out


def _own_move(s):
    import speculative_decode_verify_paged_gb300 as sa
    g = s["gscale"]
    for pool, (k, v) in zip(s["pools"], s["new"]):
        sa.spec_attn_norm_rope_append(s["plan"], s["q"], k, v, None, None, s["pos"], s["slot"], s["q"], pool["k_pool"],
                                      pool["v_pool"], s["ws"], pool.get("k_scales"), pool.get("v_scales"), g, g)
    k, v, ks, vs = s["lists"]
    scales = {} if s["case"]["kv"] == "bf16" else dict(k_scales=ks, v_scales=vs)
    sa.spec_attn_move_kv(k, v, s["table"], s["seq"], s["indptr"], s["path"], s["accepted"], s["ws"], max_seq_len=MAX_SEQ,
                         **scales)
    return _moved(s)


def _quantise(x, g):
    """bf16 rows [n, h, d] as NVFP4 against the decode scale g: (code bytes, scale bytes)."""
    x = x.float().unflatten(-1, (-1, 16))
    scale = (x.abs().amax(-1) / (6.0 * g)).clamp(max=448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    den = (_e4m3(scale) * g)[..., None]
    t = torch.where(den == 0, torch.zeros_like(x), x / den)
    # e2m1 magnitudes 0 .5 1 1.5 2 3 4 6, nearest, ties to the even code
    m = t.abs()
    code = ((m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0))
    code = code.to(torch.uint8) | (torch.signbit(t).to(torch.uint8) << 3)
    code = torch.where(den == 0, torch.zeros_like(code), code).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale


def _plain_move(s):
    c = s["case"]
    page, at = s["slot"] // c["page_size"], s["slot"] % c["page_size"]
    path = s["path"].long()
    step = torch.arange(path.shape[1], device="cuda")
    kept = step < s["accepted"][:, None]
    first = s["indptr"].long()[:-1, None]
    src, dst = s["slot"][(first + path)[kept]], s["slot"][(first + step)[kept]]
    for pool, new in zip(s["pools"], s["new"]):
        for name, x in zip(("k", "v"), new):
            parts = [(name + "_pool", x)]
            if c["kv"] == "nvfp4":
                parts = list(zip((name + "_pool", name + "_scales"), _quantise(x, s["gscale"])))
            for key, rows in parts:
                t = pool[key]
                t[page, :, at] = rows
                t[dst // c["page_size"], :, dst % c["page_size"]] = t[src // c["page_size"], :, src % c["page_size"]]
    return _moved(s)


# --------------------------------------------------------------------------- #
# What a pass cannot do without, and its result in 64 bits
# --------------------------------------------------------------------------- #
def work(case):
    op = case["op"]
    rows, ctx = _sizes(case)
    total, P = sum(rows), case["reqs"]
    if op == "tables":
        return {"bytes": total * (8 + 4 * -(-case["rows"] // 32)) + P * 8, "flops": 0}
    if op == "accept":
        return {"bytes": total * 20 + P * (8 + 16 + 4 * (case["levels"] + 4)), "flops": 0}
    hkv, d = case["hkv"], case["d"]
    row = 4 * d if case["kv"] == "bf16" else 2 * (d // 2 + d // 16)         # K and V of one key and head
    if op == "move":
        # the drafted rows in (bf16) and into the cache, then about four rows a request read and written
        return {"bytes": case["layers"] * hkv * (total * (4 * d + row) + P * 4 * 2 * row), "flops": 0}
    n, sinks, keys, pairs = case["window"], case["sinks"], 0, 0
    for w, c in zip(rows, ctx):
        lo = max(0, c - n + 1) if n else 0
        keys += c + w - lo + (min(sinks, lo) if n else 0)
        for i in range(w):
            if case["tree"]:
                at, own_keys = c + min(i, 4), min(i + 1, 5)
            else:
                at, own_keys = c + i, i + 1
            seen = c + own_keys
            if n and at + 1 - n > 0:
                seen -= max(0, at + 1 - n - sinks)
            pairs += max(1, seen)
    return {"bytes": total * case["hq"] * (4 * d + 4) + keys * hkv * row, "flops": 4 * pairs * case["hq"] * d}


def exact(case, seed):
    if case["op"] in ("tables", "accept"):
        return None                                                         # whole numbers
    s = prepare(case, seed)
    if case["op"] == "move":
        return _exact_move(case, s)
    ps, n, sinks, G, d = case["page_size"], case["window"], case["sinks"], case["hq"] // case["hkv"], case["d"]
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")

    def heads(name, table, length, h):
        """Head h of the request's keys or values, in 64 bits; unmapped pages as zeros."""
        pool = s[name + "_pool"][table, h]
        if case["kv"] == "bf16":
            x = pool.double()
        else:
            low, high = pool % 16, pool // 16
            pair = torch.stack([low, high], -1).reshape(*pool.shape[:2], d).long()
            x = torch.where(pair >= 8, -grid[pair % 8], grid[pair % 8])
            scale = s[name + "_scales"][table, h].view(torch.float8_e4m3fn).double() * s["gscale"]
            x = x * scale.repeat_interleave(16, -1)
        return x.reshape(-1, d)[:length]

    o, lse, at = [], [], 0
    for r, (w, c) in enumerate(zip(s["rows"], s["ctx"])):
        length = c + w
        table = s["table"][r, :-(-length // ps)].long().clamp(min=0)
        seen = torch.zeros(w, length, dtype=torch.bool, device="cuda")
        if case["tree"]:
            depth = _depths(s["parents"][r])
            for i in range(w):
                lo = max(0, c + depth[i] + 1 - n) if n else 0
                seen[i, lo:c] = True
                seen[i, :min(sinks, c) if n else 0] = True
                j = i
                while j >= 0:
                    seen[i, c + j] = True
                    j = s["parents"][r][j]
        else:
            for i in range(w):
                seen[i, max(0, c + i + 1 - n) if n else 0:c + i + 1] = True
                if n:
                    seen[i, :min(sinks, c + i + 1)] = True
        hidden = ~seen
        outs, sums = [], []
        for h in range(case["hq"]):
            if h % G == 0:
                k, v = heads("k", table, length, h // G), heads("v", table, length, h // G)
            x = (s["q"][at:at + w, h].double() @ k.t()) * d ** -0.5
            x[hidden] = -math.inf
            outs.append(torch.softmax(x, 1) @ v)
            sums.append(torch.logsumexp(x, 1))
        o.append(torch.stack(outs, 1))
        lse.append(torch.stack(sums, 1))
        at += w
    return [torch.cat(o), torch.cat(lse)]


def _exact_move(case, s):
    """Row by row: what every window's slots hold at last, in 64 bits."""
    holds, ptr = list(range(s["slot"].numel())), s["indptr"].tolist()       # the drafted row whose values a row's slot holds
    for r, (path, n) in enumerate(zip(s["path"].tolist(), s["accepted"].tolist())):
        for i in range(n):
            holds[ptr[r] + i] = ptr[r] + path[i]
    holds = torch.tensor(holds, device="cuda")
    out = []
    for pool, new in zip(s["pools"], s["new"]):
        for name, x in zip(("k", "v"), new):
            if case["kv"] == "nvfp4":
                out.append(_exact_nvfp4(x, s["gscale"])[holds])
                continue
            flat = pool[name + "_pool"].double().transpose(1, 2).flatten(0, 1)   # [slot, Hkv, d]
            flat[s["slot"]] = x.double()[holds]
            out.append(flat.unflatten(0, (-1, case["page_size"])).transpose(1, 2).contiguous())
    return out


def _exact_nvfp4(x, g):
    """Nearest representable values by search over the 8 magnitudes, in 64 bits."""
    x = x.double().unflatten(-1, (-1, 16))
    amax = x.abs().amax(-1, keepdim=True)
    scale = (amax / (6 * g)).clamp(max=448).float().to(torch.float8_e4m3fn).double()
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
    den = scale * g
    t = torch.where(den > 0, x.abs() / den.clamp(min=1e-300), torch.zeros_like(x))
    hi = torch.searchsorted(grid, t.contiguous()).clamp(1, 7)
    up, down = grid[hi], grid[hi - 1]
    pick_up = (t - down > up - t) | ((t - down == up - t) & (hi % 2 == 0))
    return (torch.where(pick_up, up, down) * den * torch.sign(x)).flatten(-2)
