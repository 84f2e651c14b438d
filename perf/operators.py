"""Cases of the operators around the attention call, in their plain form and as calls of the library.

Four operators of a decoder layer's step: the step's tables built on the GPU, the norm and rotation of q and k, the
same pass writing K and V into the paged cache, and cross attention to an encoder's states.  ``own`` False computes
them from elementary torch operations; ``own`` True calls the library.
"""
import math
import random

import torch

own = False

MAX_SEQ = 1 << 20          # bound on a request's length that the plans are told


# --------------------------------------------------------------------------- #
# Cases
# --------------------------------------------------------------------------- #
def _tables(name, reqs, window, ctx_lo, ctx_hi, page_size, rows, turnover, prompts):
    """``window``: most rows a running request brings; ``prompts``: most rows of a request that joins; ``turnover``: share
    of requests that end or join in this step; ``rows``: capacity of the per-row outputs (a padded batch)."""
    return {"name": name, "op": "tables", "reqs": reqs, "window": window, "ctx_lo": ctx_lo, "ctx_hi": ctx_hi,
            "page_size": page_size, "rows": rows, "turnover": turnover, "prompts": prompts}


def _rope(name, op, rows, hq, hkv, d, rot, axes, interleaved, norm, kv="bf16", page_size=16, fused=True):
    """``fused``: q, k and v are views of one projection's output rows; ``op`` "rope" or "append"."""
    return {"name": name, "op": op, "rows": rows, "hq": hq, "hkv": hkv, "d": d, "rot": rot, "axes": axes,
            "interleaved": interleaved, "norm": norm, "kv": kv, "page_size": page_size, "fused": fused}


def _cross(name, reqs, rows, ragged, kv, hq, hkv, d, fused):
    """``rows``: query rows of a request (of the longest, if ``ragged``); ``kv``: most encoder rows of a request, the
    capacity of its place in a padded batch; ``fused``: K and V are views of one projection's output rows."""
    return {"name": name, "op": "cross", "reqs": reqs, "rows": rows, "ragged": ragged, "kv": kv, "hq": hq, "hkv": hkv,
            "d": d, "fused": fused}


def listed():
    return [
        # a verify step of eight requests (the draft block's lengths and width)
        _tables("tables verify 8", 8, 9, 1024, 1600, 16, 72, 0.0, 0),
        # a large serving batch, requests ending and joining with their prompts
        _tables("tables serving 512", 512, 16, 1, 16384, 16, 16384, 0.06, 1000),
        # admission of long prompts beside running requests, larger pages
        _tables("tables prompts 61", 61, 1, 1, 8000, 64, 262144, 0.9, 8191),
        # one token of one request: plain decoding
        _rope("norm rope 1 row", "rope", 1, 24, 4, 256, 256, 1, False, True),
        # a chunk of a prompt, q and k views of the fused projection
        _rope("norm rope prompt 16384", "rope", 16384, 32, 8, 128, 128, 1, False, True),
        # an image or video prompt: time, height and width positions, pairs side by side, part of the head rotated
        _rope("rope 3 axes 5001", "rope", 5001, 24, 4, 256, 128, 3, True, False),
        # a verify window of eight requests in a model with three position axes, into the cache
        _rope("append 3 axes 72", "append", 72, 32, 8, 128, 128, 3, False, True),
        # a prompt chunk into the cache
        _rope("append prompt 8192", "append", 8192, 24, 4, 256, 256, 1, False, True),
        # the same into a 4-bit cache
        _rope("append nvfp4 4097", "append", 4097, 24, 4, 256, 64, 1, False, True, "nvfp4", 32),
        # verify windows of eight requests over an encoder's states
        _cross("cross verify 8x9", 8, 9, False, 1500, 32, 8, 128, True),
        # one token of each of 64 requests, wide heads
        _cross("cross decode 64x1", 64, 1, False, 1601, 24, 4, 256, False),
        # prompts of odd length over long states
        _cross("cross prompt 2x4097", 2, 4097, True, 4100, 32, 8, 128, True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("tables", "rope", "append", "cross"))
    hq, hkv, d = rng.choice(((24, 4, 256), (32, 8, 128), (4, 1, 64), (8, 2, 64), (12, 12, 64), (40, 8, 128),
                             (16, 1, 128), (16, 8, 256)))
    if op == "tables":
        reqs, window = _log(rng, 1, 512), rng.randint(1, 16)
        hi, prompts = _log(rng, 20, 16384), _log(rng, 1, 4000)
        turnover = rng.choice((0.0, 0.05, 0.5))
        rows = reqs * window + int(reqs * turnover + 1) * prompts
        c = _tables("", reqs, window, rng.randint(1, hi), hi, rng.choice((16, 32, 64)), min(rows, 262144), turnover,
                    prompts)
    elif op in ("rope", "append"):
        axes = rng.choice((1, 1, 2, 3))
        rot = rng.choice((d, d, d // 2, 16 * rng.randint(1, d // 16)))
        rows = _log(rng, 1, 8192 if op == "append" else 11000)
        c = _rope("", op, rows, hq, hkv, d, rot, axes, rng.random() < 0.3, rng.random() < 0.8,
                  rng.choice(("bf16", "bf16", "nvfp4")) if op == "append" else "bf16", rng.choice((16, 32, 64)),
                  rng.random() < 0.7)
    else:
        reqs, kv = _log(rng, 1, 64), _log(rng, 1, 4000)
        room = max(1, min(4000, int(2.2e9 / (reqs * kv * hq * d / 128))))   # within the largest listed case
        room = min(room, max(1, 65536 // reqs))
        c = _cross("", reqs, _log(rng, 1, room), rng.random() < 0.5, kv, hq, hkv, d, rng.random() < 0.5)
    del c["name"]
    return c


def _window_rows(case):
    """Query rows of each request of a cross attention case: fixed by the case, the first the longest."""
    if not case["ragged"]:
        return [case["rows"]] * case["reqs"]
    rng = random.Random(case["rows"] * 131 + case["reqs"])
    return [case["rows"]] + [rng.randint(max(1, case["rows"] // 2), case["rows"]) for _ in range(case["reqs"] - 1)]


# --------------------------------------------------------------------------- #
# Inputs
# --------------------------------------------------------------------------- #
def prepare(case, seed):
    return {"tables": _prepare_tables, "rope": _prepare_rope, "append": _prepare_rope,
            "cross": _prepare_cross}[case["op"]](case, seed)


def _prepare_tables(case, seed):
    rng = random.Random(seed)
    P, ps = case["reqs"], case["page_size"]
    prev, ctx, win = [], [], []
    budget = case["rows"]
    for r in range(P):
        running = rng.randint(case["ctx_lo"], case["ctx_hi"])
        tail = rng.randint(0, case["window"])            # rows of the last window that were rejected
        u = rng.random()
        if u < case["turnover"] / 2:                     # ended: its pages go back
            p, c, w = running, 0, 0
        elif u < case["turnover"] and case["prompts"]:   # joined: its prompt's rows
            p, c, w = 0, 0, rng.randint(1, case["prompts"])
        else:
            p, c, w = running, max(0, running - tail), rng.randint(1, case["window"])
        w = min(w, budget)
        budget -= w
        prev.append(p)
        ctx.append(c)
        win.append(w)
    longest = case["ctx_hi"] + case["window"] + case["prompts"]
    stride = -(-longest // ps)
    num_pages = P * stride                               # every request may grow to its full length
    held = [-(-p // ps) for p in prev]
    g = torch.Generator(device="cuda").manual_seed(seed)
    perm = torch.randperm(num_pages, generator=g, device="cuda", dtype=torch.int32)
    i32 = dict(dtype=torch.int32, device="cuda")
    held_t = torch.tensor(held, **i32)
    first = torch.cumsum(held_t, 0) - held_t
    col = torch.arange(stride, device="cuda")
    place = (first[:, None] + col).clamp(max=num_pages - 1)
    table = torch.where(col < held_t[:, None], perm[place], torch.full((), -1, **i32))
    total = sum(held)
    s = {"case": case, "ctx": torch.tensor(ctx, **i32), "win": torch.tensor(win, **i32),
         "prev": torch.tensor(prev, **i32), "free_count0": torch.tensor([num_pages - total], **i32),
         "free": torch.cat([perm[total:], perm[:total]]).contiguous(), "table": table.contiguous(),
         "seq": torch.zeros(P, **i32), "indptr": torch.zeros(P + 1, **i32), "free_count": torch.zeros(1, **i32),
         "pos": torch.zeros(case["rows"], **i32),
         "slot": torch.zeros(case["rows"], dtype=torch.int64, device="cuda"),
         "ws": torch.zeros(256, dtype=torch.uint8, device="cuda")}
    return s


def _inv_freq(rot, base=1e6):
    return [base ** (-2.0 * j / rot) for j in range(rot // 2)]


def _pair_axis(rot, axes):
    """Axis of each rotated pair: contiguous sections, the first (time) the shortest."""
    half = rot // 2
    if axes == 1:
        return [0] * half
    if axes == 2:
        return [0] * (half // 2) + [1] * (half - half // 2)
    t = half // 4
    h = (half - t) // 2
    return [0] * t + [1] * h + [2] * (half - t - h)


def _prepare_rope(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = random.Random(seed)
    n, hq, hkv, d, rot = case["rows"], case["hq"], case["hkv"], case["d"], case["rot"]

    def rand(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)

    if case["fused"]:
        qkv = rand(n, (hq + 2 * hkv) * d)
        q, k, v = (t.unflatten(1, (-1, d)) for t in qkv.split([hq * d, hkv * d, hkv * d], 1))
    else:
        q, k, v = rand(n, hq, d), rand(n, hkv, d), rand(n, hkv, d)
    start = rng.randint(0, 131072)
    if case["axes"] == 1:
        pos = start + torch.arange(n, device="cuda", dtype=torch.int32)[None]
    else:   # frames of a video: time, height, width within the frame
        side = rng.randint(8, 60)
        i = torch.arange(n, device="cuda", dtype=torch.int32)
        pos = torch.stack([start + i // (side * side), start + i // side % side, start + i % side][:case["axes"]])
    weight = lambda: 1 + 0.1 * torch.randn(d, generator=g, device="cuda") if case["norm"] else None  # noqa: E731
    s = {"case": case, "q": q, "k": k, "v": v, "pos": pos.contiguous(), "qw": weight(), "kw": weight(),
         "freq": torch.tensor(_inv_freq(rot), dtype=torch.float64, device="cuda"),
         "axis": torch.tensor(_pair_axis(rot, case["axes"]), device="cuda"),
         "q_out": torch.zeros(n, hq, d, dtype=torch.bfloat16, device="cuda")}
    ps = case["page_size"]
    pages = -(-n // ps) + 2
    if case["op"] == "rope":
        s["k_out"] = torch.zeros(n, hkv, d, dtype=torch.bfloat16, device="cuda")
    else:
        perm = torch.randperm(pages, generator=g, device="cuda")
        at = rng.randint(0, ps - 1) + torch.arange(n, device="cuda")
        s["slot"] = perm[at // ps] * ps + at % ps
        s["ws"] = torch.zeros(256, dtype=torch.uint8, device="cuda")
        if case["kv"] == "bf16":
            s["k_pool"] = torch.zeros(pages, hkv, ps, d, dtype=torch.bfloat16, device="cuda")
            s["v_pool"] = torch.zeros_like(s["k_pool"])
        else:
            s["k_pool"] = torch.zeros(pages, hkv, ps, d // 2, dtype=torch.uint8, device="cuda")
            s["k_scales"] = torch.zeros(pages, hkv, ps, d // 16, dtype=torch.uint8, device="cuda")
            s["v_pool"], s["v_scales"] = torch.zeros_like(s["k_pool"]), torch.zeros_like(s["k_scales"])
            s["gscale"] = 2.0 ** -8
            s["code_values"] = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0.0, -.5, -1, -1.5, -2, -3, -4, -6],
                                            device="cuda")
    if own:
        import speculative_decode_verify_paged_gb300 as sa
        cache = {}
        if case["op"] == "append":
            cache = dict(page_size=ps, num_pages=pages, kv_dtype=int(case["kv"] == "nvfp4"))
        s["plan"] = sa.spec_attn_norm_rope_plan_create(
            num_q_heads=hq, num_kv_heads=hkv, head_dim=d, rot_dim=rot, inv_freq=_inv_freq(rot),
            pair_axis=_pair_axis(rot, case["axes"]), num_axes=case["axes"], interleaved=int(case["interleaved"]),
            eps=1e-6, q_row_stride=q.stride(0), k_row_stride=k.stride(0), v_row_stride=v.stride(0), **cache)
    return s


def _prepare_cross(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = random.Random(seed)
    P, S, hq, hkv, d = case["reqs"], case["kv"], case["hq"], case["hkv"], case["d"]
    rows = _window_rows(case)
    indptr = [0]
    for w in rows:
        indptr.append(indptr[-1] + w)
    lens = [S] + [rng.randint(max(1, S // 4), S) for _ in range(P - 1)]
    rng.shuffle(lens)

    def rand(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)

    if case["fused"]:
        kv = rand(P * S, 2, hkv, d)
        k, v = kv[:, 0], kv[:, 1]
    else:
        k, v = rand(P * S, hkv, d), rand(P * S, hkv, d)
    i32 = dict(dtype=torch.int32, device="cuda")
    s = {"case": case, "q": rand(indptr[-1], hq, d), "k": k, "v": v, "indptr": torch.tensor(indptr, **i32),
         "kv_start": torch.arange(P, **i32) * S, "kv_len": torch.tensor(lens, **i32), "lens": lens, "max_rows": max(rows),
         "o": torch.zeros(indptr[-1], hq, d, dtype=torch.bfloat16, device="cuda"),
         "lse": torch.zeros(indptr[-1], hq, device="cuda")}
    if own:
        import speculative_decode_verify_paged_gb300 as sa
        s["plan"] = sa.spec_attn_cross_plan_create(
            num_reqs=P, total_q_rows=indptr[-1], max_q_rows=max(rows), num_q_heads=hq, num_kv_heads=hkv, head_dim=d,
            total_kv_rows=P * S, max_kv_len=S, kv_row_stride=k.stride(0))
        s["ws"] = torch.zeros(s["plan"].workspace_bytes, dtype=torch.uint8, device="cuda")
    return s


# --------------------------------------------------------------------------- #
# One pass
# --------------------------------------------------------------------------- #
def run(s):
    op = s["case"]["op"]
    if own:
        return {"tables": _own_tables, "rope": _own_rope, "append": _own_append, "cross": _own_cross}[op](s)
    return {"tables": _plain_tables, "rope": _plain_rope, "append": _plain_append, "cross": _plain_cross}[op](s)


def _own_tables(s):
    import speculative_decode_verify_paged_gb300 as sa
    sa.spec_attn_build_tables(s["ctx"], s["win"], s["prev"], s["free_count0"], s["free"], s["table"], s["seq"],
                              s["indptr"], s["free_count"], s["pos"], s["slot"], s["ws"],
                              page_size=s["case"]["page_size"], max_w=MAX_SEQ, max_seq_len=MAX_SEQ)
    return [s["table"], s["free"], s["free_count"], s["seq"], s["indptr"], s["pos"], s["slot"]]


def _plain_tables(s):
    ps, ctx, win, prev = s["case"]["page_size"], s["ctx"], s["win"], s["prev"]
    table, free, F = s["table"], s["free"], s["free_count0"].long()
    P, stride = table.shape
    num_pages, cap = free.numel(), s["slot"].numel()
    seq = ctx + win
    held, need = (prev + ps - 1) // ps, (seq + ps - 1) // ps
    new, ret = (need - held).clamp(min=0), (held - need).clamp(min=0)
    first_new, first_ret = torch.cumsum(new, 0) - new, torch.cumsum(ret, 0) - ret
    R, N = ret.sum(), new.sum()
    col = torch.arange(stride, device=table.device)
    # the returned pages on top of the stack, in request order
    returned = (col >= need[:, None]) & (col < held[:, None])
    at = torch.where(returned, F + first_ret[:, None] + col - need[:, None], 2 * num_pages)
    stack = torch.cat([free, torch.zeros(num_pages + 1, dtype=torch.int32, device=table.device)])
    stack.scatter_(0, at.reshape(-1), table.reshape(-1))
    # the new ones from its top, in request order
    grown = (col >= held[:, None]) & (col < need[:, None])
    take = (F + R - 1 - (first_new[:, None] + col - held[:, None])).clamp(0, 2 * num_pages)
    table = torch.where(grown, stack[take], table)
    F2 = F + R - N
    i = torch.arange(num_pages, device=table.device)
    free = torch.where((i >= F) & (i < F2), stack[:num_pages], free)
    indptr = torch.cat([torch.zeros(1, dtype=torch.int32, device=table.device), torch.cumsum(win, 0, dtype=torch.int32)])
    row = torch.arange(cap, device=table.device, dtype=torch.int32)
    req = (torch.searchsorted(indptr, row, right=True) - 1).clamp(max=P - 1)
    live = row < indptr[P]
    pos = torch.where(live, ctx[req] + row - indptr[req], torch.zeros_like(row))
    page = table[req, torch.where(live, pos // ps, torch.zeros_like(pos)).long()].long()
    slot = torch.where(live, page * ps + pos % ps, torch.full_like(page, -1))
    return [table, free, F2.to(torch.int32), seq, indptr, pos, slot]


def _plain_norm_rope(s, x, weight):
    """Rows of heads [n, h, d] in 32 bits, normalised and rotated; angles in 64 bits."""
    c = s["case"]
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * weight
    rot = c["rot"]
    angle = s["pos"].double()[s["axis"]].t() * s["freq"]                  # [n, rot / 2]
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    part = x[..., :rot]
    if c["interleaved"]:
        a, b = part[..., 0::2], part[..., 1::2]
        part = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = part[..., :rot // 2], part[..., rot // 2:]
        part = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([part, x[..., rot:]], -1).to(torch.bfloat16)


def _own_rope(s):
    import speculative_decode_verify_paged_gb300 as sa
    sa.spec_attn_norm_rope(s["plan"], s["q"], s["k"], s["qw"], s["kw"], s["pos"], s["q_out"], s["k_out"])
    return [s["q_out"], s["k_out"]]


def _plain_rope(s):
    return [_plain_norm_rope(s, s["q"], s["qw"]), _plain_norm_rope(s, s["k"], s["kw"])]


def _e4m3(byte):
    return byte.view(torch.float8_e4m3fn).float()


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


def _decode(s, codes, scales, page, at):
    """The values that the written slots of a 4-bit cache stand for (exact in bf16: the decode scale is a power of two)."""
    c = codes[page, :, at].long()
    v = torch.stack([s["code_values"][c & 15], s["code_values"][c >> 4]], -1).flatten(-2).unflatten(-1, (-1, 16))
    return (v * (_e4m3(scales[page, :, at]) * s["gscale"])[..., None]).flatten(-2).to(torch.bfloat16)


def _written(s, q):
    """What an append returns: the rotated queries and the cache, or the values written to a 4-bit one."""
    if s["case"]["kv"] == "bf16":
        return [q, s["k_pool"], s["v_pool"]]
    page, at = s["slot"] // s["case"]["page_size"], s["slot"] % s["case"]["page_size"]
    return [q, _decode(s, s["k_pool"], s["k_scales"], page, at), _decode(s, s["v_pool"], s["v_scales"], page, at)]


def _own_append(s):
    import speculative_decode_verify_paged_gb300 as sa
    g = s.get("gscale", 1.0)
    sa.spec_attn_norm_rope_append(s["plan"], s["q"], s["k"], s["v"], s["qw"], s["kw"], s["pos"], s["slot"], s["q_out"],
                                  s["k_pool"], s["v_pool"], s["ws"], s.get("k_scales"), s.get("v_scales"), g, g)
    return _written(s, s["q_out"])


def _plain_append(s):
    q, k = _plain_norm_rope(s, s["q"], s["qw"]), _plain_norm_rope(s, s["k"], s["kw"])
    page, at = s["slot"] // s["case"]["page_size"], s["slot"] % s["case"]["page_size"]
    if s["case"]["kv"] == "bf16":
        s["k_pool"][page, :, at] = k
        s["v_pool"][page, :, at] = s["v"]
    else:
        s["k_pool"][page, :, at], s["k_scales"][page, :, at] = _quantise(k, s["gscale"])
        s["v_pool"][page, :, at], s["v_scales"][page, :, at] = _quantise(s["v"], s["gscale"])
    return _written(s, q)


def _own_cross(s):
    import speculative_decode_verify_paged_gb300 as sa
    sa.spec_attn_run_cross(s["plan"], s["q"], s["k"], s["v"], s["indptr"], s["kv_start"], s["kv_len"], s["o"], s["lse"],
                           s["ws"])
    return [s["o"], s["lse"]]


def _plain_cross(s):
    """Padded to [request, longest window] x [request, longest states], masked, in 32 bits."""
    c = s["case"]
    P, S, hq, hkv, d = c["reqs"], c["kv"], c["hq"], c["hkv"], c["d"]
    indptr, n, G = s["indptr"].long(), s["q"].shape[0], c["hq"] // c["hkv"]
    i = torch.arange(s["max_rows"], device="cuda")
    q = s["q"][(indptr[:-1, None] + i).clamp(max=n - 1)].float()            # [P, W, Hq, d]
    q = q.unflatten(2, (hkv, G)).permute(0, 2, 3, 1, 4).reshape(P, hkv, G * len(i), d)
    j = torch.arange(S, device="cuda")
    at = s["kv_start"].long()[:, None] + j
    k, v = (t[at].permute(0, 2, 1, 3).float() for t in (s["k"], s["v"]))    # [P, Hkv, S, d]
    x = torch.matmul(q, k.transpose(2, 3)) / math.sqrt(d)
    x.masked_fill_((j >= s["kv_len"][:, None])[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    x.sub_(m).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x, v) / total
    lse = (m + torch.log(total))[..., 0]
    row = torch.arange(n, device="cuda")
    req = torch.searchsorted(indptr, row, right=True) - 1
    w = row - indptr[req]
    o = o.reshape(P, hkv, G, len(i), d)[req, :, :, w].reshape(n, hq, d).to(torch.bfloat16)
    return [o, lse.reshape(P, hkv, G, len(i))[req, :, :, w].reshape(n, hq)]


# --------------------------------------------------------------------------- #
# What a pass cannot do without, and its result in 64 bits
# --------------------------------------------------------------------------- #
def work(case):
    op = case["op"]
    if op == "tables":
        P, ps = case["reqs"], case["page_size"]
        joined = case["turnover"] / 2 if case["prompts"] else 0.0
        live = min(case["rows"], P * ((1 - case["turnover"] / 2 - joined) * (1 + case["window"]) / 2 +
                                      joined * (1 + case["prompts"]) / 2))
        # per request: three lengths in, two out; per row: position and slot out (padded rows too); a table entry read
        # for every page that holds a row
        return {"bytes": P * 20 + case["rows"] * 12 + 4 * (live / ps + P), "flops": 0}
    if op in ("rope", "append"):
        n, hq, hkv, d = case["rows"], case["hq"], case["hkv"], case["d"]
        moved = n * (hq + hkv) * d * 4 + n * 4 * case["axes"]
        if op == "append":
            row = 2 * d if case["kv"] == "bf16" else d // 2 + d // 16
            moved = n * hq * d * 4 + n * hkv * 2 * (2 * d + row) + n * (8 + 4 * case["axes"])
        return {"bytes": moved, "flops": n * (hq + hkv) * d * 8}
    rows, P = _window_rows(case), case["reqs"]
    mean = (case["kv"] + (P - 1) * (max(1, case["kv"] // 4) + case["kv"]) / 2) / P
    return {"bytes": sum(rows) * case["hq"] * (case["d"] * 4 + 4) + P * mean * case["hkv"] * case["d"] * 4,
            "flops": 4 * sum(rows) * mean * case["hq"] * case["d"]}


def exact(case, seed):
    op = case["op"]
    if op == "tables":
        return None
    s = prepare(case, seed)
    if op == "cross":
        return _exact_cross(case, s)
    turned = [_exact_heads(case, s, s["q"], s["qw"]), _exact_heads(case, s, s["k"], s["kw"])]
    if op == "rope":
        return turned
    k, v = turned[1].to(torch.bfloat16), s["v"]       # a cache holds 16-bit keys, or a quantisation of them
    if case["kv"] == "bf16":
        cache = []
        for new, pool in ((turned[1], s["k_pool"]), (v, s["v_pool"])):
            flat = pool.double().transpose(1, 2).flatten(0, 1)              # [slot, Hkv, d]
            flat[s["slot"]] = new.double()
            cache.append(flat.unflatten(0, (-1, case["page_size"])).transpose(1, 2).contiguous())
        return [turned[0]] + cache
    return [turned[0], _exact_nvfp4(k, s["gscale"]), _exact_nvfp4(v, s["gscale"])]


def _exact_heads(case, s, x, weight):
    """Complex rotation of the pairs, row block by row block, in 64 bits."""
    out = []
    angle = torch.empty(case["rows"], case["rot"] // 2, dtype=torch.float64, device="cuda")
    for j, axis in enumerate(_pair_axis(case["rot"], case["axes"])):
        angle[:, j] = s["pos"][axis].double() * _inv_freq(case["rot"])[j]
    for lo in range(0, case["rows"], 1024):
        y = x[lo:lo + 1024].double()
        if weight is not None:
            y = y / (y.square().mean(2, keepdim=True) + 1e-6).sqrt() * weight.double()
        turn = torch.polar(torch.ones_like(angle[lo:lo + 1024]), angle[lo:lo + 1024])[:, None]
        half = case["rot"] // 2
        pairs = y[:, :, :2 * half]
        if case["interleaved"]:
            z = torch.view_as_complex(pairs.unflatten(2, (half, 2)).contiguous()) * turn
            y[:, :, :2 * half] = torch.view_as_real(z).flatten(2)
        else:
            z = torch.complex(pairs[:, :, :half].contiguous(), pairs[:, :, half:].contiguous()) * turn
            y[:, :, :half], y[:, :, half:2 * half] = z.real, z.imag
        out.append(y)
    return torch.cat(out)


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


def _exact_cross(case, s):
    rows, G, d = _window_rows(case), case["hq"] // case["hkv"], case["d"]
    if sum(w * n for w, n in zip(rows, s["lens"])) * case["hq"] * d > 4e11:
        return None
    o, lse, at = [], [], 0
    for r, w in enumerate(rows):
        lo = r * case["kv"]
        q = s["q"][at:at + w].double()
        per_head = []
        for h in range(case["hq"]):
            x = q[:, h] @ s["k"][lo:lo + s["lens"][r], h // G].double().t() * d ** -0.5
            per_head.append((torch.softmax(x, 1) @ s["v"][lo:lo + s["lens"][r], h // G].double(), torch.logsumexp(x, 1)))
        o.append(torch.stack([p[0] for p in per_head], 1))
        lse.append(torch.stack([p[1] for p in per_head], 1))
        at += w
    return [torch.cat(o), torch.cat(lse)]
