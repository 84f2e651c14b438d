"""Drafted trees: positions and ancestor masks, accepted paths and the move of their keys and values, each against plain
Python on the host; whole numbers and bytes, so every comparison is exact.  Then a chain of whole steps."""
import random
import threading

import pytest
import torch

import speculative_decode_verify_paged_gb300 as sa

pytestmark = pytest.mark.gpu
I32 = dict(dtype=torch.int32, device="cuda")
I64 = dict(dtype=torch.int64, device="cuda")


@pytest.fixture(scope="module", autouse=True)
def _built():
    from speculative_decode_verify_paged_gb300 import build as libbuild
    libbuild.build()
    torch.cuda.set_device(0)


def workspace():
    return torch.zeros(256, dtype=torch.uint8, device="cuda")


def indptr_of(rows):
    out = [0]
    for w in rows:
        out.append(out[-1] + w)
    return torch.tensor(out, **I32)


def tree(rng, w, kind="any"):
    if kind == "chain":
        return [i - 1 for i in range(w)]
    if kind == "star":
        return [-1 if i == 0 else 0 for i in range(w)]
    if kind == "roots":
        return [-1] * w
    return [-1 if i == 0 or rng.random() < 0.05 else rng.randrange(max(0, i - rng.choice((1, 4, 40))), i) for i in range(w)]


def host_tables(parents, ctx, words, window, sinks):
    depth, masks = [], []
    for i, p in enumerate(parents):
        depth.append(0 if p < 0 else depth[p] + 1)
        bits, j = 0, i
        while j >= 0:
            if not window or depth[i] - depth[j] < window or ctx + depth[j] < sinks:
                bits |= 1 << j
            j = parents[j]
        masks.append([bits >> 32 * k & 0xffffffff for k in range(words)])
    return [ctx + h for h in depth], masks


def signed(words):
    return [[x - 2 ** 32 if x >= 2 ** 31 else x for x in row] for row in words]


def run_tables(trees, ctx, max_w, words, window=0, sinks=0, pad=3, ws=None, stream=None):
    rows = [len(t) for t in trees]
    n = sum(rows) + pad
    pos, mask = torch.full((n,), 99, **I32), torch.full((n, words), 99, **I32)
    ws = workspace() if ws is None else ws
    sa.spec_attn_build_tree(torch.tensor([p for t in trees for p in t] + [0] * pad, **I32),
                            torch.tensor([c + w for c, w in zip(ctx, rows)], **I32), indptr_of(rows), pos, mask, ws,
                            max_w=max_w, window_left=window, sink_keys=sinks, stream=stream)
    return pos, mask, ws


@pytest.mark.parametrize("kind", ["any", "chain", "star", "roots"])
@pytest.mark.parametrize("rows", [[1], [0, 3, 1], [31, 32, 33, 64, 65], [0, 0], [255, 7], [1024, 1]])
def test_tables(rows, kind):
    rng = random.Random(sum(rows))
    trees = [tree(rng, w, kind) for w in rows]
    ctx = [rng.randrange(5000) for _ in rows]
    max_w = max(rows + [1])
    for window, sinks, extra in ((0, 0, 0), (1, 0, 2), (3, ctx[0] + 2, 0), (2000, 7, 1)):
        words = -(-max_w // 32) + extra
        pos, mask, ws = run_tables(trees, ctx, max_w, words, window, sinks)
        want = [host_tables(t, c, words, window, sinks) for t, c in zip(trees, ctx)]
        assert pos.tolist() == [x for w in want for x in w[0]] + [0] * 3
        assert mask.tolist() == signed([x for w in want for x in w[1]] + [[0] * words] * 3)
        assert sa.spec_attn_check_device_status(ws) == 0


def test_tables_without_requests_empty_the_padding():
    pos, mask, ws = run_tables([], [], 8, 1, pad=700)
    assert not pos.any() and not mask.any()


@pytest.mark.parametrize("parent", [5, 4, 100, -2, 2 ** 31 - 1, -2 ** 31])
def test_a_bad_parent_counts_as_a_root(parent):
    t = [-1, 0, 0, 2, 3, 4]
    t[4] = parent
    pos, mask, ws = run_tables([[-1, 0], t], [10, 20], 8, 1)
    fixed = t[:4] + [-1] + t[5:]
    want = [host_tables(x, c, 1, 0, 0) for x, c in (([-1, 0], 10), (fixed, 20))]
    assert pos.tolist()[:8] == want[0][0] + want[1][0] and mask.tolist()[:8] == want[0][1] + want[1][1]
    assert sa.spec_attn_check_device_status(ws) == sa.SPEC_ATTN_DEV_BAD_TREE


@pytest.mark.parametrize("field", ["indptr", "seq"])
def test_a_bad_request_leaves_its_rows(field):
    rows = [3, 4, 2]
    parents = torch.tensor([-1, 0, 1, -1, 0, 1, 2, -1, 0], **I32)
    indptr, seq = indptr_of(rows), torch.tensor([13, 14, 12], **I32)
    if field == "indptr":
        indptr[2] = 20                    # request 1: 17 rows, request 2: -11
    else:
        seq[1] = 3
    pos, mask, ws = torch.full((9,), 99, **I32), torch.full((9, 1), 99, **I32), workspace()
    sa.spec_attn_build_tree(parents, seq, indptr, pos, mask, ws, max_w=8)
    assert pos.tolist()[:7] == [10, 11, 12, 99, 99, 99, 99]
    assert pos.tolist()[7:] == ([99, 99] if field == "indptr" else [10, 11])
    assert sa.spec_attn_check_device_status(ws) == (
        sa.SPEC_ATTN_DEV_BAD_WINDOW if field == "indptr" else sa.SPEC_ATTN_DEV_BAD_SEQ_LEN)


def host_accept(parents, draft, target, cap):
    if not parents:
        return [], -1
    path = [0]
    while len(path) < cap:
        below = [j for j, p in enumerate(parents) if p == path[-1] and j > path[-1] and draft[j] == target[path[-1]]]
        if not below:
            break
        path.append(below[0])
    return path, target[path[-1]]


def accept_case(rng, rows, kind="any", vocab=3):
    trees = [tree(rng, w, kind) for w in rows]
    draft = [[rng.randrange(vocab) for _ in t] for t in trees]
    target = [[rng.randrange(vocab) for _ in t] for t in trees]
    return trees, draft, target


def run_accept(trees, draft, target, ctx, max_w, cap, in_place=False, pad=2, ws=None, stream=None):
    rows = [len(t) for t in trees]
    flat = lambda x, **kw: torch.tensor([v for t in x for v in t] + [0] * pad, **kw)  # noqa: E731
    P = len(rows)
    seq = torch.tensor([c + w for c, w in zip(ctx, rows)], **I32)
    path, accepted, nxt = torch.full((P, cap), 99, **I32), torch.full((P,), 99, **I32), torch.full((P,), 99, **I64)
    out = seq if in_place else torch.full((P,), 99, **I32)
    ws = workspace() if ws is None else ws
    sa.spec_attn_accept_tree(flat(trees, **I32), flat(draft, **I64), flat(target, **I64), seq, indptr_of(rows), path,
                             accepted, nxt, out, ws, max_w=max_w, stream=stream)
    return path, accepted, nxt, out, ws


@pytest.mark.parametrize("kind", ["any", "chain", "star"])
@pytest.mark.parametrize("rows,cap", [([1], 1), ([0, 3, 1], 4), ([31, 32, 33, 64, 65], 9), ([64] * 8, 1),
                                      ([255, 7], 300), ([1024, 1], 1024)])
@pytest.mark.parametrize("vocab", [1, 2, 5])
def test_accept(rows, cap, kind, vocab):
    rng = random.Random(sum(rows) + vocab)
    case = accept_case(rng, rows, kind, vocab)
    ctx = [rng.randrange(5000) for _ in rows]
    for in_place in (False, True):
        path, accepted, nxt, out, ws = run_accept(*case, ctx, max(rows), cap, in_place)
        for r, (t, d, g) in enumerate(zip(*case)):
            want, last = host_accept(t, d, g, cap)
            assert path[r].tolist() == want + [-1] * (cap - len(want))
            assert (int(accepted[r]), int(nxt[r]), int(out[r])) == (len(want), last, ctx[r] + len(want))
        assert sa.spec_attn_check_device_status(ws) == 0


def test_tokens_are_compared_whole():
    """Tokens that agree in their low 32 bits are different tokens."""
    path, accepted, nxt, _, _ = run_accept([[-1, 0, 0]], [[5, 2 ** 32 + 7, 7]], [[7, 1, 2 ** 40 + 3]], [4], 4, 3)
    assert path.tolist() == [[0, 2, -1]] and nxt.tolist() == [2 ** 40 + 3]


def test_accept_reports_bad_trees_and_requests():
    t = [[-1, 5, 0], [-1, 0]]
    path, accepted, nxt, out, ws = run_accept(t, [[1, 1, 1], [1, 1]], [[1, 1, 1], [1, 1]], [10, 20], 4, 3)
    assert path.tolist() == [[0, 2, -1], [0, 1, -1]] and out.tolist() == [12, 22]
    assert sa.spec_attn_check_device_status(ws) == sa.SPEC_ATTN_DEV_BAD_TREE
    path, accepted, nxt, out, ws = run_accept(t, [[1, 1, 1], [1, 1]], [[1, 1, 1], [1, 1]], [10, -1], 2, 3)
    assert path.tolist() == [[-1] * 3] * 2 and accepted.tolist() == [0, 0] and nxt.tolist() == [-1, -1]
    assert out.tolist() == [13, 1]                        # their seq_lens
    assert sa.spec_attn_check_device_status(ws) == sa.SPEC_ATTN_DEV_BAD_WINDOW | sa.SPEC_ATTN_DEV_BAD_SEQ_LEN


class Caches:
    def __init__(self, layers, pages, hkv, d, ps, kv, interleave, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def pool(row):
            x = torch.randint(0, 256, (pages, 2, hkv, ps, row), generator=g, device="cuda", dtype=torch.uint8)
            return (x[:, 0], x[:, 1]) if interleave else (x[:, 0].contiguous(), x[:, 1].contiguous())
        self.lists = [[], [], [], []]
        for _ in range(layers):
            for i, t in enumerate(pool(2 * d if kv == "bf16" else d // 2)):
                self.lists[i].append(t.view(torch.bfloat16) if kv == "bf16" else t)
            if kv == "nvfp4":
                for i, t in enumerate(pool(d // 16)):
                    self.lists[2 + i].append(t)
        self.kv = kv

    def bytes(self):
        return [[t.contiguous().view(torch.uint8).clone() for t in x] for x in self.lists]

    def move(self, *a, **kw):
        k, v, ks, vs = self.lists
        scales = dict(k_scales=ks, v_scales=vs) if self.kv == "nvfp4" else {}
        sa.spec_attn_move_kv(k, v, *a, **scales, **kw)


def random_path(rng, w, most):
    n = rng.randint(0, min(w, most))
    return sorted(rng.sample(range(w), n))


def moved(before, table, ctx, paths, ps):
    """Every pool's bytes after the moves, from a copy of all that is read."""
    want = [[t.clone() for t in x] for x in before]
    for r, path in enumerate(paths):
        for i, j in enumerate(path):
            (p0, s0), (p1, s1) = [(int(table[r, (ctx[r] + k) // ps]), (ctx[r] + k) % ps) for k in (j, i)]
            for src, dst in zip(before, want):
                for a, b in zip(src, dst):
                    b[p1, :, s1] = a[p0, :, s0]
    return want


@pytest.mark.parametrize("kv", ["bf16", "nvfp4"])
@pytest.mark.parametrize("layers,rows,hkv,d,ps,interleave", [
    (1, [1], 1, 64, 16, False), (2, [5, 0, 64], 2, 128, 32, True), (3, [33, 20], 3, 256, 64, False),
    (1, [600, 40], 2, 64, 16, True), (65, [9, 30], 1, 64, 16, False)])
def test_move(kv, layers, rows, hkv, d, ps, interleave):
    rng = random.Random(d + layers)
    ctx = [rng.choice((0, 15, rng.randrange(200))) for _ in rows]
    need = [-(-(c + w) // ps) for c, w in zip(ctx, rows)]
    pages = sum(need) + 2
    perm = rng.sample(range(pages), pages)
    table = torch.full((len(rows), max(need) + 1), -1, dtype=torch.int32)
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = torch.tensor(perm[at:at + n], dtype=torch.int32)
        at += n
    c = Caches(layers, pages, hkv, d, ps, kv, interleave, seed=d)
    cap = 600
    for trial in range(3):
        paths = [list(range(w)) if trial == 0 else list(range(min(1, w // 2), w)) if trial == 1 else random_path(rng, w, cap)
                 for w in rows]
        before = c.bytes()
        path = torch.tensor([p + [-1] * (cap - len(p)) for p in paths], **I32)
        ws = workspace()
        c.move(table.cuda(), torch.tensor([a + w for a, w in zip(ctx, rows)], **I32), indptr_of(rows), path,
               torch.tensor([len(p) for p in paths], **I32), ws, max_seq_len=5000)
        want = moved(before, table, ctx, paths, ps)
        for a, b in zip(c.bytes(), want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
        assert sa.spec_attn_check_device_status(ws) == 0


@pytest.mark.parametrize("path,accepted,bits", [
    ([0, 2, 2], 3, sa.SPEC_ATTN_DEV_BAD_TREE), ([0, 3, 1], 3, sa.SPEC_ATTN_DEV_BAD_TREE),
    ([-1, 2, 3], 3, sa.SPEC_ATTN_DEV_BAD_TREE), ([0, 2, 6], 3, sa.SPEC_ATTN_DEV_BAD_TREE),
    ([0, 2, 3], 4, sa.SPEC_ATTN_DEV_BAD_TREE), ([0, 2, 3], -1, sa.SPEC_ATTN_DEV_BAD_TREE)])
def test_a_bad_path_moves_nothing_of_its_request(path, accepted, bits):
    c = Caches(2, 4, 2, 64, 16, "nvfp4", False, 1)
    before = c.bytes()
    table, ws = torch.tensor([[0], [1]], **I32), workspace()
    paths, n = torch.tensor([path, [1, 4, 5]], **I32), torch.tensor([accepted, 3], **I32)
    c.move(table, torch.tensor([9, 10], **I32), indptr_of([6, 6]), paths, n, ws, max_seq_len=100)
    assert sa.spec_attn_check_device_status(ws) == bits
    want = moved(before, table.cpu(), [3, 4], [[], [1, 4, 5]], 16)
    for a, b in zip(c.bytes(), want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_move_skips_bad_requests_and_pages():
    c = Caches(1, 4, 2, 64, 16, "bf16", False, 2)
    before = c.bytes()
    table, ws = torch.tensor([[0, 9], [1, 2], [3, 3]], **I32), workspace()
    paths, n = torch.tensor([[1, 4, 5]] * 3, **I32), torch.tensor([3, 3, 3], **I32)
    # request 0: its keys 14 .. 19, those from 16 on in a page that does not exist; request 1: longer than allowed
    c.move(table, torch.tensor([20, 31, 9], **I32), indptr_of([6, 6, 6]), paths, n, ws, max_seq_len=30)
    assert sa.spec_attn_check_device_status(ws) == sa.SPEC_ATTN_DEV_BAD_PAGE | sa.SPEC_ATTN_DEV_BAD_SEQ_LEN
    want = moved(before, torch.tensor([[0, 0], [0, 0], [3, 3]]), [14, 0, 3], [[1], [], [1, 4, 5]], 16)
    for a, b in zip(c.bytes(), want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_move_past_32_bits():
    """Pages 1 MiB apart in one allocation of over 4 GiB."""
    hkv, d, ps, stride = 2, 64, 16, 1 << 20
    pages = 2 ** 32 // stride + 3
    big = torch.zeros(pages * stride, dtype=torch.uint8, device="cuda").view(pages, stride)
    dense = hkv * ps * d * 2
    k, v = (big[:, i * dense:(i + 1) * dense].view(torch.bfloat16).unflatten(1, (hkv, ps, d)) for i in (0, 1))
    last = pages - 1
    new = torch.randn(2, hkv, ps, d, device="cuda").bfloat16()
    k[last], v[last] = new[0], new[1]
    ws = workspace()
    sa.spec_attn_move_kv([k], [v], torch.tensor([[last]], **I32), torch.tensor([12], **I32), indptr_of([9]),
                         torch.tensor([[2, 5, 8]], **I32), torch.tensor([3], **I32), ws, max_seq_len=16)
    assert sa.spec_attn_check_device_status(ws) == 0
    for t, n in ((k, new[0]), (v, new[1])):
        want = n.clone()
        for i, j in enumerate((2, 5, 8)):
            want[:, 3 + i] = n[:, 3 + j]
        assert torch.equal(t[last], want)


def test_refusals_write_nothing():
    t, d = [[-1, 0, 0]], [[1, 2, 3]]
    rows = torch.tensor([-1, 0, 0], **I32)
    tok, one, ptr = torch.tensor([1, 2, 3], **I64), torch.tensor([9], **I32), indptr_of([3])
    pos, mask, ws = torch.full((3,), 5, **I32), torch.full((3, 1), 5, **I32), workspace()
    path, acc, nxt, ctx = torch.full((1, 3), 5, **I32), torch.full((1,), 5, **I32), torch.full((1,), 5, **I64), one + 0
    for call in (lambda: sa.spec_attn_build_tree(rows.long(), one, ptr, pos, mask, ws, max_w=3),
                 lambda: sa.spec_attn_build_tree(rows, one, ptr, pos[:2], mask, ws, max_w=3),
                 lambda: sa.spec_attn_build_tree(rows, one, ptr.cpu(), pos, mask, ws, max_w=3),
                 lambda: sa.spec_attn_accept_tree(rows, tok.int(), tok, one, ptr, path, acc, nxt, ctx, ws, max_w=3),
                 lambda: sa.spec_attn_accept_tree(rows, tok, tok, one, ptr, path[:0], acc, nxt, ctx, ws, max_w=3)):
        with pytest.raises(ValueError):
            call()
    for call, status in (
            (lambda: sa.spec_attn_build_tree(rows, one, ptr, pos, mask, ws, max_w=33), sa.SPEC_ATTN_E_INVALID_ARG),
            (lambda: sa.spec_attn_build_tree(rows, one, ptr, pos, mask, ws, max_w=1025), sa.SPEC_ATTN_E_UNSUPPORTED),
            (lambda: sa.spec_attn_build_tree(rows, one, ptr, rows, mask, ws, max_w=3), sa.SPEC_ATTN_E_INVALID_ARG),
            (lambda: sa.spec_attn_build_tree(rows, one, ptr, pos, mask, ws[:64], max_w=3),
             sa.SPEC_ATTN_E_WORKSPACE_TOO_SMALL),
            (lambda: sa.spec_attn_accept_tree(rows, tok, tok, one, ptr, path, one, nxt, ctx, ws, max_w=3),
             sa.SPEC_ATTN_E_INVALID_ARG),
            (lambda: sa.spec_attn_accept_tree(rows, tok, tok, one, ptr, path, acc, tok[:1], ctx, ws, max_w=3),
             sa.SPEC_ATTN_E_INVALID_ARG)):
        with pytest.raises(sa.SpecAttnError) as e:
            call()
        assert e.value.status == status
    c = Caches(2, 4, 2, 64, 16, "nvfp4", False, 3)
    before = c.bytes()
    k, v, ks, vs = c.lists
    args = (torch.tensor([[0]], **I32), one, ptr, torch.tensor([[1, 2, -1]], **I32), torch.tensor([2], **I32), ws)
    for kk, vv, kw in ((k, v[:1], dict(k_scales=ks, v_scales=vs)), (k, v, dict(k_scales=ks)), (k, v, dict(v_scales=vs)),
                       (k, [v[0], v[1].cpu()], dict(k_scales=ks, v_scales=vs)), (k, v, {}),
                       (k, [v[0], v[1][:3]], dict(k_scales=ks, v_scales=vs))):
        with pytest.raises((ValueError, TypeError)):
            sa.spec_attn_move_kv(kk, vv, *args, max_seq_len=100, **kw)
    for kk, vv in (([k[0], k[0]], [v[0], k[0]]),):
        with pytest.raises(sa.SpecAttnError) as e:
            sa.spec_attn_move_kv(kk, vv, *args, max_seq_len=100, k_scales=ks, v_scales=vs)
        assert e.value.status == sa.SPEC_ATTN_E_INVALID_ARG
    torch.cuda.synchronize()
    assert bool((pos == 5).all()) and bool((mask == 5).all()) and bool((path == 5).all()) and bool((acc == 5).all())
    for a, b in zip(c.bytes(), before):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_streams_threads_and_graphs():
    """The tables and the path from two threads on streams of their own, and captured together and replayed."""
    rng = random.Random(4)
    case = accept_case(rng, [64, 30, 1, 0, 55], vocab=2)
    ctx = [rng.randrange(100) for _ in range(5)]
    want_t = run_tables(case[0], ctx, 64, 2)
    want_a = run_accept(*case, ctx, 64, 12)
    torch.cuda.synchronize()
    out = [None, None]

    def loop(i, s):
        with torch.cuda.stream(s):
            for _ in range(20):
                out[i] = run_tables(case[0], ctx, 64, 2, stream=s)[:2] + run_accept(*case, ctx, 64, 12, stream=s)[:4]
    streams = [torch.cuda.Stream() for _ in range(2)]
    threads = [threading.Thread(target=loop, args=(i, s)) for i, s in enumerate(streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for got in out:
        assert all(torch.equal(a, b) for a, b in zip(got, want_t[:2] + want_a[:4]))
    rows = [len(t) for t in case[0]]
    parents = torch.tensor([p for t in case[0] for p in t], **I32)
    draft, target = (torch.tensor([p for t in x for p in t], **I64) for x in case[1:])
    seq, ptr, ws = torch.tensor([c + w for c, w in zip(ctx, rows)], **I32), indptr_of(rows), workspace()
    n, P = sum(rows), 5
    pos, mask = torch.zeros(n, **I32), torch.zeros(n, 2, **I32)
    path, acc, nxt, new = torch.zeros(P, 12, **I32), torch.zeros(P, **I32), torch.zeros(P, **I64), torch.zeros(P, **I32)
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        sa.spec_attn_build_tree(parents, seq, ptr, pos, mask, ws, max_w=64, stream=s)
        sa.spec_attn_accept_tree(parents, draft, target, seq, ptr, path, acc, nxt, new, ws, max_w=64, stream=s)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(pos, want_t[0][:n]) and torch.equal(mask, want_t[1][:n])
    assert all(torch.equal(a, b) for a, b in zip((path, acc, nxt, new), want_a[:4]))


@pytest.mark.parametrize("kv,window,sinks", [("bf16", 0, 0), ("nvfp4", 0, 0), ("bf16", 40, 4)])
def test_steps_with_trees(kv, window, sinks):
    """Five decoding steps of a two-layer toy with trees -- tables, tree tables, rotated keys into the cache, attention,
    acceptance, move -- against a cache and an attention kept as plain tensors, in which only accepted tokens enter."""
    rng = random.Random(5)
    g = torch.Generator(device="cuda").manual_seed(5)
    P, hq, hkv, d, ps, L, W, cap = 3, 8, 2, 64, 16, 2, 21, 8
    pages = 3 * 40
    fp4 = kv == "nvfp4"
    gs = 2.0 ** -6
    shape = lambda row: (pages, hkv, ps, row)  # noqa: E731
    dt = torch.uint8 if fp4 else torch.bfloat16
    pools = [[torch.zeros(shape(d // 2 if fp4 else d), dtype=dt, device="cuda") for _ in range(L)] for _ in range(2)]
    scales = [[torch.zeros(shape(d // 16), dtype=torch.uint8, device="cuda") if fp4 else None for _ in range(L)]
              for _ in range(2)]
    table, free = torch.full((P, 40), -1, **I32), torch.randperm(pages, generator=g, device="cuda").int()
    count = torch.tensor([pages], **I32)
    ctx, prev = torch.zeros(P, **I32), torch.zeros(P, **I32)
    ws = workspace()
    nr = sa.spec_attn_norm_rope_plan_create(num_q_heads=hq, num_kv_heads=hkv, head_dim=d, inv_freq=sa.rope_inv_freq(d),
                                            page_size=ps, num_pages=pages, kv_dtype=int(fp4))
    mag = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")

    def cached(which, layer, slots):
        x = pools[which][layer][slots // ps, :, slots % ps]
        if not fp4:
            return x.double()
        c = torch.stack([x & 15, x >> 4], -1).flatten(-2).long()
        s = scales[which][layer][slots // ps, :, slots % ps].view(torch.float8_e4m3fn).double()
        return torch.where(c >= 8, -mag[c & 7], mag[c & 7]) * s.repeat_interleave(16, -1) * gs

    text = [[[] for _ in range(P)] for _ in range(2 * L)]        # accepted K, V rows of each layer and request
    for step in range(5):
        # the first step brings prompts as chains, and one request joins late
        trees = [tree(rng, rng.randint(1, W), "chain" if step == 0 else "any") for _ in range(P)]
        if step < 2:
            trees[2] = []
        rows = [len(t) for t in trees]
        n = sum(rows)
        win, seq, ptr = torch.tensor(rows, **I32), torch.zeros(P, **I32), torch.zeros(P + 1, **I32)
        pos0, slot, left = torch.zeros(n, **I32), torch.zeros(n, **I64), torch.zeros(1, **I32)
        sa.spec_attn_build_tables(ctx, win, prev, count, free, table, seq, ptr, left, pos0, slot, ws, page_size=ps,
                                  max_w=W, max_seq_len=640)
        parents = torch.tensor([p for t in trees for p in t], **I32)
        pos, mask = torch.zeros(1, n, **I32), torch.zeros(n, 1, **I32)
        sa.spec_attn_build_tree(parents, seq, ptr, pos[0], mask, ws, max_w=W, window_left=window, sink_keys=sinks)
        lens = [len(text[0][r]) for r in range(P)]
        assert seq.tolist() == [a + w for a, w in zip(lens, rows)] and sa.spec_attn_check_device_status(ws) == 0
        plan = sa.spec_attn_masked_plan_create(
            num_reqs=P, total_q_rows=n, max_w=W, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, num_pages=pages,
            block_table_stride=40, max_seq_len=640, kv_dtype=int(fp4), page_size=ps, tree=1, window_left=window,
            sink_keys=sinks)
        ws2 = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
        new = []
        for layer in range(L):
            q, k, v = (torch.randn(n, h, d, generator=g, device="cuda").bfloat16() for h in (hq, hkv, hkv))
            sa.spec_attn_norm_rope_append(nr, q, k, v, None, None, pos, slot, q, pools[0][layer], pools[1][layer], ws,
                                          scales[0][layer], scales[1][layer], gs, gs)
            o, lse = torch.zeros_like(q), torch.zeros(n, hq, device="cuda")
            sa.spec_attn_run_masked(plan, q, pools[0][layer], pools[1][layer], table, seq, ptr, mask,
                                    pos[0] if window else None, o, lse, ws2, scales[0][layer], scales[1][layer], gs, gs)
            kept = [cached(i, layer, slot) for i in (0, 1)]
            new += kept
            at = 0
            for r, t in enumerate(trees):
                depth = []
                for i, p in enumerate(t):
                    depth.append(0 if p < 0 else depth[p] + 1)
                for i in range(len(t)):
                    chain, j = [], i
                    while j >= 0:
                        chain.insert(0, at + j)
                        j = t[j]
                    cols = [text[2 * layer + a][r] + [kept[a][x] for x in chain] for a in (0, 1)]
                    where = list(range(lens[r])) + [lens[r] + h for h in range(len(chain))]
                    keep = [x for x, y in enumerate(where) if not window or y > lens[r] + depth[i] - window or y < sinks]
                    kk, vv = (torch.stack([c[x] for x in keep]).repeat_interleave(hq // hkv, 1) for c in cols)
                    x = torch.einsum("hd,shd->hs", q[at + i].double(), kk) / d ** 0.5
                    p = torch.softmax(x, 1)
                    want = torch.einsum("hs,shd->hd", p, vv)
                    # (weights and O rounded to 16 bits, twice where splits are joined: 3 x 2^-8 of the largest value)
                    assert float((o[at + i].double() - want).abs().max()) <= 3 * 2.0 ** -8 * float(vv.abs().max())
                    assert float((lse[at + i].double() - torch.logsumexp(x, 1)).abs().max()) <= 1e-3
                at += len(t)
        draft, target = (torch.randint(0, 2, (n,), generator=g, **I64) for _ in range(2))
        path, acc, nxt, new_ctx = torch.zeros(P, cap, **I32), torch.zeros(P, **I32), torch.zeros(P, **I64), torch.zeros(P, **I32)
        sa.spec_attn_accept_tree(parents, draft, target, seq, ptr, path, acc, nxt, new_ctx, ws, max_w=W)
        sa.spec_attn_move_kv(pools[0], pools[1], table, seq, ptr, path, acc, ws, max_seq_len=640,
                             **(dict(k_scales=scales[0], v_scales=scales[1]) if fp4 else {}))
        assert sa.spec_attn_check_device_status(ws) == 0 and sa.spec_attn_check_device_status(ws2) == 0
        at = 0
        for r, t in enumerate(trees):
            want, last = host_accept(t, draft.tolist()[at:at + len(t)], target.tolist()[at:at + len(t)], cap)
            assert path[r].tolist() == want + [-1] * (cap - len(want)) and int(nxt[r]) == last
            for i, x in enumerate(new):
                text[i][r] += [x[at + j] for j in want]
            at += len(t)
        assert new_ctx.tolist() == [len(x) for x in text[0]]
        # the cache holds the accepted text, in order
        for r in range(P):
            m = len(text[0][r])
            if m:
                j = torch.arange(m, device="cuda")
                slots = table[r, j // ps].long() * ps + j % ps
                for layer in range(L):
                    for i in (0, 1):
                        assert torch.equal(cached(i, layer, slots), torch.stack(text[2 * layer + i][r]))
        ctx, prev, count = new_ctx, seq, left
