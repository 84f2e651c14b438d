"""The step tables built on the GPU against a plain simulation of the rules in
Python (lists and loops): every output equal, whole buffers compared, so that
what a call must leave alone is checked as well."""
import ctypes
import os
import random
import subprocess
import threading

import pytest
import torch

import speculative_decode_verify_paged_gb300 as sa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from speculative_decode_verify_paged_gb300 import build as libbuild
    libbuild.build()
    torch.cuda.set_device(0)


def simulate(ctx, win, prev, stack, table, ps, max_rows):
    """(seq_lens, q_indptr, stack, table, positions, slots) of one step; lists in, lists out."""
    held = [-(-p // ps) for p in prev]
    seq = [c + w for c, w in zip(ctx, win)]
    need = [-(-s // ps) for s in seq]
    table = [list(row) for row in table]
    stack = list(stack)
    for r in range(len(ctx)):
        stack += table[r][need[r]:held[r]]
    for r in range(len(ctx)):
        for j in range(held[r], need[r]):
            table[r][j] = stack.pop()
    indptr, pos, slot = [0], [], []
    for r in range(len(ctx)):
        indptr.append(indptr[-1] + win[r])
        for i in range(win[r]):
            at = ctx[r] + i
            pos.append(at)
            slot.append(table[r][at // ps] * ps + at % ps)
    pad = max_rows - len(pos)
    return seq, indptr, stack, table, pos + [0] * pad, slot + [-1] * pad


class State:
    """Device buffers of a step, outputs filled with marks so that missing writes show."""

    def __init__(self, ctx, win, prev, free, table, num_pages, ps, max_rows, in_place=False):
        i32 = dict(dtype=torch.int32, device="cuda")
        self.ps = ps
        self.ctx, self.win, self.prev = (torch.tensor(x, **i32) for x in (ctx, win, prev))
        self.free = torch.full((num_pages,), -7, **i32)
        self.free[:len(free)] = torch.tensor(free, **i32)
        self.prev_count = torch.tensor([len(free)], **i32)
        self.table = torch.tensor(table, **i32).reshape(len(ctx), len(table[0]) if table else 4)
        self.seq = self.prev if in_place else torch.full((len(ctx),), -9, **i32)
        self.count = self.prev_count if in_place else torch.full((1,), -9, **i32)
        self.indptr = torch.full((len(ctx) + 1,), -9, **i32)
        self.pos = torch.full((max_rows,), -9, **i32)
        self.slot = torch.full((max_rows,), -9, dtype=torch.int64, device="cuda")
        self.ws = torch.zeros(256, dtype=torch.uint8, device="cuda")

    def run(self, **kw):
        kw = {**dict(page_size=self.ps, max_w=1 << 20, max_seq_len=1 << 30), **kw}
        sa.spec_attn_build_tables(self.ctx, self.win, self.prev, self.prev_count, self.free, self.table, self.seq,
                                  self.indptr, self.count, self.pos, self.slot, self.ws, **kw)

    def check(self, want, free_before):
        seq, indptr, stack, table, pos, slot = want
        assert sa.spec_attn_check_device_status(self.ws) == 0
        assert self.ws.count_nonzero() == 0                     # the ticket is back at 0
        assert self.seq.tolist() == seq and self.indptr.tolist() == indptr
        assert self.count.tolist() == [len(stack)]
        assert self.pos.tolist() == pos and self.slot.tolist() == slot
        got = self.table.tolist()
        assert got == table
        # the stack up to its count; what lies past the old and the new top is untouched
        now = self.free.tolist()
        assert now[:len(stack)] == stack
        top = max(len(stack), len(free_before))
        assert now[top:] == [-7] * (len(now) - top)


def draw(rng, P, ps, ctx_hi, win_hi, turnover=0.3):
    prev, ctx, win = [], [], []
    for _ in range(P):
        u = rng.random()
        p = rng.randint(0, ctx_hi)
        if u < turnover / 2:
            prev.append(p), ctx.append(0), win.append(0)
        elif u < turnover:
            prev.append(0), ctx.append(0), win.append(rng.randint(0, ctx_hi))
        else:
            c = max(0, p - rng.choice((0, 0, 1, ps - 1, ps, ps + 1, 3 * ps)))
            prev.append(p), ctx.append(c), win.append(rng.choice((0, 1, 1, rng.randint(0, win_hi))))
    return ctx, win, prev


def place(rng, prev, ps, stride, num_pages):
    pages = list(range(num_pages))
    rng.shuffle(pages)
    table = []
    for p in prev:
        n = -(-p // ps)
        table.append(pages[:n] + [-3] * (stride - n))
        del pages[:n]
    return table, pages


CASES = [
    # P, page size, longest context, longest window
    (1, 16, 0, 1), (1, 64, 5000, 16), (2, 16, 40, 40), (33, 32, 500, 16), (511, 16, 300, 9), (513, 16, 300, 9),
    (1500, 64, 200, 16), (7, 16, 9000, 9000),
]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_tables_match_the_simulation(case, in_place):
    P, ps, ctx_hi, win_hi = CASES[case]
    rng = random.Random(100 + case)
    ctx, win, prev = draw(rng, P, ps, ctx_hi, win_hi)
    stride = -(-(max(c + w for c, w in zip(ctx, win)) + max(prev) + 1) // ps)
    num_pages = P * stride
    table, free = place(rng, prev, ps, stride, num_pages)
    rows = sum(win) + rng.choice((0, 1, 700))
    s = State(ctx, win, prev, free, table, num_pages, ps, rows, in_place)
    s.run()
    s.check(simulate(ctx, win, prev, free, table, ps, rows), free)
    if not in_place:      # the same inputs again: the same answer
        s.run()
        s.check(simulate(ctx, win, prev, free, table, ps, rows), free)


@pytest.mark.parametrize("P", [255, 256, 257, 2047, 2048, 2049, 8192, 8193])
def test_request_counts_at_the_edges_of_the_split(P):
    """Around a thread's shares of the requests: one, several adjacent ones, or every 32nd."""
    ps, rng = 16, random.Random(P)
    ctx, win, prev = draw(rng, P, ps, 60, 5)
    stride = -(-(max(c + w for c, w in zip(ctx, win)) + max(prev) + 1) // ps)
    num_pages = P * stride
    table, free = place(rng, prev, ps, stride, num_pages)
    rows = sum(win) + 3
    s = State(ctx, win, prev, free, table, num_pages, ps, rows, P % 2 == 0)
    s.run()
    s.check(simulate(ctx, win, prev, free, table, ps, rows), free)


def test_returned_pages_serve_the_same_step():
    """An empty stack: the pages of requests that end go straight to one that joins."""
    ctx, win, prev = [0, 0, 5, 0], [0, 75, 1, 0], [48, 0, 16, 33]
    table, free = place(random.Random(1), prev, 16, 8, 7)
    assert free == []
    s = State(ctx, win, prev, free, table, 7, 16, 80)
    s.run()
    s.check(simulate(ctx, win, prev, free, table, 16, 80), free)


@pytest.mark.parametrize("which", ["ctx", "prev"])
def test_decode_loop_in_one_graph(which):
    """Steps of a decode loop, state updated in place, captured once and replayed; the lengths that a verify step
    would leave on the GPU are written between the replays."""
    rng = random.Random(5)
    P, ps, stride, num_pages, rows = 9, 16, 40, 9 * 40, 9 * 16 + 300
    prev = [0] * P
    table, free = place(rng, prev, ps, stride, num_pages)
    s = State([0] * P, [0] * P, prev, free, table, num_pages, ps, rows, in_place=True)
    if which == "ctx":    # seq_lens overwrite the context lengths, not the previous ones
        s.seq = s.ctx
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    for step in range(6):
        ctx, win = [], []
        for r in range(P):
            if rng.random() < 0.2:
                ctx.append(0), win.append(rng.choice((0, rng.randint(1, 30))))
            else:
                ctx.append(rng.randint(max(0, prev[r] - 15), prev[r])), win.append(rng.randint(0, 16))
        s.ctx.copy_(torch.tensor(ctx, dtype=torch.int32))
        s.win.copy_(torch.tensor(win, dtype=torch.int32))
        s.prev.copy_(torch.tensor(prev, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        want = simulate(ctx, win, prev, free, table, ps, rows)
        assert s.seq.tolist() == want[0] and s.indptr.tolist() == want[1] and s.count.tolist() == [len(want[2])]
        assert s.free[:len(want[2])].tolist() == want[2] and s.table.tolist() == want[3]
        assert s.pos.tolist() == want[4] and s.slot.tolist() == want[5]
        assert sa.spec_attn_check_device_status(s.ws) == 0
        prev, free, table = want[0], want[2], want[3]


def _refused(s, bits, **kw):
    before = [t.clone() for t in (s.free, s.table, s.prev, s.prev_count)]
    s.run(**kw)
    assert sa.spec_attn_check_device_status(s.ws) == bits
    assert s.indptr.count_nonzero() == 0 and s.pos.count_nonzero() == 0 and bool((s.slot == -1).all())
    assert torch.equal(s.free, before[0]) and torch.equal(s.table, before[1])
    assert torch.equal(s.seq, before[2]) and torch.equal(s.count, before[3])
    assert s.ws.count_nonzero() == 0


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("name,bits,change", [
    ("negative window", sa.SPEC_ATTN_DEV_BAD_WINDOW, dict(win=[3, -1, 2])),
    ("wide window", sa.SPEC_ATTN_DEV_BAD_WINDOW, dict(win=[3, 17, 2], kw=dict(max_w=16))),
    ("too many rows", sa.SPEC_ATTN_DEV_BAD_WINDOW, dict(win=[30, 31, 4])),
    ("negative context", sa.SPEC_ATTN_DEV_BAD_SEQ_LEN, dict(ctx=[10, -1, 30])),
    ("context not cached", sa.SPEC_ATTN_DEV_BAD_SEQ_LEN, dict(ctx=[10, 21, 30])),
    ("longer than the plan", sa.SPEC_ATTN_DEV_BAD_SEQ_LEN, dict(kw=dict(max_seq_len=31))),
    ("longer than the table row", sa.SPEC_ATTN_DEV_BAD_SEQ_LEN, dict(win=[3, 45, 2], kw=dict(max_w=64))),
    ("huge lengths", sa.SPEC_ATTN_DEV_BAD_SEQ_LEN, dict(prev=[10, 2 ** 31 - 1, 30], ctx=[10, 2 ** 31 - 1, 30])),
    ("out of pages", sa.SPEC_ATTN_DEV_OUT_OF_PAGES, dict(free=1, win=[8, 20, 4])),
    ("too many free pages", sa.SPEC_ATTN_DEV_BAD_FREE_LIST, dict(free=9)),
    ("negative count", sa.SPEC_ATTN_DEV_BAD_FREE_LIST, dict(free=-1)),
])
def test_refused_steps_are_empty(name, bits, change, in_place):
    prev, ctx, win = [10, 20, 30], [10, 20, 30], [3, 1, 2]
    table, free = place(random.Random(2), prev, 16, 4, 13)       # 5 pages held, 8 free
    s = State(change.get("ctx", ctx), change.get("win", win), change.get("prev", prev), free, table, 13, 16, 64, in_place)
    if "free" in change:
        s.prev_count.fill_(change["free"])
    _refused(s, bits, **{**dict(max_seq_len=64), **change.get("kw", {})})


def test_bad_page_ids_give_their_rows_no_slot():
    prev, ctx, win = [20, 20], [20, 20], [14, 2]                 # request 0 takes a page for its last two rows
    table, free = place(random.Random(3), prev, 16, 4, 12)
    bad_entry, bad_free = [list(r) for r in table], list(free)
    bad_entry[1][1] = 12                                         # the page of request 1's rows
    bad_free[-1] = -5                                            # the page that request 0 takes
    for tab, stack, rows in ((bad_entry, free, [14, 15]), (table, bad_free, [12, 13])):
        s = State(ctx, win, prev, stack, tab, 12, 16, 16)
        s.run()
        assert sa.spec_attn_check_device_status(s.ws) == sa.SPEC_ATTN_DEV_BAD_PAGE
        want = simulate(ctx, win, prev, stack, tab, 16, 16)
        assert s.slot.tolist() == [-1 if i in rows else x for i, x in enumerate(want[5])]
        assert s.table.tolist() == want[3] and s.pos.tolist() == want[4]


def test_no_requests_and_no_rows():
    s = State([], [], [], [4, 2], [], 5, 16, 3)
    s.run()
    assert s.indptr.tolist() == [0] and s.count.tolist() == [2] and s.slot.tolist() == [-1] * 3
    s = State([5], [0], [5], [4, 2], [[1, 0]], 5, 16, 0)
    s.run()
    assert s.indptr.tolist() == [0, 0] and s.seq.tolist() == [5] and sa.spec_attn_check_device_status(s.ws) == 0


def test_another_stream_and_the_largest_batch():
    """16384 requests (the limit), on a stream of its own."""
    rng = random.Random(8)
    P, ps = 16384, 16
    ctx, win, prev = draw(rng, P, ps, 60, 4)
    stride = 12
    table, free = place(rng, prev, ps, stride, P * stride)
    rows = sum(win) + 3
    s = State(ctx, win, prev, free, table, P * stride, ps, rows, True)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    s.run(stream=st)
    st.synchronize()
    s.check(simulate(ctx, win, prev, free, table, ps, rows), free)


def _large(P, in_place=False):
    """A step of P short requests, and its answer."""
    rng = random.Random(P)
    ctx, win, prev = draw(rng, P, 16, 60, 4)
    table, free = place(rng, prev, 16, 12, P * 12)
    rows = sum(win) + 3
    return State(ctx, win, prev, free, table, P * 12, 16, rows, in_place), simulate(ctx, win, prev, free, table, 16, rows), free


def test_two_threads_with_different_request_counts(tmp_path):
    """Both above 3924 requests, where a launch asks for more shared memory than a kernel has by itself: neither call
    takes it from the other's launch.  (Each on a stream of its own, with its own buffers and workspace; the calls are
    made from C, where no interpreter lock keeps them apart.)"""
    src, exe = tmp_path / "many.c", tmp_path / "many.so"
    src.write_text("""
        #include "spec_attn.h"
        typedef int (*tables_fn)(const spec_attn_tables_problem*, const int32_t*, const int32_t*, const int32_t*,
                                 const int32_t*, int32_t*, int32_t*, int32_t*, int32_t*, int32_t*, int32_t*, int64_t*,
                                 void*, size_t, spec_attn_stream_t);
        int many(tables_fn f, int n, const spec_attn_tables_problem* p, void** a, spec_attn_stream_t s) {
            int failed = 0;
            for (int i = 0; i < n; ++i)
                failed += f(p, a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[7], a[8], a[9], a[10], a[11], 256, s) != 0;
            return failed;
        }
    """)
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    subprocess.run(["gcc", "-shared", "-fPIC", "-O2", "-I", include, str(src), "-o", str(exe)], check=True)
    many = ctypes.CDLL(str(exe)).many
    many.argtypes = [ctypes.c_void_p, ctypes.c_int] + [ctypes.c_void_p] * 3
    tables = ctypes.cast(sa.load_library().spec_attn_build_tables, ctypes.c_void_p)
    steps = [_large(P) for P in (4000, 16384)]
    for s, _, _ in steps:
        s.run()                  # (the first call, with its loading of the kernel)
    torch.cuda.synchronize()
    streams, failed = [torch.cuda.Stream() for _ in steps], [None, None]

    def loop(i):
        torch.cuda.set_device(0)
        s = steps[i][0]
        prob = sa.spec_attn_tables_problem(s.ctx.numel(), s.pos.numel(), s.ps, s.free.numel(), s.table.shape[1], 1 << 20,
                                           1 << 30)
        at = (ctypes.c_void_p * 12)(*[t.data_ptr() for t in (s.ctx, s.win, s.prev, s.prev_count, s.free, s.table, s.seq,
                                                             s.indptr, s.count, s.pos, s.slot, s.ws)])
        failed[i] = many(tables, 3000, ctypes.addressof(prob), ctypes.addressof(at), streams[i].cuda_stream)
    threads = [threading.Thread(target=loop, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert failed == [0, 0]
    for s, want, free in steps:
        s.check(want, free)


def test_one_graph_with_two_request_counts():
    """A call with fewer requests between the capture of a larger one and the graph's first replay."""
    steps = [_large(P) for P in (16384, 4000)]
    torch.cuda.synchronize()
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=stream):
        for s, _, _ in steps:
            s.run(stream=stream)
    graph.replay()
    torch.cuda.synchronize()
    for s, want, free in steps:
        s.check(want, free)
