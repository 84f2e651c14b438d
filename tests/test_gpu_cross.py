"""Cross attention to dense encoder states against its formula in 64 bits.

Tolerance, from the arithmetic, for a row with A = sum_j softmax_j |v_j| and
scores x_j.  A score is a sum of exact products taken in fp32, 16 at a time (d
<= 256: at most 16 additions and one internal alignment each), so it is off by
at most E = 2^-18 max_j sum_e |q_e k_je| sm_scale (32 x 2^-23).  The exponent's
argument is rounded once (2^-24 |x|), the exponential is good to 2^-21 and the
sums of at most 2^12 terms, four chains of 2^5 a tile, to 2^-18 of themselves:
a weight is off by at most e = E + 2^-20 (8 + max |x|) of itself, and the
log-sum-exp by e.  Rounding the weights to bf16 for the second product
moves O by at most 2^-8 A, rounding O itself by 2^-8 |O|:
  |got - want| <= 2^-8 (1 + 2^-6) (|O| + A) + 2 e A."""
import math
import random
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


MARK = 77.0


class Case:
    def __init__(self, rows, lens, hq, hkv, d, starts=None, gap=3, fused=False, force_splits=0, seed=0, pad_rows=2,
                 grow=False, sm_scale=0.0, max_q=None, max_kv=None):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.rows, self.lens, self.hq, self.hkv, self.d = rows, lens, hq, hkv, d
        P, n = len(rows), sum(rows) + pad_rows
        if starts is None:       # packed, with rows of no request between and behind
            starts, at = [], gap
            for m in lens:
                starts.append(at)
                at += m + gap
        self.starts = starts
        total = max([s + m for s, m in zip(starts, lens)] + [0]) + gap
        rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        kv = torch.full((total, 2, hkv, d), float("nan"), device="cuda", dtype=torch.bfloat16)
        for s, m in zip(starts, lens):
            x = rand(m, 2, hkv, d)
            if grow:             # scores that keep growing along the range
                x[:, 0] *= torch.linspace(0.1, 12, max(m, 1), device="cuda")[:m, None, None]
            kv[s:s + m] = x.bfloat16()
        self.k, self.v = (kv[:, 0], kv[:, 1]) if fused else (kv[:, 0].contiguous(), kv[:, 1].contiguous())
        self.q = rand(n, hq, d).bfloat16()
        self.q[sum(rows):] = float("nan")
        i32 = dict(dtype=torch.int32, device="cuda")
        self.indptr = torch.tensor([sum(rows[:i]) for i in range(P + 1)], **i32)
        self.kv_start, self.kv_len = torch.tensor(starts, **i32), torch.tensor(lens, **i32)
        self.sm_scale = sm_scale or 1 / math.sqrt(d)
        self.plan = sa.spec_attn_cross_plan_create(
            num_reqs=P, total_q_rows=n, max_q_rows=max_q or max(rows + [1]), num_q_heads=hq, num_kv_heads=hkv,
            head_dim=d, total_kv_rows=total, max_kv_len=max_kv or max(lens + [0]), sm_scale=sm_scale,
            force_splits=force_splits, kv_row_stride=self.k.stride(0) if fused else 0)
        self.o = torch.full((n, hq, d), MARK, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((n, hq), MARK, device="cuda")
        self.ws = torch.full((self.plan.workspace_bytes,), 0xFF, dtype=torch.uint8, device="cuda")   # (NaN partials)
        sa.spec_attn_reset_device_status(self.ws)

    def run(self, **kw):
        sa.spec_attn_run_cross(self.plan, self.q, self.k, self.v, self.indptr, self.kv_start, self.kv_len, self.o,
                               self.lse, self.ws, **kw)

    def check(self, skip=()):
        G, at = self.hq // self.hkv, 0
        for r, (w, s, m) in enumerate(zip(self.rows, self.starts, self.lens)):
            o, lse = self.o[at:at + w].double().cpu(), self.lse[at:at + w].double().cpu()
            q = self.q[at:at + w].double().cpu()
            at += w
            if r in skip:
                assert bool((o == MARK).all()) and bool((lse == MARK).all())
                continue
            if m == 0:
                assert o.count_nonzero() == 0 and bool((lse == -math.inf).all())
                continue
            k, v = (t[s:s + m].double().cpu().repeat_interleave(G, 1) for t in (self.k, self.v))
            x = torch.einsum("whd,shd->hws", q, k) * self.sm_scale
            p = torch.softmax(x, -1)
            want, A = (torch.einsum("hws,shd->whd", p, t) for t in (v, v.abs()))
            E = 2.0 ** -18 * torch.einsum("whd,shd->hws", q.abs(), k.abs()).amax(-1) * self.sm_scale
            e = (E + 2.0 ** -20 * (8 + x.abs().amax(-1))).t()                    # [w, h]
            tol = 2.0 ** -8 * (1 + 2.0 ** -6) * (want.abs() + A) + 2 * e[..., None] * A
            bad = ~((o - want).abs() <= tol)
            assert not bad.any(), (r, int(bad.sum()), bad.nonzero()[0].tolist(), float((o - want).abs().max()))
            assert bool(((lse - torch.logsumexp(x, -1).t()).abs() <= e).all())
        assert bool((self.o[at:] == MARK).all()) and bool((self.lse[at:] == MARK).all())     # rows of no request
        assert sa.spec_attn_check_device_status(self.ws) == 0


HEADS = [(4, 1, 64), (24, 4, 256), (32, 8, 128), (40, 8, 128), (12, 12, 64), (16, 1, 128), (12, 1, 256), (3, 1, 64)]


@pytest.mark.parametrize("hq,hkv,d", HEADS)
@pytest.mark.parametrize("rows,lens", [
    ([1], [1]), ([1, 1, 1], [15, 16, 17]), ([9, 0, 5], [63, 64, 65]), ([16, 3], [0, 129]), ([7, 1, 2], [127, 128, 1000]),
])
def test_windows(hq, hkv, d, rows, lens):
    c = Case(rows, lens, hq, hkv, d, seed=hq + len(rows), fused=d == 128)
    c.run()
    c.check()


@pytest.mark.parametrize("hq,hkv,d", HEADS)
def test_prompts(hq, hkv, d):
    """More rows than a query tile holds, than two, and a remainder in the second tile of a pair."""
    wt = 128 // (hq // hkv)
    c = Case([wt + 1, 2 * wt, 3 * wt + 2, 1], [130, 31, 257, 64], hq, hkv, d, seed=d, fused=True)
    c.run()
    c.check()


@pytest.mark.parametrize("splits", [2, 3, 7])
@pytest.mark.parametrize("hq,hkv,d", [(4, 1, 64), (24, 4, 256), (32, 8, 128)])
def test_forced_splits(hq, hkv, d, splits):
    c = Case([3, 40, 8], [900, 700, 1], hq, hkv, d, force_splits=splits, seed=splits)
    c.run()
    c.check()


@pytest.mark.parametrize("hq,hkv,d,rows", [(8, 2, 64, 9), (8, 2, 64, 200), (8, 2, 128, 70), (6, 2, 256, 9), (6, 2, 256, 60)])
def test_growing_scores_move_the_reference(hq, hkv, d, rows):
    c = Case([rows], [1500], hq, hkv, d, grow=True, sm_scale=0.2, seed=7)
    c.run()
    c.check()


@pytest.mark.parametrize("splits", [1, 2, 4])
@pytest.mark.parametrize("hq,hkv,d,rows", [(8, 2, 64, 9), (8, 2, 128, 40), (6, 2, 256, 5)])
def test_infinite_scores(hq, hkv, d, rows, splits):
    """States whose scores are minus infinity weigh nothing, whole splits of them included; where all are, the softmax
    is 0 / 0 and the log-sum-exp minus infinity; one score of plus infinity makes its rows NaN."""
    c = Case([rows, rows, rows], [300, 200, 130], hq, hkv, d, force_splits=splits, seed=30)
    c.q.abs_().add_(0.5)
    c.q[sum(c.rows):] = float("nan")
    s0, s1, s2 = c.starts
    c.k[s0:s0 + 170] = -math.inf
    c.k[s1:s1 + 200] = -math.inf
    c.k[s2 + 77] = math.inf
    c.run()
    lse = c.lse[rows:2 * rows]
    assert bool((lse == -math.inf).all()) and bool(c.o[rows:2 * rows].isnan().all())
    assert bool(c.o[2 * rows:3 * rows].isnan().all())
    k, v = (t[s0 + 170:s0 + 300].double().cpu().repeat_interleave(hq // hkv, 1) for t in (c.k, c.v))
    x = torch.einsum("whd,shd->hws", c.q[:rows].double().cpu(), k) * c.sm_scale
    want = torch.einsum("hws,shd->whd", torch.softmax(x, -1), v)
    A = torch.einsum("hws,shd->whd", torch.softmax(x, -1), v.abs())
    e = (2.0 ** -20 * (8 + x.abs().amax(-1))).t()
    E = 2.0 ** -18 * torch.einsum("whd,shd->hws", c.q[:rows].double().cpu(), k.abs()).amax(-1).t() * c.sm_scale
    tol = 2.0 ** -8 * (1 + 2.0 ** -6) * (want.abs() + A) + 2 * (e + E)[..., None] * A
    assert bool(((c.o[:rows].double().cpu() - want).abs() <= tol).all())
    assert bool(((c.lse[:rows].double().cpu() - torch.logsumexp(x, -1).t()).abs() <= e + E).all())
    assert sa.spec_attn_check_device_status(c.ws) == 0


@pytest.mark.parametrize("splits", [1, 2, 3, 8])
@pytest.mark.parametrize("hq,hkv,d,rows", [(8, 2, 64, 9), (8, 2, 128, 40), (8, 2, 128, 400), (6, 2, 256, 5)])
def test_log_sum_exp_of_infinite_scores(hq, hkv, d, rows, splits):
    """ln sum exp as torch.logsumexp has it: one score of plus infinity, in the first tile or a later one, beside minus
    infinities or not, gives plus infinity; a NaN score anywhere gives NaN.  O is NaN in all of them."""
    c = Case([rows] * 5, [520] * 5, hq, hkv, d, force_splits=splits, seed=31)
    c.q.abs_().add_(0.5)
    c.q[sum(c.rows):] = float("nan")
    first, late, both, nan_after, nan_alone = c.starts
    c.k[first + 3] = math.inf
    c.k[late + 400] = math.inf
    c.k[both:both + 300] = -math.inf
    c.k[both + 301] = math.inf
    c.k[both + 519] = math.inf
    c.k[nan_after + 60] = math.inf
    c.k[nan_after + 450] = math.nan
    c.k[nan_alone + 77] = math.nan
    c.run()
    torch.cuda.synchronize()
    assert sa.spec_attn_check_device_status(c.ws) == 0
    n = 3 * rows
    assert bool((c.lse[:n] == math.inf).all()) and bool(c.lse[n:5 * rows].isnan().all())
    assert bool(c.o[:5 * rows].isnan().all())


@pytest.mark.parametrize("splits", [1, 2, 3, 5, 6, 7, 8])
@pytest.mark.parametrize("hq,hkv,d,rows", [(8, 2, 64, 9), (8, 2, 128, 40), (6, 2, 256, 5)])
def test_infinite_values(hq, hkv, d, rows, splits):
    """An infinite element of one state makes that element of its rows infinite, by the formula, and leaves the others
    as they are, whichever split the state falls to and whichever CTA combines the row."""
    c = Case([rows, rows], [600, 600], hq, hkv, d, force_splits=splits, seed=32)
    clean = c.v.clone()
    c.run()
    want = c.o.clone(), c.lse.clone()
    for at in (5, 200, 333, 480, 599):
        c.v.copy_(clean)
        c.v[c.starts[0] + at, 1, 0::3] = math.inf
        c.v[c.starts[0] + at, 1, 1::3] = -math.inf
        c.o.fill_(MARK), c.lse.fill_(MARK)
        c.run()
        heads = slice(hq // 2, hq)
        assert bool((c.o[:rows, heads, 0::3] == math.inf).all()), at
        assert bool((c.o[:rows, heads, 1::3] == -math.inf).all()), at
        c.o[:rows, heads, 0::3], c.o[:rows, heads, 1::3] = want[0][:rows, heads, 0::3], want[0][:rows, heads, 1::3]
        assert torch.equal(c.o, want[0]) and torch.equal(c.lse, want[1]), at
    assert sa.spec_attn_check_device_status(c.ws) == 0


def test_shared_and_overlapping_ranges():
    c = Case([4, 4, 30], [300, 300, 200], 8, 2, 128, starts=[5, 5, 100], seed=3)
    c.run()
    c.check()


def test_no_states_at_all():
    c = Case([3, 2], [0, 0], 8, 2, 64, starts=[0, 0], gap=0, seed=4)
    assert c.k.shape[0] == 0
    c.run()
    c.check()


def test_plan_bounds_above_the_batch():
    """max_q_rows and max_kv_len above every request's: the grid has CTAs without work."""
    c = Case([5, 1], [77, 500], 24, 4, 256, max_q=100, max_kv=5000, seed=5)
    c.run()
    c.check()
    c = Case([5, 1], [77, 500], 32, 8, 128, max_q=500, max_kv=9000, seed=5)
    c.run()
    c.check()


@pytest.mark.parametrize("hq,hkv,d", [(24, 4, 256), (32, 8, 128), (8, 8, 64)])
def test_bounds_that_bound_nothing(hq, hkv, d):
    """The largest bounds there are: the rows themselves size the launch."""
    c = Case([5, 1], [77, 500], hq, hkv, d, max_q=2 ** 31 - 1, max_kv=2 ** 31 - 1, seed=5)
    c.run()
    c.check()


def test_two_calls_at_once():
    """One plan from two threads on two streams, each with its buffers and workspace."""
    cases = [Case([9, 200], [300, 900], 8, 2, 128, seed=s) for s in (20, 21)]
    cases[1].plan = cases[0].plan
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()

    def loop(c, s):
        for _ in range(50):
            c.run(stream=s)
    threads = [threading.Thread(target=loop, args=a) for a in zip(cases, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for c in cases:
        c.check()


def test_random_batches():
    rng = random.Random(9)
    for seed in range(12):
        hq, hkv, d = rng.choice(HEADS)
        P = rng.randint(1, 6)
        rows = [rng.choice((0, 1, rng.randint(1, 16), rng.randint(1, 300))) for _ in range(P)]
        lens = [rng.choice((0, 1, rng.randint(1, 200), rng.randint(1, 1500))) for _ in range(P)]
        c = Case(rows, lens, hq, hkv, d, fused=rng.random() < 0.5, force_splits=rng.choice((0, 0, 2, 5)), seed=seed)
        c.run()
        c.check()


@pytest.mark.parametrize("hq,hkv,d,P,rows", [(6, 1, 256, 190, 1), (4, 2, 128, 250, 3), (8, 1, 64, 256, 2), (3, 3, 64, 257, 1),
                                              (16, 1, 128, 160, 9)])
def test_more_ctas_than_the_gpu_holds(hq, hkv, d, P, rows):
    """Uneven lengths, equal ones and empty ones among them: the CTAs run in order of length, the rows stay in place."""
    rng = random.Random(P)
    lens = [rng.choice((0, 1, 64, 64, 100, rng.randint(1, 400))) for _ in range(P)]
    c = Case([rng.choice((0, rows, rows)) for _ in range(P)], lens, hq, hkv, d, seed=P, max_q=rows)
    c.run()
    c.check()


@pytest.mark.parametrize("field,value,bits", [
    ("kv_len", -1, sa.SPEC_ATTN_DEV_BAD_SEQ_LEN), ("kv_len", 201, sa.SPEC_ATTN_DEV_BAD_SEQ_LEN),
    ("kv_start", -1, sa.SPEC_ATTN_DEV_BAD_SEQ_LEN), ("kv_start", 2 ** 31 - 1, sa.SPEC_ATTN_DEV_BAD_SEQ_LEN),
])
def test_a_bad_range_skips_its_request(field, value, bits):
    c = Case([4, 5, 6], [100, 200, 150], 8, 2, 64, force_splits=2, seed=6)
    getattr(c, field)[1] = value
    c.run()
    assert sa.spec_attn_check_device_status(c.ws) == bits
    c.check(skip=(1,))


def test_bad_windows_skip_their_requests():
    c = Case([4, 5, 6], [100, 200, 150], 8, 2, 64, seed=6)
    c.indptr[2] = 3               # request 1: -1 rows; request 2: 12 rows, more than the plan's 6
    c.run()
    assert sa.spec_attn_check_device_status(c.ws) == sa.SPEC_ATTN_DEV_BAD_WINDOW
    c.check(skip=(1, 2))


def test_graph_replay_other_stream_and_no_lse():
    c = Case([9, 300], [700, 1500], 32, 8, 128, fused=True, seed=8)
    c.run()
    want = c.o.clone(), c.lse.clone()
    c.o.fill_(MARK), c.lse.fill_(MARK)
    torch.cuda.synchronize()
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        c.run(stream=s)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(c.o, want[0]) and torch.equal(c.lse, want[1])
    c.check()
    c.o.fill_(MARK)
    sa.spec_attn_run_cross(c.plan, c.q, c.k, c.v, c.indptr, c.kv_start, c.kv_len, c.o, None, c.ws)
    assert torch.equal(c.o, want[0])


def test_a_plan_follows_its_buffers():
    """One plan on two sets of buffers in turn."""
    a, b = (Case([9], [200], 8, 2, 64, seed=s) for s in (10, 11))
    b.plan = a.plan
    for c in (a, b, a, b):
        c.o.fill_(MARK), c.lse.fill_(MARK)
        c.run()
        c.check()


def test_states_past_32_bits():
    """K and V rows 16 KB apart in one allocation of over 4 GiB, the range at its end."""
    d, hkv, hq, stride = 128, 2, 8, 8192
    total = 2 ** 32 // (2 * stride) + 300
    big = torch.zeros(total * stride, dtype=torch.bfloat16, device="cuda")
    view = big.view(total, stride)
    c = Case([5], [250], hq, hkv, d, starts=[0], gap=0, seed=12)
    k, v = (view[:, i * hkv * d:(i + 1) * hkv * d].unflatten(1, (hkv, d)) for i in (0, 1))
    k[total - 250:], v[total - 250:] = c.k, c.v
    plan = sa.spec_attn_cross_plan_create(num_reqs=1, total_q_rows=7, max_q_rows=5, num_q_heads=hq, num_kv_heads=hkv,
                                          head_dim=d, total_kv_rows=total, max_kv_len=250, kv_row_stride=stride)
    ws = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    sa.spec_attn_run_cross(plan, c.q, k, v, c.indptr, c.kv_start + (total - 250), c.kv_len, c.o, c.lse, ws)
    assert sa.spec_attn_check_device_status(ws) == 0
    c.check()


def test_refused_calls_write_nothing():
    c = Case([4], [100], 8, 2, 64, force_splits=1, seed=13)
    for bad in (dict(q=c.q.float()), dict(k=c.k[:, :1]), dict(kv_len=c.kv_len.long()), dict(indptr=c.indptr[:1]),
                dict(v=c.v.cpu()), dict(o=c.o[:3])):
        a = {**dict(q=c.q, k=c.k, v=c.v, indptr=c.indptr, kv_start=c.kv_start, kv_len=c.kv_len, o=c.o), **bad}
        with pytest.raises(ValueError):
            sa.spec_attn_run_cross(c.plan, *[a[n] for n in ("q", "k", "v", "indptr", "kv_start", "kv_len", "o")], c.lse,
                                   c.ws)
    with pytest.raises(sa.SpecAttnError) as e:
        sa.spec_attn_run_cross(c.plan, c.q, c.k, c.v, c.indptr, c.kv_start, c.kv_len, c.o, c.lse, c.ws[:128])
    assert e.value.status == sa.SPEC_ATTN_E_WORKSPACE_TOO_SMALL
    torch.cuda.synchronize()
    assert bool((c.o == MARK).all())


def test_overlapping_buffers_are_refused():
    """An output that shares bytes with an input or another output; rows beside the states in one buffer are apart."""
    hq, hkv, d, n, S = 4, 2, 64, 6, 100
    c = Case([n], [S], hq, hkv, d, starts=[0], gap=0, pad_rows=0, seed=14)
    c.run()
    want = c.o.clone(), c.lse.clone()
    buf = torch.full((S, 8, hkv, d), 5.0, dtype=torch.bfloat16, device="cuda")
    kv = buf[:, 2:4]
    k, v = kv[:, 0], kv[:, 1]
    k.copy_(c.k), v.copy_(c.v)
    before = buf.clone()
    plan = sa.spec_attn_cross_plan_create(num_reqs=1, total_q_rows=n, max_q_rows=n, num_q_heads=hq, num_kv_heads=hkv,
                                          head_dim=d, total_kv_rows=S, max_kv_len=S, kv_row_stride=8 * hkv * d)
    names = ("q", "k", "v", "indptr", "kv_start", "kv_len", "o", "lse", "ws")

    def run(**over):
        a = {**{x: getattr(c, x) for x in names}, **dict(k=k, v=v), **over}
        sa.spec_attn_run_cross(plan, *[a[x] for x in names])

    flat = buf.view(-1)
    rows = lambda at: flat[at:at + n * hq * d].view(n, hq, d)  # noqa: E731
    both = torch.zeros(n * hq * d + 16, dtype=torch.bfloat16, device="cuda")
    for over in (dict(o=rows(0)), dict(o=c.q), dict(q=both[8:8 + n * hq * d].view(n, hq, d), o=both[:-16].view(n, hq, d)),
                 dict(lse=flat[:2 * n * hq].view(torch.float32).view(n, hq), o=rows(0)),
                 dict(lse=c.q.view(torch.float32).flatten()[:n * hq].view(n, hq)),
                 dict(ws=c.o.view(torch.uint8).flatten()[:256]), dict(kv_len=c.lse.view(torch.int32).flatten()[:1])):
        with pytest.raises(sa.SpecAttnError) as e:
            run(**over)
        assert e.value.status == sa.SPEC_ATTN_E_INVALID_ARG
    torch.cuda.synchronize()
    assert torch.equal(buf, before)
    gap = flat[4 * hkv * d:8 * hkv * d]                  # 512 elements behind the first state: two query rows' worth
    assert gap.numel() == 2 * hq * d
    two = sa.spec_attn_cross_plan_create(num_reqs=1, total_q_rows=2, max_q_rows=n, num_q_heads=hq, num_kv_heads=hkv,
                                         head_dim=d, total_kv_rows=S, max_kv_len=S, kv_row_stride=8 * hkv * d)
    o, lse = gap.view(2, hq, d), torch.zeros(2, hq, device="cuda")
    indptr = torch.tensor([0, 2], dtype=torch.int32, device="cuda")
    sa.spec_attn_run_cross(two, c.q[:2], k, v, indptr, c.kv_start, c.kv_len, o, lse, c.ws)
    assert torch.equal(o, want[0][:2]) and torch.equal(lse, want[1][:2])
    before[0, 4:8] = buf[0, 4:8]
    assert torch.equal(buf, before)
