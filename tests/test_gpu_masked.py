"""Attention over the paged cache under tree masks and under windows with sinks, against its formula in 64 bits.

Tolerance, from the arithmetic, for a row with A = sum_j softmax_j |v_j| over the keys it sees and scores x_j.  A score is
a sum of exact products taken in fp32 (d <= 256: at most 32 additions' worth), so it is off by at most E = 2^-18 max_j
sum_e |q_e k_je| sm_scale; over a 4-bit cache q is held in fp16, which moves elements below 2^-14 by up to 2^-25: F = 2^-25
max_j sum_e |k_je| sm_scale more.  The exponent's argument is rounded once (2^-24 |x|), the exponential is good to 2^-21
and the sums to 2^-18 of themselves: a weight is off by at most e = E + F + 2^-20 (8 + max |x|) of itself, and the
log-sum-exp by e.  Rounding the weights to 16 bits for the second product moves O by at most 2^-8 A (fp16 weights below
2^-14 of the running maximum's: by 2^-25 sum |v_j|), a split's partial result held in 16 bits of its row's largest element
by 2^-12 max |v_j|, rounding O itself by 2^-8 |O|:
  |got - want| <= 2^-8 (1 + 2^-6) (|O| + A) + 2 e A + 2^-12 max |v| + 2^-25 sum |v|."""
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
MAGNITUDES = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)


def random_tree(rng, w):
    """Parents of w nodes in any order that has parents first, a second root now and then."""
    return [-1 if i == 0 or rng.random() < 0.03 else rng.randint(max(0, i - rng.choice((1, 3, 20))), i - 1)
            for i in range(w)]


class Case:
    def __init__(self, rows, ctx, hq, hkv, d, tree=False, window=0, sinks=0, kv="bf16", ps=16, interleave=False,
                 force_splits=0, seed=0, pad_rows=2, grow=False, sm_scale=0.0, max_w=None, max_len=None, extra_words=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rng = random.Random(seed)
        self.rows, self.ctx, self.hq, self.hkv, self.d, self.kv = rows, ctx, hq, hkv, d, kv
        self.tree, self.window, self.sinks, self.ps = tree, window, sinks, ps
        P, n = len(rows), sum(rows) + pad_rows
        lens = [c + w for c, w in zip(ctx, rows)]
        self.lens = lens
        # keys that a row may see; the pages that hold none of them are not mapped
        self.live = [[j < sinks or j >= c - window + 1 for j in range(m)] if window else [True] * m
                     for c, m in zip(ctx, lens)]
        stride = max([-(-m // ps) for m in lens] + [1]) + 1
        want = [[p for p in range(-(-m // ps)) if any(live[p * ps:(p + 1) * ps])] for m, live in zip(lens, self.live)]
        total = sum(len(x) for x in want)
        self.pages = total + 3
        perm = list(range(self.pages))
        rng.shuffle(perm)
        table = torch.full((P, stride), 2 ** 30, dtype=torch.int32)
        at = 0
        self.slots = []                     # slot of every live key
        for r, ps_r in enumerate(want):
            for p in ps_r:
                table[r, p] = perm[at]
                at += 1
            self.slots.append([int(table[r, j // ps]) * ps + j % ps if ok else -1 for j, ok in enumerate(self.live[r])])
        self.table = table.cuda()
        self.mag = MAGNITUDES.cuda()
        used = torch.zeros(self.pages * ps, dtype=torch.bool, device="cuda")
        used[torch.tensor([s for x in self.slots for s in x if s >= 0], dtype=torch.int64, device="cuda")] = True
        used = used.view(self.pages, 1, ps, 1)
        self.pools, self.scales, self.dense = [], [None, None], []
        self.gscale = (1.0, 1.0)
        if kv == "bf16":
            both = torch.randn(self.pages, 2, hkv, ps, d, generator=g, device="cuda").bfloat16()
            if grow:      # scores that keep growing along the context
                for r, x in enumerate(self.slots):
                    for j, s in enumerate(x):
                        if s >= 0:
                            both[s // ps, 0, :, s % ps] *= 0.1 + 12 * j / lens[r]
            both = torch.where(used[:, None], both, torch.full((), math.nan, dtype=torch.bfloat16, device="cuda"))
        else:
            self.gscale = (0.3, 0.7)
            both = torch.randint(0, 256, (self.pages, 2, hkv, ps, d // 2), generator=g, device="cuda", dtype=torch.uint8)
            sc = torch.randint(0x30, 0x40, (self.pages, 2, hkv, ps, d // 16), generator=g, device="cuda", dtype=torch.uint8)
            sc = torch.where(used[:, None], sc, torch.full((), 0x7F, dtype=torch.uint8, device="cuda"))   # NaN
            self.scales = [sc[:, 0], sc[:, 1]] if interleave else [sc[:, 0].contiguous(), sc[:, 1].contiguous()]
        self.pools = [both[:, 0], both[:, 1]] if interleave else [both[:, 0].contiguous(), both[:, 1].contiguous()]
        self.q = torch.randn(n, hq, d, generator=g, device="cuda").bfloat16()
        self.q[sum(rows):] = math.nan
        i32 = dict(dtype=torch.int32, device="cuda")
        self.indptr = torch.tensor([sum(rows[:i]) for i in range(P + 1)], **i32)
        self.seq = torch.tensor(lens, **i32)
        self.mask = self.pos = None
        words = -(-(max_w or max(rows + [1])) // 32) + extra_words
        if tree:
            self.parents = [random_tree(rng, w) for w in rows]
            self.sees, depths = [], []
            for t in self.parents:
                sets, depth = [], []
                for i, p in enumerate(t):
                    sets.append((sets[p] if p >= 0 else set()) | {i})
                    depth.append(0 if p < 0 else depth[p] + 1)
                self.sees.append(sets)
                depths.append(depth)
            self.depths = depths
            self.words = words
            self.set_masks()
            self.pos = torch.full((n,), -5, **i32)
            self.pos[:sum(rows)] = torch.tensor([c + h for c, t in zip(ctx, depths) for h in t], **i32)
        self.sm_scale = sm_scale or 1 / math.sqrt(d)
        page = both[0].numel() * both.element_size()
        self.plan = sa.spec_attn_masked_plan_create(
            num_reqs=P, total_q_rows=n, max_w=max_w or max(rows + [1]), num_q_heads=hq, num_kv_heads=hkv, head_dim=d,
            num_pages=self.pages, block_table_stride=stride, max_seq_len=max_len or max(lens + [1]),
            kv_dtype=int(kv == "nvfp4"), page_size=ps, sm_scale=sm_scale, tree=int(tree), window_left=window,
            sink_keys=sinks, mask_row_words=words if extra_words else 0, force_splits=force_splits,
            kv_page_stride=page if interleave else 0,
            scale_page_stride=2 * hkv * ps * d // 16 if interleave and kv == "nvfp4" else 0)
        self.o = torch.full((n, hq, d), MARK, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((n, hq), MARK, device="cuda")
        self.ws = torch.full((self.plan.workspace_bytes,), 0xFF, dtype=torch.uint8, device="cuda")   # (NaN partials)
        sa.spec_attn_reset_device_status(self.ws)

    def set_masks(self):
        """Mask words from ``sees``; bits past the window are set, and have to be ignored."""
        n = self.q.shape[0]
        bits = torch.zeros(n, self.words, dtype=torch.int64)
        at = 0
        for w, sets in zip(self.rows, self.sees):
            for s in sets:
                x = sum(1 << j for j in s) | ((1 << 32 * self.words) - (1 << w))
                bits[at] = torch.tensor([x >> 32 * k & 0xffffffff for k in range(self.words)])
                at += 1
        bits = torch.where(bits >= 2 ** 31, bits - 2 ** 32, bits)
        self.mask = bits.to(torch.int32).cuda()

    def run(self, **kw):
        sa.spec_attn_run_masked(self.plan, self.q, *self.pools, self.table, self.seq, self.indptr, self.mask,
                                self.pos if self.tree else None, self.o, self.lse, self.ws, *self.scales, *self.gscale,
                                **kw)

    def values(self, r, which):
        """K or V of request r [keys, Hkv, d] in 64 bits, zeros where no row sees a key."""
        slots = torch.tensor(self.slots[r], dtype=torch.int64, device="cuda")
        s = slots.clamp(min=0)
        x = self.pools[which][s // self.ps, :, s % self.ps]
        if self.kv == "bf16":
            x = x.double()
        else:
            c = torch.stack([x & 15, x >> 4], -1).flatten(-2).long()
            scale = self.scales[which][s // self.ps, :, s % self.ps].contiguous().view(torch.float8_e4m3fn).double()
            x = torch.where(c >= 8, -self.mag[c & 7], self.mag[c & 7]) * scale.repeat_interleave(16, -1)
            x = x * self.gscale[which]
        return torch.where(slots[:, None, None] >= 0, x, torch.zeros_like(x))

    def seen(self, r):
        """[rows, keys] of request r: which keys each row sees."""
        w, c, m, n = self.rows[r], self.ctx[r], self.lens[r], self.window
        j = torch.arange(m)
        out = torch.zeros(w, m, dtype=torch.bool)
        for i in range(w):
            pos = c + (self.depths[r][i] if self.tree else i)
            ok = (j < c) if self.tree else (j <= pos)
            if n:
                ok &= (j > pos - n) | (j < self.sinks)
            out[i] = ok
            if self.tree:
                out[i, [c + k for k in self.sees[r][i]]] = True
        return out.cuda()

    def check(self, skip=(), rows_skipped=()):
        G, at = self.hq // self.hkv, 0
        for r, w in enumerate(self.rows):
            o, lse = self.o[at:at + w].double(), self.lse[at:at + w].double()
            q = self.q[at:at + w].double()
            at += w
            if r in skip:
                assert bool((o == MARK).all()) and bool((lse == MARK).all())
                continue
            if w == 0:
                continue
            k, v = (self.values(r, i).repeat_interleave(G, 1) for i in (0, 1))
            seen = self.seen(r)
            x = torch.einsum("whd,shd->hws", q, k) * self.sm_scale
            x = x.masked_fill(~seen, -math.inf)
            some = seen.any(1)
            p = torch.softmax(x, -1).nan_to_num(0.0)
            want, A = (torch.einsum("hws,shd->whd", p, t) for t in (v, v.abs()))
            of = lambda t: torch.einsum("whd,shd->hws", t, k.abs()).masked_fill(~seen, 0).amax(-1)  # noqa: E731
            E = 2.0 ** -18 * of(q.abs()) * self.sm_scale
            vis = seen.double()
            vmax = torch.stack([(v.abs() * vis[i][:, None, None]).amax(0) for i in range(w)]).amax(-1, keepdim=True)
            extra = 2.0 ** -12 * vmax
            if self.kv == "nvfp4":
                E = E + 2.0 ** -25 * of(torch.ones_like(q)) * self.sm_scale
                extra = extra + 2.0 ** -25 * torch.einsum("ws,shd->whd", vis, v.abs())
            e = (E + 2.0 ** -20 * (8 + x.masked_fill(~seen, 0).abs().amax(-1))).t()                    # [w, h]
            tol = 2.0 ** -8 * (1 + 2.0 ** -6) * (want.abs() + A) + 2 * e[..., None] * A + extra
            bad = ~((o - want).abs() <= tol)
            assert not bad.any(), (r, int(bad.sum()), bad.nonzero()[0].tolist(), float((o - want).abs().max()))
            got, ref = lse[some], torch.logsumexp(x, -1).t()[some]
            assert bool(((got - ref).abs() <= e[some]).all()), float((got - ref).abs().max())
            assert bool((lse[~some] == -math.inf).all()) and o[~some].count_nonzero() == 0
        assert bool((self.o[at:] == MARK).all()) and bool((self.lse[at:] == MARK).all())     # rows of no request
        assert sa.spec_attn_check_device_status(self.ws) == 0


HEADS = [(4, 1, 64), (24, 4, 256), (32, 8, 128), (40, 8, 128), (12, 12, 64), (16, 1, 128), (12, 1, 256), (3, 1, 64)]
KV = ["bf16", "nvfp4"]


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("hq,hkv,d", HEADS)
@pytest.mark.parametrize("rows,ctx", [
    ([1], [0]), ([1, 1, 1], [14, 15, 16]), ([9, 0, 5], [54, 70, 60]), ([64, 33], [0, 129]), ([130, 1, 70], [5, 128, 1000]),
])
def test_trees(hq, hkv, d, rows, ctx, kv):
    c = Case(rows, ctx, hq, hkv, d, tree=True, kv=kv, ps=(16, 32, 64)[len(rows) - 1], seed=hq + len(rows),
             interleave=d == 128)
    c.run()
    c.check()


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("hq,hkv,d", HEADS)
@pytest.mark.parametrize("rows,ctx,window,sinks,ps", [
    ([1], [500], 100, 4, 16), ([1, 1, 1], [14, 300, 1000], 64, 16, 32), ([9, 0, 5], [500, 70, 1200], 33, 70, 16),
    ([16, 3], [0, 129], 1, 1, 64), ([70, 200], [400, 90], 48, 5, 16), ([1, 8], [700, 640], 512, 0, 64),
])
def test_windows_with_sinks(hq, hkv, d, rows, ctx, window, sinks, ps, kv):
    c = Case(rows, ctx, hq, hkv, d, window=window, sinks=sinks, kv=kv, ps=ps, seed=hq + window, interleave=ps == 32)
    c.run()
    c.check()


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("hq,hkv,d", HEADS[:4])
@pytest.mark.parametrize("window,sinks,ps", [(100, 4, 16), (3, 40, 32), (1, 0, 64), (5000, 9, 16)])
def test_trees_with_windows(hq, hkv, d, window, sinks, ps, kv):
    c = Case([40, 1, 75], [300, 64, 0], hq, hkv, d, tree=True, window=window, sinks=sinks, kv=kv, ps=ps, seed=window)
    c.run()
    c.check()


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("hq,hkv,d", HEADS)
def test_chains_without_window(hq, hkv, d, kv):
    """More rows than a query tile holds, than two, and a remainder in the second tile of a pair."""
    wt = 128 // (hq // hkv)
    c = Case([wt + 1, 2 * wt, 3 * wt + 2, 1], [130, 31, 0, 64], hq, hkv, d, kv=kv, seed=d)
    c.run()
    c.check()


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("splits", [2, 3, 7, 30])
@pytest.mark.parametrize("hq,hkv,d", [(4, 1, 64), (24, 4, 256), (32, 8, 128)])
def test_forced_splits(hq, hkv, d, splits, kv):
    c = Case([3, 70, 8], [900, 700, 1], hq, hkv, d, tree=True, force_splits=splits, kv=kv, seed=splits)
    c.run()
    c.check()
    c = Case([3, 70, 8], [900, 1500, 1], hq, hkv, d, window=800, sinks=20, force_splits=splits, kv=kv, seed=splits)
    c.run()
    c.check()


@pytest.mark.parametrize("hq,hkv,d,rows", [(8, 2, 64, 9), (8, 2, 64, 200), (8, 2, 128, 70), (6, 2, 256, 9), (6, 2, 256, 60)])
def test_growing_scores_move_the_reference(hq, hkv, d, rows):
    for tree in (False, True):
        c = Case([rows], [1500], hq, hkv, d, tree=tree, grow=True, sm_scale=0.2, seed=7)
        c.run()
        c.check()


@pytest.mark.parametrize("hq,hkv,d,rows", [(8, 2, 64, 9), (8, 2, 128, 70), (6, 2, 256, 9), (6, 2, 256, 60), (6, 1, 256, 21)])
def test_growing_scores_of_an_nvfp4_cache(hq, hkv, d, rows):
    """K's block scales grow from 2^-4 to 8 along the context."""
    for splits in (0, 1, 2):
        c = Case([rows], [1500], hq, hkv, d, tree=True, kv="nvfp4", sm_scale=0.2, force_splits=splits, seed=17)
        for j, s in enumerate(c.slots[0]):
            c.scales[0][s // c.ps, :, s % c.ps] = 0x18 + 0x38 * j // c.lens[0]
        c.run()
        c.check()


@pytest.mark.parametrize("splits", [0, 1, 3])
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 64), (32, 8, 128), (6, 2, 256)])
def test_rows_that_see_nothing(hq, hkv, d, splits):
    """Empty masks without context (whole requests, and rows between others), and rows that see one other node alone."""
    c = Case([20, 70, 3], [0, 0, 0], hq, hkv, d, tree=True, force_splits=splits, seed=3)
    c.sees[0] = [set() for _ in range(20)]
    for i in range(0, 70, 3):
        c.sees[1][i] = set()
    c.sees[1][4], c.sees[2] = {69}, [{2}, set(), {0, 2}]
    c.set_masks()
    c.run()
    c.check()


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 64), (32, 8, 128), (6, 2, 256)])
def test_keys_that_are_not_numbers_in_masked_places(hq, hkv, d, kv):
    """K of one node is NaN or infinite: the rows that do not see it come out as without, those that do are NaN."""
    c = Case([40], [100], hq, hkv, d, tree=True, kv=kv, seed=21)
    c.run()
    want = c.o.clone(), c.lse.clone()
    for node, value in ((7, math.nan), (13, math.inf)):
        s = c.slots[0][100 + node]
        if kv == "bf16":
            old = c.pools[0][s // 16, :, s % 16].clone()
            c.pools[0][s // 16, :, s % 16] = value
        else:
            old = c.scales[0][s // 16, :, s % 16].clone()
            c.scales[0][s // 16, :, s % 16] = 0x7F
        c.run()
        sees = torch.tensor([node in x for x in c.sees[0]], device="cuda")
        assert bool(sees.any()) and not bool(sees.all())
        assert bool(c.o[:40][sees].isnan().all())
        assert torch.equal(c.o[:40][~sees], want[0][:40][~sees]) and torch.equal(c.lse[:40][~sees], want[1][:40][~sees])
        if kv == "bf16":
            c.pools[0][s // 16, :, s % 16] = old
        else:
            c.scales[0][s // 16, :, s % 16] = old
    assert sa.spec_attn_check_device_status(c.ws) == 0


@pytest.mark.parametrize("splits", [1, 2, 4])
@pytest.mark.parametrize("hq,hkv,d,rows", [(8, 2, 64, 9), (8, 2, 128, 70), (6, 2, 256, 5)])
def test_infinite_scores(hq, hkv, d, rows, splits):
    """Scores of minus infinity weigh nothing, and a row of nothing else is empty; one of plus infinity makes O NaN and the
    log-sum-exp infinite; a NaN score makes both NaN."""
    c = Case([rows] * 3, [300, 200, 400], hq, hkv, d, window=2000, force_splits=splits, seed=30)
    c.q.abs_().add_(0.5)
    k = c.pools[0]

    def put(r, keys, value):
        for j in keys:
            s = c.slots[r][j]
            k[s // c.ps, :, s % c.ps] = value
    put(0, range(300 + rows), -math.inf)
    put(1, [77], math.inf)
    put(2, range(250), -math.inf)
    c.run()
    assert c.o[:rows].count_nonzero() == 0 and bool((c.lse[:rows] == -math.inf).all())
    assert bool(c.o[rows:2 * rows].isnan().all()) and bool((c.lse[rows:2 * rows] == math.inf).all())
    G = hq // hkv
    kk, v = c.values(2, 0)[250:].repeat_interleave(G, 1), c.values(2, 1)[250:].repeat_interleave(G, 1)
    q = c.q[2 * rows:3 * rows].double()
    x = (torch.einsum("whd,shd->hws", q, kk) * c.sm_scale).masked_fill(~c.seen(2)[:, 250:], -math.inf)
    want = torch.einsum("hws,shd->whd", torch.softmax(x, -1), v)
    assert float((c.o[2 * rows:3 * rows].double() - want).abs().max()) <= 2.0 ** -7 * (float(v.abs().max()))
    assert float((c.lse[2 * rows:3 * rows].double() - torch.logsumexp(x, -1).t()).abs().max()) <= 1e-3
    put(1, [150], math.nan)
    c.run()
    assert bool(c.o[rows:2 * rows].isnan().all()) and bool(c.lse[rows:2 * rows].isnan().all())
    assert sa.spec_attn_check_device_status(c.ws) == 0


def test_positions_below_the_context_count_as_its_end():
    c = Case([12], [200], 8, 2, 64, tree=True, window=50, sinks=2, seed=5)
    c.pos[:12] = torch.arange(12, device="cuda", dtype=torch.int32) * 15       # 0 .. 165, all below 200
    c.depths = [[0] * 12]
    c.run()
    c.check()
    c.pos[:12] = 2 ** 31 - 1                                                   # so far ahead that no context key is near
    c.depths = [[2 ** 30] * 12]
    c.run()
    c.check()


def test_plan_bounds_above_the_batch():
    for tree in (False, True):
        c = Case([5, 1], [77, 500], 24, 4, 256, tree=tree, max_w=100, seed=5)
        c.run()
        c.check()
        c = Case([5, 1], [77, 500], 32, 8, 128, tree=tree, max_w=500, extra_words=3, seed=5)
        c.run()
        c.check()
    c = Case([5, 1], [77, 500], 8, 2, 64, max_w=2 ** 31 - 1, max_len=2 ** 31 - 1, window=64, sinks=4, seed=5)
    c.run()
    c.check()


def test_two_calls_at_once():
    """One plan from two threads on two streams, each with its buffers and workspace."""
    cases = [Case([9, 200], [300, 900], 8, 2, 128, tree=True, seed=20) for _ in range(2)]
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


@pytest.mark.parametrize("seed", range(16))
def test_random_batches(seed):
    rng = random.Random(100 + seed)
    hq, hkv, d = rng.choice(HEADS)
    P = rng.randint(1, 6)
    rows = [rng.choice((0, 1, rng.randint(1, 16), rng.randint(1, 300))) for _ in range(P)]
    ctx = [rng.choice((0, 1, rng.randint(1, 200), rng.randint(1, 1500))) for _ in range(P)]
    window = rng.choice((0, 0, rng.randint(1, 70), rng.randint(1, 900)))
    c = Case(rows, ctx, hq, hkv, d, tree=rng.random() < 0.5, window=window, sinks=rng.choice((0, 4, rng.randint(0, 150))),
             kv=rng.choice(KV), ps=rng.choice((16, 32, 64)), interleave=rng.random() < 0.3,
             force_splits=rng.choice((0, 0, 2, 5)), seed=seed)
    c.run()
    c.check()


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("hq,hkv,d,P,rows", [(6, 1, 256, 190, 1), (4, 2, 128, 250, 3), (8, 1, 64, 300, 2), (16, 1, 128, 160, 9)])
def test_more_work_than_the_gpu_holds(hq, hkv, d, P, rows, kv):
    rng = random.Random(P)
    ctx = [rng.choice((0, 1, 64, 64, 100, rng.randint(1, 400))) for _ in range(P)]
    c = Case([rng.choice((0, rows, rows)) for _ in range(P)], ctx, hq, hkv, d, kv=kv, window=120, sinks=4, seed=P,
             max_w=rows)
    c.run()
    c.check()


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("hq,hkv,d,P", [(16, 8, 64, 45), (32, 8, 128, 45), (24, 4, 256, 45), (6, 1, 256, 256)])
def test_requests_of_all_lengths_in_rounds(hq, hkv, d, P, kv):
    """More CTAs than the GPU holds, of spans long enough that the longest requests go first: lengths of every size, equal
    ones, requests without rows or keys."""
    rng = random.Random(P + d)
    rows = [rng.choice((0, 1, 1, 2)) for _ in range(P)]
    for lens in ([rng.choice((0, 1, 63, 64, 100, 700, 700, 1400)) for _ in range(P)], [1000] * P):
        ctx = [1400] + lens[1:]
        c = Case([1] + rows[1:], ctx, hq, hkv, d, tree=True, kv=kv, seed=P)
        c.run()
        c.check()
        c.o.fill_(MARK), c.lse.fill_(MARK)
        c.seq[7] = 2 ** 30                                 # a length that cannot be
        c.run()
        at = sum(c.rows[:7])
        assert bool((c.o[at:at + c.rows[7]] == MARK).all())
        want = sa.SPEC_ATTN_DEV_BAD_SEQ_LEN if c.rows[7] else 0
        assert sa.spec_attn_check_device_status(c.ws) == want
        sa.spec_attn_reset_device_status(c.ws)
        c.seq[7] = c.lens[7]
        c.check(skip=(7,) if c.rows[7] else ())


def test_a_chain_without_a_window_is_the_window_attention():
    """Every window of up to 16 rows: the same numbers as spec_attn_run's, as far as both are rounded."""
    c = Case([9, 16, 1], [500, 33, 700], 32, 8, 128, seed=15)
    c.run()
    plan = sa.spec_attn_plan_create(num_reqs=3, total_q_rows=28, max_w=16, num_q_heads=32, num_kv_heads=8, head_dim=128,
                                    num_pages=c.pages, block_table_stride=c.table.shape[1], max_seq_len=701)
    ws = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    o, lse = torch.zeros_like(c.o), torch.zeros_like(c.lse)
    sa.spec_attn_run(plan, c.q, *c.pools, c.table, c.seq, c.indptr, o, lse, ws)
    assert float((o[:26].float() - c.o[:26].float()).abs().max()) <= 2e-2
    assert float((lse[:26] - c.lse[:26]).abs().max()) <= 1e-4


@pytest.mark.parametrize("page", [-1, 2 ** 31 - 1])
def test_bad_pages_are_reported(page):
    c = Case([4, 5], [100, 200], 8, 2, 64, tree=True, seed=6)
    c.table[1, 2] = page
    c.run()
    assert sa.spec_attn_check_device_status(c.ws) == sa.SPEC_ATTN_DEV_BAD_PAGE
    c.o[4:9], c.lse[4:9] = MARK, MARK
    c.check(skip=(1,))


@pytest.mark.parametrize("value", [4, 2 ** 31 - 1, -7])
def test_bad_lengths_skip_their_request(value):
    c = Case([4, 5, 6], [100, 200, 150], 8, 2, 64, tree=True, force_splits=2, seed=6)
    c.seq[1] = value
    c.run()
    assert sa.spec_attn_check_device_status(c.ws) == sa.SPEC_ATTN_DEV_BAD_SEQ_LEN
    c.check(skip=(1,))


def test_bad_windows_skip_their_requests():
    c = Case([4, 5, 6], [100, 200, 150], 8, 2, 64, seed=6)
    c.indptr[2] = 3               # request 1: -1 rows; request 2: 12 rows, more than the plan's 6
    c.run()
    assert sa.spec_attn_check_device_status(c.ws) == sa.SPEC_ATTN_DEV_BAD_WINDOW
    c.check(skip=(1, 2))


@pytest.mark.parametrize("kv", KV)
def test_graph_replay_other_stream_and_no_lse(kv):
    c = Case([9, 100], [700, 1500], 32, 8, 128, tree=True, kv=kv, window=900, sinks=5, seed=8)
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
    lse, c.lse = c.lse, None
    c.run()
    assert torch.equal(c.o, want[0])


def test_a_graph_follows_lengths_on_the_device():
    """A captured call replayed with shorter contexts: the same pages, fewer keys."""
    c = Case([9, 60], [700, 1500], 32, 8, 128, tree=True, seed=8)
    c.run()
    torch.cuda.synchronize()
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        c.run(stream=s)
    for cut in (300, 399):
        c.seq.sub_(cut)
        c.ctx, c.lens = [x - cut for x in c.ctx], [x - cut for x in c.lens]
        c.slots = [x[:-cut] for x in c.slots]
        c.o.fill_(MARK), c.lse.fill_(MARK)
        graph.replay()
        torch.cuda.synchronize()
        c.check()


def test_a_plan_follows_its_buffers():
    a, b = (Case([9], [200], 8, 2, 64, tree=True, seed=s) for s in (10, 10))
    b.plan = a.plan
    b.q.neg_()
    for c in (a, b, a, b):
        c.o.fill_(MARK), c.lse.fill_(MARK)
        c.run()
        c.check()


@pytest.mark.parametrize("kv", KV)
def test_pools_past_32_bits(kv):
    """Pages in an allocation of over 4 GiB, the request's at its end."""
    c = Case([5], [250], 8, 2, 128, tree=True, kv=kv, window=100, sinks=3, seed=12)
    dense = c.pools[0][0].numel() * c.pools[0].element_size()
    stride = 16 * dense
    pages = 2 ** 32 // stride + 20
    big = torch.zeros(pages * stride, dtype=torch.uint8, device="cuda")
    rows = big.view(pages, stride)
    at = pages - c.pages
    pools = []
    for i, t in enumerate(c.pools):
        v = rows[:, i * dense:(i + 1) * dense]
        v = (v.view(torch.bfloat16) if kv == "bf16" else v).unflatten(1, c.pools[0].shape[1:])
        v[at:] = t
        pools.append(v)
    c.table = torch.where(c.table < 2 ** 30, c.table + at, c.table)
    kw = {}
    if kv == "nvfp4":
        sdense = c.scales[0][0].numel()
        for i in (0, 1):
            s = torch.zeros(pages, *c.scales[0].shape[1:], dtype=torch.uint8, device="cuda")
            s[at:] = c.scales[i]
            c.scales[i] = s
        assert sdense == c.scales[0][0].numel()
    c.plan = sa.spec_attn_masked_plan_create(
        num_reqs=1, total_q_rows=7, max_w=5, num_q_heads=8, num_kv_heads=2, head_dim=128, num_pages=pages,
        block_table_stride=c.table.shape[1], max_seq_len=255, kv_dtype=int(kv == "nvfp4"), tree=1, window_left=100,
        sink_keys=3, kv_page_stride=stride, **kw)
    c.ws = torch.zeros(c.plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    c.pools = pools
    c.slots = [[s + at * 16 if s >= 0 else -1 for s in c.slots[0]]]
    c.run()
    c.check()


def test_refused_calls_write_nothing():
    c = Case([4], [100], 8, 2, 64, tree=True, window=50, seed=13)
    names = ("q", "k", "v", "table", "seq", "indptr", "mask", "pos", "o", "lse", "ws")
    ok = dict(q=c.q, k=c.pools[0], v=c.pools[1], table=c.table, seq=c.seq, indptr=c.indptr, mask=c.mask, pos=c.pos, o=c.o,
              lse=c.lse, ws=c.ws)
    for bad in (dict(q=c.q.float()), dict(k=c.pools[0][:, :1]), dict(seq=c.seq.long()), dict(indptr=c.indptr[:1]),
                dict(v=c.pools[1].cpu()), dict(o=c.o[:3]), dict(mask=c.mask[:3]), dict(pos=c.pos[:2]),
                dict(table=c.table[:, :1]), dict(mask=c.mask.long())):
        with pytest.raises(ValueError):
            sa.spec_attn_run_masked(c.plan, *[{**ok, **bad}[n] for n in names])
    for bad, status in ((dict(ws=c.ws[:128]), sa.SPEC_ATTN_E_WORKSPACE_TOO_SMALL),
                        (dict(mask=None), sa.SPEC_ATTN_E_INVALID_ARG), (dict(pos=None), sa.SPEC_ATTN_E_INVALID_ARG),
                        (dict(o=c.q), sa.SPEC_ATTN_E_INVALID_ARG),
                        (dict(lse=c.q.view(torch.float32).flatten()[:48].view(6, 8)), sa.SPEC_ATTN_E_INVALID_ARG),
                        (dict(o=c.pools[0].flatten()[:6 * 8 * 64].view(6, 8, 64)), sa.SPEC_ATTN_E_INVALID_ARG),
                        (dict(seq=c.o.view(torch.int32).flatten()[:1]), sa.SPEC_ATTN_E_INVALID_ARG),
                        (dict(mask=c.lse.view(torch.int32).flatten()[:6].view(6, 1)), sa.SPEC_ATTN_E_INVALID_ARG)):
        with pytest.raises(sa.SpecAttnError) as e:
            sa.spec_attn_run_masked(c.plan, *[{**ok, **bad}[n] for n in names])
        assert e.value.status == status
    torch.cuda.synchronize()
    assert bool((c.o == MARK).all())


@pytest.mark.parametrize("over,status", [
    (dict(num_reqs=-1), sa.SPEC_ATTN_E_INVALID_ARG), (dict(num_reqs=65536), sa.SPEC_ATTN_E_UNSUPPORTED),
    (dict(tree=2), sa.SPEC_ATTN_E_INVALID_ARG), (dict(head_dim=96), sa.SPEC_ATTN_E_UNSUPPORTED),
])
def test_plans_are_refused_with_their_status(over, status):
    prob = dict(num_reqs=1, total_q_rows=4, max_w=4, num_q_heads=8, num_kv_heads=2, head_dim=64, num_pages=4,
                block_table_stride=4, max_seq_len=60)
    with pytest.raises(sa.SpecAttnError) as e:
        sa.spec_attn_masked_plan_create(**{**prob, **over})
    assert e.value.status == status


@pytest.mark.parametrize("scale", [0.0, -0.3, math.inf, math.nan])
def test_bad_global_scales_are_refused(scale):
    c = Case([4], [100], 8, 2, 64, tree=True, kv="nvfp4", seed=13)
    for scales in ((scale, 0.7), (0.3, scale)):
        c.gscale = scales
        with pytest.raises(sa.SpecAttnError) as e:
            c.run()
        assert e.value.status == sa.SPEC_ATTN_E_INVALID_ARG
    torch.cuda.synchronize()
    assert bool((c.o == MARK).all())


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("hq,hkv,d,rows,ctx", [(32, 8, 128, [64] * 10, 700), (32, 8, 128, [128] * 4, 900), (8, 1, 64, [40] * 170, 90),
                                               (24, 4, 256, [21] * 45, 150), (16, 1, 128, [300, 2, 90, 40] * 6, 400)])
def test_every_shape_of_launch(hq, hkv, d, rows, ctx, kv):
    """Two query tiles a CTA, CTAs that share an SM, more CTAs than fit: the plans that larger batches get."""
    rng = random.Random(d + len(rows))
    c = Case(rows, [rng.randint(ctx // 2, ctx) for _ in rows], hq, hkv, d, tree=True, kv=kv, seed=d)
    c.run()
    c.check()
    c = Case(rows, [rng.randint(ctx // 2, ctx) for _ in rows], hq, hkv, d, window=200, sinks=7, kv=kv, ps=32, seed=d)
    c.run()
    c.check()
