"""Attention under masks with more than 8 splits: the second kernel joins them sixteen at a time, with a running maximum and
sum between.  Requests of exactly 16, 17 and more splits beside requests of one, maxima that move from batch to batch,
batches that hold nothing, infinite and NaN scores in either batch; against the formula in 64 bits, as in
test_gpu_masked.py (whose tolerance counts the 16 bits of a split's row)."""
import math

import pytest
import torch

import speculative_decode_verify_paged_gb300 as sa
from test_gpu_masked import Case, KV

pytestmark = pytest.mark.gpu
SHAPES = [(8, 2, 64), (32, 8, 128), (6, 2, 256)]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from speculative_decode_verify_paged_gb300 import build as libbuild
    libbuild.build()
    torch.cuda.set_device(0)


def joined(c, splits):
    """The plan leaves ``splits`` partial rows a (row, head): (log-sum, largest) and d 16-bit elements each."""
    pairs = splits * c.q.shape[0] * c.hq
    assert splits > 8 and c.plan.workspace_bytes == 256 + -(-pairs * 8 // 256) * 256 + pairs * c.d * 2


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("splits", [9, 16, 17, 33, 40])
@pytest.mark.parametrize("hq,hkv,d", SHAPES)
def test_batches_of_splits(hq, hkv, d, splits, kv):
    """One tile a split; requests that end within, at and one key past every border between batches."""
    most = 64 * splits
    lens = sorted({n for n in (1, 63, 64 * 15 + 1, 64 * 16, 64 * 16 + 1, 64 * 32, 64 * 32 + 7, most - 5) if n < most} | {most})
    rows = [1, 3, 40, 8, 1, 2, 9, 5][:len(lens)]
    for tree in (True, False):
        c = Case([min(w, n) for w, n in zip(rows, lens)], [n - min(w, n) for w, n in zip(rows, lens)], hq, hkv, d, tree=tree,
                 force_splits=splits, kv=kv, seed=splits)
        joined(c, splits)
        c.run()
        c.check()


@pytest.mark.parametrize("splits", [9, 17, 33])
@pytest.mark.parametrize("hq,hkv,d", SHAPES)
def test_maxima_that_move_between_batches(hq, hkv, d, splits):
    """Scores that grow along the context, and the same keys backwards."""
    n = 64 * splits
    for back in (False, True):
        c = Case([5, 20], [n - 5, n - 40], hq, hkv, d, tree=True, grow=True, sm_scale=0.2, force_splits=splits, seed=7)
        if back:
            k = c.pools[0]
            for r, slots in enumerate(c.slots):
                s = torch.tensor(slots, device="cuda")
                old = k[s // c.ps, :, s % c.ps].clone()
                k[s // c.ps, :, s % c.ps] = old.flip(0)
        joined(c, splits)
        c.run()
        c.check()


@pytest.mark.parametrize("splits", [17, 33])
def test_growing_scores_of_an_nvfp4_cache(splits):
    for hq, hkv, d in SHAPES:
        c = Case([5, 20], [64 * splits - 5, 64 * splits - 40], hq, hkv, d, tree=True, kv="nvfp4", sm_scale=0.2,
                 force_splits=splits, seed=17)
        for r, slots in enumerate(c.slots):
            for j, s in enumerate(slots):
                c.scales[0][s // c.ps, :, s % c.ps] = 0x18 + 0x38 * j // c.lens[r]
        joined(c, splits)
        c.run()
        c.check()


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("splits", [9, 17, 33])
@pytest.mark.parametrize("hq,hkv,d", SHAPES)
def test_batches_that_hold_nothing(hq, hkv, d, splits, kv):
    """A tree's rows so far ahead of the window that they see no key of the context but, in the second case, its first:
    every split but the last (and the first) is empty for them.  Other rows see all of it."""
    n = 64 * splits
    for sinks in (0, 3):
        c = Case([12, 3], [n - 12, n - 70], hq, hkv, d, tree=True, window=n, sinks=sinks, force_splits=splits, kv=kv, seed=5)
        for r, at in ((0, 0), (1, 12)):
            for i in range(0, c.rows[r], 2):
                c.pos[at + i] = 2 ** 31 - 1
                c.depths[r][i] = 2 ** 30
        joined(c, splits)
        c.run()
        c.check()


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("splits", [9, 18])
@pytest.mark.parametrize("hq,hkv,d", SHAPES)
def test_rows_that_see_nothing(hq, hkv, d, splits, kv):
    """No context; nodes that see nothing, one node far away, or their ancestors."""
    w = 64 * splits - 30
    c = Case([w, 3], [0, 0], hq, hkv, d, tree=True, force_splits=splits, kv=kv, seed=3)
    for i in range(0, w, 3):
        c.sees[0][i] = set()
    for i in range(1, w, 3):
        c.sees[0][i] = {(i * 7) % w}
    c.sees[1] = [{2}, set(), {0, 2}]
    c.set_masks()
    joined(c, splits)
    c.run()
    c.check()


@pytest.mark.parametrize("splits", [9, 17, 33])
@pytest.mark.parametrize("tree", [True, False])
@pytest.mark.parametrize("hq,hkv,d,rows", [(8, 2, 64, 9), (8, 2, 128, 70), (6, 2, 256, 5)])
def test_infinite_scores(hq, hkv, d, rows, tree, splits):
    """As with few splits: minus infinity weighs nothing, plus infinity makes O NaN and the log-sum-exp infinite, NaN both
    NaN; in the first batch, the last split, and both."""
    n = 64 * splits
    ctx = [n - rows, n - rows - 1, n - rows - 7]
    last = n - rows - 8                                     # (a key of the context, in the last splits)
    gone = 64 * (splits - 3) + 5
    c = Case([rows] * 3, ctx, hq, hkv, d, tree=tree, window=0 if tree else 2 * n, force_splits=splits, seed=30)
    c.q.abs_().add_(0.5)
    k, clean = c.pools[0], c.pools[0].clone()

    def put(r, keys, value):
        s = torch.tensor([c.slots[r][j] for j in keys], device="cuda")
        k[s // c.ps, :, s % c.ps] = value
    G = hq // hkv
    put(0, range(n), -math.inf)
    put(2, range(gone), -math.inf)
    for keys in ([77], [last], [77, last]):
        put(1, keys, math.inf)
        c.run()
        assert c.o[:rows].count_nonzero() == 0 and bool((c.lse[:rows] == -math.inf).all())
        assert bool(c.o[rows:2 * rows].isnan().all()) and bool((c.lse[rows:2 * rows] == math.inf).all())
        kk, v = (c.values(2, i)[gone:].repeat_interleave(G, 1) for i in (0, 1))
        x = torch.einsum("whd,shd->hws", c.q[2 * rows:3 * rows].double(), kk) * c.sm_scale
        x = x.masked_fill(~c.seen(2)[:, gone:], -math.inf)
        want = torch.einsum("hws,shd->whd", torch.softmax(x, -1), v)
        # (weights, a split's row and O rounded: 2^-8, 2^-12 and 2^-8 of the largest value at most)
        assert float((c.o[2 * rows:3 * rows].double() - want).abs().max()) <= 2.0 ** -6 * float(v.abs().max())
        assert float((c.lse[2 * rows:3 * rows].double() - torch.logsumexp(x, -1).t()).abs().max()) <= 1e-3
        for extra in ([150], [last - 3]):
            put(1, extra, math.nan)
            c.run()
            assert bool(c.o[rows:2 * rows].isnan().all()) and bool(c.lse[rows:2 * rows].isnan().all())
            put(1, extra, 1.0)
        s = torch.tensor([c.slots[1][j] for j in keys], device="cuda")
        k[s // c.ps, :, s % c.ps] = clean[s // c.ps, :, s % c.ps]
    assert sa.spec_attn_check_device_status(c.ws) == 0


@pytest.mark.parametrize("splits", [9, 17])
@pytest.mark.parametrize("hq,hkv,d", SHAPES)
def test_nan_scales_of_an_nvfp4_cache(hq, hkv, d, splits):
    n = 64 * splits
    c = Case([6], [n - 6], hq, hkv, d, kv="nvfp4", force_splits=splits, seed=31)
    for j in (3, n - 70):
        s = c.slots[0][j]
        old = c.scales[0][s // c.ps, :, s % c.ps].clone()
        c.scales[0][s // c.ps, :, s % c.ps] = 0x7F
        c.run()
        assert bool(c.o[:6].isnan().all()) and bool(c.lse[:6].isnan().all())
        c.scales[0][s // c.ps, :, s % c.ps] = old
    c.run()
    c.check()


def test_the_join_repeats_itself():
    """Two runs, and a replayed capture, give the same bits."""
    c = Case([9, 60], [64 * 33 - 9, 900], 32, 8, 128, tree=True, force_splits=33, seed=8)
    c.run()
    want = c.o.clone(), c.lse.clone()
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        c.run(stream=s)
    for again in (c.run, graph.replay):
        c.o.fill_(0), c.lse.fill_(0)
        c.ws[256:] = 0xFF
        torch.cuda.synchronize()
        again()
        torch.cuda.synchronize()
        assert torch.equal(c.o[:69], want[0][:69]) and torch.equal(c.lse[:69], want[1][:69])
