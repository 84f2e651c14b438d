"""Attention under masks in every shape of launch: each case asserts, from its plan, that it takes the kernel it is here for
(query tiles a CTA, CTAs an SM, how splits are joined, the longest requests first) and compares with the formula in 64 bits
as test_gpu_masked.py does.  Then two query tiles a CTA in earnest, which only batches of many rows over long contexts get."""
import math
import random

import pytest
import torch

import speculative_decode_verify_paged_gb300 as sa
from test_gpu_masked import KV, MARK, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from speculative_decode_verify_paged_gb300 import build as libbuild
    libbuild.build()
    torch.cuda.set_device(0)


def takes(c, tiles, ctas, join=None, first=None):
    i = c.plan.info
    assert (i["query_tiles"], i["ctas_per_sm"]) == (tiles, ctas), i
    assert join is None or i["join"] == join, i
    assert first is None or i["longest_first"] == first, i


FEW = ([9, 40], [1500, 700])
MANY = ([9, 1, 0, 5] * 6, [1500, 700, 64, 1] * 6)
PAIRS = ([200, 3, 131, 128, 0], [2000, 0, 17, 640, 100])


@pytest.mark.parametrize("tree", [True, False])
@pytest.mark.parametrize("splits,join", [(1, 0), (3, 1), (12, 2)])
@pytest.mark.parametrize("hq,hkv,d,kv,batch,tiles,ctas", [
    (8, 2, 64, "bf16", FEW, 1, 1), (16, 8, 64, "bf16", MANY, 1, 2), (8, 2, 128, "bf16", FEW, 1, 1),
    (32, 8, 128, "bf16", MANY, 1, 2), (16, 8, 128, "bf16", PAIRS, 2, 1), (6, 2, 256, "bf16", FEW, 1, 1),
    (8, 2, 64, "nvfp4", FEW, 1, 1), (32, 8, 128, "nvfp4", FEW, 1, 1), (6, 2, 256, "nvfp4", FEW, 1, 1)])
def test_every_kernel_with_every_join(hq, hkv, d, kv, batch, tiles, ctas, splits, join, tree):
    c = Case(*batch, hq, hkv, d, tree=tree, kv=kv, force_splits=splits, seed=d + splits)
    takes(c, tiles, ctas, join)
    c.run()
    c.check()


@pytest.mark.parametrize("hq,hkv,d,kv,longest,splits,tiles,ctas,join", [
    (16, 8, 64, "bf16", 1400, 1, 1, 2, 0), (16, 8, 64, "bf16", 9000, 3, 1, 2, 1), (4, 4, 64, "bf16", 46000, 12, 1, 2, 2),
    (32, 8, 128, "bf16", 1400, 1, 1, 2, 0), (24, 4, 256, "bf16", 6000, 3, 1, 1, 1), (16, 8, 64, "nvfp4", 1400, 1, 1, 1, 0),
    (32, 8, 128, "nvfp4", 1400, 1, 1, 1, 0), (24, 4, 256, "nvfp4", 6000, 3, 1, 1, 1)])
def test_the_longest_first_with_every_join(hq, hkv, d, kv, longest, splits, tiles, ctas, join):
    rng = random.Random(longest)
    P = 45
    rows = [rng.choice((0, 1, 1, 3)) for _ in range(P)]
    ctx = [rng.choice((0, 1, 63, 64, 200, 700, 700, 1300)) for _ in range(P)]
    rows[30], ctx[30] = 2, longest
    c = Case(rows, ctx, hq, hkv, d, tree=True, kv=kv, force_splits=splits, seed=P)
    takes(c, tiles, ctas, join, 1)
    c.run()
    c.check()


PAIR_BATCHES = [
    (16, 8, PAIRS),                                                                       # tiles of 64 rows
    (32, 8, ([70, 1, 33, 32, 64, 65, 31, 40], [2000, 64, 0, 1300, 640, 127, 1999, 5])),   # 32
    (16, 1, ([257, 16, 9, 8, 100], [2000, 5, 700, 63, 1000])),                            # 8
    (4, 4, ([257, 128, 129, 1] * 4, [2000, 0, 500, 1500] * 4)),                           # 128
    (40, 8, ([257, 51], [2000, 1111])),                                                   # 25, of 125 pairs
    (12, 4, ([200, 85, 43, 84, 126, 42, 41, 1], [2000, 9, 0, 640, 63, 65, 1000, 129])),   # 42, of 126 pairs
]


@pytest.mark.parametrize("tree", [True, False])
@pytest.mark.parametrize("hq,hkv,batch", PAIR_BATCHES)
def test_two_query_tiles(hq, hkv, batch, tree):
    for ps, seed in ((16, 1), (64, 2)):
        c = Case(*batch, hq, hkv, 128, tree=tree, ps=ps, interleave=ps == 64, seed=seed)
        takes(c, 2, 1)
        c.run()
        c.check()


@pytest.mark.parametrize("hq,hkv,rows,ctx,window,sinks,tree", [
    (16, 8, [1000, 300, 70], [500, 900, 0], 500, 4, True), (32, 8, [1000, 129], [500, 1400], 500, 70, True),
    (32, 8, [2049], [3952], 2048, 4, False), (16, 1, [1000, 8, 500], [500, 1000, 3], 500, 0, True),
    (32, 8, [2049, 100, 1], [3952, 3000, 5000], 2048, 200, False)])
@pytest.mark.parametrize("splits", [0, 2, 12])
def test_two_query_tiles_under_windows(hq, hkv, rows, ctx, window, sinks, tree, splits):
    c = Case(rows, ctx, hq, hkv, 128, tree=tree, window=window, sinks=sinks, ps=32, force_splits=splits, seed=window)
    takes(c, 2, 1)
    c.run()
    c.check()


def test_two_query_tiles_with_scores_that_grow():
    for tree in (True, False):
        c = Case(*PAIRS, 16, 8, 128, tree=tree, grow=True, sm_scale=0.2, seed=7)
        takes(c, 2, 1)
        c.run()
        c.check()


@pytest.mark.parametrize("splits", [1, 2, 12])
def test_two_query_tiles_and_rows_that_see_nothing(splits):
    """Rows of either tile, and whole warps of them, that see nothing; rows that see one other node alone."""
    c = Case([200, 128, 70, 131, 9], [0, 2000, 0, 500, 0], 16, 8, 128, tree=True, force_splits=splits, seed=3)
    takes(c, 2, 1)
    for r, which in ((0, range(0, 200, 3)), (2, range(70)), (4, range(9))):
        for i in which:
            c.sees[r][i] = set()
    c.sees[0][4], c.sees[0][199] = {150}, {0}
    c.set_masks()
    c.run()
    c.check()


@pytest.mark.parametrize("splits", [1, 3, 12])
def test_two_query_tiles_and_keys_that_are_not_numbers(splits):
    c = Case(*PAIRS, 16, 8, 128, tree=True, force_splits=splits, seed=21)
    takes(c, 2, 1)
    c.run()
    want = c.o.clone(), c.lse.clone()
    k = c.pools[0]
    for node, value in ((7, math.nan), (130, math.inf), (65, -math.inf)):
        s = c.slots[0][2000 + node]
        old = k[s // 16, :, s % 16].clone()
        k[s // 16, :, s % 16] = value
        c.run()
        sees = torch.tensor([node in x for x in c.sees[0]], device="cuda")
        assert bool(sees.any()) and not bool(sees.all())
        assert bool(c.o[:200][sees].isnan().all())         # (q has both signs: an infinite key gives infinity - infinity)
        keep = torch.cat([~sees, torch.ones(c.o.shape[0] - 200, dtype=torch.bool, device="cuda")])
        assert torch.equal(c.o[keep], want[0][keep]) and torch.equal(c.lse[keep], want[1][keep])
        k[s // 16, :, s % 16] = old
    assert sa.spec_attn_check_device_status(c.ws) == 0


@pytest.mark.parametrize("splits", [1, 3, 12])
def test_two_query_tiles_and_infinite_scores(splits):
    """-inf in all of a request's keys, +inf in one of another's, NaN beside it."""
    c = Case([200] * 5, [2000, 300, 1000, 5, 700], 16, 8, 128, force_splits=splits, seed=30)
    takes(c, 2, 1)
    c.q.abs_().add_(0.5)

    def put(r, keys, value):
        s = torch.tensor([c.slots[r][j] for j in keys], device="cuda")
        c.pools[0][s // c.ps, :, s % c.ps] = value
    put(2, range(1200), -math.inf)
    put(1, [77], math.inf)
    c.run()
    assert c.o[400:600].count_nonzero() == 0 and bool((c.lse[400:600] == -math.inf).all())
    assert bool(c.o[200:400].isnan().all()) and bool((c.lse[200:400] == math.inf).all())
    put(1, [150], math.nan)
    c.run()
    assert bool(c.o[200:400].isnan().all()) and bool(c.lse[200:400].isnan().all())
    assert bool(c.o[:200].isfinite().all()) and bool(c.o[600:1000].isfinite().all())
    assert sa.spec_attn_check_device_status(c.ws) == 0


def test_two_query_tiles_and_bad_requests():
    for field, bits in (("page", sa.SPEC_ATTN_DEV_BAD_PAGE), ("seq", sa.SPEC_ATTN_DEV_BAD_SEQ_LEN),
                        ("indptr", sa.SPEC_ATTN_DEV_BAD_WINDOW)):
        c = Case(*PAIRS, 16, 8, 128, tree=True, seed=6)
        takes(c, 2, 1)
        if field == "page":
            c.table[2, 3] = -1
        elif field == "seq":
            c.seq[2] = 2 ** 31 - 1
        else:
            c.indptr[3] = 202                              # request 2: -1 rows, request 3: more than the plan's 200
        c.run()
        assert sa.spec_attn_check_device_status(c.ws) == bits
        if field == "page":
            c.o[203:334], c.lse[203:334] = MARK, MARK
        c.check(skip=(2, 3) if field == "indptr" else (2,))


def test_two_query_tiles_replayed_with_other_lengths():
    """A captured call; then shorter contexts, so that CTAs and splits drop out."""
    c = Case(*PAIRS, 16, 8, 128, tree=True, force_splits=3, seed=8)
    takes(c, 2, 1, 1)
    c.run()
    want = c.o.clone()
    torch.cuda.synchronize()
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        c.run(stream=s)
    c.o.fill_(MARK)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(c.o[:462], want[:462])
    for cut in ([900, 0, 17, 600, 3], [1100, 0, 0, 40, 0]):
        c.seq.sub_(torch.tensor(cut, dtype=torch.int32, device="cuda"))
        c.ctx, c.lens = [x - y for x, y in zip(c.ctx, cut)], [x - y for x, y in zip(c.lens, cut)]
        c.slots = [x[:m] for x, m in zip(c.slots, c.lens)]
        c.o.fill_(MARK), c.lse.fill_(MARK)
        graph.replay()
        torch.cuda.synchronize()
        c.check()


@pytest.mark.parametrize("kv", KV)
def test_runs_repeat_themselves(kv):
    """Every shape gives the same bits again."""
    for batch, hq, hkv, d in ((FEW, 8, 2, 64), (MANY, 16, 8, 64), (MANY, 32, 8, 128), (PAIRS, 16, 8, 128), (FEW, 6, 2, 256)):
        for splits in (0, 1, 3, 12):
            c = Case(*batch, hq, hkv, d, tree=True, kv=kv, force_splits=splits, seed=9)
            c.run()
            want = c.o.clone(), c.lse.clone()
            for _ in range(5):
                c.o.fill_(MARK), c.lse.fill_(MARK)
                c.run()
                assert torch.equal(c.o, want[0]) and torch.equal(c.lse, want[1])
