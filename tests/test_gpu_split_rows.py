"""Rows of splits that wait in 16 bits, with values below the smallest normal number and with streams of keys that cancel.

A split's row is held as fp16 of a scale that is its largest element, but not below 2^-126 (under masks) or 2^-124 over its
sum of weights (the draft's windows).  A row whose values are all below 2^-126 may also be taken as zeros by the products:
such results are compared to 2^-126."""
import math

import pytest
import torch

import speculative_decode_verify_paged_gb300 as sa
from test_gpu_masked import Case

pytestmark = pytest.mark.gpu
TINY = 2.0 ** -126


@pytest.fixture(scope="module", autouse=True)
def _built():
    from speculative_decode_verify_paged_gb300 import build as libbuild
    libbuild.build()
    torch.cuda.set_device(0)


def make_tiny(c, keys):
    """V of the first ``keys`` keys of every request below 2^-126, every other element exactly 0."""
    for r, slots in enumerate(c.slots):
        for j, s in enumerate(slots[:keys]):
            at = (s // c.ps, slice(None), s % c.ps)
            c.pools[1][at] = (c.pools[1][at].double() * 2.0 ** -130).bfloat16()
            c.pools[1][at][..., ::2] = 0


def attention(c):
    """[rows, Hq, d] in 64 bits."""
    G, out, at = c.hq // c.hkv, [], 0
    for r, w in enumerate(c.rows):
        k, v = (c.values(r, i).repeat_interleave(G, 1) for i in (0, 1))
        x = torch.einsum("whd,shd->hws", c.q[at:at + w].double(), k) * c.sm_scale
        out.append(torch.einsum("hws,shd->whd", torch.softmax(x.masked_fill(~c.seen(r), -math.inf), -1), v))
        at += w
    return torch.cat(out)


@pytest.mark.parametrize("splits", [1, 3, 9, 12, 17])
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 64), (32, 8, 128), (6, 2, 256)])
def test_values_below_the_normal_range_under_masks(hq, hkv, d, splits):
    c = Case([3, 9], [1200, 1400], hq, hkv, d, tree=True, force_splits=splits, seed=splits)
    make_tiny(c, 1409)
    c.run()
    assert float((c.o[:12].double() - attention(c)).abs().max()) <= TINY
    # the first keys only: their splits' rows are joined with others of ordinary size
    c = Case([3, 9], [1200, 1400], hq, hkv, d, tree=True, force_splits=splits, seed=splits)
    make_tiny(c, 700)
    c.run()
    c.check()


@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 64), (32, 8, 128), (6, 2, 256)])
def test_one_smallest_normal_element_among_zeros(hq, hkv, d):
    """Eight keys of equal weight, one element of 2^-126 among them: the row's largest is 2^-129."""
    c = Case([1], [64 * 17 - 1], hq, hkv, d, force_splits=17, seed=2)
    c.q[:1] = 0
    for j, s in enumerate(c.slots[0][:64]):
        c.pools[1][s // c.ps, :, s % c.ps] = 0
    s = c.slots[0][5]
    c.pools[1][s // c.ps, :, s % c.ps, 3] = TINY
    c.run()
    c.check()


@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 64), (32, 8, 128)])
def test_streams_of_keys_that_cancel(hq, hkv, d):
    """Nine splits of two tiles of 64 keys, of equal weights: the first tile's values are 4096 sixty-three times, the
    second's -4096, and one key of the first is s = 1 + e / 64.  All sums are exact in 32 bits, so that a split's row is
    s / 128, off by at most 2^-12 of its largest element, below 2 / 128, and the result rounded once."""
    c = Case([1], [9 * 128 - 1], hq, hkv, d, force_splits=9, seed=3)
    c.q[:1] = 0
    e = 1 + (torch.arange(d, device="cuda") % 64) / 64
    for j, s in enumerate(c.slots[0]):
        big = 4096.0 if j % 128 < 64 else -4096.0
        c.pools[1][s // c.ps, :, s % c.ps] = (e if j % 128 == 63 else e * 0 if j % 128 == 127 else e * 0 + big).bfloat16()
    c.run()
    want = (e.double() / 128).expand(hq, d)
    assert bool(((c.o[0].double() - want).abs() <= 2.0 ** -8 * want + (2.0 ** -12 + 2.0 ** -20) * 2 / 128).all())
    assert float((c.lse[0].double() - math.log(9 * 128)).abs().max()) <= 1e-5


@pytest.mark.parametrize("kv", ["bf16", "nvfp4"])
@pytest.mark.parametrize("mode", ["cuda_core", "tcgen05", "w_invariant"])
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 64), (32, 8, 128), (6, 2, 256)])
def test_values_below_the_normal_range_in_windows(hq, hkv, d, mode, kv):
    """The same for the draft's windows, split by either kernel; a 4-bit cache by its global scale."""
    for keys in (1409, 700):
        if kv == "nvfp4" and keys == 700:
            continue
        c = Case([3, 9], [1200, 1400], hq, hkv, d, kv=kv, seed=5)
        if kv == "bf16":
            make_tiny(c, keys)
        else:
            c.gscale = (0.3, 2.0 ** -140)
        over = dict(w_invariant=1, fixed_keys_per_split=128) if mode == "w_invariant" else dict(
            force_splits=11, kernel_variant=sa.SPEC_ATTN_VARIANT_TCGEN05 if mode == "tcgen05" else
            sa.SPEC_ATTN_VARIANT_CUDA_CORE)
        plan = sa.spec_attn_plan_create(
            num_reqs=2, total_q_rows=c.q.shape[0], max_w=9, num_q_heads=hq, num_kv_heads=hkv, head_dim=d,
            num_pages=c.pages, block_table_stride=c.table.shape[1], max_seq_len=1409, kv_dtype=int(kv == "nvfp4"), **over)
        assert plan.info["max_splits"] > 1
        ws = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
        sa.spec_attn_run(plan, c.q, *c.pools, c.table, c.seq, c.indptr, c.o, c.lse, ws, *c.scales, *c.gscale)
        assert sa.spec_attn_check_device_status(ws) == 0
        tol = TINY if keys == 1409 else 2.0 ** -6 * float(c.pools[1].nan_to_num(0).abs().max())
        assert float((c.o[:12].double() - attention(c)).abs().max()) <= tol
