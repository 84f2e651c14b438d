"""Rows of splits that wait in 16 bits, with values below the smallest normal number.

A split's row is held as fp16 of a scale that is its largest element, at least 2^-126.  A row whose values are all below
that may also be taken as zeros by the products: such results are compared to 2^-126."""
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
