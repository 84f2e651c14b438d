"""Calls of the attention under masks at the edges of its documentation: tables that end with the last request's last page,
scales whose product leaves the range of fp32."""
import pytest
import torch

import speculative_decode_verify_paged_gb300 as sa
from test_gpu_masked import MARK, Case, KV

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from speculative_decode_verify_paged_gb300 import build as libbuild
    libbuild.build()
    torch.cuda.set_device(0)


def call(c, table):
    """The C call, with a table of its own."""
    at = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    status = sa.load_library().spec_attn_run_masked(
        c.plan.handle, at(c.q), at(c.pools[0]), at(c.pools[1]), at(c.scales[0]), at(c.scales[1]), *c.gscale, at(table),
        at(c.seq), at(c.indptr), at(c.mask), at(c.pos), at(c.o), at(c.lse), at(c.ws), c.ws.numel(),
        torch.cuda.current_stream().cuda_stream)
    assert status == sa.SPEC_ATTN_OK


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 3)])
@pytest.mark.parametrize("splits", [0, 2, 12])
def test_a_table_that_ends_with_the_last_page(kv, window, sinks, splits):
    """Entries past a request's pages are never read: the last row of the table holds no more than its pages."""
    for lens in ([900, 20], [20, 900], [5]):
        rows = [min(4, n) for n in lens]
        c = Case(rows, [n - w for n, w in zip(lens, rows)], 8, 2, 64, tree=True, kv=kv, window=window, sinks=sinks,
                 force_splits=splits, seed=3)
        P, stride = c.table.shape
        stride2 = 200                                      # (rows far longer than any request)
        c.plan = sa.spec_attn_masked_plan_create(
            num_reqs=P, total_q_rows=c.q.shape[0], max_w=max(rows), num_q_heads=8, num_kv_heads=2, head_dim=64,
            num_pages=c.pages, block_table_stride=stride2, max_seq_len=max(lens), kv_dtype=int(kv == "nvfp4"), tree=1,
            window_left=window, sink_keys=sinks, force_splits=splits)
        c.ws = torch.zeros(c.plan.workspace_bytes, dtype=torch.uint8, device="cuda")
        table = torch.full((P, stride2), -1, dtype=torch.int32, device="cuda")
        table[:, :stride] = c.table
        used = (P - 1) * stride2 + -(-lens[-1] // 16)
        call(c, table.flatten()[:used].clone())
        c.check()


@pytest.mark.parametrize("kv,sm_scale,k_gscale", [
    ("nvfp4", 0.05, 2.0 ** -149), ("nvfp4", 2.0 ** -100, 2.0 ** -60), ("bf16", 2.0 ** 128 - 2.0 ** 104, 1.0),
    ("nvfp4", 2.0 ** 100, 2.0 ** 60)])
def test_scales_whose_product_is_zero_or_infinite_are_refused(kv, sm_scale, k_gscale):
    c = Case([4], [100], 8, 2, 64, tree=True, kv=kv, sm_scale=sm_scale, seed=13)
    c.gscale = (k_gscale, 1.0)
    with pytest.raises(sa.SpecAttnError) as e:
        c.run()
    assert e.value.status == sa.SPEC_ATTN_E_INVALID_ARG
    torch.cuda.synchronize()
    assert bool((c.o == MARK).all())
