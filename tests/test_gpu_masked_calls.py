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


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("hq,hkv,d,rows,ctx", [
    (8, 2, 64, [9, 40], [1500, 700]), (16, 8, 128, [200, 3, 131, 128, 0], [2000, 0, 17, 640, 100]),
    (6, 2, 256, [9, 40], [1500, 700]), (32, 8, 128, [1] * 30, [700] * 30)])
def test_no_lse(hq, hkv, d, rows, ctx, kv):
    for splits in (1, 3, 12):
        c = Case(rows, ctx, hq, hkv, d, tree=True, kv=kv, force_splits=splits, seed=1)
        c.run()
        want = c.o.clone()
        c.o.fill_(MARK)
        c.lse = None
        c.run()
        assert torch.equal(c.o, want) and sa.spec_attn_check_device_status(c.ws) == 0


@pytest.mark.parametrize("tree", [0, 1])
def test_as_many_requests_as_there_may_be(tree):
    """65535 requests of one key each: O is the key's value, LSE its score."""
    P, hq, hkv, d = 65535, 2, 1, 64
    g = torch.Generator(device="cuda").manual_seed(2)
    i32 = dict(dtype=torch.int32, device="cuda")
    q = torch.randn(P, hq, d, generator=g, device="cuda").bfloat16()
    k, v = (torch.randn(P, hkv, 16, d, generator=g, device="cuda").bfloat16() for _ in range(2))
    table = torch.randperm(P, generator=g, device="cuda").int()[:, None].contiguous()
    plan = sa.spec_attn_masked_plan_create(num_reqs=P, total_q_rows=P, max_w=1, num_q_heads=hq, num_kv_heads=hkv, head_dim=d,
                                           num_pages=P, block_table_stride=1, max_seq_len=16, tree=tree)
    o, lse = torch.zeros_like(q), torch.zeros(P, hq, device="cuda")
    ws = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    sa.spec_attn_run_masked(plan, q, k, v, table, torch.ones(P, **i32), torch.arange(P + 1, **i32),
                            torch.ones(P, 1, **i32) if tree else None, None, o, lse, ws)
    assert sa.spec_attn_check_device_status(ws) == 0
    at = table[:, 0].long()
    assert torch.equal(o, v[at, :, 0].expand(P, hq, d))
    want = (q.double() * k[at, :, 0].double()).sum(-1) / 8
    assert float((lse.double() - want).abs().max()) <= 2.0 ** -18 * float((q.double() * k[at, :, 0].double()).abs().sum(-1).max())


@pytest.mark.parametrize("splits", [1, 2, 9])
def test_rows_past_32_bits(splits):
    """A prompt of 2^20 + 40 rows of 16 x 128 under a window of 100 keys and 4 sinks: 4 GiB of q and of O (and with nine
    splits 36 GiB of partial rows); rows from its start, its middle and its end."""
    n, hq, d, window, sinks = 2 ** 20 + 40, 16, 128, 100, 4
    g = torch.Generator(device="cuda").manual_seed(2)
    i32 = dict(dtype=torch.int32, device="cuda")
    pages = -(-n // 64)
    q = torch.empty(n, hq, d, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    k, v = (torch.empty(pages, 1, 64, d, dtype=torch.bfloat16, device="cuda").normal_(generator=g) for _ in range(2))
    table = torch.randperm(pages, generator=g, device="cuda").int()[None].contiguous()
    plan = sa.spec_attn_masked_plan_create(num_reqs=1, total_q_rows=n, max_w=n, num_q_heads=hq, num_kv_heads=1, head_dim=d,
                                           num_pages=pages, block_table_stride=pages, max_seq_len=n, page_size=64,
                                           window_left=window, sink_keys=sinks, force_splits=splits)
    o, lse = torch.zeros_like(q), torch.zeros(n, hq, device="cuda")
    ws = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    sa.spec_attn_run_masked(plan, q, k, v, table, torch.tensor([n], **i32), torch.tensor([0, n], **i32), None, None, o, lse, ws)
    assert sa.spec_attn_check_device_status(ws) == 0
    for row in (0, 3, 99, 100, 104, 2 ** 19 + 7, 2 ** 20 - 1, 2 ** 20, n - 1):
        j = torch.tensor([x for x in range(row + 1) if x > row - window or x < sinks], device="cuda")
        kk, vv = (t[table[0, j // 64].long(), 0, j % 64].double() for t in (k, v))
        x = q[row].double() @ kk.t() / d ** 0.5
        want = torch.softmax(x, 1) @ vv
        # (weights and O in bf16: 2^-8 of sum p |v| and of O; a split's row 2^-12 of the largest value)
        tol = 2.0 ** -8 * (1 + 2.0 ** -6) * (want.abs() + torch.softmax(x, 1) @ vv.abs()) + 2.0 ** -11 * vv.abs().max()
        assert bool(((o[row].double() - want).abs() <= tol).all()), row
        assert float((lse[row].double() - torch.logsumexp(x, 1)).abs().max()) <= 1e-4
