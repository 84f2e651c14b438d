"""The chain a decoder layer runs -- step tables, norm and rotation into the
cache, attention -- against a state kept on the host alone: tables by the rules
in lists and loops, rotated rows at those positions, the oracle's append into
those slots, and the oracle's attention over the cache that comes of it.  The
host is given lengths and projections, and nothing the chain computed.  Tables
and cache bytes are equal; the attention keeps the bounds of its own parity
tests (O within 1e-2 and 1e-3 on average, LSE within 1e-4)."""
import math
import random

import numpy as np
import pytest
import torch

import oracle
import speculative_decode_verify_paged_gb300 as sa
from speculative_decode_verify_paged_gb300 import workloads as W
from test_gpu_norm_rope import _bytes, _cache, close, formula
from test_gpu_step_tables import simulate

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from speculative_decode_verify_paged_gb300 import build as libbuild
    libbuild.build()
    oracle.build()
    torch.cuda.set_device(0)


# (ctx, window) of the two requests at each step: both admitted with prompts; a window each, 5 keys of request 0
# rejected; request 1 rolled back over a page border, its pages returned; request 0 grows into them; request 1 ends
STEPS = [([0, 0], [75, 31]), ([70, 31], [9, 4]), ([79, 10], [1, 2]), ([80, 12], [16, 16]), ([96, 0], [1, 0])]


@pytest.mark.parametrize("kv,interleave", [(W.KV_BF16, False), (W.KV_BF16, True), (W.KV_NVFP4, False), (W.KV_NVFP4, True)])
def test_the_chain_against_a_cache_kept_on_the_host(kv, interleave):
    hq, hkv, d, ps, P, pages, stride, cap = 8, 2, 128, 16, 2, 11, 8, 120
    i32 = dict(dtype=torch.int32, device="cuda")
    g = 0.0625 if kv == W.KV_NVFP4 else 1.0
    pools = _cache(pages, hkv, ps, d, kv, interleave)
    host = [_np_of(p) for p in pools]
    strides = dict(kv_page_stride=pools[0].stride(0) * pools[0].element_size())
    if kv == W.KV_NVFP4:
        strides["scale_page_stride"] = pools[2].stride(0)
    freq = sa.rope_inv_freq(d)
    plan = sa.spec_attn_norm_rope_plan_create(num_q_heads=hq, num_kv_heads=hkv, head_dim=d, inv_freq=freq, kv_dtype=kv,
                                              page_size=ps, num_pages=pages, **strides)
    attn = sa.spec_attn_plan_create(num_reqs=P, total_q_rows=cap, max_w=16, num_q_heads=hq, num_kv_heads=hkv, head_dim=d,
                                    num_pages=pages, block_table_stride=stride, max_seq_len=stride * ps, kv_dtype=kv,
                                    page_size=ps, **strides)
    ws = torch.zeros(attn.workspace_bytes, dtype=torch.uint8, device="cuda")
    stack = list(range(pages))
    random.Random(1).shuffle(stack)
    tab, prev = [[-1] * stride for _ in range(P)], [0] * P
    free, count, table = torch.tensor(stack, **i32), torch.tensor([pages], **i32), torch.tensor(tab, **i32)
    seq, indptr = torch.zeros(P, **i32), torch.zeros(P + 1, **i32)
    pos, slot = torch.zeros(cap, **i32), torch.zeros(cap, dtype=torch.int64, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(2)
    qw, kw = (1 + 0.3 * torch.randn(d, generator=gen, device="cuda") for _ in range(2))
    for ctx, win in STEPS:
        # on the GPU
        q, k, v = (torch.randn(cap, h, d, generator=gen, device="cuda").bfloat16() for h in (hq, hkv, hkv))
        q_rot = torch.full_like(q, 77.0)
        o = torch.full((cap, hq, d), 77.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((cap, hq), 77.0, device="cuda")
        sa.spec_attn_build_tables(torch.tensor(ctx, **i32), torch.tensor(win, **i32), seq, count, free, table, seq,
                                  indptr, count, pos, slot, ws, page_size=ps, max_w=128, max_seq_len=stride * ps)
        sa.spec_attn_norm_rope_append(plan, q, k, v, qw, kw, pos[None], slot, q_rot, pools[0], pools[1], ws,
                                      *(pools[2:] or [None, None]), g, g)
        if max(win) <= 16:
            sa.spec_attn_run(attn, q_rot, pools[0], pools[1], table, seq, indptr, o, lse, ws,
                             *(pools[2:] or [None, None]), g, g)
        assert sa.spec_attn_check_device_status(ws) == 0
        # on the host
        new_seq, ptr, stack, tab, at, _ = simulate(ctx, win, prev, stack, tab, ps, cap)
        prev, n = new_seq, ptr[-1]
        at_t = torch.tensor([at[:n]], **i32)
        q_ref, k_ref = torch.zeros_like(q[:n]), torch.zeros_like(k[:n])
        sa.spec_attn_norm_rope(plan, q[:n], k[:n], qw, kw, at_t, q_ref, k_ref)
        for x, w, got in ((q[:n], qw, q_ref), (k[:n], kw, k_ref)):
            close(got, *formula(x, w, at_t, freq, [0] * (d // 2), d, 0, 1e-6, 1.0))
        req = [r for r in range(P) for _ in range(win[r])]
        # (the oracle appends windows of up to 16 rows: a request a row)
        host = oracle.append_kv(num_kv_heads=hkv, head_dim=d, page_size=ps, kv_dtype=kv, k_new=k_ref.cpu(),
                                v_new=v[:n].cpu(), k_pool=host[0], v_pool=host[1], k_scales=(host + [None] * 2)[2],
                                v_scales=(host + [None] * 2)[3], k_gscale=g, v_gscale=g,
                                block_table=np.array([tab[r] for r in req], dtype=np.int32),
                                seq_lens=np.array(at[:n], dtype=np.int32) + 1,
                                q_indptr=np.arange(n + 1, dtype=np.int32))
        host = [p for p in host if p is not None]
        # both
        assert seq.tolist() == new_seq and indptr.tolist() == ptr and count.tolist() == [len(stack)]
        assert free[:len(stack)].tolist() == stack and table.tolist() == tab
        assert torch.equal(q_rot[:n], q_ref) and bool((q_rot[n:] == 77.0).all())
        for got, want in zip(pools, host):
            assert np.array_equal(_bytes(got), want.view(np.uint8).reshape(-1))
        if max(win) > 16:
            continue
        o_ref, lse_ref, _ = oracle.run(num_q_heads=hq, num_kv_heads=hkv, head_dim=d, page_size=ps, num_pages=pages,
                                       mask_mode=0, kv_dtype=kv, sm_scale=1 / math.sqrt(d), q=q_ref.cpu(),
                                       k_pool=host[0], v_pool=host[1], k_scales=(host + [None] * 2)[2],
                                       v_scales=(host + [None] * 2)[3], k_gscale=g, v_gscale=g,
                                       block_table=np.array(tab, dtype=np.int32),
                                       seq_lens=np.array(new_seq, dtype=np.int32), q_indptr=np.array(ptr, dtype=np.int32))
        err = np.abs(o[:n].float().cpu().numpy() - o_ref)
        assert err.max() <= 1e-2 and err.mean() <= 1e-3, (err.max(), err.mean())
        rel = np.abs(lse[:n].cpu().numpy() - lse_ref) / np.maximum(1.0, np.abs(lse_ref))
        assert rel.max() <= 1e-4
        assert bool((o[n:] == 77.0).all()) and bool((lse[n:] == 77.0).all())


def _np_of(t):
    t = t.cpu().contiguous()
    return t.view(torch.int16).numpy().view(np.uint16) if t.dtype == torch.bfloat16 else t.numpy()
