"""Norm and rotation of q and k (and the same into the paged cache) against
their formulas in 64 bits.

Tolerance, from the arithmetic: one rounding to bf16 moves a value by at most
2^-8 of itself.  Before it everything is fp32: the sum of squares (chains of at
most 16 products and 4 additions) and its root are within 2^-19, the products
with root and weight and the rotation's product and sum within 5 x 2^-24, cos
and sin within 2^-22 of one (argument rounding 2^-24 x pi and 2 ulp).  In all
2^-17 of the magnitude that the rotated pair has covers it:
  |got - want| <= 2^-8 (1 + 2^-8) |want| + 2^-17 (|a| + |b|)."""
import math

import numpy as np
import pytest
import torch

import oracle
import speculative_decode_verify_paged_gb300 as sa
from speculative_decode_verify_paged_gb300 import workloads as W

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from speculative_decode_verify_paged_gb300 import build as libbuild
    libbuild.build()
    oracle.build()
    torch.cuda.set_device(0)


def formula(x, weight, pos, freq, axis, rot, interleaved, eps, scale):
    """(want, magnitude of each element's pair) in 64 bits; x [n, h, d], pos [axes, n]."""
    y = x.double().cpu()
    if weight is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * weight.double().cpu()
    want, mag = y.clone(), y.abs()
    half = rot // 2
    for j in range(half):
        i0, i1 = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
        t = pos[axis[j]].double().cpu() * freq[j]
        c, s = torch.cos(t)[:, None] * scale, torch.sin(t)[:, None] * scale
        a, b = y[..., i0], y[..., i1]
        want[..., i0], want[..., i1] = a * c - b * s, a * s + b * c
        mag[..., i0] = mag[..., i1] = (a.abs() + b.abs()) * abs(scale)
    return want, mag


def close(got, want, mag):
    got = got.double().cpu()
    bad = (got - want).abs() > 2.0 ** -8 * (1 + 2.0 ** -8) * want.abs() + 2.0 ** -17 * mag
    assert not bad.any(), (int(bad.sum()), (got - want).abs()[bad].max().item())


class Case:
    def __init__(self, n, hq, hkv, d, rot=None, axes=1, interleaved=0, norm=True, seed=0, fused=False, eps=1e-6,
                 scale=1.0, far=0, **plan):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rot = d if rot is None else rot
        rand = lambda *s: (torch.randn(*s, generator=g, device="cuda") * 2).to(torch.bfloat16)  # noqa: E731
        if fused:
            qkv = rand(n, (hq + 2 * hkv) * d)
            self.q, self.k, self.v = (t.unflatten(1, (-1, d)) for t in qkv.split([hq * d, hkv * d, hkv * d], 1))
            plan.update(q_row_stride=qkv.shape[1], k_row_stride=qkv.shape[1], v_row_stride=qkv.shape[1])
        else:
            self.q, self.k, self.v = rand(n, hq, d), rand(n, hkv, d), rand(n, hkv, d)
        w = lambda: 1 + 0.3 * torch.randn(d, generator=g, device="cuda") if norm else None  # noqa: E731
        self.qw, self.kw = w(), w()
        self.pos = (torch.randint(0, 5000, (axes, n), generator=g, device="cuda") + far).to(torch.int32)
        self.freq = sa.rope_inv_freq(rot, 1e6) if rot else []
        self.axis = [j % axes for j in range(rot // 2)]
        self.args = (self.pos, self.freq, self.axis, rot, interleaved, eps, scale)
        self.plan = sa.spec_attn_norm_rope_plan_create(
            num_q_heads=hq, num_kv_heads=hkv, head_dim=d, rot_dim=rot, inv_freq=self.freq,
            pair_axis=self.axis if axes > 1 else None, num_axes=axes, interleaved=interleaved, eps=eps,
            rot_scale=scale, **plan)
        mark = lambda *s: torch.full(s, 77.0, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        self.q_out, self.k_out = mark(n, hq, d), mark(n, hkv, d)

    def run(self, **kw):
        sa.spec_attn_norm_rope(self.plan, self.q, self.k, self.qw, self.kw, self.pos, self.q_out, self.k_out, **kw)

    def check(self):
        close(self.q_out, *formula(self.q, self.qw, *self.args))
        close(self.k_out, *formula(self.k, self.kw, *self.args))


SHAPES = [
    # rows, Hq, Hkv, d, rotated, axes, interleaved, norm, fused
    (1, 4, 1, 64, 64, 1, 0, True, False),
    (1, 24, 4, 256, 256, 1, 0, True, True),
    (3, 5, 3, 64, 16, 1, 0, True, False),          # heads that do not fill a warp, one rotating lane
    (7, 1, 1, 128, 48, 2, 0, True, True),          # an odd number of rotating pieces
    (17, 40, 8, 128, 128, 3, 0, True, True),
    (9, 16, 1, 256, 64, 1, 1, True, False),
    (5, 12, 12, 64, 32, 4, 1, False, True),
    (33, 32, 8, 128, 128, 1, 1, True, False),
    (4, 3, 2, 256, 0, 1, 0, True, False),          # the norm alone
    (4, 3, 2, 128, 128, 1, 0, False, True),        # the rotation alone
    (700, 24, 4, 256, 128, 3, 0, True, True),
    (4999, 8, 2, 64, 64, 1, 0, True, True),        # more rows than resident warps
]


@pytest.mark.parametrize("case", range(len(SHAPES)))
def test_norm_rope_matches_the_formula(case):
    n, hq, hkv, d, rot, axes, inter, norm, fused = SHAPES[case]
    c = Case(n, hq, hkv, d, rot, axes, inter, norm, seed=case, fused=fused)
    c.run()
    c.check()


@pytest.mark.parametrize("far", [2 ** 31 - 6000, 10 ** 6, -3000])
def test_far_and_negative_positions(far):
    """2^-53 of the 64-bit oracle's own angle at 2^31 is 2^-22: inside the tolerance."""
    c = Case(40, 4, 2, 128, far=far, seed=3, scale=1.3)
    c.run()
    c.check()


@pytest.mark.parametrize("norm,value", [(True, 0.0), (True, 1e-30), (True, 3e38), (False, 3e38)])
def test_extreme_values(norm, value):
    """Zero rows give zeros; a sum of squares past fp32 gives 0 (x times 1 / inf), as the fp32 formula does."""
    c = Case(2, 2, 1, 64, norm=norm, seed=4)
    c.q.fill_(value)
    c.k.fill_(value)
    c.run()
    if norm and value > 1e30:
        assert c.q_out.count_nonzero() == 0 and c.k_out.count_nonzero() == 0
    elif not norm:
        assert not torch.isnan(c.q_out).any()
    else:
        c.check()


def test_nan_stays_in_its_head():
    c = Case(3, 4, 2, 64, seed=5)
    c.q[1, 2, 7] = float("nan")
    c.k[0, 0, 3] = float("inf")
    c.run()
    nan = torch.isnan(c.q_out).any(-1)
    assert nan.nonzero().tolist() == [[1, 2]]
    assert torch.isnan(c.k_out).any(-1).nonzero().tolist() == [[0, 0]]


def test_in_place_on_the_fused_rows():
    a = Case(37, 24, 4, 256, 64, seed=6, fused=True)
    a.run()
    row = 24 * 256 + 8 * 256
    b = Case(37, 24, 4, 256, 64, seed=6, fused=True, q_out_row_stride=row, k_out_row_stride=row)
    v = b.v.clone()
    b.q_out, b.k_out = b.q, b.k
    b.run()
    assert torch.equal(a.q_out, b.q) and torch.equal(a.k_out, b.k) and torch.equal(v, b.v)


def test_one_side_alone_and_no_rows():
    full = Case(6, 8, 2, 128, seed=7)
    full.run()
    p = dict(head_dim=128, inv_freq=full.freq)
    q_only = sa.spec_attn_norm_rope_plan_create(num_q_heads=8, num_kv_heads=0, **p)
    out = torch.zeros_like(full.q)
    sa.spec_attn_norm_rope(q_only, full.q, None, full.qw, None, full.pos, out, None)
    assert torch.equal(out, full.q_out)
    k_only = sa.spec_attn_norm_rope_plan_create(num_q_heads=0, num_kv_heads=2, **p)
    out = torch.zeros_like(full.k)
    sa.spec_attn_norm_rope(k_only, None, full.k, None, full.kw, full.pos, None, out)
    assert torch.equal(out, full.k_out)
    e = Case(0, 8, 2, 128)
    e.run()


def test_weights_of_a_larger_buffer():
    """Weights need no more than their type's alignment; a side without heads has no rows to be in place."""
    c = Case(33, 8, 2, 128, seed=31)
    c.run()
    want = c.q_out.clone(), c.k_out.clone()
    packed = torch.zeros(2 * 128 + 3, device="cuda")
    packed[1:129], packed[130:258] = c.qw, c.kw
    c.q_out.fill_(77.0), c.k_out.fill_(77.0)
    sa.spec_attn_norm_rope(c.plan, c.q, c.k, packed[1:129], packed[130:258], c.pos, c.q_out, c.k_out)
    assert torch.equal(c.q_out, want[0]) and torch.equal(c.k_out, want[1])
    plan = sa.spec_attn_norm_rope_plan_create(num_q_heads=0, num_kv_heads=2, head_dim=128, rot_dim=0, inv_freq=[],
                                              q_row_stride=512)
    sa.spec_attn_norm_rope(plan, None, c.k, None, c.kw, None, None, c.k_out)


def test_graph_replay_and_another_stream():
    c = Case(50, 24, 4, 256, seed=8)
    c.run()
    want = c.q_out.clone(), c.k_out.clone()
    c.q_out.zero_(), c.k_out.zero_()
    torch.cuda.synchronize()
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=s):
        c.run(stream=s)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(c.q_out, want[0]) and torch.equal(c.k_out, want[1])


# --------------------------------------------------------------------------- #
# into the cache
# --------------------------------------------------------------------------- #
def _bytes(t):
    t = t.detach().cpu().contiguous()
    return (t.view(torch.int16) if t.dtype == torch.bfloat16 else t).numpy().view(np.uint8).reshape(-1)


def _cache(pages, hkv, ps, d, kv, interleave):
    """K and V pools (and scales) full of marks: dense, or sharing one allocation page by page."""
    rows = [(d, torch.bfloat16)] if kv == W.KV_BF16 else [(d // 2, torch.uint8), (d // 16, torch.uint8)]
    out = []
    for row, kind in rows:
        both = torch.full((pages, 2, hkv, ps, row), 9, device="cuda", dtype=kind)
        out += [both[:, 0], both[:, 1]] if interleave else [both[:, 0].contiguous(), both[:, 1].contiguous()]
    return out


@pytest.mark.parametrize("kv,interleave", [(W.KV_BF16, False), (W.KV_BF16, True), (W.KV_NVFP4, False),
                                           (W.KV_NVFP4, True)])
@pytest.mark.parametrize("hq,hkv,d,rot,ps", [(8, 2, 64, 64, 16), (24, 4, 256, 256, 32), (5, 3, 128, 48, 64)])
def test_append_bytes_equal_norm_rope_then_the_oracle_append(kv, interleave, hq, hkv, d, rot, ps):
    """Windows of ragged widths at ragged lengths: the cache bytes are the oracle's append of the rows that
    spec_attn_norm_rope gives, and no other byte changes; q comes out the same bits."""
    ctx, win = [0, 13, 40, 1000 % (3 * ps)], [3, 16, 0, 9]
    n = sum(win)
    pages = sum(-(-(c + w) // ps) for c, w in zip(ctx, win)) + 3
    stride = max(-(-(c + w) // ps) for c, w in zip(ctx, win))
    rng = np.random.default_rng(11)
    perm, table, slots, at = rng.permutation(pages), np.full((4, stride), -1, dtype=np.int32), [], 0
    for r in range(4):
        m = -(-(ctx[r] + win[r]) // ps)
        table[r, :m] = perm[at:at + m]
        at += m
        slots += [int(table[r, p // ps]) * ps + p % ps for p in range(ctx[r], ctx[r] + win[r])]
    g = 2.0 ** -5 if kv == W.KV_NVFP4 else 1.0
    pools = _cache(pages, hkv, ps, d, kv, interleave)
    size = pools[0].element_size()
    strides = dict(kv_page_stride=2 * hkv * ps * pools[0].shape[-1] * size) if interleave else {}
    if interleave and kv == W.KV_NVFP4:
        strides["scale_page_stride"] = 2 * hkv * ps * d // 16
    c = Case(n, hq, hkv, d, rot, seed=12, fused=True, kv_dtype=kv, page_size=ps, num_pages=pages, **strides)
    c.run()                                       # q_out and k_out of the pass without a cache
    want_q = c.q_out.clone()
    host = [None if i >= len(pools) else pools[i].cpu().contiguous() for i in range(4)]
    ref = oracle.append_kv(num_kv_heads=hkv, head_dim=d, page_size=ps, kv_dtype=kv, k_new=c.k_out.cpu(),
                           v_new=c.v.cpu().contiguous(), k_pool=host[0], v_pool=host[1], k_scales=host[2],
                           v_scales=host[3], k_gscale=g, v_gscale=g, block_table=torch.from_numpy(table),
                           seq_lens=torch.tensor([a + b for a, b in zip(ctx, win)], dtype=torch.int32),
                           q_indptr=torch.tensor(np.cumsum([0] + win), dtype=torch.int32))
    c.q_out.fill_(77.0)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    sa.spec_attn_norm_rope_append(c.plan, c.q, c.k, c.v, c.qw, c.kw, c.pos, torch.tensor(slots, device="cuda"), c.q_out,
                                  pools[0], pools[1], ws, *(pools[2:] or [None, None]), g, g)
    assert sa.spec_attn_check_device_status(ws) == 0
    assert torch.equal(c.q_out, want_q)
    for got, want in zip(pools, ref):
        assert np.array_equal(_bytes(got), want.view(np.uint8).reshape(-1))


@pytest.mark.parametrize("kv", [W.KV_BF16, W.KV_NVFP4])
def test_padded_and_bad_rows_are_skipped_whole(kv):
    hq, hkv, d, ps, pages = 4, 2, 64, 16, 5
    n = 9
    pools = _cache(pages, hkv, ps, d, kv, False)
    before = [p.clone() for p in pools]
    c = Case(n, hq, hkv, d, seed=13, kv_dtype=kv, page_size=ps, num_pages=pages)
    c.run()
    want = c.q_out.clone()
    c.q_out.fill_(77.0)
    slot = torch.tensor([3, -1, 79, 80, 2 ** 40, -2 ** 60, 17, -1, -1], device="cuda")
    live = [0, 2, 6]
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    sa.spec_attn_norm_rope_append(c.plan, c.q, c.k, c.v, c.qw, c.kw, c.pos, slot, c.q_out, *pools[:2], ws,
                                  *(pools[2:] or [None, None]), 0.25, 0.25)
    assert sa.spec_attn_check_device_status(ws) == sa.SPEC_ATTN_DEV_BAD_PAGE
    for i in range(n):
        assert torch.equal(c.q_out[i], want[i]) if i in live else bool((c.q_out[i] == 77.0).all())
    for p, b in zip(pools, before):
        touched = (p != b).flatten(3).any(3).any(1).flatten().nonzero().flatten().tolist()
        assert set(touched) <= {int(slot[i]) for i in live}
        if p.shape[-1] != d // 16:
            assert set(touched) == {int(slot[i]) for i in live}


def test_slots_past_32_bits_of_bytes():
    """A pool of more than 4 GiB: the last page's slots, written and nothing near their 32-bit images."""
    hq, hkv, d, ps = 1, 4, 256, 16
    page = hkv * ps * d * 2
    pages = (2 ** 32 + 2 ** 28) // page
    k_pool = torch.zeros(pages, hkv, ps, d, dtype=torch.bfloat16, device="cuda")
    c = Case(2, hq, hkv, d, seed=14, page_size=ps, num_pages=pages)
    c.run()
    slot = torch.tensor([pages * ps - 1, 2 ** 32 // page * ps + 3], device="cuda")
    v_pool = torch.zeros_like(k_pool)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    sa.spec_attn_norm_rope_append(c.plan, c.q, c.k, c.v, c.qw, c.kw, c.pos, slot, c.q_out, k_pool, v_pool, ws)
    assert sa.spec_attn_check_device_status(ws) == 0
    for i, s in enumerate(slot.tolist()):
        assert torch.equal(k_pool[s // ps, :, s % ps], c.k_out[i])
        assert torch.equal(v_pool[s // ps, :, s % ps], c.v[i])
    assert k_pool.flatten(1).any(1).sum() == 2 and v_pool.flatten(1).any(1).sum() == 2


def test_refused_calls_write_nothing():
    c = Case(4, 4, 2, 64, seed=15, page_size=16, num_pages=2)
    pools = _cache(2, 2, 16, 64, W.KV_BF16, False)
    slot = torch.arange(4, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    no_cache = Case(4, 4, 2, 64, seed=15)
    lib = sa.load_library()
    st = lib.spec_attn_norm_rope_append(            # the plan has no cache
        no_cache.plan.handle, 4, *[t.data_ptr() for t in (c.q, c.k, c.v, c.qw, c.kw, c.pos, slot, c.q_out, *pools)], None,
        None, 1.0, 1.0, ws.data_ptr(), 256, None)
    assert st == sa.SPEC_ATTN_E_INVALID_ARG
    with pytest.raises(ValueError):                     # (nor do its shapes fit)
        sa.spec_attn_norm_rope_append(no_cache.plan, c.q, c.k, c.v, c.qw, c.kw, c.pos, slot, c.q_out, *pools, ws)
    with pytest.raises(ValueError):                     # positions of another length
        sa.spec_attn_norm_rope(c.plan, c.q, c.k, c.qw, c.kw, c.pos[:, :3].contiguous(), c.q_out, c.k_out)
    with pytest.raises(ValueError):                     # weights in another type
        sa.spec_attn_norm_rope(c.plan, c.q, c.k, c.qw.bfloat16(), c.kw, c.pos, c.q_out, c.k_out)
    with pytest.raises(ValueError):                     # rows not at the plan's stride
        sa.spec_attn_norm_rope(c.plan, torch.cat([c.q, c.q], 1)[:, :4], c.k, c.qw, c.kw, c.pos, c.q_out, c.k_out)
    with pytest.raises(ValueError):                     # 32-bit slots
        sa.spec_attn_norm_rope_append(c.plan, c.q, c.k, c.v, c.qw, c.kw, c.pos, slot.int(), c.q_out, *pools, ws)
    with pytest.raises(sa.SpecAttnError):               # in place at another stride
        other = Case(4, 4, 2, 64, seed=15, q_out_row_stride=512)
        sa._check(lib.spec_attn_norm_rope(other.plan.handle, 4, c.q.data_ptr(), c.k.data_ptr(), None, None,
                                          c.pos.data_ptr(), c.q.data_ptr(), c.k_out.data_ptr(), None), "in place")
    torch.cuda.synchronize()
    assert bool((c.q_out == 77.0).all()) and bool((c.k_out == 77.0).all())
    assert all(bool((p == 9).all()) for p in pools)


# --------------------------------------------------------------------------- #
# the chain: tables, norm and rotation into the cache, attention
# --------------------------------------------------------------------------- #
@pytest.mark.parametrize("kv", [W.KV_BF16, W.KV_NVFP4])
def test_tables_then_append_then_attention(kv):
    """Two requests are admitted with prompts, then verify a window, lengths never leaving the GPU: the attention's
    rows match the oracle's attention over the cache that the oracle builds from the same rows."""
    hq, hkv, d, ps, P = 8, 2, 128, 16, 2
    pages, stride, cap = 40, 16, 200
    i32 = dict(dtype=torch.int32, device="cuda")
    g = 0.0625 if kv == W.KV_NVFP4 else 1.0
    pools = [p.zero_() for p in _cache(pages, hkv, ps, d, kv, False)]
    plan = sa.spec_attn_norm_rope_plan_create(num_q_heads=hq, num_kv_heads=hkv, head_dim=d,
                                              inv_freq=sa.rope_inv_freq(d), kv_dtype=kv, page_size=ps, num_pages=pages)
    attn = sa.spec_attn_plan_create(num_reqs=P, total_q_rows=cap, max_w=16, num_q_heads=hq, num_kv_heads=hkv,
                                    head_dim=d, num_pages=pages, block_table_stride=stride, max_seq_len=stride * ps,
                                    kv_dtype=kv, page_size=ps)
    ws = torch.zeros(attn.workspace_bytes, dtype=torch.uint8, device="cuda")
    free = torch.randperm(pages, generator=torch.Generator().manual_seed(1)).to(**i32)
    count, table = torch.tensor([pages], **i32), torch.full((P, stride), -1, **i32)
    seq, indptr = torch.zeros(P, **i32), torch.zeros(P + 1, **i32)
    pos, slot = torch.zeros(cap, **i32), torch.zeros(cap, dtype=torch.int64, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(2)
    o = torch.zeros(cap, hq, d, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(cap, hq, device="cuda")
    w = torch.ones(d, device="cuda")
    for ctx, win in (([0, 0], [75, 31]), ([70, 31], [9, 4])):     # the second step drops 5 rejected keys
        sa.spec_attn_build_tables(torch.tensor(ctx, **i32), torch.tensor(win, **i32), seq, count, free, table, seq,
                                  indptr, count, pos, slot, ws, page_size=ps, max_w=128, max_seq_len=stride * ps)
        q, k, v = (torch.randn(cap, h, d, generator=gen, device="cuda").bfloat16() for h in (hq, hkv, hkv))
        q_rot = torch.zeros_like(q)
        sa.spec_attn_norm_rope_append(plan, q, k, v, w, w, pos[None], slot, q_rot, pools[0], pools[1], ws,
                                      *(pools[2:] or [None, None]), g, g)
    sa.spec_attn_run(attn, q_rot, pools[0], pools[1], table, seq, indptr, o, lse, ws, *(pools[2:] or [None, None]), g, g)
    assert sa.spec_attn_check_device_status(ws) == 0
    assert seq.tolist() == [79, 35] and indptr.tolist() == [0, 9, 13]
    n = 13
    host = [None if i >= len(pools) else pools[i].cpu() for i in range(4)]
    o_ref, lse_ref, _ = oracle.run(num_q_heads=hq, num_kv_heads=hkv, head_dim=d, page_size=ps, num_pages=pages,
                                   mask_mode=0, kv_dtype=kv, sm_scale=1 / math.sqrt(d), q=q_rot[:n].cpu(),
                                   k_pool=host[0], v_pool=host[1], k_scales=host[2], v_scales=host[3], k_gscale=g,
                                   v_gscale=g, block_table=table.cpu(), seq_lens=seq.cpu(), q_indptr=indptr.cpu())
    err = np.abs(o[:n].float().cpu().numpy() - o_ref)
    assert err.max() <= 1e-2 and err.mean() <= 1e-3, (err.max(), err.mean())
    rel = np.abs(lse[:n].cpu().numpy() - lse_ref) / np.maximum(1.0, np.abs(lse_ref))
    assert rel.max() <= 1e-4
    # and the last step's rows are where the table says
    k_rot = torch.zeros_like(k)
    sa.spec_attn_norm_rope(plan, q, k, w, w, pos[None], torch.zeros_like(q), k_rot)
    if kv == W.KV_BF16:
        for i in range(n):
            s = int(slot[i])
            assert torch.equal(pools[0][s // ps, :, s % ps], k_rot[i]) and torch.equal(pools[1][s // ps, :, s % ps], v[i])


@pytest.mark.parametrize("seed,gscale", [(0, 2.0 ** -6), (1, 0.3), (2, 1.0 / 2688), (3, 7.5e-6), (4, 1e-25), (5, 3e24),
                                         (6, 2.0 ** -8 * (2 - 2.0 ** -23))])
def test_quantised_values_of_every_range(seed, gscale):
    """V goes into a 4-bit cache as it is: rows of wide range, dyadic values on rounding borders, zeros of both signs,
    tiny and clipped blocks, against the oracle's own divisions, byte for byte -- for decode scales in the middle of
    the range, at its ends (where a block's quotients are divisions) and with a significand of ones."""
    hkv, d, ps, n = 4, 256, 16, 512
    k, v = W.window_kv_rows(n, hkv, d, seed=60 + seed)
    pools = _cache(n // ps, hkv, ps, d, W.KV_NVFP4, False)
    host = [p.cpu().contiguous() for p in pools]
    plan = sa.spec_attn_norm_rope_plan_create(num_q_heads=1, num_kv_heads=hkv, head_dim=d, rot_dim=0, inv_freq=[],
                                              kv_dtype=1, page_size=ps, num_pages=n // ps)
    q = torch.zeros(n, 1, d, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    sa.spec_attn_norm_rope_append(plan, q, k.cuda(), v.cuda(), None, None, torch.zeros(1, n, dtype=torch.int32, device="cuda"),
                                  torch.arange(n, device="cuda"), q, *pools[:2], ws, *pools[2:], gscale, gscale)
    assert sa.spec_attn_check_device_status(ws) == 0
    # (32 requests of 16 rows at context 0: their slots are the rows' numbers)
    ref = oracle.append_kv(num_kv_heads=hkv, head_dim=d, page_size=ps, kv_dtype=1, k_new=k, v_new=v, k_pool=host[0],
                           v_pool=host[1], k_scales=host[2], v_scales=host[3], k_gscale=gscale, v_gscale=gscale,
                           block_table=torch.arange(n // 16, dtype=torch.int32)[:, None].contiguous(),
                           seq_lens=torch.full((n // 16,), 16, dtype=torch.int32),
                           q_indptr=torch.arange(n // 16 + 1, dtype=torch.int32) * 16)
    for got, want in zip(pools, ref):
        assert np.array_equal(_bytes(got), want.view(np.uint8).reshape(-1))


def test_overlapping_buffers_are_refused():
    """An output that shares bytes with an input it is not in the place of, or with another output."""
    n, hq, hkv, d, ps, pages = 6, 4, 4, 64, 16, 2
    c = Case(n, hq, hkv, d, seed=16, page_size=ps, num_pages=pages)
    c.run()
    want = c.q_out.clone(), c.k_out.clone()
    buf = torch.full((2 * n + 2, hq, d), 5.0, dtype=torch.bfloat16, device="cuda")

    def norm_rope(**over):
        a = {**dict(q=c.q, k=c.k, qw=c.qw, kw=c.kw, pos=c.pos, q_out=buf[:n], k_out=buf[n:2 * n]), **over}
        sa.spec_attn_norm_rope(c.plan, *[a[x] for x in ("q", "k", "qw", "kw", "pos", "q_out", "k_out")])

    as_pos = buf.view(torch.int32).flatten()[:n].view(1, n)
    for over in (dict(q=buf[1:n + 1]), dict(k=buf[:n]), dict(k=buf[n + 1:2 * n + 1]), dict(k_out=buf[n - 1:2 * n - 1]),
                 dict(q=buf[n:2 * n]), dict(qw=buf.view(torch.float32).flatten()[:d]), dict(pos=as_pos),
                 dict(q=buf[:n], k_out=buf[:n])):
        with pytest.raises(sa.SpecAttnError) as e:
            norm_rope(**over)
        assert e.value.status == sa.SPEC_ATTN_E_INVALID_ARG
    pools = _cache(pages, hkv, ps, d, W.KV_BF16, False)
    slot, ws = torch.arange(n, device="cuda"), torch.zeros(256, dtype=torch.uint8, device="cuda")

    def append(**over):
        a = {**dict(q=c.q, k=c.k, v=c.v, qw=c.qw, kw=c.kw, pos=c.pos, slot=slot, q_out=buf[:n], k_pool=pools[0],
                    v_pool=pools[1], ws=ws), **over}
        sa.spec_attn_norm_rope_append(c.plan, *a.values())

    as_rows = pools[0].view(-1)[5 * d:5 * d + n * hkv * d].view(n, hkv, d)
    for over in (dict(v_pool=pools[0]), dict(k=as_rows), dict(v=as_rows), dict(q_out=as_rows), dict(v=buf[:n]),
                 dict(k=buf[1:n + 1]), dict(slot=buf.view(torch.int64).flatten()[:n]),
                 dict(ws=buf.view(torch.uint8).flatten()[:256])):
        with pytest.raises(sa.SpecAttnError) as e:
            append(**over)
        assert e.value.status == sa.SPEC_ATTN_E_INVALID_ARG
    torch.cuda.synchronize()
    assert bool((buf == 5.0).all()) and all(bool((p == 9).all()) for p in pools)
    norm_rope()
    assert torch.equal(buf[:n], want[0]) and torch.equal(buf[n:2 * n], want[1]) and bool((buf[2 * n:] == 5.0).all())


def test_outputs_between_the_rows_of_their_inputs():
    """Rows of one buffer that lie between each other at two strides are apart: outputs in the gaps of the inputs' rows,
    and every second row of a wider stride."""
    n, hq, hkv, d = 9, 2, 1, 64
    a = Case(n, hq, hkv, d, seed=17)
    a.run()
    wide = torch.full((n, 512), 3.0, dtype=torch.bfloat16, device="cuda")
    q, k, q_out = wide[:, :128].unflatten(1, (hq, d)), wide[:, 128:192].unflatten(1, (hkv, d)), wide[:, 256:384].unflatten(1, (hq, d))
    long = torch.full((2 * n, 512), 3.0, dtype=torch.bfloat16, device="cuda")
    k_out = long[::2, 64:128].unflatten(1, (hkv, d))
    q.copy_(a.q), k.copy_(a.k)
    plan = sa.spec_attn_norm_rope_plan_create(num_q_heads=hq, num_kv_heads=hkv, head_dim=d, inv_freq=a.freq, eps=1e-6,
                                              q_row_stride=512, k_row_stride=512, q_out_row_stride=512,
                                              k_out_row_stride=1024)
    sa.spec_attn_norm_rope(plan, q, k, a.qw, a.kw, a.pos, q_out, k_out)
    assert torch.equal(q_out, a.q_out) and torch.equal(k_out, a.k_out) and torch.equal(q, a.q) and torch.equal(k, a.k)
    assert bool((wide[:, 384:] == 3.0).all()) and bool((long[1::2] == 3.0).all())
