"""Calls of the tree's operators that their documentation allows: the accepted path written over the lengths, and the move
behind it, for which the caller keeps the lengths of before; a last request that cannot be."""
import random

import pytest
import torch

import speculative_decode_verify_paged_gb300 as sa
from test_gpu_tree import Caches, I32, I64, accept_case, host_accept, indptr_of, moved, workspace

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from speculative_decode_verify_paged_gb300 import build as libbuild
    libbuild.build()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("kv", ["bf16", "nvfp4"])
def test_lengths_written_in_place_and_a_kept_copy(kv):
    rng = random.Random(9)
    rows, ctx, cap = [20, 1, 33], [40, 7, 0], 8
    trees, draft, target = accept_case(rng, rows, vocab=2)
    c = Caches(2, 20, 2, 64, 16, kv, False, 4)
    before = c.bytes()
    table = torch.arange(18, dtype=torch.int32).view(3, 6)
    flat = lambda x, **kw: torch.tensor([v for t in x for v in t], **kw)  # noqa: E731
    seq, ptr, ws = torch.tensor([a + w for a, w in zip(ctx, rows)], **I32), indptr_of(rows), workspace()
    kept = seq.clone()
    path, taken, nxt = torch.zeros(3, cap, **I32), torch.zeros(3, **I32), torch.zeros(3, **I64)
    sa.spec_attn_accept_tree(flat(trees, **I32), flat(draft, **I64), flat(target, **I64), seq, ptr, path, taken, nxt, seq, ws,
                             max_w=33)
    c.move(table.cuda(), kept, ptr, path, taken, ws, max_seq_len=96)
    paths = [host_accept(t, d, g, cap)[0] for t, d, g in zip(trees, draft, target)]
    assert seq.tolist() == [a + len(p) for a, p in zip(ctx, paths)] and any(p != list(range(len(p))) for p in paths)
    for a, b in zip(c.bytes(), moved(before, table, ctx, paths, 16)):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    # the new lengths in their place lie before key 0 for a context shorter than what was not accepted: refused there
    c.move(table[2:].cuda(), seq[2:], indptr_of(rows[2:]), path[2:], taken[2:], ws, max_seq_len=96)
    assert sa.spec_attn_check_device_status(ws) == sa.SPEC_ATTN_DEV_BAD_SEQ_LEN


@pytest.mark.parametrize("end", [5, -1])
def test_a_last_window_below_zero_leaves_the_others_rows(end):
    """The rows from q_indptr[P] on are other requests' then, of more CTAs than the GPU holds at once."""
    P, w = 2000, 1024
    i = torch.arange(w, **I32)
    parents = torch.where(i > 0, 0, -1).int().repeat(P)                        # stars
    ptr = torch.arange(P + 1, **I32) * w
    ptr[P] = end
    pos, mask, ws = torch.full((P * w,), 99, **I32), torch.full((P * w, 32), 99, **I32), workspace()
    sa.spec_attn_build_tree(parents, torch.full((P,), w + 7, **I32), ptr, pos, mask, ws, max_w=w)
    assert sa.spec_attn_check_device_status(ws) == sa.SPEC_ATTN_DEV_BAD_WINDOW
    pos = pos.view(P, w)
    assert bool((pos[:-1] == 7 + (i > 0)).all()) and bool((pos[-1] == 99).all())
    mask = mask.view(P, w, 32)
    want = torch.zeros(w, 32, dtype=torch.int64, device="cuda")
    want[i.long(), i.long() // 32] = 1 << (i.long() % 32)
    want[:, 0] |= 1
    want = torch.where(want >= 2 ** 31, want - 2 ** 32, want).int()
    assert bool((mask[:-1] == want).all()) and bool((mask[-1] == 99).all())
