"""The accepted path written over the lengths, and the move behind it: the caller keeps the lengths of before."""
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
