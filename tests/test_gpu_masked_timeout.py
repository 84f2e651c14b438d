"""The time-out path of the bounded waits of the attention under masks, made to run out without any fault: with the stall hook
no K is copied, every wait behind it gives up after about a second, the CTAs free their tensor memory and the call raises
SPEC_ATTN_DEV_WAIT_TIMEOUT in the device-status word.  The same plan afterwards is right again, and so is a call whose CTAs
take the tensor memory of every SM."""
import pytest
import torch

import speculative_decode_verify_paged_gb300 as sa
from test_gpu_masked import MARK, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from speculative_decode_verify_paged_gb300 import build as libbuild
    libbuild.build()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("kv,hq,hkv,d,rows,ctx,splits", [
    ("bf16", 8, 2, 64, [3, 9], [2000, 200], 1), ("bf16", 32, 8, 128, [3, 9], [2000, 200], 3),
    ("bf16", 6, 2, 256, [3, 9], [2000, 200], 12), ("bf16", 16, 1, 128, [300], [900], 1),
    ("bf16", 16, 8, 128, [200] * 5, [1900] * 5, 1), ("bf16", 4, 2, 64, [1] * 100, [100] * 100, 1), ("nvfp4", 8, 2, 64, [3, 9], [2000, 200], 1),
    ("nvfp4", 32, 8, 128, [3, 9], [2000, 200], 3), ("nvfp4", 6, 2, 256, [3, 9], [2000, 200], 12),
])
def test_waits_that_run_out_set_the_status_and_leave_the_context_usable(kv, hq, hkv, d, rows, ctx, splits):
    c = Case(rows, ctx, hq, hkv, d, tree=True, kv=kv, force_splits=splits, seed=4)
    info = c.plan.info
    assert info["max_splits"] == (splits if splits < 4 else 11) and info["query_tiles"] == 1 + (len(rows) == 5)
    assert info["ctas_per_sm"] == 1 + (len(rows) == 100)
    c.plan.set_test_stall(1)
    c.run()
    torch.cuda.synchronize()
    assert sa.spec_attn_check_device_status(c.ws) == sa.SPEC_ATTN_DEV_WAIT_TIMEOUT
    c.plan.set_test_stall(0)
    c.o.fill_(MARK), c.lse.fill_(MARK)
    c.run()
    c.check()
    full = Case([1] * 400, [70] * 400, 6, 1, 256, seed=1)
    full.run()
    full.check()
