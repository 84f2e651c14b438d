"""CPU-side checks of the masked plan's info and of its stall hook: the binding's struct has the header's layout, and what is
no plan is refused; and numbers that the problem's fields do not hold."""
import ctypes
import os
import subprocess

import pytest

import speculative_decode_verify_paged_gb300 as sa
from speculative_decode_verify_paged_gb300 import build as libbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return sa.load_library()


def test_the_struct_matches_the_header_layout(tmp_path):
    names = [f[0] for f in sa.spec_attn_masked_plan_info._fields_]
    lines = ['printf("size %zu\\n", sizeof(spec_attn_masked_plan_info));']
    lines += [f'printf("{n} %zu\\n", offsetof(spec_attn_masked_plan_info, {n}));' for n in names]
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "spec_attn.h"\nint main(void) {\n    '
                   + "\n    ".join(lines) + "\n    return 0;\n}\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    out = dict(line.split() for line in subprocess.run([str(exe)], capture_output=True, text=True,
                                                        check=True).stdout.splitlines())
    assert int(out["size"]) == ctypes.sizeof(sa.spec_attn_masked_plan_info)
    for n in names:
        assert int(out[n]) == getattr(sa.spec_attn_masked_plan_info, n).offset, n


def test_null_arguments(lib):
    info = sa.spec_attn_masked_plan_info()
    assert lib.spec_attn_masked_plan_get_info(None, ctypes.byref(info)) == sa.SPEC_ATTN_E_INVALID_ARG
    assert lib.spec_attn_masked_plan_get_info(None, None) == sa.SPEC_ATTN_E_INVALID_ARG
    for stall in (0, 1, 2):
        assert lib.spec_attn_masked_plan_set_test_stall(None, stall) == sa.SPEC_ATTN_E_INVALID_ARG


@pytest.mark.parametrize("over", [dict(window_left=2 ** 32), dict(sink_keys=2 ** 32 + 4), dict(max_w=2 ** 32 + 1),
                                  dict(tree=2 ** 32), dict(force_splits=-2 ** 32), dict(max_seq_len=2 ** 64 + 60),
                                  dict(kv_page_stride=2 ** 64), dict(num_reqs=2 ** 32 + 1), dict(head_dim=2 ** 32 + 64)])
def test_numbers_that_their_fields_do_not_hold_are_refused(lib, over):
    prob = dict(num_reqs=1, total_q_rows=4, max_w=4, num_q_heads=8, num_kv_heads=2, head_dim=64, num_pages=4,
                block_table_stride=4, max_seq_len=60)
    with pytest.raises(sa.SpecAttnError) as e:
        sa.spec_attn_masked_plan_create(**{**prob, **over})
    assert e.value.status == sa.SPEC_ATTN_E_UNSUPPORTED
