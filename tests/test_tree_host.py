"""CPU-side checks of the tree calls and of the masked attention: the binding's structs have the header's layout, and the
host checks refuse bad problems and pointers before any GPU work."""
import ctypes
import os
import subprocess

import pytest
import torch

import speculative_decode_verify_paged_gb300 as sa
from speculative_decode_verify_paged_gb300 import build as libbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BAD, UNSUPPORTED = sa.SPEC_ATTN_E_INVALID_ARG, sa.SPEC_ATTN_E_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return sa.load_library()


@pytest.mark.parametrize("cstruct", ["spec_attn_masked_problem", "spec_attn_tree_problem", "spec_attn_move_problem"])
def test_structs_match_the_header_layout(tmp_path, cstruct):
    pystruct = getattr(sa, cstruct)
    names = [f[0] for f in pystruct._fields_]
    lines = [f'printf("size %zu\\n", sizeof({cstruct}));']
    lines += [f'printf("{n} %zu\\n", offsetof({cstruct}, {n}));' for n in names]
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "spec_attn.h"\nint main(void) {\n    '
                   + "\n    ".join(lines) + "\n    return 0;\n}\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    out = dict(line.split() for line in subprocess.run([str(exe)], capture_output=True, text=True,
                                                        check=True).stdout.splitlines())
    assert int(out["size"]) == ctypes.sizeof(pystruct)
    for n in names:
        assert int(out[n]) == getattr(pystruct, n).offset, n


@pytest.mark.parametrize("over,status", [
    (dict(num_reqs=-1), BAD), (dict(num_reqs=65536), UNSUPPORTED), (dict(total_q_rows=-1), BAD),
    (dict(total_q_rows=2 ** 30 + 1), UNSUPPORTED), (dict(max_w=0), BAD), (dict(num_q_heads=6, num_kv_heads=4), BAD),
    (dict(num_q_heads=34, num_kv_heads=2), UNSUPPORTED), (dict(head_dim=96), UNSUPPORTED), (dict(head_dim=0), BAD),
    (dict(page_size=48), UNSUPPORTED), (dict(page_size=128), UNSUPPORTED), (dict(num_pages=0), BAD),
    (dict(num_pages=2 ** 27), UNSUPPORTED), (dict(block_table_stride=-1), BAD),
    (dict(block_table_stride=2 ** 27), UNSUPPORTED), (dict(kv_dtype=2), BAD), (dict(sm_scale=-1.0), BAD),
    (dict(sm_scale=float("nan")), BAD), (dict(sm_scale=float("inf")), BAD), (dict(tree=2), BAD),
    (dict(window_left=-1), BAD), (dict(sink_keys=-1), BAD), (dict(tree=1, max_w=65, mask_row_words=2), BAD),
    (dict(mask_row_words=-1), BAD), (dict(force_splits=-1), BAD), (dict(max_seq_len=2 ** 31), UNSUPPORTED),
    (dict(max_seq_len=-1), BAD), (dict(kv_page_stride=4096), BAD), (dict(kv_page_stride=8200), BAD),
    (dict(kv_dtype=1, scale_page_stride=264), BAD), (dict(kv_dtype=1, kv_page_stride=2056), BAD),
])
def test_masked_plan_refuses_bad_problems(lib, over, status):
    prob = dict(num_reqs=2, total_q_rows=8, max_w=4, num_q_heads=8, num_kv_heads=2, head_dim=128, page_size=16,
                num_pages=20, block_table_stride=10, kv_dtype=0, sm_scale=0.0, tree=0, window_left=0, sink_keys=0,
                mask_row_words=0, force_splits=0, max_seq_len=160, kv_page_stride=0, scale_page_stride=0)
    prob.update(over)
    pr = sa.spec_attn_masked_problem(*[prob[f[0]] for f in sa.spec_attn_masked_problem._fields_])
    h = ctypes.c_void_p()
    assert lib.spec_attn_masked_plan_create(ctypes.byref(pr), ctypes.byref(h), None) == status
    assert not h.value


def test_null_arguments(lib):
    assert lib.spec_attn_masked_plan_create(None, None, None) == BAD
    assert lib.spec_attn_run_masked(*([None] * 6), 1.0, 1.0, *([None] * 8), 0, None) == BAD
    assert lib.spec_attn_masked_plan_destroy(None) == sa.SPEC_ATTN_OK
    assert lib.spec_attn_build_tree(*([None] * 7), 0, None) == BAD
    assert lib.spec_attn_accept_tree(*([None] * 11), 0, None) == BAD
    assert lib.spec_attn_move_kv(*([None] * 11), 0, None) == BAD


# (host checks come before any CUDA call, so made-up addresses do)
def _tree(lib, call, names, over=None, ptr=None, ws_bytes=256):
    prob = dict(num_reqs=4, total_rows=64, max_w=32, mask_row_words=0, window_left=0, sink_keys=0, path_stride=8, reserved=0)
    prob.update(over or {})
    at = {n: 0x10000 * (i + 1) for i, n in enumerate(names)}
    at.update(ptr or {})
    pr = sa.spec_attn_tree_problem(*[prob[f[0]] for f in sa.spec_attn_tree_problem._fields_])
    return getattr(lib, call)(ctypes.byref(pr), *[at[n] for n in names], ws_bytes, None)


BUILD = ("spec_attn_build_tree", ["parents", "seq_lens", "q_indptr", "positions", "row_mask", "workspace"])
ACCEPT = ("spec_attn_accept_tree", ["parents", "draft_tokens", "target_tokens", "seq_lens", "q_indptr", "path",
                                    "accept_lens", "next_tokens", "ctx_lens", "workspace"])


@pytest.mark.parametrize("call,names", [BUILD, ACCEPT])
@pytest.mark.parametrize("over,status", [
    (dict(num_reqs=-1), BAD), (dict(num_reqs=65536), UNSUPPORTED), (dict(total_rows=-1), BAD), (dict(max_w=0), BAD),
    (dict(max_w=1025), UNSUPPORTED), (dict(reserved=1), BAD), (dict(max_w=33, mask_row_words=1), BAD),
    (dict(window_left=-1), BAD), (dict(sink_keys=-1), BAD),
])
def test_tree_calls_refuse_bad_problems(lib, call, names, over, status):
    assert _tree(lib, call, names, over) == status


def test_accept_refuses_an_empty_path(lib):
    assert _tree(lib, *ACCEPT, dict(path_stride=0)) == BAD


@pytest.mark.parametrize("call,names", [BUILD, ACCEPT])
def test_tree_calls_refuse_bad_pointers(lib, call, names):
    for i, n in enumerate(names):
        assert _tree(lib, call, names, ptr={n: None}) == BAD, n
        assert _tree(lib, call, names, ptr={n: 0x10000 * (i + 1) + 2}) == BAD, n
    assert _tree(lib, call, names, ws_bytes=255) == sa.SPEC_ATTN_E_WORKSPACE_TOO_SMALL


@pytest.mark.parametrize("call,names,ptr", [
    (*BUILD, dict(positions=0x10000)), (*BUILD, dict(positions=0x50010)), (*BUILD, dict(row_mask=0x20000)),
    (*BUILD, dict(row_mask=0x60000 - 64)), (*ACCEPT, dict(path=0x10000)), (*ACCEPT, dict(accept_lens=0x60010)),
    (*ACCEPT, dict(next_tokens=0x30000)), (*ACCEPT, dict(ctx_lens=0x40004)), (*ACCEPT, dict(ctx_lens=0x50000)),
    (*ACCEPT, dict(accept_lens=0x40000, ctx_lens=0x40000)),
])
def test_tree_calls_refuse_overlaps(lib, call, names, ptr):
    assert _tree(lib, call, names, ptr=ptr) == BAD


MOVE = ["block_table", "seq_lens", "q_indptr", "path", "accept_lens", "workspace"]


def _move(lib, over=None, ptr=None, pools=None, ws_bytes=256):
    prob = dict(num_reqs=4, num_layers=2, num_kv_heads=2, head_dim=64, page_size=16, num_pages=8, block_table_stride=4,
                kv_dtype=1, path_stride=8, reserved=0, max_seq_len=64, kv_page_stride=0, scale_page_stride=0)
    prob.update(over or {})
    at = {n: 0x10000 * (i + 1) for i, n in enumerate(MOVE)}
    at.update(ptr or {})
    lists = [[0x1000000 * (4 * i + l + 1) for l in range(2)] for i in range(4)]
    for (i, l), v in (pools or {}).items():
        lists[i][l] = v
    arrays = [(ctypes.c_void_p * 2)(*x) for x in lists]
    pr = sa.spec_attn_move_problem(*[prob[f[0]] for f in sa.spec_attn_move_problem._fields_])
    return lib.spec_attn_move_kv(ctypes.byref(pr), *arrays, *[at[n] for n in MOVE], ws_bytes, None)


@pytest.mark.parametrize("over,status", [
    (dict(num_reqs=-1), BAD), (dict(num_reqs=65536), UNSUPPORTED), (dict(num_layers=-1), BAD), (dict(num_kv_heads=0), BAD),
    (dict(num_kv_heads=65536), UNSUPPORTED), (dict(head_dim=96), UNSUPPORTED), (dict(page_size=8), UNSUPPORTED),
    (dict(num_pages=-1), BAD), (dict(num_pages=2 ** 27), UNSUPPORTED), (dict(block_table_stride=2 ** 27), UNSUPPORTED),
    (dict(kv_dtype=2), BAD), (dict(path_stride=0), BAD), (dict(reserved=1), BAD), (dict(max_seq_len=2 ** 31), UNSUPPORTED),
    (dict(kv_page_stride=512), BAD), (dict(kv_page_stride=1032), BAD), (dict(scale_page_stride=64), BAD),
])
def test_move_refuses_bad_problems(lib, over, status):
    assert _move(lib, over) == status


def test_move_refuses_bad_pointers(lib):
    for i, n in enumerate(MOVE):
        assert _move(lib, ptr={n: None}) == BAD, n
        assert _move(lib, ptr={n: 0x10000 * (i + 1) + 2}) == BAD, n
    for i in range(4):
        for l in range(2):
            assert _move(lib, pools={(i, l): None}) == BAD
            assert _move(lib, pools={(i, l): 0x900008}) == BAD
    assert _move(lib, ws_bytes=255) == sa.SPEC_ATTN_E_WORKSPACE_TOO_SMALL
    assert _move(lib, pools={(0, 1): 0x10000}) == BAD              # a pool over the block table
    assert _move(lib, pools={(1, 1): 0x2000000}) == BAD            # V over K of its layer


def test_native_calls_refuse_cpu_tensors(lib):
    i = torch.zeros(4, dtype=torch.int32)
    ws = torch.zeros(256, dtype=torch.uint8)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        sa.spec_attn_build_tree(i, i, i, i, i[:, None], ws, max_w=4)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        sa.spec_attn_accept_tree(i, i.long(), i.long(), i, i, i[None], i, i.long(), i, ws, max_w=4)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        sa.spec_attn_move_kv([i], [i], i[None], i, i, i[None], i, ws, max_seq_len=4)
    with pytest.raises(TypeError):
        sa.spec_attn_move_kv(i, i, i[None], i, i, i[None], i, ws, max_seq_len=4)
    calls = sa._native()
    for f in (calls.run_masked, calls.build_tree, calls.accept_tree, calls.move_kv):
        with pytest.raises(TypeError):
            f(())
    with pytest.raises(TypeError, match="not a plan"):
        calls.run_masked((1, 2), *([None] * 16))
