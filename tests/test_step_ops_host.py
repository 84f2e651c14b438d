"""CPU-side checks of the entry points around the attention call: the binding's
structs have the header's layout, the host checks refuse bad problems and
pointers before any GPU work, and the rotation helpers give the usual tables."""
import ctypes
import os
import subprocess

import pytest
import torch

import speculative_decode_verify_paged_gb300 as sa
from speculative_decode_verify_paged_gb300 import build as libbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return sa.load_library()


STRUCTS = [("spec_attn_tables_problem", sa.spec_attn_tables_problem),
           ("spec_attn_norm_rope_problem", sa.spec_attn_norm_rope_problem),
           ("spec_attn_cross_problem", sa.spec_attn_cross_problem)]


@pytest.mark.parametrize("cstruct,pystruct", STRUCTS)
def test_structs_match_the_header_layout(tmp_path, cstruct, pystruct):
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


# --------------------------------------------------------------------------- #
# step tables: host checks come before any CUDA call, so made-up addresses do
# --------------------------------------------------------------------------- #
def _tables(lib, over=None, ptr=None, ws_bytes=256):
    prob = dict(num_reqs=4, max_rows=64, page_size=16, num_pages=100, block_table_stride=20, max_w=16, max_seq_len=320)
    prob.update(over or {})
    names = ["ctx_lens", "window_lens", "prev_seq_lens", "prev_free_count", "free_pages", "block_table", "seq_lens",
             "q_indptr", "free_count", "positions", "slot_map", "workspace"]
    at = {n: 0x10000 * (i + 1) for i, n in enumerate(names)}
    at.update(ptr or {})
    pr = sa.spec_attn_tables_problem(*[prob[f[0]] for f in sa.spec_attn_tables_problem._fields_])
    return lib.spec_attn_build_tables(ctypes.byref(pr), *[at[n] for n in names], ws_bytes, None)


@pytest.mark.parametrize("over,status", [
    (dict(num_reqs=-1), sa.SPEC_ATTN_E_INVALID_ARG),
    (dict(num_reqs=16385), sa.SPEC_ATTN_E_UNSUPPORTED),
    (dict(max_rows=-1), sa.SPEC_ATTN_E_INVALID_ARG),
    (dict(max_w=0), sa.SPEC_ATTN_E_INVALID_ARG),
    (dict(page_size=48), sa.SPEC_ATTN_E_UNSUPPORTED),
    (dict(page_size=0), sa.SPEC_ATTN_E_UNSUPPORTED),
    (dict(max_seq_len=2 ** 31), sa.SPEC_ATTN_E_UNSUPPORTED),
    (dict(block_table_stride=2 ** 27), sa.SPEC_ATTN_E_UNSUPPORTED),      # 2^31 keys a row
    (dict(num_pages=-5), sa.SPEC_ATTN_E_INVALID_ARG),
])
def test_tables_refuse_bad_problems(lib, over, status):
    assert _tables(lib, over) == status


@pytest.mark.parametrize("ptr", [
    dict(ctx_lens=None), dict(window_lens=None), dict(prev_seq_lens=None), dict(prev_free_count=None),
    dict(free_pages=None), dict(block_table=None), dict(seq_lens=None), dict(q_indptr=None), dict(free_count=None),
    dict(positions=None), dict(slot_map=None), dict(workspace=None),
    dict(ctx_lens=0x10002), dict(slot_map=0xb0004), dict(workspace=0xc0010),
    dict(seq_lens=0x10004),                 # overlaps ctx_lens without being it
    dict(seq_lens=0x20000),                 # is window_lens
    dict(q_indptr=0x30000),                 # is prev_seq_lens
    dict(free_count=0x50000),               # lies in free_pages
    dict(positions=0xb0000),                # lies in slot_map
])
def test_tables_refuse_bad_pointers(lib, ptr):
    assert _tables(lib, ptr=ptr) == sa.SPEC_ATTN_E_INVALID_ARG


def test_tables_refuse_a_small_workspace(lib):
    assert _tables(lib, ws_bytes=255) == sa.SPEC_ATTN_E_WORKSPACE_TOO_SMALL
    assert lib.spec_attn_build_tables(None, *([None] * 12), 0, None) == sa.SPEC_ATTN_E_INVALID_ARG


# --------------------------------------------------------------------------- #
# norm and rotation
# --------------------------------------------------------------------------- #
def _nr_create(lib, over=None, freq=None, axis=None):
    prob = dict(num_q_heads=8, num_kv_heads=2, head_dim=128, rot_dim=128, interleaved=0, num_axes=1, eps=1e-6,
                rot_scale=1.0, q_row_stride=0, k_row_stride=0, v_row_stride=0, q_out_row_stride=0,
                k_out_row_stride=0, kv_dtype=0, page_size=0, num_pages=0, reserved=0, kv_page_stride=0,
                scale_page_stride=0)
    prob.update(over or {})
    pr = sa.spec_attn_norm_rope_problem(*[prob[f[0]] for f in sa.spec_attn_norm_rope_problem._fields_])
    freq = sa.rope_inv_freq(256) if freq is None else freq
    arr = (ctypes.c_double * 128)(*freq[:128])
    ax = None if axis is None else (ctypes.c_uint8 * 128)(*axis)
    h = ctypes.c_void_p()
    st = lib.spec_attn_norm_rope_plan_create(ctypes.byref(pr), arr, ax, ctypes.byref(h))
    assert not h.value
    return st


@pytest.mark.parametrize("over,status", [
    (dict(num_q_heads=-1), sa.SPEC_ATTN_E_INVALID_ARG),
    (dict(num_q_heads=0, num_kv_heads=0), sa.SPEC_ATTN_E_INVALID_ARG),
    (dict(num_q_heads=5000), sa.SPEC_ATTN_E_UNSUPPORTED),
    (dict(head_dim=96), sa.SPEC_ATTN_E_UNSUPPORTED),
    (dict(rot_dim=144), sa.SPEC_ATTN_E_INVALID_ARG),
    (dict(rot_dim=24), sa.SPEC_ATTN_E_UNSUPPORTED),
    (dict(rot_dim=-16), sa.SPEC_ATTN_E_INVALID_ARG),
    (dict(interleaved=2), sa.SPEC_ATTN_E_INVALID_ARG),
    (dict(num_axes=0), sa.SPEC_ATTN_E_INVALID_ARG),
    (dict(num_axes=5), sa.SPEC_ATTN_E_INVALID_ARG),
    (dict(eps=-1.0), sa.SPEC_ATTN_E_INVALID_ARG),
    (dict(eps=float("nan")), sa.SPEC_ATTN_E_INVALID_ARG),
    (dict(rot_scale=float("inf")), sa.SPEC_ATTN_E_INVALID_ARG),
    (dict(q_row_stride=1016), sa.SPEC_ATTN_E_INVALID_ARG),       # below the dense row (1024)
    (dict(k_row_stride=260), sa.SPEC_ATTN_E_INVALID_ARG),        # not a multiple of 8
    (dict(v_row_stride=-8), sa.SPEC_ATTN_E_INVALID_ARG),
    (dict(q_out_row_stride=8), sa.SPEC_ATTN_E_INVALID_ARG),
    (dict(reserved=1), sa.SPEC_ATTN_E_INVALID_ARG),
    (dict(page_size=48, num_pages=4), sa.SPEC_ATTN_E_UNSUPPORTED),
    (dict(page_size=16, num_pages=0), sa.SPEC_ATTN_E_INVALID_ARG),
    (dict(page_size=16, num_pages=4, kv_dtype=2), sa.SPEC_ATTN_E_INVALID_ARG),
    (dict(page_size=16, num_pages=4, kv_page_stride=4096), sa.SPEC_ATTN_E_INVALID_ARG),    # dense: 8192 B
    (dict(page_size=16, num_pages=4, kv_dtype=1, scale_page_stride=264), sa.SPEC_ATTN_E_INVALID_ARG),
])
def test_norm_rope_plan_refuses_bad_problems(lib, over, status):
    assert _nr_create(lib, over) == status


def test_norm_rope_plan_refuses_bad_frequencies_and_axes(lib):
    good = sa.rope_inv_freq(256)
    for bad in (float("nan"), float("inf"), -1.0, 2.0 ** 20):
        assert _nr_create(lib, freq=[bad] + good[1:]) == sa.SPEC_ATTN_E_INVALID_ARG
    assert _nr_create(lib, dict(num_axes=3), axis=[3] + [0] * 127) == sa.SPEC_ATTN_E_INVALID_ARG
    with pytest.raises(ValueError):
        sa.spec_attn_norm_rope_plan_create(num_q_heads=8, num_kv_heads=2, head_dim=128, inv_freq=good[:63])
    with pytest.raises(ValueError):
        sa.spec_attn_norm_rope_plan_create(num_q_heads=8, num_kv_heads=2, head_dim=128, inv_freq=good[:64],
                                           pair_axis=[0] * 63)


def test_null_arguments(lib):
    assert lib.spec_attn_norm_rope_plan_create(None, None, None, None) == sa.SPEC_ATTN_E_INVALID_ARG
    assert lib.spec_attn_norm_rope(None, 1, *([None] * 8)) == sa.SPEC_ATTN_E_INVALID_ARG
    assert lib.spec_attn_norm_rope_append(None, 1, *([None] * 12), 1.0, 1.0, None, 0,
                                          None) == sa.SPEC_ATTN_E_INVALID_ARG
    assert lib.spec_attn_norm_rope_plan_destroy(None) == sa.SPEC_ATTN_OK


def test_rope_helpers():
    assert sa.rope_inv_freq(4, 100.0) == [1.0, 0.1]
    assert sa.rope_pair_axis((2, 3, 1)) == [0, 0, 1, 1, 1, 2]
    assert sa.rope_pair_axis((2, 3, 1), interleaved=True) == [0, 1, 2, 0, 1, 1]


def test_cpu_tensors_are_refused(lib):
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="ctx_lens must be a CUDA tensor"):
        sa.spec_attn_build_tables(i, i, i, i[:1], i, i[None].expand(4, 4), i, i, i[:1], i, i.long(),
                                  torch.zeros(256, dtype=torch.uint8), max_seq_len=64)


def test_native_calls_count_their_arguments(lib):
    calls = sa._native()
    for f in (calls.build_tables, calls.norm_rope, calls.norm_rope_append, calls.run_cross):
        with pytest.raises(TypeError):
            f(())
    with pytest.raises(TypeError, match="not a plan"):
        calls.norm_rope((1, 2), *([None] * 8))


# --------------------------------------------------------------------------- #
# cross attention
# --------------------------------------------------------------------------- #
@pytest.mark.parametrize("over,status", [
    (dict(num_reqs=-1), sa.SPEC_ATTN_E_INVALID_ARG),
    (dict(num_reqs=65536), sa.SPEC_ATTN_E_UNSUPPORTED),
    (dict(total_q_rows=-1), sa.SPEC_ATTN_E_INVALID_ARG),
    (dict(max_q_rows=0), sa.SPEC_ATTN_E_INVALID_ARG),
    (dict(num_q_heads=6, num_kv_heads=4), sa.SPEC_ATTN_E_INVALID_ARG),
    (dict(num_q_heads=34, num_kv_heads=2), sa.SPEC_ATTN_E_UNSUPPORTED),
    (dict(head_dim=96), sa.SPEC_ATTN_E_UNSUPPORTED),
    (dict(total_kv_rows=-1), sa.SPEC_ATTN_E_INVALID_ARG),
    (dict(total_q_rows=2 ** 30 + 1), sa.SPEC_ATTN_E_UNSUPPORTED),
    (dict(total_kv_rows=2 ** 30 + 1), sa.SPEC_ATTN_E_UNSUPPORTED),
    (dict(max_kv_len=-1), sa.SPEC_ATTN_E_INVALID_ARG),
    (dict(sm_scale=-0.5), sa.SPEC_ATTN_E_INVALID_ARG),
    (dict(sm_scale=float("nan")), sa.SPEC_ATTN_E_INVALID_ARG),
    (dict(force_splits=-1), sa.SPEC_ATTN_E_INVALID_ARG),
    (dict(force_splits=9), sa.SPEC_ATTN_E_UNSUPPORTED),           # a cluster has at most 8 CTAs
    (dict(kv_row_stride=248), sa.SPEC_ATTN_E_INVALID_ARG),      # below the dense row (256)
    (dict(kv_row_stride=260), sa.SPEC_ATTN_E_INVALID_ARG),      # not a multiple of 8
])
def test_cross_plan_refuses_bad_problems(lib, over, status):
    prob = dict(num_reqs=2, total_q_rows=8, max_q_rows=4, num_q_heads=8, num_kv_heads=2, head_dim=128,
                total_kv_rows=100, max_kv_len=60, sm_scale=0.0, force_splits=0, kv_row_stride=0)
    prob.update(over)
    pr = sa.spec_attn_cross_problem(*[prob[f[0]] for f in sa.spec_attn_cross_problem._fields_])
    h = ctypes.c_void_p()
    assert lib.spec_attn_cross_plan_create(ctypes.byref(pr), ctypes.byref(h), None) == status
    assert not h.value


def test_cross_null_arguments(lib):
    assert lib.spec_attn_cross_plan_create(None, None, None) == sa.SPEC_ATTN_E_INVALID_ARG
    assert lib.spec_attn_run_cross(*([None] * 10), 0, None) == sa.SPEC_ATTN_E_INVALID_ARG
    assert lib.spec_attn_cross_plan_destroy(None) == sa.SPEC_ATTN_OK
