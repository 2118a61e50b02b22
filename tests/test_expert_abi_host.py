"""Host-side checks of include/tk_expert.h that need no GPU: strict C99, every
declared symbol exported and bound, bad arguments rejected before any HIP call
(fake, never-dereferenced device addresses)."""
import inspect
import os
import re
import subprocess

import pytest

import moe_activation_bit_amd as tk

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "tk_expert.h")
OK, INVALID, UNSUPPORTED = tk.TkStatus.TK_OK, tk.TkStatus.TK_ERR_INVALID_ARG, tk.TkStatus.TK_ERR_UNSUPPORTED
INF, NAN = float("inf"), float("nan")
BF16, FP32, FP8, FP4 = tk.TK_DTYPE_BF16, tk.TK_DTYPE_FP32, tk.TK_DTYPE_FP8, tk.TK_DTYPE_FP4
A, B, C, D, E, F, G, H = (0x7000_0000_0000 + i * 0x0100_0000_0000 for i in range(8))


def test_header_is_strict_c99_and_its_symbols_are_bound(tmp_path):
    src = tmp_path / "h.c"
    src.write_text('#include "tk_expert.h"\nint main(void) { return TK_DTYPE_FP4 == TK_DTYPE_FP8; }\n')
    subprocess.run(["gcc", "-std=c99", "-pedantic", "-Wall", "-Wextra", "-Werror", "-fsyntax-only",
                    "-I" + os.path.join(ROOT, "include"), str(src)], check=True)
    text = open(HEADER).read()
    declared = {m.group(1): m.group(2) for m in re.finditer(r"^tk_status (tk_\w+)\(([^;]*)\);", text, re.M)}
    assert sorted(declared) == ["tk_expert_gemm", "tk_expert_gemm_dgrad", "tk_expert_gemm_wgrad",
                                "tk_swiglu_backward", "tk_swiglu_checkpoint_fp8"]
    lib = tk.load_library()
    for name, args in declared.items():
        assert hasattr(lib, name) and name in tk.SIGNATURES and name in tk.__all__
        names = [a.split()[-1].lstrip("*") for a in args.replace("\n", " ").split(",")]
        assert names == list(inspect.signature(getattr(tk, name)).parameters)
        assert len(names) == len(tk.SIGNATURES[name][1])
    assert tk.TK_DTYPE_FP4 == int(re.search(r"#define TK_DTYPE_FP4 (\d+)", text).group(1))


def gemm(**kw):
    a = dict(x=A, x_scales=B, x_dtype=FP8, x_scale_fmt=1, x_group=128, x_rows=16, row_index=C, expert_offsets=D,
             n_rows=64, w=E, w_scales=F, w_dtype=FP4, w_scale_fmt=1, w_group=32, experts=8, out_features=512,
             in_features=1024, out_dtype=BF16, out=G, stream=0)
    a.update(kw)
    return tk.tk_expert_gemm(**a)


def plain(**kw):
    return gemm(**dict(dict(x_scales=None, x_dtype=BF16, w_scales=None, w_dtype=BF16), **kw))


@pytest.mark.parametrize("kw", [
    dict(n_rows=-1), dict(n_rows=2 ** 31), dict(x_rows=-1), dict(x_rows=2 ** 31), dict(experts=0), dict(experts=-1),
    dict(out_features=0), dict(out_features=12), dict(out_features=-8), dict(in_features=0), dict(in_features=24),
    dict(out_features=2 ** 20 + 8), dict(in_features=2 ** 20 + 32), dict(x_dtype=FP32), dict(x_dtype=FP4),
    dict(x_dtype=-1), dict(w_dtype=FP32), dict(w_dtype=4), dict(out_dtype=FP8), dict(out_dtype=-1),
    dict(x_scale_fmt=5), dict(w_scale_fmt=-1), dict(x_group=-128), dict(x_group=96), dict(w_group=48),
    dict(x=None), dict(x_scales=None), dict(w=None), dict(w_scales=None), dict(out=None), dict(expert_offsets=None),
    dict(row_index=None), dict(x=A + 8), dict(w=E + 8), dict(out=G + 8), dict(row_index=C + 2),
    dict(expert_offsets=D + 1), dict(x_scale_fmt=0, x_scales=B + 2), dict(w_scale_fmt=0, w_group=128, w_scales=F + 1),
    dict(out=A), dict(out=B), dict(out=C), dict(out=D), dict(out=E + 1024), dict(out=F + 16),
], ids=str)
def test_gemm_invalid_arguments(kw):
    assert gemm(**kw) == INVALID


@pytest.mark.parametrize("kw", [dict(in_features=1028), dict(x=None), dict(w=None), dict(out=A + 64), dict(x=A + 2)],
                         ids=str)
def test_gemm_bf16_invalid_arguments(kw):
    assert plain(**kw) == INVALID


@pytest.mark.parametrize("kw", [
    dict(experts=513), dict(x_dtype=BF16), dict(w_dtype=BF16), dict(out_dtype=FP32), dict(x_scale_fmt=2),
    dict(w_scale_fmt=4), dict(x_group=16), dict(w_group=8), dict(x_scale_fmt=0, x_group=64),
    dict(w_scale_fmt=0, w_group=32),
], ids=str)
def test_gemm_unsupported(kw):
    assert gemm(**kw) == UNSUPPORTED


def test_gemm_empty():
    assert gemm(n_rows=0) == OK
    assert gemm(n_rows=0, x_rows=0, x=None, x_scales=None, w=None, w_scales=None, out=None, row_index=None) == OK
    assert plain(n_rows=0, out_dtype=FP32, x_scale_fmt=9, w_group=-5) == OK  # ignored for bf16
    assert gemm(n_rows=0, experts=1, expert_offsets=None) == OK


def dgrad(**kw):
    a = dict(dy=A, dy_rows=16, row_index=B, expert_offsets=C, n_rows=64, w=D, experts=8, out_features=512,
             in_features=1000, out_dtype=BF16, dx=E, stream=0)
    a.update(kw)
    return tk.tk_expert_gemm_dgrad(**a)


@pytest.mark.parametrize("kw", [
    dict(n_rows=-1), dict(dy_rows=-1), dict(experts=0), dict(out_features=4), dict(in_features=1001), dict(out_dtype=2),
    dict(dy=None), dict(w=None), dict(dx=None), dict(row_index=None), dict(expert_offsets=None), dict(dy=A + 2),
    dict(w=D + 8), dict(dx=E + 4), dict(row_index=B + 1), dict(dx=A), dict(dx=B), dict(dx=C + 16), dict(dx=D),
], ids=str)
def test_dgrad_invalid_arguments(kw):
    assert dgrad(**kw) == INVALID


def test_dgrad_empty_and_unsupported():
    assert dgrad(experts=513) == UNSUPPORTED
    assert dgrad(n_rows=0) == OK
    assert dgrad(n_rows=0, dy=None, w=None, dx=None, dy_rows=0, row_index=None) == OK


def wgrad(**kw):
    a = dict(dy=A, dy_rows=64, dy_index=None, x=B, x_scales=C, x_dtype=FP8, x_group=128, x_rows=16, x_index=D,
             expert_offsets=E, n_rows=64, experts=8, out_features=512, in_features=1024, accumulate=0, out_dtype=FP32,
             dw=F, stream=0)
    a.update(kw)
    return tk.tk_expert_gemm_wgrad(**a)


@pytest.mark.parametrize("kw", [
    dict(n_rows=-1), dict(dy_rows=-1), dict(dy_rows=63), dict(x_rows=-1), dict(x_index=None), dict(experts=0),
    dict(out_features=4), dict(in_features=1016), dict(x_dtype=FP4), dict(out_dtype=2), dict(x_group=-8), dict(x_group=96), dict(dy=None), dict(x=None), dict(x_scales=None),
    dict(dw=None), dict(expert_offsets=None), dict(dy=A + 8), dict(x=B + 8), dict(dw=F + 8), dict(x_index=D + 2),
    dict(dw=A), dict(dw=B), dict(dw=C), dict(dw=D), dict(dw=E), dict(dw=None, n_rows=0),
], ids=str)
def test_wgrad_invalid_arguments(kw):
    assert wgrad(**kw) == INVALID


def test_wgrad_accumulate_is_a_truth_value():
    lib = tk.load_library()
    assert lib.tk_expert_gemm_wgrad(A, 64, None, B, C, FP8, 128, 16, D, E, 64, 8, 512, 1024, 2, FP32, F, None) == INVALID


def test_wgrad_empty_and_unsupported():
    assert wgrad(experts=513) == UNSUPPORTED
    assert wgrad(x_group=4) == UNSUPPORTED
    assert wgrad(n_rows=0, accumulate=1) == OK
    assert wgrad(n_rows=0, accumulate=1, dy=None, x=None, x_scales=None, dy_rows=0) == OK


def checkpoint(**kw):
    a = dict(x=A, topk_weight=B, n=4, hidden=1024, group_size=128, clamp_limit=INF, scale_fmt=1, codes=C, scales=D,
             x_codes=E, x_scales=F, stream=0)
    a.update(kw)
    return tk.tk_swiglu_checkpoint_fp8(**a)


@pytest.mark.parametrize("kw", [
    dict(n=-1), dict(n=2 ** 31), dict(hidden=0), dict(hidden=12), dict(group_size=-8), dict(group_size=12),
    dict(group_size=96), dict(clamp_limit=0.0), dict(clamp_limit=-1.0), dict(clamp_limit=NAN), dict(scale_fmt=5),
    dict(scale_fmt=-1), dict(x=None), dict(codes=None), dict(scales=None), dict(x_codes=None), dict(x_scales=None),
    dict(x=A + 8), dict(topk_weight=B + 2), dict(codes=C + 4), dict(x_codes=E + 4), dict(scale_fmt=0, scales=D + 2),
    dict(scale_fmt=0, x_scales=F + 2), dict(codes=A), dict(scales=B), dict(x_codes=C + 8), dict(x_scales=E + 8191),
], ids=str)
def test_checkpoint_invalid_arguments(kw):
    assert checkpoint(**kw) == INVALID


def test_checkpoint_empty_and_unsupported():
    assert checkpoint(group_size=0) == UNSUPPORTED
    assert checkpoint(group_size=1024) == UNSUPPORTED
    assert checkpoint(hidden=960, group_size=96) == UNSUPPORTED
    assert checkpoint(scale_fmt=2, scales=D) == UNSUPPORTED
    assert checkpoint(n=0) == OK
    assert checkpoint(n=0, x=None, codes=None, scales=None, x_codes=None, x_scales=None, topk_weight=None) == OK


def backward(**kw):
    a = dict(dy=A, h=B, h_scales=C, h_dtype=FP8, scale_fmt=1, group_size=128, topk_weight=D, n=4, hidden=1024,
             clamp_limit=INF, dh=E, dweight=F, y=G, stream=0)
    a.update(kw)
    return tk.tk_swiglu_backward(**a)


@pytest.mark.parametrize("kw", [
    dict(n=-1), dict(n=2 ** 31), dict(hidden=0), dict(hidden=12), dict(hidden=2 ** 18 + 8), dict(h_dtype=FP32),
    dict(h_dtype=FP4), dict(clamp_limit=0.0), dict(clamp_limit=NAN), dict(scale_fmt=5), dict(scale_fmt=-1),
    dict(group_size=-8), dict(group_size=12), dict(group_size=96), dict(dy=None), dict(h=None), dict(h_scales=None),
    dict(dh=None), dict(dy=A + 8), dict(h=B + 8), dict(dh=E + 8), dict(y=G + 8), dict(dweight=F + 2),
    dict(topk_weight=D + 2), dict(scale_fmt=0, h_scales=C + 2), dict(dh=A), dict(dh=B), dict(dh=B, h_dtype=BF16, dy=B),
    dict(dh=B + 16, h_dtype=BF16), dict(y=A + 16), dict(y=B), dict(y=E + 64), dict(dweight=D), dict(dweight=C),
], ids=str)
def test_backward_invalid_arguments(kw):
    assert backward(**kw) == INVALID


def test_backward_empty_and_unsupported():
    assert backward(scale_fmt=2) == UNSUPPORTED
    assert backward(n=0) == OK
    assert backward(n=0, h_dtype=BF16, dh=B, y=A, h_scales=None, scale_fmt=7) == OK
    assert backward(n=0, dy=None, h=None, h_scales=None, dh=None, dweight=None, y=None, topk_weight=None) == OK


def test_more_tiles_than_a_launch_holds():
    """Refused before any HIP call, whichever tiles the sizes choose."""
    far = 1 << 60
    for rows, columns in ((2 ** 31 - 1, 2 ** 20), (2 ** 31 - 1, 2 ** 17)):
        assert gemm(n_rows=rows, out_features=columns, out=far) == UNSUPPORTED
        assert plain(n_rows=rows, out_features=columns, out=far) == UNSUPPORTED
        assert dgrad(n_rows=rows, in_features=columns, dx=far) == UNSUPPORTED
    assert plain(n_rows=2 ** 28, experts=512, out_features=2 ** 20, out=far, x_rows=2 ** 28) == UNSUPPORTED
    assert wgrad(experts=512, out_features=2 ** 20, in_features=2 ** 20, dw=far, x_group=0) == UNSUPPORTED
