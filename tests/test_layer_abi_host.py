"""Host-side checks of include/tk_layer.h that need no GPU: strict C99, every
declared symbol exported and bound, bad arguments rejected before any HIP call
(fake, never-dereferenced device addresses)."""
import os
import re
import subprocess

import pytest

import moe_activation_bit_amd as tk

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "tk_layer.h")
OK, INVALID, UNSUPPORTED = tk.TkStatus.TK_OK, tk.TkStatus.TK_ERR_INVALID_ARG, tk.TkStatus.TK_ERR_UNSUPPORTED
INF, NAN = float("inf"), float("nan")
A, B, C, D, E, F, G, H = (0x7000_0000_0000 + i * 0x0100_0000_0000 for i in range(8))


def test_header_is_strict_c99_and_its_symbols_are_bound(tmp_path):
    src = tmp_path / "h.c"
    src.write_text('#include "tk_layer.h"\nint main(void) { return TK_SCORE_SIGMOID + TK_DTYPE_FP8 == 0; }\n')
    subprocess.run(["gcc", "-std=c99", "-pedantic", "-Wall", "-Wextra", "-Werror", "-fsyntax-only",
                    "-I" + os.path.join(ROOT, "include"), str(src)], check=True)
    text = open(HEADER).read()
    names = sorted(set(re.findall(r"^tk_status (tk_\w+)\(", text, re.M)))
    assert names == ["tk_expert_gemv_fp4", "tk_rmsnorm_backward", "tk_rmsnorm_cast_fp8", "tk_route",
                     "tk_route_backward"]
    lib = tk.load_library()
    for name in names:
        assert hasattr(lib, name) and name in tk.SIGNATURES and name in tk.__all__ and callable(getattr(tk, name))
    assert tk.TK_RMSNORM_PARTS == int(re.search(r"#define TK_RMSNORM_PARTS (\d+)", text).group(1))
    assert tk.TK_DTYPE_FP8 == int(re.search(r"#define TK_DTYPE_FP8 (\d+)", text).group(1))


def norm(**kw):
    a = dict(x=A, residual=B, in_dtype=0, weight=C, n=4, hidden=1024, eps=1e-6, group_size=128, scale_fmt=0,
             residual_out=D, y=E, rstd=F, codes=G, scales=H, stream=0)
    a.update(kw)
    return tk.tk_rmsnorm_cast_fp8(**a)


@pytest.mark.parametrize("kw", [
    dict(n=-1), dict(n=2 ** 31), dict(hidden=0), dict(hidden=12), dict(hidden=-8), dict(in_dtype=2), dict(in_dtype=-1),
    dict(eps=-1e-6), dict(eps=NAN), dict(eps=INF), dict(group_size=-8), dict(group_size=12), dict(group_size=96),
    dict(scale_fmt=5), dict(scale_fmt=-1), dict(x=None), dict(weight=None), dict(codes=None), dict(scales=None),
    dict(codes=None, scales=None, residual_out=None, y=None, rstd=None), dict(x=A + 8), dict(residual=B + 4),
    dict(weight=C + 4), dict(residual_out=D + 8), dict(y=E + 2), dict(rstd=F + 2), dict(codes=G + 4),
    dict(scales=H + 2), dict(scales=H + 4, scale_fmt=tk.TK_SCALE_FP32_COLMAJOR), dict(residual_out=A + 16),
    dict(y=A), dict(codes=B + 64), dict(rstd=C), dict(scales=G + 8), dict(y=D + 32), dict(y=B),
], ids=str)
def test_norm_invalid_arguments(kw):
    assert norm(**kw) == INVALID


def test_norm_empty_and_unsupported():
    assert norm(n=0) == OK
    assert norm(n=0, x=None, weight=None, codes=None, scales=None, residual_out=None, y=None, rstd=None) == OK
    assert norm(n=0, residual_out=A) == OK
    assert norm(hidden=32776, group_size=0) == UNSUPPORTED
    assert norm(n=0, hidden=32768, group_size=0, in_dtype=1) == OK


def norm_bwd(**kw):
    a = dict(dy=A, h=B, in_dtype=0, weight=C, rstd=D, dresidual=E, n=4, hidden=1024, dx=F, dweight=G, workspace=H,
             stream=0)
    a.update(kw)
    return tk.tk_rmsnorm_backward(**a)


@pytest.mark.parametrize("kw", [
    dict(n=-1), dict(n=2 ** 31), dict(hidden=0), dict(hidden=20), dict(in_dtype=2), dict(dy=None), dict(h=None),
    dict(weight=None), dict(rstd=None), dict(dx=None), dict(workspace=None), dict(dy=A + 8), dict(h=B + 2),
    dict(weight=C + 8), dict(rstd=D + 2), dict(dresidual=E + 4), dict(dx=F + 8), dict(dweight=G + 4),
    dict(workspace=H + 8), dict(dx=B), dict(dx=A + 16), dict(dweight=C), dict(workspace=G + 64), dict(workspace=F),
], ids=str)
def test_norm_backward_invalid_arguments(kw):
    assert norm_bwd(**kw) == INVALID


def test_norm_backward_empty_and_unsupported():
    assert norm_bwd(n=0, dweight=None) == OK  # nothing to write, no launch
    assert norm_bwd(n=0, dweight=None, dx=A) == OK
    assert norm_bwd(hidden=32776) == UNSUPPORTED


def route(**kw):
    a = dict(logits=A, in_dtype=1, bias=B, tokens=4, experts=256, k=8, n_group=8, topk_group=4, scoring=0, normalise=1,
             scale=2.5, topk_idx=C, topk_weight=D, stream=0)
    a.update(kw)
    return tk.tk_route(**a)


@pytest.mark.parametrize("kw", [
    dict(tokens=-1), dict(tokens=2 ** 31), dict(experts=0), dict(k=0), dict(k=257), dict(in_dtype=2), dict(scoring=2),
    dict(scoring=-1), dict(n_group=0), dict(n_group=3), dict(topk_group=0), dict(topk_group=9), dict(k=129),
    dict(experts=8, n_group=8, topk_group=8, k=2), dict(scale=NAN), dict(scale=INF), dict(logits=None),
    dict(topk_idx=None), dict(topk_weight=None), dict(logits=A + 2), dict(logits=A + 1, in_dtype=0), dict(bias=B + 2),
    dict(topk_idx=C + 2), dict(topk_weight=D + 1), dict(topk_idx=A + 64), dict(topk_weight=B), dict(topk_weight=C + 8),
], ids=str)
def test_route_invalid_arguments(kw):
    assert route(**kw) == INVALID


def test_route_empty_and_unsupported():
    assert route(tokens=0) == OK
    assert route(tokens=0, logits=None, bias=None, topk_idx=None, topk_weight=None) == OK
    assert route(experts=576, n_group=8) == UNSUPPORTED
    assert route(experts=256, n_group=1, topk_group=1, k=65) == UNSUPPORTED
    assert route(tokens=0, in_dtype=0, logits=A + 2) == OK


def route_bwd(**kw):
    a = dict(dweight=A, topk_idx=B, logits=C, in_dtype=1, tokens=4, experts=256, k=8, scoring=0, normalise=1, scale=2.5,
             dlogits=D, stream=0)
    a.update(kw)
    return tk.tk_route_backward(**a)


@pytest.mark.parametrize("kw", [
    dict(tokens=-1), dict(experts=0), dict(k=0), dict(k=257), dict(in_dtype=3), dict(scoring=2), dict(scale=-INF),
    dict(dweight=None), dict(topk_idx=None), dict(logits=None), dict(dlogits=None), dict(dweight=A + 2),
    dict(topk_idx=B + 1), dict(logits=C + 2), dict(dlogits=D + 2), dict(dlogits=C), dict(dlogits=A), dict(dlogits=B + 16),
], ids=str)
def test_route_backward_invalid_arguments(kw):
    assert route_bwd(**kw) == INVALID


def test_route_backward_empty_and_unsupported():
    assert route_bwd(tokens=0) == OK
    assert route_bwd(experts=513) == UNSUPPORTED
    assert route_bwd(k=65) == UNSUPPORTED


def gemv(**kw):
    a = dict(x=A, x_scales=B, x_dtype=tk.TK_DTYPE_FP8, x_scale_fmt=0, x_group=128, topk_idx=C, tokens=4, k=8, x_slots=0,
             codes=D, scales=E, scale_fmt=1, group_size=32, experts=16, out_features=512, in_features=1024, out_dtype=0,
             out=F, stream=0)
    a.update(kw)
    return tk.tk_expert_gemv_fp4(**a)


@pytest.mark.parametrize("kw", [
    dict(x_dtype=1), dict(x_dtype=3), dict(out_dtype=2), dict(scale_fmt=5), dict(scale_fmt=-1), dict(x_scale_fmt=9),
    dict(tokens=-1), dict(k=0), dict(tokens=2 ** 28), dict(topk_idx=None), dict(experts=0), dict(experts=32769),
    dict(out_features=0), dict(out_features=2 ** 24 + 1), dict(in_features=0), dict(in_features=1040), dict(in_features=-32),
    dict(group_size=-32), dict(group_size=96), dict(x_group=-128), dict(x_group=384), dict(x=None), dict(x_scales=None),
    dict(codes=None), dict(scales=None), dict(out=None), dict(x=A + 8), dict(codes=D + 8), dict(topk_idx=C + 2),
    dict(out=F + 1), dict(out=F + 2, out_dtype=1), dict(scales=E + 2, scale_fmt=0, group_size=128), dict(x_scales=B + 2),
    dict(out=A), dict(out=D + 32), dict(out=E), dict(out=C), dict(out=B),
], ids=str)
def test_gemv_invalid_arguments(kw):
    assert gemv(**kw) == INVALID


def test_gemv_empty_and_unsupported():
    assert gemv(tokens=0) == OK
    assert gemv(tokens=0, k=1, topk_idx=None, x_dtype=0, x_scales=None, x_group=7) == OK
    assert gemv(k=65) == UNSUPPORTED
    assert gemv(group_size=16) == UNSUPPORTED
    assert gemv(group_size=32, scale_fmt=0) == UNSUPPORTED
    assert gemv(x_group=32) == UNSUPPORTED
    assert gemv(tokens=0, x_group=32, x_scale_fmt=1) == OK
    for fmt in (tk.TK_SCALE_FP32_COLMAJOR, tk.TK_SCALE_UE8M0_COLMAJOR, tk.TK_SCALE_UE8M0_PACKED):
        assert gemv(scale_fmt=fmt) == UNSUPPORTED and gemv(x_scale_fmt=fmt) == UNSUPPORTED


def test_no_norm_kernel_that_no_call_reaches():
    """Four steps a wave means more than 32 of them in a row, so nine waves or more: no form for 256 threads."""
    names = set(re.findall(rb"rmsnorm_cast_kernelILb[01]ELi(\d)ELi\dELi\dELi(\d+)EE", open(tk.LIB_PATH, "rb").read()))
    assert names == {(b"1", b"256"), (b"1", b"1024"), (b"2", b"256"), (b"2", b"1024"), (b"4", b"1024")}


@pytest.mark.parametrize("gone", ["_cuda_getCurrentRawStream", "_cuda_getDevice"])
def test_the_default_stream_without_torchs_private_functions(monkeypatch, gone):
    import types

    import torch
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: types.SimpleNamespace(cuda_stream=77))
    monkeypatch.delattr(torch._C, gone, raising=False)
    assert tk._current_stream() == 77
