"""The operators of include/tk_expert.h at the ends of what they take."""
import numpy as np
import pytest
import torch

import expert_ref as ex
import layer_ref as ref
import moe_activation_bit_amd as tk
import test_gpu_expert_products as products

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
OK = tk.TkStatus.TK_OK
BF16, FP32, FP8, FP4 = tk.TK_DTYPE_BF16, tk.TK_DTYPE_FP32, tk.TK_DTYPE_FP8, tk.TK_DTYPE_FP4
INF = float("inf")


def say(*a):
    print("[gpu-case]", *a, flush=True)


@pytest.mark.parametrize("gather_dy", [False, True])
@pytest.mark.parametrize("out_f,in_f,group", [(264, 256, 0), (264, 256, 32), (136, 64, 0), (136, 64, 8)], ids=str)
def test_wgrad_rows_of_none_take_no_scale(out_f, in_f, group, gather_dy):
    """An entry of x_index that names no row is a row of zeros whatever the scales of x's first row are; a NaN
    among the scales reaches the columns of its group in the experts that have its row."""
    say("scales of rows of none", out_f, in_f, group, gather_dy)
    rng = np.random.default_rng(out_f + group + gather_dy)
    counts = [30, 70, 41]
    off, n, x_rows = products.offsets_of(counts), sum(counts), 37
    index = rng.integers(1, x_rows, n).astype(np.int32)  # nobody's: row 0
    index[[3, 29, 30, 64, 99, 140]] = [-1, x_rows, -1, 2 ** 31 - 1, -2 ** 31, -1]
    index[index == 36] = 1  # the last expert's alone
    index[120] = 36
    codes = products.whole_codes(rng, (x_rows, in_f))
    scales = rng.integers(125, 130, (x_rows, in_f // (group or in_f))).astype(np.uint8)
    scales[0], scales[36, 0] = 255, 255
    dy_rows = 19 if gather_dy else n
    dyi = rng.integers(0, dy_rows, n).astype(np.int32) if gather_dy else None
    dy = products.whole(rng, (dy_rows, out_f))
    dy[dy == 0] = 1
    x = ex.coded(codes, scales, True)
    with np.errstate(invalid="ignore"):
        want = ex.wgrad(dy, dyi, x, index, off, n, np.zeros((3, out_f, in_f)))[0]
    dw = torch.ones((3, out_f, in_f), device=DEV)
    assert tk.tk_expert_gemm_wgrad(products.bf16(dy), dy_rows, products.dev(dyi), products.dev(codes), products.dev(scales),
                                   FP8, group, x_rows, products.dev(index), products.dev(off), n, 3, out_f, in_f, 0, FP32,
                                   dw) == OK
    got = products.host(dw, False)
    first = group or in_f
    assert np.isfinite(want[:2]).all() and np.isnan(want[2, :, :first]).all() and np.isfinite(want[2, :, first:]).all()
    assert np.array_equal(got, want.astype(np.float32), equal_nan=True)


def backward_rows(n, hidden, fp8, gen):
    """n rows of dy and h, few distinct ones, on the device."""
    dy = torch.randn((64, hidden), generator=gen, device=DEV).to(torch.bfloat16)
    dy = dy.repeat((n + 63) // 64, 1)[:n].contiguous()
    if fp8:
        h = torch.randint(0, 120, (64, 2 * hidden), generator=gen, device=DEV, dtype=torch.uint8)
        scales = torch.randint(110, 125, (n, 1), generator=gen, device=DEV, dtype=torch.uint8)
    else:
        h, scales = torch.randn((64, 2 * hidden), generator=gen, device=DEV).to(torch.bfloat16), None
    return dy, h.repeat((n + 63) // 64, 1)[:n].contiguous(), scales


@pytest.mark.parametrize("n,hidden,fp8", [(2 ** 26 + 5, 8, True), (2 ** 22 + 7, 8, False), (2 ** 21 + 3, 520, True),
                                          (2 ** 20 + 9, 1032, True)], ids=str)
def test_backward_of_more_rows_than_workgroups(n, hidden, fp8):
    """2^32 work-items are the most that a launch holds: rows beyond the grid's are taken by the same workgroups."""
    say("backward rows", n, hidden, fp8)
    gen = torch.Generator(device=DEV).manual_seed(n)
    dy, h, scales = backward_rows(n, hidden, fp8, gen)
    weight = torch.rand(n, generator=gen, device=DEV)
    kind, fmt, group = (FP8, 1, 0) if fp8 else (BF16, 0, 0)

    def outputs(rows):
        return (torch.zeros((rows, 2 * hidden), dtype=torch.bfloat16, device=DEV), torch.zeros(rows, device=DEV),
                torch.zeros((rows, hidden), dtype=torch.bfloat16, device=DEV))

    whole = outputs(n)
    assert tk.tk_swiglu_backward(dy, h, scales, kind, fmt, group, weight, n, hidden, 2.0, *whole) == OK
    most = 1 << 19  # rows that one pass of the grid takes at any width
    part = outputs(most)
    for lo in range(0, n, most):
        rows = min(most, n - lo)
        assert tk.tk_swiglu_backward(dy[lo:], h[lo:], scales[lo:] if fp8 else None, kind, fmt, group, weight[lo:], rows,
                                     hidden, 2.0, *part) == OK
        for a, b in zip(whole, part):
            assert torch.equal(a[lo:lo + rows], b[:rows])


@pytest.mark.parametrize("clamp", [INF, 2.5])
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("n,hidden,group", [(37, 1024, 128), (5, 520, 8), (64, 96, 32), (130, 1536, 512),
                                            (16390, 2048, 128)])
def test_checkpoint_has_the_bits_of_two_calls_with_nan_too(n, hidden, group, fmt, clamp):
    """A NaN or an infinity among the inputs leaves what the two calls leave, in its group and in the others."""
    say("checkpoint NaN", n, hidden, group, fmt, clamp)
    gen = torch.Generator(device=DEV).manual_seed(n + hidden)
    x = (torch.randn((n, 2 * hidden), generator=gen, device=DEV) * 3).to(torch.bfloat16)
    at = torch.rand(x.shape, generator=gen, device=DEV)
    for i, bits in enumerate((0x7FC0, 0x7F81, -0x40, 0x7F80, -0x80)):  # NaN of either sign, infinities
        x.view(torch.int16).masked_fill_((at >= i * 3e-3) & (at < (i + 1) * 3e-3), bits)
    weight = torch.rand(n, generator=gen, device=DEV)

    def buffers(cols):
        return (torch.full((n + 1, cols), 0xA5, dtype=torch.uint8, device=DEV),
                torch.full((n + 1, cols // group), 77, dtype=torch.uint8 if fmt else torch.float32, device=DEV))

    (c0, s0), (c1, s1) = buffers(hidden), buffers(hidden)
    (xc0, xs0), (xc1, xs1) = buffers(2 * hidden), buffers(2 * hidden)
    assert tk.tk_swiglu_cast_fp8(x, weight, n, hidden, group, clamp, fmt, c0, s0) == OK
    assert tk.tk_cast_fp8(x, 0, n, 2 * hidden, group, fmt, xc0, xs0) == OK
    assert tk.tk_swiglu_checkpoint_fp8(x, weight, n, hidden, group, clamp, fmt, c1, s1, xc1, xs1) == OK
    torch.cuda.synchronize()
    for a, b in ((c0, c1), (s0, s1), (xc0, xc1), (xs0, xs1)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_no_rows_and_no_address():
    """x or dy of no rows has no address (torch's is 0): every index names none, every result is zero."""
    off = products.dev(np.array([0, 70, 80], np.int32))
    index = products.dev(np.arange(80, dtype=np.int32))
    none = torch.empty((0, 64), dtype=torch.bfloat16, device=DEV)
    codes = torch.empty((0, 64), dtype=torch.uint8, device=DEV)
    scales = torch.empty((0, 2), dtype=torch.uint8, device=DEV)
    assert none.data_ptr() == codes.data_ptr() == scales.data_ptr() == 0
    w = torch.ones((2, 64, 64), dtype=torch.bfloat16, device=DEV)
    y = torch.ones((80, 64), device=DEV)
    assert tk.tk_expert_gemm(none, None, BF16, 0, 0, 0, index, off, 80, w, None, BF16, 0, 0, 2, 64, 64, FP32, y) == OK
    assert not y.any()
    y.fill_(1)
    assert tk.tk_expert_gemm_dgrad(none, 0, index, off, 80, w, 2, 64, 64, FP32, y) == OK
    assert not y.any()
    w8 = torch.full((128, 64), 0x38, dtype=torch.uint8, device=DEV)
    for x_group, w_group in ((32, 32), (0, 32), (32, 0)):
        ws = torch.full((128, 64 // (w_group or 64)), 127, dtype=torch.uint8, device=DEV)
        out = torch.ones((80, 64), dtype=torch.bfloat16, device=DEV)
        assert tk.tk_expert_gemm(codes, scales, FP8, 1, x_group, 0, index, off, 80, w8, ws, FP8, 1, w_group, 2, 64, 64,
                                 BF16, out) == OK
        assert not out.any()
    dy = torch.ones((80, 64), dtype=torch.bfloat16, device=DEV)
    start = torch.arange(2 * 64 * 64, device=DEV, dtype=torch.float32).view(2, 64, 64)
    for accumulate in (0, 1):
        for args in ((dy, 80, None, none, None, BF16, 0, 0, index), (none, 0, index, dy, None, BF16, 0, 80, None),
                     (dy, 80, None, codes, scales, FP8, 32, 0, index), (none, 0, index, none, None, BF16, 0, 0, index)):
            dw = start.clone()
            assert tk.tk_expert_gemm_wgrad(*args, off, 80, 2, 64, 64, accumulate, FP32, dw) == OK
            assert torch.equal(dw, start if accumulate else torch.zeros_like(start))


@pytest.mark.parametrize("counts,out_f", [([9, 5], 72), ([90, 40], 1032), ([300, 90], 8200)], ids=str)
@pytest.mark.parametrize("x_group,w_group", [(0, 0), (32, 32), (0, 32), (128, 0), (64, 64)], ids=str)
def test_gemm_scale_bytes_at_the_ends(x_group, w_group, counts, out_f):
    """Scales of 2^-127 to 2^127 against each other, over every tile size: the product of a row's two scales is
    anything that a result of normal size may have (of groups against one a row, which the sum with the groups' scales
    meets later, those that leave this sum in fp32's range); byte 255 is a NaN in its row (its column) alone."""
    say("scale bytes", x_group, w_group, counts, out_f)
    rng = np.random.default_rng(out_f + x_group + w_group)
    off, n, e, in_f = products.offsets_of(counts), sum(counts), 2, 512


    def operand(rows, first, small, large, group, other):
        """Scale bytes of the rows of expert 0 (`first` of them) and of expert 1."""
        byte = np.array([(small if r < first else large)[r % len(small)] for r in range(rows)])
        if group and not other:
            byte = np.clip(byte, 20, 227)
        scales = np.repeat(byte[:, None], in_f // (group or in_f), 1).astype(np.uint8)
        scales[3] = 255
        codes = products.whole_codes(rng, (rows, in_f))
        return codes, scales, ex.coded(codes, scales, True)

    xc, xs, x = operand(n, counts[0], (0, 3, 60), (254, 251, 200), x_group, w_group)
    wc, ws, w = operand(e * out_f, out_f, (254, 190), (0, 40), w_group, x_group)
    out = torch.zeros((n, out_f), dtype=torch.int16, device=DEV)
    assert tk.tk_expert_gemm(products.dev(xc), products.dev(xs), FP8, 1, x_group, n, None, products.dev(off), n,
                             products.dev(wc), products.dev(ws), FP8, 1, w_group, e, out_f, in_f, BF16, out) == OK
    got = products.host(out, True)
    with np.errstate(all="ignore"):
        want = np.concatenate([x[lo:hi] @ w[i * out_f:(i + 1) * out_f].T for i, (lo, hi) in enumerate(ex.spans(off, n))])
        want = ref.round_bf16(want.astype(np.float32))  # whole numbers times powers of two: exact before the rounding
    normal = np.isnan(want) | (want == 0) | (np.abs(want) >= 2.0 ** -126)
    assert np.isnan(want).sum() > n and normal.mean() > 0.9
    assert np.array_equal(got[normal], want[normal], equal_nan=True)


@pytest.mark.parametrize("out_f,in_f,group", [(200, 256, 0), (200, 256, 16), (24, 256, 0), (24, 256, 8)], ids=str)
def test_wgrad_scale_bytes_at_the_ends(out_f, in_f, group):
    """Every code under every scale byte, one row an expert: the value as bf16 holds it (below 2^-133 rounded, from
    2^128 on infinite, byte 255 a NaN) times a power of two."""
    say("wgrad scale bytes", out_f, in_f, group)
    codes = np.tile(np.arange(256, dtype=np.uint8), (256, 1))
    scales = np.repeat(np.arange(256, dtype=np.uint8)[:, None], in_f // (group or in_f), 1)
    off = np.arange(257, dtype=np.int32)
    for power in (0, 40, -40):
        dy = np.full((256, out_f), 2.0 ** power, np.float32)
        dw = torch.zeros((256, out_f, in_f), device=DEV)
        assert tk.tk_expert_gemm_wgrad(products.bf16(dy), 256, None, products.dev(codes), products.dev(scales), FP8, group,
                                       256, None, products.dev(off), 256, 256, out_f, in_f, 0, FP32, dw) == OK
        got = products.host(dw, False)
        with np.errstate(all="ignore"):
            x = ref.round_bf16(ex.coded(codes, scales, True).astype(np.float32))
            want = (x.astype(np.float64) * 2.0 ** power).astype(np.float32)
        for row in range(256):
            for o in (0, out_f - 1):
                assert np.array_equal(got[row, o], want[row], equal_nan=True), (power, row, o)
