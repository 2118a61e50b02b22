"""The kernels of include/tk_expert.h that the sizes of the other tests do not
choose: every number of row blocks and several turns of scales in the products
of codes, steps cut short in their larger tiles, the weights' gradient with both
indices and with none, the checkpoint's launches of four steps a wave."""
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


def values(codes, scales, u8, fp4):
    """ex.coded on the device, in 64 bits."""
    if fp4:
        table = torch.from_numpy(ref.E2M1).to(DEV)
        v = torch.stack([table[(codes & 15).int()], table[(codes >> 4).int()]], -1).flatten(1)
    else:
        v = torch.from_numpy(ex.E4M3).to(DEV)[codes.int()]
    s = torch.from_numpy(ref.e8m0_value(np.arange(256))).to(DEV)[scales.int()] if u8 else scales.double()
    return v * s.repeat_interleave(v.shape[1] // s.shape[1], 1)


def operand(gen, rows, cols, kind, group, fp4=False):
    """Codes of whole (FP4: half) numbers with power-of-two scales 2^-1 .. 2, and their values."""
    if fp4:
        codes = torch.randint(0, 256, (rows, cols // 2), generator=gen, device=DEV, dtype=torch.uint8)
    else:
        whole = torch.tensor([0x00, 0x38, 0x40, 0x44, 0x48, 0xB8, 0xC0, 0xC4, 0xC8], dtype=torch.uint8, device=DEV)
        codes = whole[torch.randint(0, 9, (rows, cols), generator=gen, device=DEV)]
    power = torch.randint(0, 3, (rows, cols // (group or cols)), generator=gen, device=DEV)
    u8 = kind == "ue8m0"
    scales = (power + 126).to(torch.uint8) if u8 else torch.tensor([0.5, 1.0, 2.0], device=DEV)[power]
    return codes, scales, values(codes, scales, u8, fp4)


def check_codes(seed, counts, out_f, in_f, x_kind, w_kind, fp4):
    """The product of every row, some found by an index, bit for bit: no sum is rounded before bf16 (of 128 products
    the smallest unit is 2^-3 and the largest 96, well within what the instruction keeps)."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    rng = np.random.default_rng(seed)
    off, n, e = products.offsets_of(counts, 1), sum(counts) + 4, len(counts)
    xc, xs, x = operand(gen, n, in_f, *x_kind)
    wc, ws, w = operand(gen, e * out_f, in_f, *w_kind, fp4=fp4)
    w = w.view(e, out_f, in_f)
    for index in (None, products.index_of(rng, n, n, True)):
        out = torch.full((n, out_f), 7.0, dtype=torch.bfloat16, device=DEV)
        want = out.double()
        for i, (lo, hi) in enumerate(ex.spans(off, n)):
            if index is None:
                rows = x[lo:hi]
            else:
                at = torch.from_numpy(index[lo:hi].astype(np.int64)).to(DEV)
                good = (at >= 0) & (at < n)
                rows = torch.where(good[:, None], x[torch.where(good, at, 0)], 0.0)
            want[lo:hi] = rows @ w[i].t().contiguous()
        assert tk.tk_expert_gemm(xc, xs, FP8, 1 if x_kind[0] == "ue8m0" else 0, x_kind[1], n, products.dev(index),
                                 products.dev(off), n, wc, ws, FP4 if fp4 else FP8, 1 if w_kind[0] == "ue8m0" else 0,
                                 w_kind[1], e, out_f, in_f, BF16, out) == OK
        assert torch.equal(want.float().double(), want)  # the case's sums fit fp32
        assert torch.equal(out, want.float().to(torch.bfloat16))


U0, U32, U128, F0, F128, F256 = (("ue8m0", 0), ("ue8m0", 32), ("ue8m0", 128), ("fp32", 0), ("fp32", 128), ("fp32", 256))
PAIRS = [(U128, U128), (U128, U32), (U32, U128), (U32, U32), (F128, F128), (F256, F128), (F0, F0), (U0, F0), (U128, U0),
         (F0, U128), (F128, U32), (U128, F128)]


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("x_kind,w_kind", PAIRS, ids=str)
def test_codes_every_number_of_row_blocks(x_kind, w_kind, fp4):
    """256 x 256 tiles with one to eight blocks of 32 rows; 8 steps of scales (two turns) and 12 (three)."""
    say("row blocks of codes", x_kind, w_kind, fp4)
    for in_f in (1024, 1536):
        check_codes(in_f + fp4, [20, 64, 96, 130, 160, 161, 223, 256, 290], 4104, in_f, x_kind, w_kind, fp4)


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("x_kind,w_kind", PAIRS, ids=str)
def test_codes_several_turns_in_smaller_tiles(x_kind, w_kind, fp4):
    say("turns of codes", x_kind, w_kind, fp4)
    check_codes(1 + fp4, [33, 64, 0, 65, 40, 71], 2824, 1536, x_kind, w_kind, fp4)  # 128 columns x 64 rows
    check_codes(3 + fp4, [0, 17, 16, 0, 2], 72, 2560, x_kind, w_kind, fp4)          # 64 x 16


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("in_f", [32, 288, 416, 672, 1184])
@pytest.mark.parametrize("x_kind,w_kind", [(F0, F0), (U0, U0), (F0, U0)], ids=str)
def test_codes_steps_cut_short_in_every_tile(x_kind, w_kind, in_f, fp4):
    say("short steps of codes", x_kind, w_kind, in_f, fp4)
    check_codes(in_f + fp4, [20, 64, 96, 130, 160, 161, 223, 256, 290], 4104, in_f, x_kind, w_kind, fp4)
    check_codes(in_f + fp4, [33, 64, 0, 65, 40, 71], 2824, in_f, x_kind, w_kind, fp4)
    check_codes(in_f + fp4, [0, 17, 16, 0, 2], 72, in_f, x_kind, w_kind, fp4)


@pytest.mark.parametrize("accumulate", [0, 1])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("shape", [(264, 208), (520, 336), (136, 208)], ids=str)
@pytest.mark.parametrize("name", ["few_behind", "mid", "large", "many"])
def test_wgrad_with_both_indices_and_with_none(name, shape, gather, fp8, accumulate):
    say("wgrad indices", name, shape, gather, fp8, accumulate)
    rng = np.random.default_rng(len(name) * 149 + shape[0] + shape[1] + gather)
    off, n, e = products.layout(name)
    out_f, in_f = shape
    dy_rows, x_rows = (29, 31) if gather else (n, n)
    dyi = products.index_of(rng, n, dy_rows, True) if gather else None
    xi = products.index_of(rng, n, x_rows, True) if gather else None
    dy = products.whole(rng, (dy_rows, out_f))
    for group in (0, 16) if fp8 else (0,):
        if fp8:
            codes = products.whole_codes(rng, (x_rows, in_f))
            scales = rng.integers(125, 130, (x_rows, in_f // (group or in_f))).astype(np.uint8)
            x, xd, sd = ex.coded(codes, scales, True), products.dev(codes), products.dev(scales)
        else:
            x = products.whole(rng, (x_rows, in_f))
            xd, sd = products.bf16(x), None
        for bf in (False, True):
            start = products.whole(rng, (e, out_f, in_f), 100)
            dw = products.bf16(start) if bf else products.dev(start)
            assert tk.tk_expert_gemm_wgrad(products.bf16(dy), dy_rows, products.dev(dyi), xd, sd, FP8 if fp8 else BF16,
                                           group, x_rows, products.dev(xi), products.dev(off), n, e, out_f, in_f,
                                           accumulate, BF16 if bf else FP32, dw) == OK
            want = ex.wgrad(dy, dyi, x, xi, off, n, start if accumulate else np.zeros_like(start))[0]
            products.same_or(products.host(dw, bf), want, bf)


@pytest.mark.parametrize("clamp", [INF, 2.5])
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("n,hidden,group", [(16384, 2048, 128), (16401, 2040, 8), (8192, 4096, 512), (3277, 10240, 64)])
def test_checkpoint_of_four_steps_a_wave(n, hidden, group, fmt, clamp):
    say("checkpoint of four steps", n, hidden, group, fmt, clamp)
    gen = torch.Generator(device=DEV).manual_seed(n + hidden)
    x = (torch.randn((n, 2 * hidden), generator=gen, device=DEV) * 3).to(torch.bfloat16)
    x[1] = 0
    x[2, :hidden] = 0
    for weight in (None, torch.rand(n, generator=gen, device=DEV)):
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
            assert torch.equal(a, b)
