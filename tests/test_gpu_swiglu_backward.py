"""The SwiGLU step that leaves a checkpoint against the two calls that it is, bit
for bit, and SwiGLU's gradient against its statement in 64 bits and against
differences."""
import numpy as np
import pytest
import torch

import expert_ref as ex
import layer_ref as ref
import moe_activation_bit_amd as tk

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
OK = tk.TkStatus.TK_OK
INF = float("inf")


def say(*a):
    print("[gpu-case]", *a, flush=True)


def dev(a):
    if a is None:
        return None
    return torch.from_numpy(np.ascontiguousarray(a.view(np.int16) if a.dtype == np.uint16 else a)).to(DEV)


def bf16_host(t):
    return ref.bf16_value(t.cpu().numpy().view(np.uint16))


@pytest.mark.parametrize("clamp", [INF, 2.5])
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("n,hidden,group", [(1, 8, 8), (3, 24, 8), (37, 1024, 128), (349, 7168, 128), (5, 520, 8),
                                            (130, 1536, 512), (64, 96, 32), (1000, 2048, 64), (9, 4096, 256)])
def test_checkpoint_has_the_bits_of_two_calls(n, hidden, group, fmt, clamp):
    say("checkpoint", n, hidden, group, fmt, clamp)
    rng = np.random.default_rng(n + hidden)
    x = dev(ref.bf16_bits(rng.standard_normal((n, 2 * hidden)) * 3))
    if n > 3:
        x[1] = 0
        x[2, :hidden] = 0
    for weight in (None, dev(rng.random(n).astype(np.float32))):
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


def backward(dy, h, scales, h_dtype, fmt, group, weight, n, hidden, clamp, want_dweight=True, want_y=True):
    dh = torch.zeros((n, 2 * hidden), dtype=torch.int16, device=DEV)
    dweight = torch.zeros(n, device=DEV) if want_dweight else None
    y = torch.zeros((n, hidden), dtype=torch.int16, device=DEV) if want_y else None
    assert tk.tk_swiglu_backward(dy, h, scales, h_dtype, fmt, group, weight, n, hidden, clamp, dh, dweight, y) == OK
    torch.cuda.synchronize()
    return bf16_host(dh), None if dweight is None else dweight.cpu().numpy(), None if y is None else bf16_host(y)


def check(got, dy, h, weight, clamp):
    """Roundings: s to 4 units in the last place (the exponential, the sum and the reciprocal with its refinement,
    2^-22 together), then at most seven fp32 operations for each result, s + a(1 - s) losing up to twice its own
    size to cancellation (its terms' magnitudes count); one rounding to bf16, whose smallest step is 2^-133; and
    g sigma(g) beyond -87 off by up to 1.4e-36.  dweight: a term's roundings and those of the sum over hidden terms."""
    want, dw, y, mag = ex.swiglu_backward(dy, h, weight, clamp)
    _, (g, u, gc, uc, s, w) = ex.swiglu(h, weight, clamp)
    half = h.shape[1] // 2
    rel, tiny = 16 * 2.0 ** -24, 2e-36 * (1 + np.abs(dy * w) * (1 + np.abs(uc)))
    size = np.concatenate([np.abs(dy * w * uc) * (s + np.abs(gc * s) * (1 - s)) * (g <= clamp), np.abs(want[:, half:])],
                          1)
    bad = np.abs(got[0] - want) > ref.UB16 * np.abs(want) + (1 + ref.UB16) * rel * size + np.tile(tiny, 2)
    assert not bad.any(), (np.argwhere(bad)[:3], got[0][bad][:3], want[bad][:3])
    if got[1] is not None:
        assert np.all(np.abs(got[1] - dw) <= (16 + half) * 2.0 ** -24 * mag + tiny.sum(1))
    if got[2] is not None:
        assert np.all(np.abs(got[2] - y) <= ref.UB16 * np.abs(y) + (1 + ref.UB16) * rel * np.abs(y) + tiny)


SIZES = [(1, 8), (5, 24), (3, 512), (7, 520), (9, 1024), (6, 1032), (130, 2048), (33, 7168)]


@pytest.mark.parametrize("clamp", [INF, 1.5])
@pytest.mark.parametrize("n,hidden", SIZES)
def test_backward_from_bf16(n, hidden, clamp):
    say("backward bf16", n, hidden, clamp)
    rng = np.random.default_rng(n * hidden)
    h = ref.round_bf16(rng.standard_normal((n, 2 * hidden)) * 3)
    h[0, :3] = [0.0, 1.5, -1.5]  # a gate at the limit passes its gradient
    h[0, hidden:hidden + 3] = [1.5, -1.5, 0.0]
    dy = ref.round_bf16(rng.standard_normal((n, hidden)))
    for weight in (None, rng.random(n).astype(np.float32)):
        got = backward(dev(ref.bf16_bits(dy)), dev(ref.bf16_bits(h)), None, tk.TK_DTYPE_BF16, 0, 0, dev(weight), n,
                       hidden, clamp)
        check(got, dy, h, weight, clamp)


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("n,hidden,group", [(1, 8, 8), (5, 24, 48), (5, 24, 16), (3, 512, 0), (9, 1024, 128),
                                            (6, 1032, 24), (130, 2048, 128), (33, 7168, 2048), (4, 7168, 0)])
def test_backward_from_checkpoint(n, hidden, group, fmt):
    say("backward fp8", n, hidden, group, fmt)
    rng = np.random.default_rng(n * hidden + group)
    x = dev(ref.bf16_bits(rng.standard_normal((n, 2 * hidden)) * 3))
    codes = torch.zeros((n, 2 * hidden), dtype=torch.uint8, device=DEV)
    scales = torch.zeros((n, 2 * hidden // (group or 2 * hidden)), dtype=torch.uint8 if fmt else torch.float32, device=DEV)
    assert tk.tk_cast_fp8(x, 0, n, 2 * hidden, group, fmt, codes, scales) == OK
    torch.cuda.synchronize()
    h = ex.coded(codes.cpu().numpy(), scales.cpu().numpy(), bool(fmt)).astype(np.float32)  # as code * scale rounds
    dy = ref.round_bf16(rng.standard_normal((n, hidden)))
    weight = rng.random(n).astype(np.float32)
    for clamp in (INF, 2.0):
        got = backward(dev(ref.bf16_bits(dy)), codes, scales, tk.TK_DTYPE_FP8, fmt, group, dev(weight), n, hidden, clamp)
        check(got, dy, h, weight, clamp)


def test_far_gates():
    """Gates where e^-g leaves fp32's range, and results that bf16 holds with few bits."""
    g = np.array([0.0, -0.0, 87.0, -87.0, 88.0, -88.0, 100.0, -100.0, 1e30, -1e30, 3e38, -3e38, 1e-30, -1e-38, 20.0,
                  -20.0], np.float32)
    hidden = len(g)
    h = ref.round_bf16(np.concatenate([g, np.ones(hidden, np.float32)])[None])
    dy = np.full((1, hidden), 0.5, np.float32)
    got = backward(dev(ref.bf16_bits(dy)), dev(ref.bf16_bits(h)), None, 0, 0, 0, None, 1, hidden, INF)
    check((got[0], None, got[2]), dy, h, None, INF)


def test_nan_shows_in_its_own_places():
    rng = np.random.default_rng(2)
    n, hidden = 5, 1024
    h = rng.standard_normal((n, 2 * hidden)).astype(np.float32)
    h[1, 7] = np.nan
    dy = rng.standard_normal((n, hidden)).astype(np.float32)
    dh, dw, y = backward(dev(ref.bf16_bits(dy)), dev(ref.bf16_bits(h)), None, 0, 0, 0, None, n, hidden, INF)
    assert np.argwhere(np.isnan(dh)).tolist() == [[1, 7], [1, hidden + 7]]
    assert np.argwhere(np.isnan(dw)).tolist() == [[1]] and np.argwhere(np.isnan(y)).tolist() == [[1, 7]]


def test_in_place_and_without_outputs():
    rng = np.random.default_rng(4)
    n, hidden = 33, 1536
    h = dev(ref.bf16_bits(rng.standard_normal((n, 2 * hidden))))
    dy = dev(ref.bf16_bits(rng.standard_normal((n, hidden))))
    w = dev(rng.random(n).astype(np.float32))
    dh, dw, y = backward(dy, h, None, 0, 0, 0, w, n, hidden, 1.0)
    only, _, _ = backward(dy, h, None, 0, 0, 0, w, n, hidden, 1.0, False, False)
    assert np.array_equal(only, dh)
    dw2 = torch.zeros(n, device=DEV)
    assert tk.tk_swiglu_backward(dy, h, None, 0, 0, 0, w, n, hidden, 1.0, h, dw2, dy) == OK
    torch.cuda.synchronize()
    assert np.array_equal(bf16_host(h), dh) and np.array_equal(bf16_host(dy), y) and np.array_equal(dw2.cpu().numpy(), dw)
