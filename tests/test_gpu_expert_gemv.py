"""tk_expert_gemv_fp4 on the GPU against the plain 64-bit reference: bit for bit
on inputs whose products and sums are exact in fp32 in any order, and within the
bound of an fp32 sum in any order on random ones."""
import numpy as np
import pytest
import torch

import layer_ref as ref
import moe_activation_bit_amd as tk
import oracle

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
OK = tk.TkStatus.TK_OK
PAD = 256
FP32, UE8M0 = tk.TK_SCALE_FP32, tk.TK_SCALE_UE8M0


def say(*a):
    print("[gpu-case]", *a, flush=True)


def up(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def run(xk, x, xs, xg, idx, tokens, k, slots, codes, scales, u8, group, out_bf16, stream=None):
    E, out, inner = codes.shape[0], codes.shape[1], codes.shape[2] * 2
    item = 2 if out_bf16 else 4
    n = tokens * k * out * item
    buf = torch.full((n + 2 * PAD,), 0xC3, dtype=torch.uint8, device=DEV)
    xd = up(x.view(np.int16)) if xk == "bf16" else up(x)
    rc = tk.tk_expert_gemv_fp4(xd, up(xs), tk.TK_DTYPE_BF16 if xk == "bf16" else tk.TK_DTYPE_FP8,
                               UE8M0 if xk == "fp8e" else FP32, xg, up(idx), tokens, k, slots, up(codes), up(scales),
                               UE8M0 if u8 else FP32, group, E, out, inner,
                               tk.TK_DTYPE_BF16 if out_bf16 else tk.TK_DTYPE_FP32, buf.data_ptr() + PAD, stream)
    assert rc == OK, tk.tk_status_str(rc)
    torch.cuda.synchronize()
    o = buf.cpu().numpy()
    assert (o[:PAD] == 0xC3).all() and (o[PAD + n:] == 0xC3).all(), "canary"
    return o[PAD:PAD + n].view(np.uint16 if out_bf16 else np.float32).reshape(tokens * k, out)


E4M3_WHOLE = [int(np.flatnonzero(ref.e4m3_values() == v)[0]) for v in range(-4, 5)]


def make(seed, tokens, k, E, out, inner, xk, xg, slots, u8, group, exact, dense=False):
    """exact: whole activations up to 4, weights of half steps up to 6 with scales of 1, 2 and 4: every product and
    every sum up to 2^23 of them is a multiple of 1/2 below 2^23."""
    rng = np.random.default_rng(seed)
    rows = tokens * k if slots else tokens
    codes = rng.integers(0, 256, (E, out, inner // 2), dtype=np.uint8)
    G, XG = inner // (group or inner), inner // (xg or inner)
    if u8:
        scales = rng.integers(127, 130, (E, out, G)).astype(np.uint8) if exact else rng.integers(115, 125, (E, out, G)).astype(np.uint8)
    else:
        scales = (2.0 ** rng.integers(0, 3, (E, out, G)) if exact else 0.01 + rng.random((E, out, G))).astype(np.float32)
    xs = None
    if xk == "bf16":
        x = ref.bf16_bits(rng.integers(-4, 5, (rows, inner)).astype(np.float32) if exact else rng.standard_normal((rows, inner)))
    else:
        x = np.array(E4M3_WHOLE, np.uint8)[rng.integers(0, 9, (rows, inner))] if exact else rng.integers(0, 256, (rows, inner)).astype(np.uint8)
        x = np.where((x & 0x7F) == 0x7F, 0x30, x).astype(np.uint8)
        if xk == "fp8e":
            xs = (rng.integers(127, 129, (rows, XG)) if exact else rng.integers(120, 126, (rows, XG))).astype(np.uint8)
        else:
            xs = (2.0 ** rng.integers(0, 2, (rows, XG)) if exact else 0.01 + rng.random((rows, XG))).astype(np.float32)
    idx = None if dense else np.stack([rng.permutation(max(E, k))[:k] % E for _ in range(tokens)]).astype(np.int32)
    return x, xs, idx, codes, scales


def check(got, out_bf16, want, mag, inner, exact):
    if exact:
        assert mag.max() < 2 ** 22
        w32 = want.astype(np.float32)
        assert np.array_equal(w32, want)
        assert np.array_equal(got, ref.bf16_bits(w32) if out_bf16 else w32 + np.float32(0)), "exact sums differ"
        return
    v = (ref.bf16_value(got) if out_bf16 else got).astype(np.float64)
    # an fp32 sum of `inner` exact products in any order, each with up to three scale roundings
    bound = ref.U32 * (inner + 3) * mag + (ref.UB16 * (1 + 2.0 ** -7) * np.abs(want) if out_bf16 else 0)
    err = np.abs(v - want)
    assert np.all(err <= bound), f"off by {np.max(err / np.maximum(bound, 1e-300)):.2f} of the bound"
    # and in norm: independent roundings of random products grow with the root of their number
    assert np.linalg.norm(err) <= (8 * ref.U32 * np.sqrt(inner) + (ref.UB16 if out_bf16 else 0)) * np.linalg.norm(mag if not out_bf16 else want) + 1e-30


CASES = [  # tokens, k, experts, out, in, x, x group, slots, u8, group
    (1, 1, 1, 16, 32, "bf16", 0, 0, True, 32), (1, 1, 3, 1, 32, "fp8", 0, 0, True, 0), (1, 2, 4, 17, 96, "fp8e", 32, 0, True, 32),
    (1, 8, 16, 300, 7168, "fp8", 128, 0, True, 32), (3, 4, 8, 129, 2016, "bf16", 0, 1, True, 0),
    (16, 8, 8, 70, 2048, "fp8", 0, 1, True, 32), (17, 2, 4, 33, 1024, "bf16", 0, 0, False, 128),
    (5, 6, 64, 64, 512, "fp8e", 0, 0, False, 0), (2, 3, 5, 50, 4096, "fp8", 128, 1, False, 256),
    (4, 2, 2, 31, 160, "fp8e", 32, 1, True, 32), (1, 64, 64, 40, 256, "bf16", 0, 0, True, 64),
    (40, 2, 3, 48, 384, "fp8", 128, 0, True, 128), (70, 1, 2, 20, 544, "bf16", 0, 0, True, 0),
    (64, 8, 32, 24, 1024, "fp8e", 128, 0, True, 32), (2, 2, 4, 1024, 1056, "fp8", 0, 0, True, 32),
    (9, 8, 12, 96, 7168, "bf16", 0, 1, True, 32), (1, 8, 8, 37, 384, "fp8", 384, 0, False, 384),
    (3, 2, 4, 45, 4128, "bf16", 0, 0, True, 32), (1, 4, 4, 2048, 64, "bf16", 0, 0, True, 32),
    (20, 5, 6, 33, 640, "fp8", 128, 1, False, 128), (33, 3, 4, 19, 8192, "fp8e", 32, 0, True, 256),
]


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("out_bf16", [True, False])
def test_gemv(case, out_bf16):
    tokens, k, E, out, inner, xk, xg, slots, u8, group = case
    say("gemv", case, out_bf16)
    for exact in (True, False):
        x, xs, idx, codes, scales = make(tokens + out, tokens, k, E, out, inner, xk, xg, slots, u8, group, exact)
        want, mag = ref.gemv(ref.x_values(x, xs, xk), idx, k, slots, ref.fp4_values(codes, scales, u8))
        check(run(xk, x, xs, xg, idx, tokens, k, slots, codes, scales, u8, group, out_bf16), out_bf16, want, mag, inner, exact)


@pytest.mark.parametrize("tokens", [1, 2, 3, 7, 16, 17, 33, 64, 65, 100])
@pytest.mark.parametrize("xk,xg,u8,group", [("bf16", 0, True, 32), ("fp8", 128, False, 128), ("fp8e", 32, True, 32), ("fp8", 0, True, 0),
                                            ("bf16", 0, False, 0)])
def test_dense(tokens, xk, xg, u8, group):
    say("gemv dense", tokens, xk, xg, u8, group)
    out, inner = 75, 1280
    for exact in (True, False):
        x, xs, _, codes, scales = make(tokens, tokens, 1, 1, out, inner, xk, xg, 0, u8, group, exact, dense=True)
        want, mag = ref.gemv(ref.x_values(x, xs, xk), np.zeros((tokens, 1), int), 1, 0, ref.fp4_values(codes, scales, u8))
        check(run(xk, x, xs, xg, None, tokens, 1, 0, codes, scales, u8, group, False), False, want, mag, inner, exact)


@pytest.mark.parametrize("inner", [32, 96, 160, 288, 992, 2016, 4128])
@pytest.mark.parametrize("xk", ["bf16", "fp8", "fp8e"])
@pytest.mark.parametrize("u8", [True, False])
def test_one_scale_a_row_of_any_width(inner, xk, u8):
    say("gemv one scale a row", inner, xk, u8)
    tokens, k, E, out = 5, 2, 3, 37
    for exact in (True, False):
        x, xs, idx, codes, scales = make(inner, tokens, k, E, out, inner, xk, 0, 0, u8, 0, exact)
        want, mag = ref.gemv(ref.x_values(x, xs, xk), idx, k, 0, ref.fp4_values(codes, scales, u8))
        check(run(xk, x, xs, 0, idx, tokens, k, 0, codes, scales, u8, 0, False), False, want, mag, inner, exact)


def test_absent_repeated_and_crowded():
    say("gemv routing")
    E, out, inner, k = 6, 34, 256, 4
    for xk, xg in (("bf16", 0), ("fp8", 128)):
        for slots in (0, 1):
            x, xs, idx, codes, scales = make(8, 50, k, E, out, inner, xk, xg, slots, True, 32, True)
            idx[0] = -1                        # a token that goes nowhere
            idx[1] = [2, 2, 2, 2]              # one expert four times
            idx[2] = [-1, 5, 6, 2 ** 31 - 1]   # dropped and out of range
            idx[3] = [-2 ** 31, 0, 0, 1]
            idx[10:] = 3                       # 160 rows of one expert
            want, mag = ref.gemv(ref.x_values(x, xs, xk), idx, k, slots, ref.fp4_values(codes, scales, True))
            check(run(xk, x, xs, xg, idx, 50, k, slots, codes, scales, True, 32, False), False, want, mag, inner, True)


def test_rows_do_not_depend_on_the_batch():
    say("gemv batch")
    E, out, inner, k = 8, 100, 2048, 2
    for xk, xg, u8, group in (("bf16", 0, True, 32), ("fp8", 128, True, 32), ("fp8e", 32, True, 64), ("fp8", 0, False, 128)):
        x, xs, idx, codes, scales = make(4, 40, k, E, out, inner, xk, xg, 0, u8, group, False)
        all_ = run(xk, x, xs, xg, idx, 40, k, 0, codes, scales, u8, group, False)
        again = run(xk, x, xs, xg, idx, 40, k, 0, codes, scales, u8, group, False)
        assert np.array_equal(all_, again)
        for t in (0, 17, 39):
            one = run(xk, x[t:t + 1], None if xs is None else xs[t:t + 1], xg, idx[t:t + 1], 1, k, 0, codes, scales, u8, group, False)
            assert np.array_equal(one, all_[t * k:(t + 1) * k])


def test_extreme_scales_and_special_values():
    say("gemv extremes")
    out, inner = 32, 128
    codes = np.full((1, out, inner // 2), 0x22, np.uint8)  # every weight 1
    x = ref.bf16_bits(np.ones((1, inner), np.float32))
    for byte, want in ((0, 2.0 ** -120), (1, 2.0 ** -119), (246, 2.0 ** 126)):
        scales = np.full((1, out, inner // 32), byte, np.uint8)
        got = run("bf16", x, None, 0, None, 1, 1, 0, codes, scales, True, 32, False)
        assert np.all(got == np.float32(want)), byte
    # a NaN scale, a NaN activation and an infinite one reach their own results and no others
    scales = np.full((1, out, inner // 32), 127, np.uint8)
    scales[0, 3, 1] = 255
    xn = ref.bf16_value(x).repeat(3, 0)
    xn[1, 5], xn[2, 7] = np.nan, np.inf
    got = run("bf16", ref.bf16_bits(xn), None, 0, None, 3, 1, 0, codes, scales, True, 32, False)
    assert np.isnan(got[0, 3]) and np.all(np.delete(got[0], 3) == inner)
    assert np.isnan(got[1]).all()
    assert np.all(np.delete(got[2], 3) == np.inf)
    xc = np.full((2, inner), 0x38, np.uint8)  # E4M3 1.0
    xc[1, 9] = 0x7F
    got = run("fp8", xc, np.ones((2, 1), np.float32), 0, None, 2, 1, 0, codes, scales, True, 32, False)
    assert np.isnan(got[0, 3]) and np.all(np.delete(got[0], 3) == inner) and np.isnan(got[1]).all()


def test_weights_from_the_cast():
    """Weights as tk_cast_fp4 leaves them, activations as tk_cast_fp8 does."""
    say("gemv cast")
    rng = np.random.default_rng(0)
    E, out, inner, tokens, k = 4, 96, 1024, 3, 2
    w = rng.standard_normal((E * out, inner)).astype(np.float32)
    x = rng.standard_normal((tokens, inner)).astype(np.float32)
    idx = np.array([[0, 3], [1, 2], [3, 1]], np.int32)
    for sfmt, group, xg in ((UE8M0, 32, 128), (FP32, 128, 0)):
        codes = torch.empty((E * out, inner // 2), dtype=torch.uint8, device=DEV)
        scales = torch.empty((E * out, inner // group), dtype=torch.uint8 if sfmt == UE8M0 else torch.float32, device=DEV)
        xc = torch.empty((tokens, inner), dtype=torch.uint8, device=DEV)
        xs = torch.empty((tokens, inner // (xg or inner)), dtype=torch.float32, device=DEV)
        y = torch.empty((tokens * k, out), dtype=torch.float32, device=DEV)
        assert tk.tk_cast_fp4(up(w), tk.TK_DTYPE_FP32, E * out, inner, group, sfmt, codes, scales) == OK
        assert tk.tk_cast_fp8(up(x), tk.TK_DTYPE_FP32, tokens, inner, xg, FP32, xc, xs) == OK
        assert tk.tk_expert_gemv_fp4(xc, xs, tk.TK_DTYPE_FP8, FP32, xg, up(idx), tokens, k, 0, codes, scales, sfmt, group, E, out,
                                     inner, tk.TK_DTYPE_FP32, y) == OK
        torch.cuda.synchronize()
        oc, os_ = oracle.cast(w, group, oracle.FP4, oracle.SCALE_UE8M0 if sfmt == UE8M0 else oracle.SCALE_FP32)
        xo, xso = oracle.cast(x, xg, oracle.FP8, oracle.SCALE_FP32)
        wv = ref.fp4_values(oc.reshape(E, out, -1), os_.reshape(E, out, -1), sfmt == UE8M0)
        want, mag = ref.gemv(ref.x_values(xo, xso.reshape(tokens, -1), "fp8"), idx, k, 0, wv)
        check(y.cpu().numpy(), False, want, mag, inner, False)


def want_on_gpu(xk, x, xs, idx, k, slots, codes, scales, u8):
    """ref.gemv's results by 64-bit products on the GPU, an expert at a time."""
    xv, lut = up(ref.x_values(x, xs, xk)), up(ref.E2M1)
    rows = up(idx.reshape(-1))
    out, mag = (torch.zeros((len(rows), codes.shape[1]), dtype=torch.float64, device=DEV) for _ in range(2))
    for e in range(codes.shape[0]):
        mine = torch.nonzero(rows == e)[:, 0]
        if len(mine):
            c = up(codes[e]).to(torch.int64)
            w = torch.stack([lut[c & 15], lut[c >> 4]], -1).reshape(codes.shape[1], -1)
            sc = up(ref.e8m0_value(scales[e]) if u8 else scales[e].astype(np.float64))
            w = (w.reshape(*sc.shape, -1) * sc[..., None]).reshape(w.shape).t().contiguous()
            v = xv[mine if slots else mine // k]
            out[mine], mag[mine] = v @ w, v.abs() @ w.abs()
    return out.cpu().numpy(), mag.cpu().numpy()


# Launches of 2048 workgroups and more, whose waves go through two tiles of weight rows, and of 4096, four: every kind of
# activation and of scale, whole steps of 256 columns and others, rows of weights that end inside a wave's tiles,
# one pass over an expert's rows and several, x rows that stay in LDS from tile to tile and ones staged again for each.
TILED = [  # as CASES; experts of 0: one matrix for all rows
    (40, 8, 64, 4100, 512, "fp8", 128, 0, True, 32), (64, 16, 64, 2050, 1024, "bf16", 0, 0, True, 32),
    (64, 8, 64, 4099, 544, "fp8e", 32, 1, True, 32), (48, 8, 64, 4097, 768, "fp8", 128, 0, False, 128),
    (40, 8, 32, 4101, 1280, "bf16", 0, 1, False, 0), (9, 64, 64, 2077, 2560, "fp8", 0, 0, True, 32),
    (200, 4, 16, 8200, 288, "fp8", 0, 0, True, 0), (33, 16, 64, 2100, 256, "fp8e", 0, 0, False, 128),
    (32, 8, 64, 4096, 1024, "fp8e", 128, 0, True, 32), (20, 16, 64, 2049, 512, "fp8", 256, 0, True, 64),
    (512, 1, 0, 8210, 1280, "fp8", 128, 0, True, 32), (272, 1, 0, 8196, 4384, "bf16", 0, 0, True, 32),
    (272, 1, 0, 8190, 4608, "fp8", 128, 0, True, 32), (600, 1, 0, 7000, 640, "fp8e", 32, 0, False, 128),
]


@pytest.mark.parametrize("case", TILED, ids=str)
def test_several_tiles_a_wave(case):
    tokens, k, E, out, inner, xk, xg, slots, u8, group = case
    say("gemv tiles", case)
    for exact in (True, False):
        x, xs, idx, codes, scales = make(out + inner, tokens, k, max(E, 1), out, inner, xk, xg, slots, u8, group, exact, dense=not E)
        if E:
            idx[0], idx[1, 0], idx[tokens // 2:tokens // 2 + 3] = -1, E, 5 % E  # absent, out of range, crowded
        chosen = np.zeros((tokens, 1), np.int32) if idx is None else idx
        want, mag = want_on_gpu(xk, x, xs, chosen, k, slots, codes, scales, u8)
        for out_bf16 in (False, True):
            got = run(xk, x, xs, xg, idx, tokens, k, slots, codes, scales, u8, group, out_bf16)
            check(got, out_bf16, want, mag, inner, exact)
            assert not got[chosen.reshape(-1) < 0].any()


@pytest.mark.parametrize("xk,xg", [("bf16", 0), ("fp8", 128), ("fp8", 0), ("fp8e", 32)])
@pytest.mark.parametrize("u8,group,inner", [(True, 32, 2048), (True, 128, 2048), (False, 128, 2048), (True, 32, 2016), (False, 0, 2016)])
def test_rows_do_not_depend_on_the_batch_however_the_columns_are_shared(xk, xg, u8, group, inner):
    """One token: four waves share a row's columns.  Two: two do.  Sixteen and 40: one wave takes them all, two tiles one
    after the other.  The parts and their order stay."""
    say("gemv batch and waves", xk, xg, u8, group, inner)
    E, out, k, T = 64, 2048, 8, 40
    xg = xg if xg == 0 or inner % xg == 0 else 0
    x, xs, idx, codes, scales = make(inner + group, T, k, E, out, inner, xk, xg, 0, u8, group, False)
    idx[39] = idx[3]
    cd, sd = up(codes), up(scales)

    def rows(lo, hi):
        y = torch.empty(((hi - lo) * k, out), device=DEV)
        xd = up(x[lo:hi].view(np.int16)) if xk == "bf16" else up(x[lo:hi])
        rc = tk.tk_expert_gemv_fp4(xd, None if xs is None else up(xs[lo:hi]), tk.TK_DTYPE_BF16 if xk == "bf16" else tk.TK_DTYPE_FP8,
                                   UE8M0 if xk == "fp8e" else FP32, xg, up(idx[lo:hi]), hi - lo, k, 0, cd, sd,
                                   UE8M0 if u8 else FP32, group, E, out, inner, tk.TK_DTYPE_FP32, y)
        assert rc == OK, tk.tk_status_str(rc)
        return y.cpu().numpy()

    whole = rows(0, T)
    for lo, hi in ((0, 1), (17, 18), (39, 40), (3, 5), (8, 12), (16, 32)):
        assert np.array_equal(rows(lo, hi).view(np.uint32), whole[lo * k:hi * k].view(np.uint32)), (lo, hi)


@pytest.mark.parametrize("byte", [0, 1, 2, 3, 4, 100, 254])
def test_activations_at_the_ends_of_bf16(byte):
    """FP8 activations with UE8M0 scales are taken as bf16 numbers: exact but for what lies below 2^-133, half of whose
    steps are rounded to even, or past the largest number, which fp32 does not hold either."""
    say("gemv activations", byte)
    out, inner = 16, 128
    code = np.array([c for c in range(256) if c & 127 != 127], np.uint8)
    x = np.zeros((len(code), inner), np.uint8)
    x[:, 37] = code
    scale = 247 - max(0, byte - 60)  # of the weights, 1 by their codes: results between 2^-80 and 2^80
    got = run("fp8e", x, np.full((len(code), 1), byte, np.uint8), 0, None, len(code), 1, 0, np.full((1, out, inner // 2), 0x22, np.uint8),
              np.full((1, out, inner // 32), scale, np.uint8), True, 32, False)
    v = ref.e4m3_values()[code] * 2.0 ** (byte - 127)
    near = np.round(v * 2.0 ** 133) * 2.0 ** -133
    assert byte > 2 or (near != v).any()
    want = np.where(np.abs(v) < 2.0 ** 128, near * 2.0 ** (scale - 127), np.copysign(np.inf, v)).astype(np.float32)
    assert np.array_equal(got, np.repeat(want[:, None], out, 1) + np.float32(0))


@pytest.mark.parametrize("inner", [32, 96, 128, 384, 640, 256, 512])
def test_infinite_scales_of_rows_that_end_inside_a_step(inner):
    """An infinite fp32 scale makes infinities of its products, and no NaN of the columns past a row's end."""
    say("gemv infinite scales", inner)
    out, inf = 20, np.float32(np.inf)
    codes = np.full((1, out, inner // 2), 0x22, np.uint8)  # every weight 1
    codes[0, 1::2] = 0xAA                                  # or -1
    sign = np.where(np.arange(out) % 2, -1.0, 1.0)
    one8, one16 = np.full((3, inner), 0x38, np.uint8), ref.bf16_bits(np.ones((3, inner), np.float32))
    for group in (0, 128) if inner % 128 == 0 else (0,):
        scales = np.ones((1, out, inner // (group or inner)), np.float32)
        scales[0, 4:, -1] = inf
        want = np.tile(np.where(np.arange(out) < 4, sign * inner, sign * inf), (3, 1)).astype(np.float32)
        for xk, x, xs in (("bf16", one16, None), ("fp8", one8, np.ones((3, 1), np.float32)), ("fp8e", one8, np.full((3, 1), 127, np.uint8))):
            got = run(xk, x, xs, 0, None, 3, 1, 0, codes, scales, False, group, False)
            assert np.array_equal(got, want), (xk, group)
    if inner % 128 == 0:  # of the activations
        xs = np.ones((3, inner // 128), np.float32)
        xs[1, -1] = inf
        want = np.tile(sign * inner, (3, 1)).astype(np.float32)
        want[1] = sign * inf
        for u8, scales in ((True, np.full((1, out, inner // 32), 127, np.uint8)), (False, np.ones((1, out, inner // 128), np.float32))):
            got = run("fp8", one8, xs, 128, None, 3, 1, 0, codes, scales, u8, 32 if u8 else 128, False)
            assert np.array_equal(got, want), u8
