"""tk_rmsnorm_cast_fp8 and tk_rmsnorm_backward on the GPU against the plain
64-bit reference.  The forward is op-by-op fp32 from the stored rstd on, so its
y and, through the oracle's cast, its codes and scales are compared bit for bit
once rstd is within its own rounding; bounds elsewhere count roundings."""
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


def say(*a):
    print("[gpu-case]", *a, flush=True)


def up(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


class Out:
    """An output buffer with canaries on both sides; `at` is its address."""

    def __init__(self, nbytes, like=None):
        self.n = nbytes
        self.buf = torch.full((nbytes + 2 * PAD,), 0xC3, dtype=torch.uint8, device=DEV)
        self.at = self.buf.data_ptr() + PAD
        if like is not None:
            self.buf[PAD:PAD + nbytes] = torch.from_numpy(np.ascontiguousarray(like).view(np.uint8).reshape(-1)).to(DEV)

    def get(self, dtype):
        o = self.buf.cpu().numpy()
        assert (o[:PAD] == 0xC3).all() and (o[PAD + self.n:] == 0xC3).all(), "canary overwritten"
        return o[PAD:PAD + self.n].view(dtype)


def make(seed, n, hidden, bf16, residual, spread=1.0):
    rng = np.random.default_rng(seed)

    def draw(sigma):
        a = (sigma * rng.standard_normal((n, hidden))).astype(np.float32)
        return ref.bf16_bits(a) if bf16 else a

    return draw(spread), draw(4 * spread) if residual else None, (1 + 0.25 * rng.standard_normal(hidden)).astype(np.float32)


def value(a, bf16):
    return None if a is None else ref.bf16_value(a) if bf16 else a


SCALE_LD = {0: None, 1: None, 2: 4, 3: 16, 4: 4}


def scale_bytes(fmt, n, groups):
    if fmt in (0, 1):
        return n * groups * (4 if fmt == 0 else 1)
    ld = -(-n // SCALE_LD[fmt]) * SCALE_LD[fmt]
    return groups * ld * 4 if fmt == 2 else groups * ld if fmt == 3 else -(-groups // 4) * ld * 4


def rows_of_scales(buf, fmt, n, groups):
    """A scale buffer in any layout as row-major [n, groups]."""
    if fmt == 0:
        return buf.view(np.float32).reshape(n, groups)
    if fmt == 1:
        return buf.reshape(n, groups)
    ld = -(-n // SCALE_LD[fmt]) * SCALE_LD[fmt]
    if fmt == 2:
        return np.ascontiguousarray(buf.view(np.float32).reshape(groups, ld)[:, :n].T)
    if fmt == 3:
        return np.ascontiguousarray(buf.reshape(groups, ld)[:, :n].T)
    b = buf.reshape(-1, ld, 4)[:, :n]  # [ceil(G/4), n, 4]
    return np.ascontiguousarray(b.transpose(1, 0, 2).reshape(n, -1)[:, :groups])


def run_norm(x, res, w, bf16, eps, group, fmt, in_place=None, codes=True, keep=True, stream=None):
    n, hidden = x.shape
    item, G = 2 if bf16 else 4, hidden // (group or hidden)
    xd, rd, wd = Out(x.nbytes, x), None if res is None else Out(res.nbytes, res), up(w)
    h = {"x": xd, "res": rd}.get(in_place) or Out(n * hidden * item)
    y, rstd = Out(n * hidden * 2), Out(n * 4)
    c, s = Out(n * hidden), Out(scale_bytes(fmt, n, G))
    rc = tk.tk_rmsnorm_cast_fp8(xd.at, rd and rd.at, tk.TK_DTYPE_BF16 if bf16 else tk.TK_DTYPE_FP32, wd, n, hidden, eps,
                                group, fmt, h.at, y.at if keep else None, rstd.at if keep else None,
                                c.at if codes else None, s.at if codes else None, stream)
    assert rc == OK, tk.tk_status_str(rc)
    torch.cuda.synchronize()
    out = {"h": h.get(np.uint16 if bf16 else np.float32).reshape(n, hidden)}
    y_, rstd_, c_, s_ = y.get(np.uint16), rstd.get(np.float32), c.get(np.uint8), s.get(np.uint8)
    if keep:
        out["y"], out["rstd"] = y_.reshape(n, hidden), rstd_
    if codes:
        out["codes"], out["scales"] = c_.reshape(n, hidden), rows_of_scales(s_, fmt, n, G)
    return out


def check_norm(x, res, w, bf16, eps, group, fmt, got):
    h = ref.norm_stream(value(x, bf16), value(res, bf16), bf16)
    assert np.array_equal(value(got["h"], bf16), h), "stream"
    rstd, y = ref.norm(h, w, eps)
    # rstd: computed in 64 bits and rounded once
    assert np.all(np.abs(got["rstd"] - rstd) <= ref.U32 * (1 + 2.0 ** -10) * rstd), "rstd"
    y32 = (h * got["rstd"][:, None]) * w  # fp32, one rounding an operation
    assert y32.dtype == np.float32
    assert np.array_equal(got["y"], ref.bf16_bits(y32)), "y"
    codes, scales = oracle.cast(y32, group, oracle.FP8, oracle.SCALE_FP32 if fmt in (0, 2) else oracle.SCALE_UE8M0)
    assert np.array_equal(got["codes"], codes), "codes"
    assert np.array_equal(got["scales"].view(np.uint8).reshape(-1), scales.view(np.uint8).reshape(-1)), "scales"
    # and straight from the 64-bit y: half a step of E4M3 (of its smallest step below 2^-6), the scale's and
    # y's few fp32 roundings
    G = group or x.shape[1]
    sv = (scales if scales.dtype == np.float32 else ref.e8m0_value(scales)).astype(np.float64).reshape(x.shape[0], -1, 1)
    v = ref.e4m3_values()[codes].reshape(x.shape[0], -1, G) * sv
    yy = y.reshape(v.shape)
    assert np.all(np.abs(v - yy) <= np.abs(yy) * (ref.UE4M3 + 8 * ref.U32) + sv * 2.0 ** -10 * (1 + 8 * ref.U32)), "value"


SHAPES = [  # n, hidden, group, scale format
    (1, 8, 0, 0), (1, 7168, 128, 0), (3, 64, 8, 1), (7, 200, 40, 0), (5, 520, 0, 1), (33, 1024, 128, 2),
    (8, 7168, 128, 0), (2, 2016, 96, 3), (17, 1536, 768, 4), (4, 4096, 512, 1), (9, 8192, 0, 2), (3, 16384, 1024, 0),
    (2, 32768, 256, 4), (1, 32760, 0, 0), (2, 32752, 16376, 1), (19, 2056, 8, 0), (6, 7168, 896, 3), (5, 24, 24, 0),
    # more rows: a lane holds several steps of its row, or a wave the whole of it
    (2049, 8, 8, 0), (2050, 1000, 0, 1), (2051, 2048, 128, 4), (2048, 2304, 96, 0), (2063, 4104, 24, 3),
    (2200, 7168, 128, 1), (2048, 512, 32, 2),
]


@pytest.mark.parametrize("n,hidden,group,fmt", SHAPES)
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("residual", [True, False])
def test_norm(n, hidden, group, fmt, bf16, residual):
    say("norm", n, hidden, group, fmt, bf16, residual)
    x, res, w = make(n * 7 + hidden, n, hidden, bf16, residual)
    check_norm(x, res, w, bf16, 1e-6, group, fmt, run_norm(x, res, w, bf16, 1e-6, group, fmt))


@pytest.mark.parametrize("bf16", [True, False])
def test_norm_zero_rows_large_and_tiny_values(bf16):
    say("norm values", bf16)
    n, hidden = 12, 1032
    x, res, w = make(5, n, hidden, bf16, True)
    to = ref.bf16_bits if bf16 else (lambda a: a.astype(np.float32))
    xv, rv = value(x, bf16).copy(), value(res, bf16).copy()
    xv[0] = rv[0] = 0                               # a padding row
    xv[1], rv[1] = xv[2], -xv[2]                    # cancels to zero
    xv[3] *= np.float32(1e30); rv[3] *= np.float32(1e30)    # squares past fp32
    xv[4] *= np.float32(1e-30); rv[4] = 0           # squares below fp32
    xv[5, 1:] = 0; rv[5, 1:] = 0                    # one value
    w[7] = 0
    x, res = to(xv), to(rv)
    for group, fmt in ((0, 0), (24, 1), (8, 3), (344, 0)):
        got = run_norm(x, res, w, bf16, 1e-6, group, fmt)
        check_norm(x, res, w, bf16, 1e-6, group, fmt, got)
        assert not got["codes"][0].any() and not got["scales"][0].any()
    assert np.isfinite(got["scales"]).all()


def test_norm_nan_and_infinity_show():
    say("norm nan")
    x, _, w = make(6, 4, 512, True, False)
    xv = ref.bf16_value(x)
    xv[1, 3], xv[2, 5] = np.nan, np.inf
    for group, fmt in ((0, 0), (64, 0), (64, 1), (0, 1)):
        got = run_norm(ref.bf16_bits(xv), None, w, True, 1e-6, group, fmt)
        assert np.isnan(got["rstd"][1]) and got["rstd"][2] == 0
        assert ((got["codes"][1] & 0x7F) == 0x7F).all()
        assert (got["codes"][2, 5] & 0x7F) == 0x7F and not (np.delete(got["codes"][2], 5) & 0x7F).any()
        clean = run_norm(x, None, w, True, 1e-6, group, fmt)
        for r in (0, 3):  # the rows beside are untouched
            assert np.array_equal(got["codes"][r], clean["codes"][r]) and np.array_equal(got["scales"][r], clean["scales"][r])


def test_norm_rows_do_not_depend_on_their_number():
    say("norm batch")
    x, res, w = make(8, 2100, 2304, True, True)
    for group, fmt in ((0, 0), (96, 1), (128, 0)):
        all_ = run_norm(x, res, w, True, 1e-5, group, fmt)
        for lo, hi in ((0, 1), (7, 9), (2000, 2100)):
            part = run_norm(x[lo:hi], res[lo:hi], w, True, 1e-5, group, fmt)
            for m in part:
                assert np.array_equal(part[m], all_[m][lo:hi]), m


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("n", [5, 2100])
def test_norm_in_place_and_optional_outputs(bf16, n):
    say("norm in place", bf16, n)
    x, res, w = make(9, n, 1024, bf16, True)
    want = run_norm(x, res, w, bf16, 1e-6, 128, 0)
    for place in ("x", "res"):
        got = run_norm(x, res, w, bf16, 1e-6, 128, 0, in_place=place)
        assert all(np.array_equal(got[m], want[m]) for m in want)
    got = run_norm(x, res, w, bf16, 1e-6, 128, 0, keep=False)
    assert all(np.array_equal(got[m], want[m]) for m in got)
    got = run_norm(x, res, w, bf16, 1e-6, 128, 0, codes=False)
    assert all(np.array_equal(got[m], want[m]) for m in got)


# ---- backward -----------------------------------------------------------------------------------


def run_backward(dy, h, w, rstd, dres, bf16, place=None, dweight=True):
    n, hidden = dy.shape
    dyd, hd, wd, rd = Out(dy.nbytes, dy), up(h), up(w), up(rstd)
    dd = None if dres is None else Out(dres.nbytes, dres)
    dx = {"dy": dyd, "dres": dd}.get(place) or Out(dy.nbytes)
    dw = Out(hidden * 4)
    ws = Out(min(n, tk.TK_RMSNORM_PARTS) * hidden * 4)
    rc = tk.tk_rmsnorm_backward(dyd.at, hd, tk.TK_DTYPE_BF16 if bf16 else tk.TK_DTYPE_FP32, wd, rd, dd and dd.at, n,
                                hidden, dx.at, dw.at if dweight else None, ws.at if dweight else None)
    assert rc == OK, tk.tk_status_str(rc)
    torch.cuda.synchronize()
    ws.get(np.uint8)
    return dx.get(np.uint16 if bf16 else np.float32).reshape(n, hidden), dw.get(np.float32)


def check_backward(dy, h, w, rstd, dres, bf16, dx, dw):
    n, hidden = dy.shape
    dyv, hv, rv = value(dy, bf16), value(h, bf16), value(dres, bf16)
    want, want_w = ref.norm_backward(dyv, hv, w, rstd, rv)
    r = rstd.astype(np.float64)[:, None]
    a, g = np.abs(hv * r), np.abs(dyv.astype(np.float64) * w)
    mag = (g * a).mean(1, keepdims=True)
    # roundings: a and g one each, a product three; a sum of `hidden` terms at most the additions on one lane
    # (32) + over the lanes (6) + over the waves (16); the last steps' own on what they add
    terms = r * (g * 4 + a * mag * (32 + 6 + 16 + 8)) + (np.abs(rv) if rv is not None else 0)
    bound = ref.U32 * terms + (ref.UB16 if bf16 else ref.U32) * np.abs(want) * (1 + 2.0 ** -7) + 2.0 ** -133
    err = np.abs(value(dx, bf16).astype(np.float64) - want)
    assert np.all(err <= bound), f"dx off by {np.max(err / bound):.2f} of its bound"
    # rows one after the other in a part, then 32 parts in order and 16 sums of those
    depth = -(-n // tk.TK_RMSNORM_PARTS) + 32 + 16 + 4
    bound_w = ref.U32 * depth * (np.abs(dyv.astype(np.float64)) * a).sum(0)
    err = np.abs(dw - want_w)
    assert np.all(err <= bound_w), f"dweight off by {np.max(err / bound_w):.2f} of its bound"


BWD_SHAPES = [(1, 8), (2, 24), (1, 7168), (5, 520), (33, 1024), (600, 64), (1025, 2016), (513, 4096), (40, 8200),
              (9, 16384), (3, 32768), (2, 32760), (1600, 7168)]


@pytest.mark.parametrize("n,hidden", BWD_SHAPES)
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("skip", [True, False])
def test_backward(n, hidden, bf16, skip):
    say("norm backward", n, hidden, bf16, skip)
    dy, dres, w = make(n + hidden, n, hidden, bf16, skip)
    h, _, _ = make(n + hidden + 1, n, hidden, bf16, False, 4.0)
    rstd = ref.norm(value(h, bf16), w, 1e-6)[0].astype(np.float32)
    dx, dw = run_backward(dy, h, w, rstd, dres, bf16)
    check_backward(dy, h, w, rstd, dres, bf16, dx, dw)


def test_backward_of_the_forward_is_the_difference_quotient():
    say("norm backward differences")
    n, hidden, eps = 6, 264, 1e-5
    x, res, w = make(3, n, hidden, False, True)
    f = run_norm(x, res, w, False, eps, 0, 0)
    dy = make(4, n, hidden, False, False)[0]
    dx, dw = run_backward(dy, f["h"], w, f["rstd"], None, False)
    rng, t = np.random.default_rng(5), 1e-4
    h = f["h"].astype(np.float64)
    e = float(np.float32(eps))
    for _ in range(4):
        u, v = rng.standard_normal(h.shape), rng.standard_normal(hidden)

        def loss(s):
            hh = h + s * u
            return (dy * hh / np.sqrt(np.square(hh).mean(1, keepdims=True) + e) * (w + s * v)).sum()

        slope, got = (loss(t) - loss(-t)) / (2 * t), (dx * u).sum() + (dw * v).sum()
        # fp32 gradients of about 1600 terms of order 1 (half a step each, times some ten roundings), and t^2
        assert abs(slope - got) <= 1600 * 10 * ref.U32 + 1e-5


def test_backward_in_place_without_dweight_and_empty():
    say("norm backward variants")
    for bf16 in (True, False):
        dy, dres, w = make(11, 700, 2048, bf16, True)
        h = make(12, 700, 2048, bf16, False, 4.0)[0]
        rstd = ref.norm(value(h, bf16), w, 1e-6)[0].astype(np.float32)
        dx, dw = run_backward(dy, h, w, rstd, dres, bf16)
        for place in ("dy", "dres"):
            dx2, dw2 = run_backward(dy, h, w, rstd, dres, bf16, place)
            assert np.array_equal(dx, dx2) and np.array_equal(dw, dw2)
        dx2, _ = run_backward(dy, h, w, rstd, dres, bf16, dweight=False)
        assert np.array_equal(dx, dx2)
    dw = torch.full((2048,), 7.0, device=DEV)
    assert tk.tk_rmsnorm_backward(None, None, 0, None, None, None, 0, 2048, None, dw, None) == OK
    assert not dw.any()


@pytest.mark.parametrize("hidden", [8, 512, 520, 1024, 4096, 8192, 8200, 16392, 32768])
@pytest.mark.parametrize("bf16", [True, False])
def test_backward_rows_do_not_depend_on_their_number(hidden, bf16):
    say("norm backward batch", hidden, bf16)
    n = 1100
    dy, dres, w = make(hidden, n, hidden, bf16, True)
    h = make(hidden + 1, n, hidden, bf16, False, 4.0)[0]
    rstd = ref.norm(value(h, bf16), w, 1e-6)[0].astype(np.float32)
    for skip in (dres, None):
        whole, _ = run_backward(dy, h, w, rstd, skip, bf16)
        for rows in (slice(0, 1), slice(3, 40), slice(76, 1100)):
            part, _ = run_backward(dy[rows], h[rows], w, rstd[rows], None if skip is None else skip[rows], bf16)
            assert np.array_equal(whole[rows], part), rows


@pytest.mark.parametrize("n,hidden", [(3, 8), (32, 64), (255, 1016), (257, 2048), (1023, 1024), (1024, 72), (1025, 72), (700, 7168),
                                      (33, 16384), (64, 20480)])
@pytest.mark.parametrize("bf16", [True, False])
def test_backward_of_few_rows(n, hidden, bf16):
    say("norm backward few rows", n, hidden, bf16)
    dy, dres, w = make(n * hidden, n, hidden, bf16, True)
    h = make(n * hidden + 1, n, hidden, bf16, False, 4.0)[0]
    rstd = ref.norm(value(h, bf16), w, 1e-6)[0].astype(np.float32)
    dx, dw = run_backward(dy, h, w, rstd, dres, bf16)
    check_backward(dy, h, w, rstd, dres, bf16, dx, dw)
    for place in ("dy", "dres"):
        dx2, dw2 = run_backward(dy, h, w, rstd, dres, bf16, place)
        assert np.array_equal(dx, dx2) and np.array_equal(dw, dw2), place


@pytest.mark.parametrize("n,hidden", [(1025, 8), (1031, 168), (4099, 504), (1030, 512), (1037, 520), (2500, 1016), (1100, 1024),
                                      (1026, 1032), (1030, 16392), (1025, 32768)])
@pytest.mark.parametrize("bf16", [True, False])
def test_backward_of_narrow_and_wide_rows(n, hidden, bf16):
    say("norm backward narrow and wide", n, hidden, bf16)
    dy, dres, w = make(n + hidden, n, hidden, bf16, True)
    h = make(n + hidden + 1, n, hidden, bf16, False, 4.0)[0]
    rstd = ref.norm(value(h, bf16), w, 1e-6)[0].astype(np.float32)
    dx, dw = run_backward(dy, h, w, rstd, dres, bf16)
    check_backward(dy, h, w, rstd, dres, bf16, dx, dw)
    dx2, dw2 = run_backward(dy, h, w, rstd, dres, bf16, "dy")
    assert np.array_equal(dx, dx2) and np.array_equal(dw, dw2)
    few, _ = run_backward(dy[-9:], h[-9:], w, rstd[-9:], dres[-9:], bf16)
    assert np.array_equal(dx[-9:], few)


def test_backward_without_dweight_of_any_width():
    say("norm backward without dweight")
    for n, hidden in ((5, 32768), (1200, 24), (700, 1024), (3, 16392), (2000, 520)):
        dy, dres, w = make(n, n, hidden, True, True)
        h = make(n + 1, n, hidden, True, False, 4.0)[0]
        rstd = ref.norm(value(h, True), w, 1e-6)[0].astype(np.float32)
        want, _ = run_backward(dy, h, w, rstd, dres, True)
        got, _ = run_backward(dy, h, w, rstd, dres, True, dweight=False)
        assert np.array_equal(got, want), (n, hidden)


def border_rows(hidden):
    """fp32 rows whose sums of squares lie within a few units of the 64-bit last place of where 1/rms rounds to the next
    fp32 number, and differ by four of those units with the order of the sum: eight squares just below 2^-53 count
    beside each other, and not one by one beside a 1."""
    steps = -(-hidden // 512)
    half = (steps + 1) // 2
    r = np.float32(np.sqrt(hidden / 1.4))
    mid = (float(r) + float(np.nextafter(r, np.float32(0)))) / 2
    rows = np.zeros((49, hidden), np.float32)
    for j in range(49):
        rows[j, 0] = 1
        rows[j, half * 512:half * 512 + 8] = np.nextafter(np.float32(2.0 ** -26.5), np.float32(0))
        rest = hidden / mid ** 2 - 1 + (j - 24 - 2) * 2.0 ** -52
        for i in range(3):  # what is left of the sum, by squares of fp32 numbers
            a = np.float32(np.sqrt(rest))
            if float(a) ** 2 > rest:
                a = np.nextafter(a, np.float32(0))
            rows[j, 512 + 8 * i] = a
            rest -= float(a) ** 2
    return rows


@pytest.mark.parametrize("hidden", [2560, 7168, 8192])
def test_norm_rows_do_not_depend_on_their_number_at_a_rounding_border(hidden):
    say("norm batch border", hidden)
    x = border_rows(hidden)
    w = np.ones(hidden, np.float32)
    few = run_norm(x, None, w, False, 0.0, 0, 0)
    many = run_norm(np.tile(x, (21, 1)), None, w, False, 0.0, 0, 0)
    # the sums' last bits decide on the way to fp32: both neighbours appear
    assert len(np.unique(few["rstd"])) == 2
    for m in few:
        assert np.array_equal(np.tile(few[m], (21,) + (1,) * (few[m].ndim - 1)), many[m]), m


@pytest.mark.parametrize("hidden", [2304, 7168, 12288])
def test_norm_fp32_rows_of_many_magnitudes_do_not_depend_on_their_number(hidden):
    say("norm batch fp32", hidden)
    rng = np.random.default_rng(hidden)
    x = (rng.standard_normal((1100, hidden)) * 2.0 ** rng.integers(-40, 40, (1100, hidden))).astype(np.float32)
    w = (1 + 0.25 * rng.standard_normal(hidden)).astype(np.float32)
    whole = run_norm(x, None, w, False, 1e-6, 128, 0)
    for lo, hi in ((0, 1), (600, 1100)):
        part = run_norm(x[lo:hi], None, w, False, 1e-6, 128, 0)
        for m in part:
            assert np.array_equal(part[m], whole[m][lo:hi]), m


@pytest.mark.parametrize("n,hidden", [(333, 1024), (1024, 1024), (512, 8192), (300, 16384), (1030, 16392), (1600, 20480),   # columns summed apart
                                      (4099, 504), (16000, 512), (5000, 1016), (9001, 2048),                               # several rows a workgroup
                                      (1025, 4096), (3000, 7168), (1100, 8192), (600, 12616)])                             # one
@pytest.mark.parametrize("bf16", [True, False])
def test_backward_dweight_within_its_roundings(n, hidden, bf16):
    """Two roundings a product, then the longest chain of additions: up to 256 parts of the rows one after the other in
    each, eight rows of a workgroup, 16 parts in order and 16 sums of those; or 32 or 64 parts in batches of eight."""
    say("norm backward dweight", n, hidden, bf16)
    dy, _, w = make(n + hidden, n, hidden, bf16, False)
    h, _, _ = make(n + hidden + 1, n, hidden, bf16, False, 4.0)
    rstd = ref.norm(value(h, bf16), w, 1e-6)[0].astype(np.float32)
    _, dw = run_backward(dy, h, w, rstd, None, bf16)
    terms = value(dy, bf16).astype(np.float64) * (value(h, bf16) * rstd.astype(np.float64)[:, None])
    depth = 2 + max(-(-n // 256) + 8 + 16 + 16, -(-n // (32 * 8)) + 8 + 2 + 16)
    assert np.all(np.abs(dw - terms.sum(0)) <= ref.U32 * depth * np.abs(terms).sum(0))
    # and in norm: roundings of random terms are independent, so that their sum grows with the root of the depth
    assert np.linalg.norm(dw - terms.sum(0)) <= ref.U32 * np.sqrt(depth) * np.linalg.norm(np.abs(terms).sum(0))
