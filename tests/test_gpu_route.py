"""tk_route and tk_route_backward on the GPU against the plain 64-bit reference:
indices equal, weights within their one rounding, gradients within bounds that
count roundings."""
import numpy as np
import pytest
import torch

import layer_ref as ref
import moe_activation_bit_amd as tk

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
OK = tk.TkStatus.TK_OK
PAD = 64


def say(*a):
    print("[gpu-case]", *a, flush=True)


def up(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def make(seed, T, E, bf16, masked=0.0, sigma=2.0):
    rng = np.random.default_rng(seed)
    x = (sigma * rng.standard_normal((T, E))).astype(np.float32)
    x[rng.random((T, E)) < masked] = -np.inf
    return ref.round_bf16(x) if bf16 else x, (0.1 * rng.standard_normal(E)).astype(np.float32)


def run_route(x, bf16, bias, k, ng, tg, softmax, normalise, scale=2.5):
    T, E = x.shape
    idx = torch.full((T * k + 2 * PAD,), -77, dtype=torch.int32, device=DEV)
    w = torch.full((T * k + 2 * PAD,), -77.0, dtype=torch.float32, device=DEV)
    xd = up(ref.bf16_bits(x).view(np.int16)) if bf16 else up(x)
    rc = tk.tk_route(xd, tk.TK_DTYPE_BF16 if bf16 else tk.TK_DTYPE_FP32, up(bias), T, E, k, ng, tg,
                     tk.TK_SCORE_SOFTMAX if softmax else tk.TK_SCORE_SIGMOID, normalise, scale,
                     idx.data_ptr() + 4 * PAD, w.data_ptr() + 4 * PAD)
    assert rc == OK, tk.tk_status_str(rc)
    torch.cuda.synchronize()
    i, ww = idx.cpu().numpy(), w.cpu().numpy()
    for a in (i, ww):
        assert (a[:PAD] == -77).all() and (a[PAD + T * k:] == -77).all(), "canary"
    return i[PAD:PAD + T * k].reshape(T, k), ww[PAD:PAD + T * k].reshape(T, k)


def check_route(x, bias, k, ng, tg, softmax, normalise, got, scale=2.5):
    idx, w = ref.route(x, bias, k, ng, tg, softmax, normalise, scale)
    assert np.array_equal(got[0], idx), f"indices differ at {np.argwhere(got[0] != idx)[:3].tolist()}"
    assert np.array_equal(np.isnan(got[1]), np.isnan(w))
    # computed in 64 bits and rounded once (2^-149: half the smallest fp32 step, and room for its 64-bit error)
    assert np.all(np.isnan(w) | (np.abs(got[1] - w) <= ref.U32 * (1 + 2.0 ** -10) * np.abs(w) + 2.0 ** -149)), "weights"


SHAPES = [  # experts, k, groups, kept groups
    (1, 1, 1, 1), (2, 2, 1, 1), (8, 2, 1, 1), (33, 5, 1, 1), (60, 4, 1, 1), (64, 6, 1, 1), (64, 64, 1, 1), (100, 3, 1, 1),
    (128, 8, 1, 1), (129, 9, 1, 1), (160, 6, 1, 1), (256, 8, 1, 1), (256, 16, 1, 1), (256, 17, 1, 1), (300, 8, 1, 1),
    (384, 8, 1, 1), (512, 8, 1, 1), (512, 64, 1, 1), (500, 33, 1, 1),
    (256, 8, 8, 4), (256, 8, 8, 1), (256, 8, 8, 8), (256, 8, 4, 2), (256, 4, 2, 1), (160, 6, 8, 3), (96, 5, 3, 2),
    (72, 4, 8, 2), (64, 8, 32, 4), (512, 8, 16, 8), (512, 8, 256, 9), (100, 7, 5, 2), (128, 16, 8, 4), (64, 4, 4, 2),
    (192, 8, 8, 4), (14, 3, 7, 2),
]


@pytest.mark.parametrize("E,k,ng,tg", SHAPES)
@pytest.mark.parametrize("softmax", [False, True])
def test_route(E, k, ng, tg, softmax):
    say("route", E, k, ng, tg, softmax)
    for n, (T, bf16, with_bias, normalise, masked) in enumerate([
            (1, False, True, 1, 0.0), (37, False, True, 1, 0.0), (64, True, False, 0, 0.0), (18, True, True, 0, 0.3),
            (13, False, False, 1, 0.9), (5, True, True, 1, 0.99)]):
        x, bias = make(E * 100 + k + n, T, E, bf16, masked)
        b = bias if with_bias else None
        check_route(x, b, k, ng, tg, softmax, normalise, run_route(x, bf16, b, k, ng, tg, softmax, normalise))


@pytest.mark.parametrize("E,k,ng,tg", [
    (96, 4, 3, 2), (384, 8, 3, 2), (192, 8, 3, 1), (130, 6, 13, 5), (33, 4, 11, 4), (45, 5, 9, 3), (500, 8, 10, 4),
    (30, 4, 15, 15), (12, 3, 6, 3), (510, 16, 15, 8), (496, 8, 16, 4), (40, 16, 5, 5), (306, 7, 6, 2), (62, 2, 2, 1),
])
@pytest.mark.parametrize("softmax", [False, True])
def test_route_groups_of_any_size(E, k, ng, tg, softmax):
    say("route any groups", E, k, ng, tg, softmax)
    for n, (T, bf16, with_bias, normalise, masked) in enumerate([
            (1, False, True, 1, 0.0), (41, False, False, 1, 0.0), (22, True, True, 0, 0.3), (9, False, True, 1, 0.97)]):
        x, bias = make(E * 100 + k + n, T, E, bf16, masked)
        b = bias if with_bias else None
        check_route(x, b, k, ng, tg, softmax, normalise, run_route(x, bf16, b, k, ng, tg, softmax, normalise))
    # every key equal, and whole groups masked
    x = np.zeros((5, E), np.float32)
    x[1, :E // ng] = -np.inf
    x[2, E // ng:] = -np.inf
    x[3] = -np.inf
    x[4, ::2] = -np.inf
    check_route(x, None, k, ng, tg, softmax, 1, run_route(x, False, None, k, ng, tg, softmax, 1))


@pytest.mark.parametrize("E,k,ng,tg", [(256, 8, 8, 4), (64, 6, 1, 1), (512, 8, 16, 8), (160, 6, 8, 3), (128, 8, 1, 1), (96, 4, 3, 2)])
@pytest.mark.parametrize("spread", [0, 2.0 ** -25, 2.0 ** -23, 2.0 ** -21, 2.0 ** -19, 2.0 ** -16])
@pytest.mark.parametrize("offset", [0.0, 1.0, -1000.0])
def test_route_keys_that_nearly_tie(E, k, ng, tg, spread, offset):
    """Scores that the bias brings to within a few units of each other's last place: an order that only exact scores
    tell, or (offset) that the sum's rounding makes a tie."""
    say("route near ties", E, k, ng, tg, spread, offset)
    T = 48
    rng = np.random.default_rng(E + k)
    x = (3 * rng.standard_normal((T, E))).astype(np.float32)
    x[:, 1:] = x[:1, 1:]  # one bias for all: the rows' other logits are equal
    x[:, 0] += 8 * rng.random(T).astype(np.float32)
    s = ref.scores(x[:1], False)[0]
    bias = (offset + 0.7 - s + spread * rng.standard_normal(E)).astype(np.float32)
    for T_ in (T, 3):
        check_route(x[:T_], bias, k, ng, tg, False, 1, run_route(x[:T_], False, bias, k, ng, tg, False, 1))
    # values of groups that cancel: keys of opposite signs
    if ng > 1:
        per = E // ng
        b = bias.copy()
        b[::per] += 500
        b[1::per] -= 500
        for g in range(ng):
            b[g * per + 2:(g + 1) * per] -= 2000
        check_route(x, b, min(k, 2 * tg), ng, tg, False, 1, run_route(x, False, b, min(k, 2 * tg), ng, tg, False, 1))


@pytest.mark.parametrize("E,k,ng,tg", [(256, 8, 8, 4), (64, 6, 1, 1), (512, 8, 16, 8), (160, 8, 8, 3)])
def test_route_ties_extremes_and_masks(E, k, ng, tg):
    say("route values", E, k, ng, tg)
    rng = np.random.default_rng(E)
    x, bias = make(E, 24, E, False)
    x[0] = 0.0                                         # every expert ties
    x[1] = rng.integers(-2, 3, E)                      # many ties
    x[2] = -np.inf                                     # nothing remains
    x[3] = -np.inf
    x[3, E // 2] = 1.0                                 # one remains
    x[4] = 40 + rng.standard_normal(E)                 # sigmoid saturates: equal rounded scores
    x[5] = -300 - 50 * rng.random(E)                   # scores below fp32
    x[6] = -3e38
    x[7] = np.where(rng.random(E) < 0.5, 3e38, -3e38)
    x[8, ::2] = -np.inf
    x[9] = np.where(np.arange(E) < E - 1, -np.inf, -1000.0)
    x[10, 3] = np.nan
    x[11] = np.nan
    x[12, 5] = np.inf
    x[13, 1], x[13, 2] = np.inf, -np.inf
    x[14] = np.finfo(np.float32).tiny * rng.standard_normal(E)
    x[15] = -0.0
    x[15, ::3] = 0.0
    b2 = bias.copy()
    b2[::5] = -np.inf                                  # masked by the bias
    b2[3] = 3e38
    for softmax in (False, True):
        for normalise in (0, 1):
            for b in (None, bias, b2, np.zeros(E, np.float32)):
                check_route(x, b, k, ng, tg, softmax, normalise, run_route(x, False, b, k, ng, tg, softmax, normalise))


def test_route_tokens_do_not_depend_on_their_number():
    say("route batch")
    x, bias = make(1, 3000, 256, False)
    i, w = run_route(x, False, bias, 8, 8, 4, False, 1)
    for lo, hi in ((0, 1), (5, 8), (2990, 3000)):
        i2, w2 = run_route(x[lo:hi], False, bias, 8, 8, 4, False, 1)
        assert np.array_equal(i[lo:hi], i2) and np.array_equal(w[lo:hi].view(np.uint32), w2.view(np.uint32))


def test_route_large():
    say("route large")
    for E, k, ng, tg, softmax, bf16, masked in ((256, 8, 8, 4, False, False, 0.0), (64, 6, 1, 1, True, True, 0.1)):
        x, bias = make(2, 20000, E, bf16, masked)
        b = bias if ng > 1 else None
        check_route(x, b, k, ng, tg, softmax, ng > 1, run_route(x, bf16, b, k, ng, tg, softmax, ng > 1))


# ---- backward -----------------------------------------------------------------------------------


def run_backward(dw, idx, x, bf16, softmax, normalise, scale=2.5):
    T, E = x.shape
    k, item = idx.shape[1], 2 if bf16 else 4
    out = torch.full((T * E * item + 2 * PAD,), 0xC3, dtype=torch.uint8, device=DEV)
    xd = up(ref.bf16_bits(x).view(np.int16)) if bf16 else up(x)
    rc = tk.tk_route_backward(up(dw), up(idx), xd, tk.TK_DTYPE_BF16 if bf16 else tk.TK_DTYPE_FP32, T, E, k,
                              tk.TK_SCORE_SOFTMAX if softmax else tk.TK_SCORE_SIGMOID, normalise, scale,
                              out.data_ptr() + PAD)
    assert rc == OK, tk.tk_status_str(rc)
    torch.cuda.synchronize()
    o = out.cpu().numpy()
    assert (o[:PAD] == 0xC3).all() and (o[PAD + T * E * item:] == 0xC3).all(), "canary"
    body = o[PAD:PAD + T * E * item]
    return (ref.bf16_value(body.view(np.uint16)) if bf16 else body.view(np.float32)).reshape(T, E)


def check_backward(dw, idx, x, bf16, softmax, normalise, got):
    want, mag = ref.route_backward(dw, idx, x, softmax, normalise, 2.5)
    live = x[np.isfinite(x)]
    reach = float(live.max() - live.min()) if live.size else 0.0
    # an fp32 exponential's argument is off by half a step of its size, twice where a score is a ratio of them;
    # the sums' depth is 8 additions on a lane and 6 over the lanes, twice; some 16 roundings besides
    bound = ref.U32 * mag * (3 * reach + 2 * 14 + 16) + (ref.UB16 if bf16 else ref.U32) * np.abs(want) + 2.0 ** -126
    err = np.abs(got - want)
    assert np.all(err <= bound), f"off by {np.max(err / bound):.2f} of the bound"


@pytest.mark.parametrize("E,k", [(1, 1), (8, 2), (33, 5), (64, 6), (100, 8), (160, 6), (256, 8), (300, 64), (512, 8)])
@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("normalise", [0, 1])
def test_backward(E, k, softmax, normalise):
    say("route backward", E, k, softmax, normalise)
    for n, (T, bf16, masked) in enumerate([(1, False, 0.0), (41, False, 0.0), (23, True, 0.0), (18, False, 0.4)]):
        rng = np.random.default_rng(E * 10 + k + n)
        x, _ = make(E + n, T, E, bf16, masked)
        idx, _ = ref.route(x, None, k, 1, 1, softmax, normalise, 2.5)
        idx[rng.random(idx.shape) < 0.05] = -1
        dw = rng.standard_normal((T, k)).astype(np.float32)
        check_backward(dw, idx, x, bf16, softmax, normalise, run_backward(dw, idx, x, bf16, softmax, normalise))


@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("normalise", [0, 1])
def test_backward_absent_repeated_and_extreme(softmax, normalise):
    say("route backward values", softmax, normalise)
    rng = np.random.default_rng(3)
    x, _ = make(7, 12, 48, False)
    idx = np.argsort(-x, axis=1, kind="stable")[:, :6].astype(np.int32)
    idx[0] = -1                                   # every slot absent
    idx[1, 2:] = [idx[1, 0], 48, -5, idx[1, 1]]   # repeats and entries out of range
    x[2] = -200 - 5 * rng.random(48)              # scores below fp32 share the weight all the same
    x[3] = 60 + rng.standard_normal(48)           # saturated
    x[4, idx[4, 1:]] = -np.inf                    # masked but for one
    dw = rng.standard_normal((12, 6)).astype(np.float32)
    dw[5] = 0
    got = run_backward(dw, idx, x, False, softmax, normalise)
    check_backward(dw, idx, x, False, softmax, normalise, got)
    assert not got[0].any() and not got[5].any()


@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("normalise", [0, 1])
def test_backward_of_the_forward_is_the_difference_quotient(softmax, normalise):
    say("route backward differences", softmax, normalise)
    x, bias = make(9, 16, 64, False, sigma=1.0)
    idx, _ = run_route(x, False, bias, 6, 8, 4, softmax, normalise)
    rng, t = np.random.default_rng(1), 1e-4
    dw = rng.standard_normal(idx.shape).astype(np.float32)
    g = run_backward(dw, idx, x, False, softmax, normalise).astype(np.float64)
    for _ in range(4):
        u = rng.standard_normal(x.shape)

        def loss(s):
            p = ref.scores(x.astype(np.float64) + s * u, softmax)
            w = np.take_along_axis(p, idx.astype(np.int64), 1)
            return 2.5 * (dw * (w / w.sum(1, keepdims=True) if normalise else w)).sum()

        # about 100 terms of order 1, some 30 roundings each, and t^2
        assert abs((loss(t) - loss(-t)) / (2 * t) - (g * u).sum()) <= 100 * 30 * ref.U32 + 1e-6


def check_backward_in_64_bits(dw, idx, x, bf16, softmax, normalise, got):
    """Half a step of the result's type, however much the formula's differences cancel: everything before it is in 64
    bits (an exponential's argument of up to 2^11 is off by 2^-53 of its size, some 30 roundings besides: 2^-40 of the
    terms' magnitudes).  Softmax over all experts: its fp32 exponentials are off by u, half a step for each unit of
    their arguments and two for their own; so is a result, and by u of sum_i s_i |d_e - d_i|, what its difference is
    the sum of; an unchosen expert's takes two more roundings."""
    want, mag = ref.route_backward(dw, idx, x, softmax, normalise, 2.5)
    steps, more = ref.U32, 0.0
    if softmax and not normalise:
        u = ref.U32 * (float(x.max() - x.min()) + 2)
        d = np.zeros(x.shape)
        for t, row in enumerate(idx):
            for j, e in enumerate(row):
                if e >= 0:
                    d[t, e] = 2.5 * float(dw[t, j])
        s = ref.scores(x, True)
        steps, more = 3 * ref.U32 + 2 * u, u * s * (s[:, None, :] * np.abs(d[:, :, None] - d[:, None, :])).sum(2)
    bound = ((ref.UB16 + steps) if bf16 else steps) * (1 + 2.0 ** -10) * np.abs(want) + more + 2.0 ** -40 * mag + 2.0 ** -133
    err = np.abs(got - want)
    assert np.all(err <= bound), f"off by {np.max(err / bound):.2f} of the bound"


@pytest.mark.parametrize("E,k", [(8, 1), (8, 2), (64, 2), (100, 6), (256, 8), (512, 16), (64, 17), (300, 33)])
@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("normalise", [0, 1])
def test_backward_whose_differences_cancel(E, k, softmax, normalise):
    """Gradients that are nearly equal for all chosen experts, and experts that take nearly all of the weight: d - dot
    is a small difference of large numbers."""
    say("route backward cancelling", E, k, softmax, normalise)
    rng = np.random.default_rng(E + k)
    for n, (bf16, spread, lead) in enumerate([(False, 1e-3, 0.0), (False, 1e-6, 0.0), (False, 1.0, 9.0), (False, 1.0, 16.0),
                                              (True, 1e-3, 0.0), (True, 1.0, 9.0)]):
        x, _ = make(E + k + n, 37, E, bf16)
        x[np.arange(37), rng.integers(0, E, 37)] += np.float32(lead)
        x = ref.round_bf16(x) if bf16 else x
        idx, _ = ref.route(x, None, k, 1, 1, softmax, normalise, 2.5)
        idx[rng.random(idx.shape) < 0.02] = -1
        dw = (1 + spread * rng.standard_normal((37, k))).astype(np.float32)
        check_backward_in_64_bits(dw, idx, x, bf16, softmax, normalise, run_backward(dw, idx, x, bf16, softmax, normalise))


@pytest.mark.parametrize("k", [2, 20])
@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("normalise", [0, 1])
def test_backward_shows_nan_in_its_own_token(k, softmax, normalise):
    say("route backward nan", k, softmax, normalise)
    x, _ = make(5, 6, 64, False)
    idx, _ = ref.route(x, None, k, 1, 1, softmax, normalise, 2.5)
    dw = np.random.default_rng(1).standard_normal((6, k)).astype(np.float32)
    clean = run_backward(dw, idx, x, False, softmax, normalise)
    xn, dn = x.copy(), dw.copy()
    xn[1, idx[1, 1]] = np.nan
    if softmax:
        xn[2, idx[2, 0]] = np.inf
    dn[4, 1] = np.nan
    got = run_backward(dn, idx, xn, False, softmax, normalise)
    for t in (1, 4) + ((2,) if softmax else ()):
        assert np.isnan(got[t, idx[t, 1 if t != 2 else 0]]), t
    for t in (0, 3, 5):
        assert np.array_equal(got[t], clean[t])


# With the shapes above every form of the kernels: 64 experts by eight and by four tokens a wave, the compiled-in counts
# and the others in one to four lists a lane, each with top-8 and another k, and one token a wave at every 64 experts.
MORE_SHAPES = [
    (64, 8, 1, 1), (64, 3, 1, 1), (64, 8, 8, 4), (64, 8, 4, 2), (64, 8, 16, 16), (64, 12, 1, 1), (64, 5, 2, 1),
    (33, 8, 1, 1), (100, 8, 1, 1), (128, 6, 1, 1), (128, 8, 8, 2), (160, 8, 1, 1), (192, 8, 1, 1), (192, 6, 8, 4),
    (200, 8, 1, 1), (200, 6, 1, 1), (256, 6, 1, 1), (256, 6, 8, 4), (256, 6, 8, 8), (300, 6, 1, 1), (384, 6, 1, 1),
    (384, 8, 8, 4), (500, 8, 1, 1), (500, 6, 1, 1), (512, 6, 1, 1), (512, 6, 16, 8), (100, 20, 1, 1), (150, 20, 1, 1),
    (300, 17, 1, 1), (384, 17, 1, 1), (448, 17, 1, 1), (40, 8, 20, 10), (12, 8, 1, 1), (8, 8, 4, 4),
]


@pytest.mark.parametrize("E,k,ng,tg", MORE_SHAPES)
@pytest.mark.parametrize("softmax", [False, True])
def test_route_every_form(E, k, ng, tg, softmax):
    say("route every form", E, k, ng, tg, softmax)
    for n, (T, bf16, with_bias, normalise, masked) in enumerate([
            (1, False, True, 1, 0.0), (75, False, False, 0, 0.0), (66, True, True, 1, 0.2), (35, False, True, 0, 0.95),
            (50, True, False, 1, 0.5)]):
        x, bias = make(E * 1000 + k * 10 + n, T, E, bf16, masked)
        b = bias if with_bias else None
        check_route(x, b, k, ng, tg, softmax, normalise, run_route(x, bf16, b, k, ng, tg, softmax, normalise))
    # ties (of all, and of a few values), empty rows, one expert left, NaN and infinities
    rng = np.random.default_rng(E + k)
    x, bias = make(E + k, 40, E, False)
    x[0], x[1], x[2] = 0.0, -np.inf, -np.inf
    x[2, E - 1] = 3.0
    x[3:20] = rng.integers(-2, 3, (17, E))
    x[20:30][rng.random((10, E)) < 0.9] = -np.inf
    x[30, E // 2], x[31, 0] = np.nan, np.inf
    x[32] = 40 + rng.standard_normal(E)
    x[33] = -300 - 50 * rng.random(E)
    for b in (None, np.zeros(E, np.float32), bias):
        check_route(x, b, k, ng, tg, softmax, 1, run_route(x, False, b, k, ng, tg, softmax, 1))


@pytest.mark.parametrize("E,k,ng,tg", [(64, 8, 1, 1), (64, 8, 8, 4), (64, 6, 1, 1), (256, 8, 8, 4), (512, 8, 16, 8), (160, 6, 8, 3),
                                       (96, 4, 3, 2), (100, 8, 1, 1), (300, 20, 1, 1)])
@pytest.mark.parametrize("spread", [0, 2.0 ** -27, 2.0 ** -24, 2.0 ** -20, 2.0 ** -16])
@pytest.mark.parametrize("softmax", [False, True])
def test_route_scores_that_nearly_tie(E, k, ng, tg, spread, softmax):
    say("route near ties of either score", E, k, ng, tg, spread, softmax)
    for seed in range(6):
        rng = np.random.default_rng(E + k + seed)
        x = np.repeat((2 * rng.standard_normal((1, E))).astype(np.float32), 11, 0)
        s = ref.scores(x[:1], softmax)[0]
        bias = (0.7 - s + spread * rng.standard_normal(E)).astype(np.float32)
        check_route(x, bias, k, ng, tg, softmax, 1, run_route(x, False, bias, k, ng, tg, softmax, 1))
