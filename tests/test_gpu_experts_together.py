"""The operators of include/tk_expert.h together and where they are run from: the
training step of examples/moe_train.py stage by stage against plain statements
in 64 bits, the products against their gradients, HIP graphs replayed with eager
work in between, two streams at once, offsets past 32 bits, and values that have
to stay in their own rows."""
import os
import sys

import numpy as np
import pytest
import torch

import expert_ref as ex
import layer_ref as ref
import moe_activation_bit_amd as tk
import oracle
import test_gpu_expert_products as products
import test_gpu_swiglu_backward as swiglu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import moe_train  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
OK = tk.TkStatus.TK_OK
BF16, FP32, FP8, FP4 = tk.TK_DTYPE_BF16, tk.TK_DTYPE_FP32, tk.TK_DTYPE_FP8, tk.TK_DTYPE_FP4


def say(*a):
    print("[gpu-case]", *a, flush=True)


def host(t):
    torch.cuda.synchronize()
    return ref.bf16_value(t.cpu().view(torch.int16).numpy().view(np.uint16)) if t.dtype == torch.bfloat16 else t.cpu().numpy()


def bits(t):
    return t.cpu().view(torch.int16).numpy().view(np.uint16)


@pytest.fixture(scope="module", autouse=True)
def _table():
    assert tk.tk_init(0) == OK  # SwiGLU's, before any capture


def batch(tokens, hidden, experts, k, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn((tokens, hidden), generator=gen, device=DEV).to(torch.bfloat16)
    dout = torch.randn((tokens, hidden), generator=gen, device=DEV).to(torch.bfloat16)
    weight, idx = torch.rand((tokens, experts), generator=gen, device=DEV).topk(k, dim=-1)
    idx = idx.to(torch.int32)
    idx[torch.rand(idx.shape, generator=gen, device=DEV) < 0.1] = -1  # dropped slots
    return x, dout, idx.contiguous(), weight.contiguous()


@pytest.mark.parametrize("tokens,clamp", [(1, float("inf")), (37, 1.0), (300, float("inf"))])
def test_training_step_stage_by_stage(tokens, clamp):
    say("training step", tokens, clamp)
    hidden, inter, experts, k = 256, 384, 8, 3
    b = moe_train.Experts(tokens, hidden, inter, experts, k, clamp)
    x, dout, idx, weight = batch(tokens, hidden, experts, k, tokens)
    for t in (b.h, b.z, b.dact, b.dh, b.drow):
        t.zero_()  # rows past the last are read by the steps between the products
    b.forward(x, idx, weight)
    dx, dweight = b.backward(dout)
    torch.cuda.synchronize()
    n, off, token, pos = b.rows, host(b.offsets), host(b.token), host(b.pos)
    live = np.arange(n) < off[-1]
    rpos, roff = oracle.topk_to_pos(host(idx), experts)
    assert np.array_equal(pos, rpos) and np.array_equal(off, roff)
    for t in range(tokens):
        for j in range(k):
            if pos[t, j] >= 0:
                assert token[pos[t, j]] == t and host(b.weight)[pos[t, j]] == host(weight)[t, j]
    assert np.all(token[~live] == -1)

    def product(codes, scales, index, w, out, got):
        xv = ex.coded(host(codes), host(scales), True)
        wv = ex.coded(host(w[0]).reshape(experts * out, -1), host(w[1]).reshape(experts * out, -1), True)
        wv = wv.reshape(experts, out, -1)
        want, mag = ex.gemm(xv, index, off, n, wv, np.zeros(got.shape))
        lost = np.zeros_like(want)
        for c in range(0, xv.shape[1], 128):  # what 128 products may lose below the largest of them
            for e, (lo, hi) in enumerate(ex.spans(off, n)):
                a = np.abs(ex.take(xv, index, lo, hi)[:, c:c + 128])
                for r in range(lo, hi):
                    lost[r] += 128 * 2.0 ** -13 * (a[r - lo] * np.abs(wv[e][:, c:c + 128])).max(1)
        products.check_sum(got, True, want, mag, 3 * xv.shape[1] // 128, lost)

    product(b.x8, b.x8s, token, b.gate_up8, 2 * inter, host(b.h))
    codes, scales, _ = oracle.swiglu_cast(bits(b.h), host(b.weight), moe_train.GROUP,
                                          None if clamp == float("inf") else clamp, 8, 1)
    assert np.array_equal(host(b.a8), codes) and np.array_equal(host(b.a8s), scales)
    product(b.a8, b.a8s, None, b.down8, hidden, host(b.z))

    zero = np.zeros
    w_down, w_gate = host(b.down).astype(np.float64), host(b.gate_up).astype(np.float64)
    dy = host(dout).astype(np.float64)
    want, mag = ex.dgrad(dy, token, off, n, w_down, zero((n, inter)))
    products.check_sum(host(b.dact), True, want, mag, hidden)
    most = max(hi - lo for lo, hi in ex.spans(off, n))
    want, mag = ex.wgrad(dy, token, ex.coded(host(b.a8), host(b.a8s), True), None, off, n, zero(w_down.shape))
    products.check_sum(host(b.ddown), False, want, mag, most)
    h = ex.coded(host(b.h8), host(b.h8s), True).astype(np.float32)
    swiglu.check((host(b.dh), host(b.drow_weight), None), host(b.dact), h, host(b.weight), clamp)
    dh = host(b.dh).astype(np.float64)
    want, mag = ex.dgrad(dh, None, off, n, w_gate, zero((n, hidden)))
    products.check_sum(host(b.drow), True, want, mag, 2 * inter)
    want, mag = ex.wgrad(dh, None, ex.coded(host(b.x8), host(b.x8s), True), token, off, n, zero(w_gate.shape))
    products.check_sum(host(b.dgate_up), False, want, mag, most)
    got = oracle.moe_reduce(bits(b.drow), pos, host(b.ones), None, 1.0, True)
    assert np.array_equal(bits(dx), got)
    want = np.where(pos < 0, 0, host(b.drow_weight)[np.maximum(pos, 0)])
    assert np.array_equal(host(dweight), want.astype(np.float32))
    # a second micro-batch is added
    first = host(b.ddown), host(b.dgate_up)
    b.backward(dout, accumulate=True)
    for a, t in zip(first, (b.ddown, b.dgate_up)):
        assert np.array_equal(host(t), a + a)


def test_products_and_gradients_are_adjoint():
    """sum dy (W x) = sum (W^T dy) x = sum (dy x^T) W, exactly, in whole numbers."""
    rng = np.random.default_rng(1)
    counts = [30, 0, 71, 5]
    off, n, e, out_f, in_f = products.offsets_of(counts), sum(counts), 4, 200, 216
    x, dy = products.whole(rng, (n, in_f)), products.whole(rng, (n, out_f))
    w = products.whole(rng, (e, out_f, in_f))
    y, dx = torch.zeros((n, out_f), device=DEV), torch.zeros((n, in_f), device=DEV)
    dw = torch.zeros((e, out_f, in_f), device=DEV)
    xd, dyd, wd, offd = products.bf16(x), products.bf16(dy), products.bf16(w), products.dev(off)
    assert tk.tk_expert_gemm(xd, None, BF16, 0, 0, n, None, offd, n, wd, None, BF16, 0, 0, e, out_f, in_f, FP32, y) == OK
    assert tk.tk_expert_gemm_dgrad(dyd, n, None, offd, n, wd, e, out_f, in_f, FP32, dx) == OK
    assert tk.tk_expert_gemm_wgrad(dyd, n, None, xd, None, BF16, 0, n, None, offd, n, e, out_f, in_f, 0, FP32, dw) == OK
    sums = [(a.astype(np.int64) * b.astype(np.int64)).sum() for a, b in
            ((dy, host(y)), (x, host(dx)), (w, host(dw)))]
    assert sums[0] == sums[1] == sums[2]


def test_prefill_and_decode_with_the_same_weights():
    """The rows of tk_expert_gemm and of tk_expert_gemv_fp4 from the same 4-bit weights and FP8 activations."""
    rng = np.random.default_rng(2)
    tokens, k, e, out_f, in_f = 24, 4, 8, 320, 512
    xc, xs, x = products.fp8_operand(rng, tokens, in_f, "ue8m0", 128)
    wc, ws, w = products.fp8_operand(rng, e * out_f, in_f, "ue8m0", 32, fp4=True)
    idx = np.argsort(rng.random((tokens, e)), axis=1)[:, :k].astype(np.int32)
    idx[3, 1] = idx[7, 0] = -1
    args = [products.dev(a) for a in (xc, xs, idx, wc, ws)]
    pos, off = (torch.zeros(s, dtype=torch.int32, device=DEV) for s in ((tokens, k), (e + 1,)))
    assert tk.tk_topk_to_pos(args[2], tokens, k, e, pos, off) == OK
    n = tokens * k
    token = np.full(n, -1, np.int32)
    p = host(pos)
    token[p[p >= 0]] = np.nonzero(p >= 0)[0]
    rows = torch.zeros((n, out_f), dtype=torch.bfloat16, device=DEV)
    slots = torch.zeros((n, out_f), dtype=torch.bfloat16, device=DEV)
    assert tk.tk_expert_gemm(args[0], args[1], FP8, 1, 128, tokens, products.dev(token), off, n, args[3], args[4], FP4, 1,
                             32, e, out_f, in_f, BF16, rows) == OK
    assert tk.tk_expert_gemv_fp4(args[0], args[1], FP8, 1, 128, args[2], tokens, k, 0, args[3], args[4], 1, 32, e, out_f,
                                 in_f, BF16, slots) == OK
    rows, slots = host(rows), host(slots).reshape(tokens, k, out_f)
    for t in range(tokens):
        for j in range(k):
            assert np.array_equal(slots[t, j], rows[p[t, j]] if p[t, j] >= 0 else np.zeros(out_f))


def test_graph_replays():
    tokens, hidden, inter, experts, k = 130, 256, 256, 8, 2
    b = moe_train.Experts(tokens, hidden, inter, experts, k)
    x, dout, idx, weight = batch(tokens, hidden, experts, k, 5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b.forward(x, idx, weight)
        b.backward(dout)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = b.forward(x, idx, weight)
        dx, dweight = b.backward(dout)
    eager = moe_train.Experts(tokens, hidden, inter, experts, k)
    for seed in (6, 7, 8):
        nx, ndout, nidx, nweight = batch(tokens, hidden, experts, k, seed)
        for a, c in ((x, nx), (dout, ndout), (idx, nidx), (weight, nweight)):
            a.copy_(c)
        graph.replay()
        want = eager.forward(nx, nidx, nweight)
        wdx, wdweight = eager.backward(ndout)
        live = int(host(b.offsets)[-1])
        for a, c in ((out, want), (dx, wdx), (dweight, wdweight), (b.ddown, eager.ddown), (b.dgate_up, eager.dgate_up),
                     (b.a8[:live], eager.a8[:live]), (b.h8[:live], eager.h8[:live])):
            torch.cuda.synchronize()
            assert torch.equal(a, c)


def test_two_streams_at_once():
    hidden, inter, experts, k = 512, 256, 16, 4
    blocks, streams, data, want = [], [], [], []
    for i, tokens in enumerate((200, 333)):
        blocks.append(moe_train.Experts(tokens, hidden, inter, experts, k, seed=i))
        data.append(batch(tokens, hidden, experts, k, 20 + i))
        streams.append(torch.cuda.Stream())
        x, dout, idx, weight = data[i]
        out = blocks[i].forward(x, idx, weight).clone()
        dx, _ = blocks[i].backward(dout)
        want.append((out, dx.clone(), blocks[i].ddown.clone(), blocks[i].dgate_up.clone()))
    torch.cuda.synchronize()
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                x, dout, idx, weight = data[i]
                blocks[i].forward(x, idx, weight)
                blocks[i].backward(dout)
    torch.cuda.synchronize()
    for b, w in zip(blocks, want):
        for a, c in zip((b.out, b.dx, b.ddown, b.dgate_up), w):
            assert torch.equal(a, c)


def test_nan_stays_in_its_rows():
    """Rows behind the last expert's, other experts' rows and unnamed rows of x may hold anything."""
    rng = np.random.default_rng(9)
    off = np.array([2, 40, 40, 103], np.int32)
    n, e, out_f, in_f = 110, 3, 136, 104
    x, dy, w = (rng.standard_normal(s).astype(np.float32) for s in ((n, in_f), (n, out_f), (e, out_f, in_f)))
    live = (np.arange(n) >= 2) & (np.arange(n) < 103)
    x[~live] = dy[~live] = np.nan
    x[50], dy[60] = np.nan, np.inf  # rows of the last expert
    w[1] = np.nan                   # an expert without rows
    y, dx = torch.zeros((n, out_f), device=DEV), torch.zeros((n, in_f), device=DEV)
    dw = torch.full((e, out_f, in_f), 7.0, device=DEV)
    xd, dyd, wd, offd = products.bf16(x), products.bf16(dy), products.bf16(w), products.dev(off)
    assert tk.tk_expert_gemm(xd, None, BF16, 0, 0, n, None, offd, n, wd, None, BF16, 0, 0, e, out_f, in_f, FP32, y) == OK
    assert tk.tk_expert_gemm_dgrad(dyd, n, None, offd, n, wd, e, out_f, in_f, FP32, dx) == OK
    assert tk.tk_expert_gemm_wgrad(dyd, n, None, xd, None, BF16, 0, n, None, offd, n, e, out_f, in_f, 0, FP32, dw) == OK
    y, dx, dw = host(y), host(dx), host(dw)
    rows = np.arange(n)
    assert np.array_equal(rows[np.isnan(y).any(1)], [50]) and np.isnan(y[50]).all()
    assert np.array_equal(rows[~np.isfinite(dx).all(1)], [60])
    assert not y[~live].any() and not dx[~live].any()
    assert np.isfinite(dw[0]).all() and not dw[1].any() and np.isnan(dw[2]).all()
    # a gather that leaves the NaN rows of x out
    index = np.where(live, 2 + rng.integers(0, 38, n), 0).astype(np.int32)
    y = torch.zeros((n, out_f), device=DEV)
    assert tk.tk_expert_gemm(xd, None, BF16, 0, 0, n, products.dev(index), offd, n, wd, None, BF16, 0, 0, e, out_f, in_f,
                             FP32, y) == OK
    assert np.isfinite(host(y)).all()


def test_no_rows_to_take():
    """x and dy of no rows: every index names none, every result is zero."""
    off = products.dev(np.array([0, 70, 80], np.int32))
    index = products.dev(np.arange(80, dtype=np.int32))
    w = torch.ones((2, 64, 64), dtype=torch.bfloat16, device=DEV)
    none = torch.empty((0, 64), dtype=torch.bfloat16, device=DEV)
    y = torch.ones((80, 64), device=DEV)
    x = torch.ones((80, 64), dtype=torch.bfloat16, device=DEV)  # a place of its own, of which no row is named
    assert tk.tk_expert_gemm(x, None, BF16, 0, 0, 0, index, off, 80, w, None, BF16, 0, 0, 2, 64, 64, FP32, y) == OK
    assert not host(y).any()
    y.fill_(1)
    assert tk.tk_expert_gemm_dgrad(x, 0, index, off, 80, w, 2, 64, 64, FP32, y) == OK
    assert not host(y).any()
    dw = torch.ones((2, 64, 64), device=DEV)
    assert tk.tk_expert_gemm_wgrad(x, 0, index, x, None, BF16, 0, 80, None, off, 80, 2, 64, 64, 0, FP32, dw) == OK
    assert not host(dw).any() and none.numel() == 0
    codes = torch.zeros((2 * 64, 64), dtype=torch.uint8, device=DEV)
    scales = torch.full((2 * 64, 2), 127, dtype=torch.uint8, device=DEV)
    out = torch.ones((80, 64), dtype=torch.bfloat16, device=DEV)
    assert tk.tk_expert_gemm(codes, scales, FP8, 1, 32, 0, index, off, 80, codes, scales, FP8, 1, 32, 2, 64, 64, BF16,
                             out) == OK
    assert not host(out).any()


def test_scales_at_any_address():
    """UE8M0 scales aligned to a byte only."""
    rng = np.random.default_rng(12)
    off, n, e = products.layout("mid")
    out_f, in_f = 72, 256
    for group in (32, 128):
        xc, xs, x = products.fp8_operand(rng, n, in_f, "ue8m0", group)
        wc, ws, w = products.fp8_operand(rng, e * out_f, in_f, "ue8m0", group)

        def shifted(a):
            t = torch.zeros(a.size + 1, dtype=torch.uint8, device=DEV)
            t[1:] = torch.from_numpy(a.reshape(-1)).to(DEV)
            return t[1:]

        out = torch.zeros((n, out_f), dtype=torch.int16, device=DEV)
        assert tk.tk_expert_gemm(products.dev(xc), shifted(xs), FP8, 1, group, n, None, products.dev(off), n,
                                 products.dev(wc), shifted(ws), FP8, 1, group, e, out_f, in_f, BF16, out) == OK
        want = ex.gemm(x, None, off, n, w.reshape(e, out_f, in_f), np.zeros((n, out_f)))[0]
        products.same_or(products.host(out, True), want, True)


def test_offsets_past_32_bits():
    """x, weights and results of more than 4 GiB: the last rows and the last expert."""
    say("offsets past 32 bits")
    n, k_, out_f = 600_000, 4096, 64  # x of 4.9 GB
    gen = torch.Generator(device=DEV).manual_seed(3)
    x = torch.zeros((n, k_), dtype=torch.bfloat16, device=DEV)
    tail = torch.randint(-3, 4, (300, k_), generator=gen, device=DEV).to(torch.bfloat16)
    x[-300:] = tail
    w = torch.randint(-3, 4, (1, out_f, k_), generator=gen, device=DEV).to(torch.bfloat16)
    out = torch.zeros((n, out_f), device=DEV)
    want = tail.cpu().double() @ w[0].cpu().double().t()
    assert tk.tk_expert_gemm(x, None, BF16, 0, 0, n, None, None, n, w, None, BF16, 0, 0, 1, out_f, k_, FP32, out) == OK
    assert torch.equal(out[-300:].cpu().double(), want) and not out[:-300].any()
    index = torch.arange(n - 300, n, dtype=torch.int32, device=DEV)  # the same rows found by an index
    few = torch.zeros((300, out_f), device=DEV)
    assert tk.tk_expert_gemm(x, None, BF16, 0, 0, n, index, None, 300, w, None, BF16, 0, 0, 1, out_f, k_, FP32, few) == OK
    assert torch.equal(few.cpu().double(), want)
    dy = torch.randint(-3, 4, (300, out_f), generator=gen, device=DEV).to(torch.bfloat16)
    dw = torch.zeros((1, out_f, k_), device=DEV)
    assert tk.tk_expert_gemm_wgrad(dy, 300, None, x, None, BF16, 0, n, index, None, 300, 1, out_f, k_, 0, FP32, dw) == OK
    assert torch.equal(dw[0].cpu().double(), dy.cpu().double().t() @ tail.cpu().double())
    big = torch.zeros((n, k_), dtype=torch.bfloat16, device=DEV)  # a result of 4.9 GB
    wide = torch.randint(-3, 4, (1, k_, 64), generator=gen, device=DEV).to(torch.bfloat16)
    rows = torch.zeros((n, 64), dtype=torch.bfloat16, device=DEV)
    rows[-300:] = dy
    assert tk.tk_expert_gemm(rows, None, BF16, 0, 0, n, None, None, n, wide, None, BF16, 0, 0, 1, k_, 64, BF16, big) == OK
    want = (dy.cpu().double() @ wide[0].cpu().double().t()).to(torch.bfloat16)
    assert torch.equal(big[-300:].cpu(), want) and not big[:1000].any() and not big[n // 2:n // 2 + 1000].any()
    del x, big, rows, out
    e = 300  # weights of 5 GB
    we = torch.zeros((e, 2048, k_), dtype=torch.bfloat16, device=DEV)
    we[-1] = torch.randint(-3, 4, (2048, k_), generator=gen, device=DEV).to(torch.bfloat16)
    off = torch.zeros(e + 1, dtype=torch.int32, device=DEV)
    off[-1] = 300
    out = torch.zeros((300, 2048), device=DEV)
    assert tk.tk_expert_gemm(tail, None, BF16, 0, 0, 300, None, off, 300, we, None, BF16, 0, 0, e, 2048, k_, FP32, out) == OK
    assert torch.equal(out.cpu().double(), tail.cpu().double() @ we[-1].cpu().double().t())
    dx = torch.zeros((300, k_), device=DEV)
    dy = torch.randint(-3, 4, (300, 2048), generator=gen, device=DEV).to(torch.bfloat16)
    assert tk.tk_expert_gemm_dgrad(dy, 300, None, off, 300, we, e, 2048, k_, FP32, dx) == OK
    assert torch.equal(dx.cpu().double(), dy.cpu().double() @ we[-1].cpu().double())
    dw = torch.ones((e, 2048, k_), device=DEV)
    assert tk.tk_expert_gemm_wgrad(dy, 300, None, tail, None, BF16, 0, 300, None, off, 300, e, 2048, k_, 0, FP32, dw) == OK
    assert torch.equal(dw[-1].cpu().double(), dy.cpu().double().t() @ tail.cpu().double()) and not dw[:-1].any()


def test_swiglu_offsets_past_32_bits():
    n, hidden = 280_000, 4096  # h of 4.6 GB
    h = torch.zeros((n, 2 * hidden), dtype=torch.bfloat16, device=DEV)
    dy = torch.zeros((n, hidden), dtype=torch.bfloat16, device=DEV)
    gen = torch.Generator(device=DEV).manual_seed(4)
    h[-5:] = torch.randn((5, 2 * hidden), generator=gen, device=DEV).to(torch.bfloat16)
    dy[-5:] = torch.randn((5, hidden), generator=gen, device=DEV).to(torch.bfloat16)
    codes = torch.empty((n, hidden), dtype=torch.uint8, device=DEV)
    x_codes = torch.empty((n, 2 * hidden), dtype=torch.uint8, device=DEV)
    scales, x_scales = (torch.empty((n, c // 128), dtype=torch.uint8, device=DEV) for c in (hidden, 2 * hidden))
    assert tk.tk_swiglu_checkpoint_fp8(h, None, n, hidden, 128, float("inf"), 1, codes, scales, x_codes, x_scales) == OK
    few = [torch.empty_like(t[-5:]) for t in (codes, scales, x_codes, x_scales)]
    assert tk.tk_swiglu_checkpoint_fp8(h[-5:].clone(), None, 5, hidden, 128, float("inf"), 1, *few) == OK
    torch.cuda.synchronize()
    for a, c in zip(few, (codes, scales, x_codes, x_scales)):
        assert torch.equal(a, c[-5:])
    dh, dw = torch.empty_like(h), torch.empty(n, device=DEV)
    assert tk.tk_swiglu_backward(dy, x_codes, x_scales, FP8, 1, 128, None, n, hidden, float("inf"), dh, dw, None) == OK
    dh5, dw5 = torch.empty_like(h[-5:]), torch.empty(5, device=DEV)
    assert tk.tk_swiglu_backward(dy[-5:].clone(), few[2], few[3], FP8, 1, 128, None, 5, hidden, float("inf"), dh5, dw5,
                                 None) == OK
    torch.cuda.synchronize()
    assert torch.equal(dh[-5:], dh5) and torch.equal(dw[-5:], dw5) and not dh[:1000].any()


def test_rows_do_not_depend_on_others():
    """A row's result is the same bits whatever the other rows of its expert are, over every tile size."""
    rng = np.random.default_rng(21)
    e, out_f, in_f = 2, 8200, 520
    w = products.bf16(rng.standard_normal((e, out_f, in_f)).astype(np.float32))
    x = rng.standard_normal((600, in_f)).astype(np.float32)
    seen = None
    for counts in ([1, 0], [20, 3], [70, 9], [590, 10]):
        off, n = products.offsets_of(counts), sum(counts)
        y = torch.zeros((n, out_f), device=DEV)
        assert tk.tk_expert_gemm(products.bf16(x[:n]), None, BF16, 0, 0, n, None, products.dev(off), n, w, None, BF16, 0,
                                 0, e, out_f, in_f, FP32, y) == OK
        row = host(y)[0]
        seen = row if seen is None else seen
        assert np.array_equal(row, seen)


@pytest.mark.parametrize("counts,out_f", [([20, 13], 72), ([90, 40], 8200), ([700, 900], 4104)])
def test_rows_of_none_are_zero_whatever_the_weights_hold(counts, out_f):
    """Over every tile size; a NaN among the weights reaches the other rows."""
    rng = np.random.default_rng(30)
    e, in_f = 2, 128
    off, n = products.offsets_of(counts), sum(counts)
    index = rng.integers(0, n, n).astype(np.int32)
    none = rng.random(n) < 0.3
    index[none] = rng.choice([-1, n, 2**31 - 1], none.sum())
    x = rng.standard_normal((n, in_f)).astype(np.float32)
    w = rng.standard_normal((e, out_f, in_f)).astype(np.float32)
    w[:, 5, 7] = np.nan
    dw, di = products.dev(off), products.dev(index)
    y = torch.ones((n, out_f), device=DEV)
    assert tk.tk_expert_gemm(products.bf16(x), None, BF16, 0, 0, n, di, dw, n, products.bf16(w), None, BF16, 0, 0, e, out_f,
                             in_f, FP32, y) == OK
    y = host(y)
    assert not y[none].any() and np.isnan(y[~none][:, 5]).all() and np.isfinite(np.delete(y[~none], 5, 1)).all()
    wt = np.ascontiguousarray(np.swapaxes(w, 1, 2))  # [e, in_f, out_f]: rows of in_f values against it
    y = torch.ones((n, out_f), device=DEV)
    assert tk.tk_expert_gemm_dgrad(products.bf16(x), n, di, dw, n, products.bf16(wt), e, in_f, out_f, FP32, y) == OK
    y = host(y)
    assert not y[none].any() and np.isnan(y[~none][:, 5]).all() and np.isfinite(np.delete(y[~none], 5, 1)).all()
    codes = rng.integers(0, 120, (n, in_f), dtype=np.uint8)
    wcodes = rng.integers(0, 120, (e, out_f, in_f), dtype=np.uint8)
    wcodes[:, 5, 7] = 0x7F
    for group in (32, 64, 0):  # 64: the scales' own kernel
        g = in_f // (group or in_f)
        xs, ws = (torch.full((r, g), 127, dtype=torch.uint8, device=DEV) for r in (n, e * out_f))
        out = torch.ones((n, out_f), dtype=torch.bfloat16, device=DEV)
        assert tk.tk_expert_gemm(products.dev(codes), xs, FP8, 1, group, n, di, dw, n, products.dev(wcodes), ws, FP8, 1,
                                 group, e, out_f, in_f, BF16, out) == OK
        y = host(out)
        assert not y[none].any() and np.isnan(y[~none][:, 5]).all() and np.isfinite(np.delete(y[~none], 5, 1)).all()
