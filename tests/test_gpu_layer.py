"""The operators of include/tk_layer.h together and where they are run from: the
block of examples/moe_block.py stage by stage against plain statements in 64
bits (and the oracle's bits for the steps it has), HIP graphs replayed several
times with eager work in between, streams other than the default one, and
tensors whose offsets pass 32 bits."""
import os
import sys

import numpy as np
import pytest
import torch

import layer_ref as ref
import moe_activation_bit_amd as tk
import oracle
import test_gpu_expert_gemv as gemv
import test_gpu_rmsnorm as rmsnorm
import test_gpu_route as route

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import moe_block  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
OK = tk.TkStatus.TK_OK
BF16, FP32, FP8 = tk.TK_DTYPE_BF16, tk.TK_DTYPE_FP32, tk.TK_DTYPE_FP8


def say(*a):
    print("[gpu-case]", *a, flush=True)


def bits(t):
    return t.detach().cpu().view(torch.int16).numpy().view(np.uint16)


def host(t):
    return bits(t) if t.dtype == torch.bfloat16 else t.detach().cpu().numpy()


@pytest.fixture(scope="module", autouse=True)
def _table():
    assert tk.tk_init(0) == OK  # the fused SwiGLU step's, before any capture


def block(tokens, seed=0):
    b = moe_block.MoeBlock(tokens, 512, 256, 16, 4, groups=4, keep=2, seed=seed)
    gen = torch.Generator(device=DEV).manual_seed(seed + 1)
    x = torch.randn(b.x.shape, generator=gen, device=DEV).to(torch.bfloat16)
    r = (3 * torch.randn(b.x.shape, generator=gen, device=DEV)).to(torch.bfloat16)
    return b, x, r


def start(b, x, r):
    b.x.copy_(x)
    b.residual.copy_(r)


# ---- the block ----------------------------------------------------------------------------------


@pytest.mark.parametrize("tokens", [1, 5, 33])
def test_block_stage_by_stage(tokens):
    say("block", tokens)
    b, x, r = block(tokens)
    start(b, x, r)
    b.decode()
    torch.cuda.synchronize()
    got = {"h": host(b.residual), "rstd": host(b.rstd), "y": host(b.y), "codes": host(b.codes), "scales": host(b.scales)}
    rmsnorm.check_norm(host(x), host(r), host(b.norm_weight), True, b.eps, moe_block.X_GROUP, 0, got)
    y, w = ref.bf16_value(got["y"]).astype(np.float64), host(b.router).astype(np.float64)
    logits = host(b.logits)
    assert np.all(np.abs(logits - y @ w.T) <= ref.U32 * (b.hidden + 2) * (np.abs(y) @ np.abs(w).T))
    route.check_route(logits, host(b.bias), b.k, b.groups, b.keep, False, 1, (host(b.idx), host(b.weight)), b.scale)
    idx = host(b.idx)

    def product(codes, scales, slots, weights, out, inner):
        want, mag = ref.gemv(ref.x_values(codes, scales, "fp8"), idx, b.k, slots,
                             ref.fp4_values(host(weights[0]), host(weights[1]), True))
        gemv.check(host(out), True, want, mag, inner, False)

    product(got["codes"], got["scales"], 0, b.gate_up, b.h, b.hidden)
    act, act_scales, _ = oracle.swiglu_cast(host(b.h), None, moe_block.X_GROUP, None, 8, tk.TK_SCALE_FP32)
    assert np.array_equal(host(b.act), act) and np.array_equal(host(b.act_scales), act_scales)
    product(act, act_scales, 1, b.down, b.z, b.inter)
    out = oracle.moe_reduce(host(b.z), host(b.pos).reshape(tokens, b.k), host(b.weight), None, 1.0, True)
    assert np.array_equal(host(b.out), out)


def test_block_gradients():
    say("block gradients")
    b, x, r = block(37)
    start(b, x, r)
    b.route()
    gen = torch.Generator(device=DEV).manual_seed(9)
    dweight = torch.randn(b.weight.shape, generator=gen, device=DEV)
    dstream = torch.randn(b.x.shape, generator=gen, device=DEV).to(torch.bfloat16)
    dx, dnorm, drouter = b.router_gradients(dweight, dstream)
    torch.cuda.synchronize()
    # the whole way in 64 bits, from the values the forward pass stored (y rounded to bf16 for the router's)
    h, y, w = ref.bf16_value(host(b.residual)), ref.bf16_value(host(b.y)).astype(np.float64), host(b.router).astype(np.float64)
    rstd, _ = ref.norm(h, host(b.norm_weight), b.eps)
    dlogits, mag = ref.route_backward(host(dweight), host(b.idx), host(b.logits), False, 1, b.scale)
    want_dx, want_dnorm = ref.norm_backward(dlogits @ w, h, host(b.norm_weight), rstd, ref.bf16_value(host(dstream)))
    want_drouter = dlogits.T @ y
    # dlogits is off by some 60 half steps of fp32 of its terms; dy is rounded to bf16 once (which dx and dnorm
    # see in norm: independent roundings), dx once more
    off = 64 * ref.U32 * mag

    def near(got, want, bound):
        assert np.linalg.norm(got - want) <= bound, (np.linalg.norm(got - want), bound)

    near(host(drouter), want_drouter, np.linalg.norm(off.T @ np.abs(y)) + ref.U32 * 40 * np.linalg.norm(mag.T @ np.abs(y)))
    dy = dlogits @ w
    scaled = np.abs(dy) * np.abs(host(b.norm_weight)) * rstd[:, None]
    # the norm's gradient subtracts a projection: it does not lengthen a row
    near(ref.bf16_value(host(dx)), want_dx, (ref.UB16 + 64 * ref.U32) * (np.linalg.norm(scaled) + np.linalg.norm(want_dx))
         + 64 * ref.U32 * np.linalg.norm((mag @ np.abs(w)) * rstd[:, None]) * 2)
    a = np.abs(h * rstd[:, None])
    near(host(dnorm), want_dnorm, ref.UB16 * np.linalg.norm((np.abs(dy) * a).sum(0))
         + 128 * ref.U32 * np.linalg.norm(((mag @ np.abs(w)) * a).sum(0)))


def test_block_as_a_graph():
    say("block graph")
    b, x, r = block(3)
    inputs = [(torch.roll(x, i, 0), torch.roll(r, 2 * i, 1)) for i in range(4)]
    want = []
    for xi, ri in inputs:
        start(b, xi, ri)
        b.decode()
        want.append([t.clone() for t in (b.out, b.residual, b.idx, b.weight, b.z)])
    graph = b.capture()
    for i in (0, 1, 2, 3, 1, 0):
        start(b, *inputs[i])
        for t in (b.out, b.z, b.h, b.act, b.codes, b.logits, b.weight):
            t.view(torch.uint8).fill_(0xA5)
        b.idx.fill_(-1)
        graph.replay()
        torch.cuda.synchronize()
        for got, w in zip((b.out, b.residual, b.idx, b.weight, b.z), want[i]):
            assert torch.equal(got.view(torch.uint8), w.view(torch.uint8)), f"replay of input {i}"
        (x.float() @ x.float().t()).sum().item()  # eager work between the replays


# ---- each operator by itself --------------------------------------------------------------------


def calls(n=70, hidden=1024, experts=64, k=6, out=200):
    """name -> (inputs, outputs, call): each call reads its inputs and writes its outputs."""
    gen = torch.Generator(device=DEV).manual_seed(4)

    def randn(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=gen, device=DEV).to(dtype)

    def empty(*shape, dtype=torch.float32):
        return torch.empty(shape, dtype=dtype, device=DEV)

    b16, u8, i32 = torch.bfloat16, torch.uint8, torch.int32
    x, res, w = randn(n, hidden, dtype=b16), randn(n, hidden, dtype=b16), randn(hidden)
    h, y, rstd, codes, scales = (empty(n, hidden, dtype=b16), empty(n, hidden, dtype=b16), empty(n),
                                 empty(n, hidden, dtype=u8), empty(n, hidden // 128))
    dy, rs = randn(n, hidden, dtype=b16), randn(n).abs()
    dx, dw, parts = empty(n, hidden, dtype=b16), empty(hidden), empty(min(n, tk.TK_RMSNORM_PARTS), hidden)
    logits, bias, idx, weight = randn(n, experts), randn(experts), empty(n, k, dtype=i32), empty(n, k)
    dweight, dlogits = randn(n, k), empty(n, experts)
    chosen = torch.argsort(randn(n, experts), 1)[:, :k].to(i32).contiguous()
    wc = torch.randint(0, 256, (experts, out, hidden // 2), generator=gen, device=DEV, dtype=torch.int32).to(u8)
    ws = torch.randint(110, 130, (experts, out, hidden // 32), generator=gen, device=DEV, dtype=torch.int32).to(u8)
    prod = empty(n * k, out)
    return {
        "norm": ([x, res, w], [h, y, rstd, codes, scales], lambda s=None: tk.tk_rmsnorm_cast_fp8(
            x, res, BF16, w, n, hidden, 1e-6, 128, 0, h, y, rstd, codes, scales, s)),
        "norm backward": ([dy, x, w, rs, res], [dx, dw], lambda s=None: tk.tk_rmsnorm_backward(
            dy, x, BF16, w, rs, res, n, hidden, dx, dw, parts, s)),
        "route": ([logits, bias], [idx, weight], lambda s=None: tk.tk_route(
            logits, FP32, bias, n, experts, k, 8, 4, tk.TK_SCORE_SIGMOID, 1, 2.5, idx, weight, s)),
        "route backward": ([dweight, chosen, logits], [dlogits], lambda s=None: tk.tk_route_backward(
            dweight, chosen, logits, FP32, n, experts, k, tk.TK_SCORE_SOFTMAX, 0, 2.5, dlogits, s)),
        "products": ([x, chosen, wc, ws], [prod], lambda s=None: tk.tk_expert_gemv_fp4(
            x, None, BF16, 0, 0, chosen, n, k, 0, wc, ws, tk.TK_SCALE_UE8M0, 32, experts, out, hidden, FP32, prod, s)),
    }


def same(outs, want):
    return all(torch.equal(o.view(torch.uint8), w.view(torch.uint8)) for o, w in zip(outs, want))


def poison(outs):
    for o in outs:
        o.view(torch.uint8).fill_(0xA5)


def test_graphs_replayed_beside_an_eager_graph_of_the_same_leaves():
    say("operators in one graph")
    ops = calls()
    # an eager graph of the norm's and the router's inputs lives while the backward calls are captured
    leaves = [ops["norm backward"][0][1].float().requires_grad_(), ops["route"][0][0].clone().requires_grad_()]
    alive = (leaves[0] * torch.rsqrt(leaves[0].square().mean(1, keepdim=True) + 1e-6)).square().sum() + leaves[1].sigmoid().sum()
    want = {}
    for name, (_, outs, call) in ops.items():
        assert call() == OK
        want[name] = [o.clone() for o in outs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _, _, call in ops.values():
            assert call() == OK
    for _ in range(4):
        for _, outs, _ in ops.values():
            poison(outs)
        graph.replay()
        torch.cuda.synchronize()
        for name, (_, outs, _) in ops.items():
            assert same(outs, want[name]), name
        assert (leaves[0].detach() @ leaves[0].detach().t()).sum().isfinite()
    alive.backward()
    assert all(leaf.grad.isfinite().all() for leaf in leaves)


@pytest.mark.parametrize("explicit", [False, True])
def test_on_another_stream(explicit):
    """Inputs that a side stream fills late, on which the call then runs: an operator that ran elsewhere would read
    what was there before."""
    say("operators on a side stream", explicit)
    ops = calls()
    side, slow = torch.cuda.Stream(), torch.randn(4096, 4096, device=DEV)
    for name, (ins, outs, call) in ops.items():
        assert call() == OK
        torch.cuda.synchronize()
        want, kept = [o.clone() for o in outs], [i.clone() for i in ins]
        poison(outs)
        for i in ins:
            i.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for _ in range(8):
                slow @ slow
            for i, v in zip(ins, kept):
                i.copy_(v)
            if not explicit:
                assert call() == OK
        if explicit:
            assert call(side.cuda_stream) == OK
        side.synchronize()
        assert same(outs, want), name


# ---- offsets that pass 32 bits ------------------------------------------------------------------


def test_norm_offsets_past_32_bits():
    say("norm, 2^31 elements and more")
    n, hidden = 131072 + 40, 16384  # 2^31 elements at row 131072
    x = torch.empty(n, hidden, dtype=torch.bfloat16, device=DEV)
    x[:4096].normal_(generator=torch.Generator(device=DEV).manual_seed(1))
    for i in range(4096, n, 4096):
        x[i:i + 4096] = x[:min(4096, n - i)]
    w = torch.randn(hidden, device=DEV)

    def forward(x):
        n = len(x)
        outs = (torch.empty(n, device=DEV), torch.empty(n, hidden, dtype=torch.uint8, device=DEV),
                torch.empty(n, hidden // 128, device=DEV))
        assert tk.tk_rmsnorm_cast_fp8(x, None, BF16, w, n, hidden, 1e-6, 128, 0, None, None, outs[0], outs[1], outs[2]) == OK
        return outs

    def backward(x, rstd):
        dx = torch.empty_like(x)
        assert tk.tk_rmsnorm_backward(x, x, BF16, w, rstd, None, len(x), hidden, dx, None, None) == OK
        return dx

    whole, part = forward(x), forward(x[-40:].clone())
    for a, b in zip(whole, part):
        assert torch.equal(a[-40:], b)
    dx = backward(x, whole[0])
    assert torch.equal(dx[-40:], backward(x[-40:].clone(), part[0]))
    assert torch.equal(dx[:8], dx[4096:4104])


def test_routing_offsets_past_32_bits():
    say("routing, 2^31 logits and more")
    T, E, k = (1 << 31) // 512 + 24, 512, 8
    x = torch.empty(T, E, dtype=torch.bfloat16, device=DEV)
    x[:65536].normal_(generator=torch.Generator(device=DEV).manual_seed(2))
    for i in range(65536, T, 65536):
        x[i:i + 65536] = x[:min(65536, T - i)]

    def both(x):
        T = len(x)
        idx, w = torch.empty(T, k, dtype=torch.int32, device=DEV), torch.empty(T, k, device=DEV)
        assert tk.tk_route(x, BF16, None, T, E, k, 1, 1, tk.TK_SCORE_SOFTMAX, 1, 1.0, idx, w) == OK
        d = torch.empty_like(x)
        assert tk.tk_route_backward(w, idx, x, BF16, T, E, k, tk.TK_SCORE_SOFTMAX, 0, 1.0, d) == OK
        return idx, w, d

    for a, b in zip(both(x), both(x[-24:].clone())):
        assert torch.equal(a[-24:].view(torch.uint8), b.view(torch.uint8))


def test_weight_offsets_past_32_bits():
    say("products, 2^32 bytes of weights and more")
    E, out, inner, k = 160, 4096, 16384, 2
    gen = torch.Generator(device=DEV).manual_seed(3)
    codes = torch.empty(E, out, inner // 2, dtype=torch.uint8, device=DEV)
    for e in range(E):
        codes[e].random_(0, 256, generator=gen)
    scales = torch.empty(E, out, inner // 32, dtype=torch.uint8, device=DEV).random_(115, 125, generator=gen)
    x = torch.randn(3, inner, generator=gen, device=DEV).to(torch.bfloat16)
    idx = torch.tensor([[159, 0], [128, 159], [-1, 127]], dtype=torch.int32, device=DEV)
    got = torch.empty(6, out, device=DEV)
    assert codes.numel() > 1 << 32
    assert tk.tk_expert_gemv_fp4(x, None, BF16, 0, 0, idx, 3, k, 0, codes, scales, tk.TK_SCALE_UE8M0, 32, E, out, inner,
                                 FP32, got) == OK
    for r, e in enumerate(idx.flatten().tolist()):
        if e < 0:
            assert not got[r].any()
            continue
        one = torch.full((1, k), -1, dtype=torch.int32, device=DEV)
        one[0, 0] = 0
        want = torch.empty(k, out, device=DEV)
        assert tk.tk_expert_gemv_fp4(x[r // k].clone(), None, BF16, 0, 0, one, 1, k, 0, codes[e].clone(), scales[e].clone(),
                                     tk.TK_SCALE_UE8M0, 32, 1, out, inner, FP32, want) == OK
        assert torch.equal(got[r], want[0]), (r, e)


# ---- addresses aligned to an element and no more --------------------------------------------------


def shifted(t, by=1):
    """A copy of t that begins `by` elements after a 256-byte boundary."""
    buf = torch.empty(t.numel() + by, dtype=t.dtype, device=DEV)
    buf[by:] = t.reshape(-1)
    out = buf[by:].view(t.shape)
    assert out.data_ptr() % 256 == by * t.element_size()
    return out


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,k,ng,tg", [(64, 6, 1, 1), (64, 8, 8, 4), (128, 8, 1, 1), (256, 8, 8, 4), (160, 6, 1, 1), (512, 8, 1, 1), (100, 5, 1, 1), (256, 20, 1, 1)])
def test_routing_at_any_elements_address(dtype, E, k, ng, tg):
    say("routing, shifted", dtype, E, k, ng, tg)
    T = 37
    gen = torch.Generator(device=DEV).manual_seed(E + k)
    x = (2 * torch.randn(T, E, generator=gen, device=DEV)).to(dtype)
    bias, dw = torch.randn(E, generator=gen, device=DEV) * .1, torch.randn(T, k, generator=gen, device=DEV)
    code = FP32 if dtype == torch.float32 else BF16
    for softmax in (0, 1):
        for norm in (0, 1):
            got = []
            for place in (lambda t: t, shifted):
                idx, w, d = (place(torch.zeros(shape, dtype=t, device=DEV)) for shape, t in
                             (((T, k), torch.int32), ((T, k), torch.float32), ((T, E), dtype)))
                xs = place(x)
                assert tk.tk_route(xs, code, place(bias), T, E, k, ng, tg, softmax, norm, 2.5, idx, w) == OK
                assert tk.tk_route_backward(place(dw), idx, xs, code, T, E, k, softmax, norm, 2.5, d) == OK
                got.append((idx, w, d))
            for a, b in zip(*got):
                assert torch.equal(a, b)


@pytest.mark.parametrize("u8,group", [(True, 32), (True, 128), (False, 128), (False, 0)])
@pytest.mark.parametrize("x8", [False, True])
def test_products_at_any_elements_address(u8, group, x8):
    say("products, shifted", u8, group, x8)
    T, k, E, out, inner = 5, 2, 4, 70, 1024
    gen = torch.Generator(device=DEV).manual_seed(group + x8)
    if x8:
        x, xs = torch.randint(0, 120, (T, inner), generator=gen, device=DEV, dtype=torch.int32).to(torch.uint8), torch.rand(T, inner // 128, generator=gen, device=DEV)
    else:
        x, xs = torch.randn(T, inner, generator=gen, device=DEV).to(torch.bfloat16), None
    codes = torch.randint(0, 256, (E, out, inner // 2), generator=gen, device=DEV, dtype=torch.int32).to(torch.uint8)
    G = inner // (group or inner)
    sc = torch.randint(118, 124, (E, out, G), generator=gen, device=DEV, dtype=torch.int32).to(torch.uint8) if u8 else torch.rand(E, out, G, generator=gen, device=DEV)
    idx = torch.randint(0, E, (T, k), generator=gen, device=DEV, dtype=torch.int32)
    for dtype in (torch.bfloat16, torch.float32):
        got = []
        for place in (lambda t: t, shifted):
            y = place(torch.zeros(T * k, out, dtype=dtype, device=DEV))
            assert tk.tk_expert_gemv_fp4(x, None if xs is None else place(xs), FP8 if x8 else BF16, 0, 128 if x8 else 0, place(idx), T, k, 0,
                                         codes, place(sc), 1 if u8 else 0, group, E, out, inner, FP32 if dtype == torch.float32 else BF16, y) == OK
            got.append(y)
        assert torch.equal(*got)
        # weights at 16 bytes past a boundary, through the caches instead of past them
        y = torch.empty_like(got[0])
        assert tk.tk_expert_gemv_fp4(x, xs, FP8 if x8 else BF16, 0, 128 if x8 else 0, idx, T, k, 0, shifted(codes, 16), sc, 1 if u8 else 0, group,
                                     E, out, inner, FP32 if dtype == torch.float32 else BF16, y) == OK
        assert torch.equal(y, got[0])
