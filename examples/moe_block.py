"""One MoE block around this library's calls: a step of decoding with 4-bit
expert weights, eager or as a HIP graph, and the gradients that reach the
router and the norm.

    python examples/moe_block.py [--tokens 1] [--experts 64] [--k 8] [--hidden 7168] [--inter 2048] [--steps 50]

prints the time of a decode step, eager and replayed from a graph, and the rate
at which the chosen experts' weights are read."""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import moe_activation_bit_amd as tk  # noqa: E402

W_GROUP, X_GROUP = 32, 128  # columns a scale: of the weights (UE8M0), of the activations (fp32)


def call(fn, *args):
    rc = fn(*args)
    if rc != tk.TkStatus.TK_OK:
        raise RuntimeError(f"{fn.__name__}: {tk.tk_status_str(rc)}")


class MoeBlock:
    """Weights and buffers of a block, for `tokens` tokens at a time."""

    def __init__(self, tokens, hidden, inter, experts, k, groups=1, keep=1, eps=1e-6, scale=2.5, seed=0, device="cuda"):
        self.tokens, self.hidden, self.inter, self.experts, self.k = tokens, hidden, inter, experts, k
        self.groups, self.keep, self.eps, self.scale = groups, keep, eps, scale
        gen = torch.Generator(device=device).manual_seed(seed)

        def randn(*shape, std=1.0):
            return torch.randn(shape, generator=gen, device=device) * std

        def empty(*shape, dtype=torch.bfloat16):
            return torch.empty(shape, dtype=dtype, device=device)

        self.norm_weight = 1 + randn(hidden, std=0.1)
        self.router = randn(experts, hidden, std=hidden ** -0.5)
        self.bias = randn(experts, std=0.01)
        # 4-bit weights, [experts, out, in/2] and a scale for each W_GROUP columns, laid out once
        self.gate_up = self._quantise(randn, empty, 2 * inter, hidden)
        self.down = self._quantise(randn, empty, hidden, inter)

        rows = tokens * k
        self.x = empty(tokens, hidden)         # this block's input: what attention added
        self.residual = empty(tokens, hidden)  # the residual stream, updated in place
        self.y, self.y32 = empty(tokens, hidden), empty(tokens, hidden, dtype=torch.float32)
        self.rstd = empty(tokens, dtype=torch.float32)
        self.codes = empty(tokens, hidden, dtype=torch.uint8)
        self.scales = empty(tokens, hidden // X_GROUP, dtype=torch.float32)
        self.logits = empty(tokens, experts, dtype=torch.float32)
        self.idx, self.weight = empty(tokens, k, dtype=torch.int32), empty(tokens, k, dtype=torch.float32)
        self.h = empty(rows, 2 * inter)
        self.act = empty(rows, inter, dtype=torch.uint8)
        self.act_scales = empty(rows, inter // X_GROUP, dtype=torch.float32)
        self.z = empty(rows, hidden)
        self.pos = torch.arange(rows, dtype=torch.int32, device=device)  # slot j of token t is row t*k + j
        self.out = empty(tokens, hidden)

    def _quantise(self, randn, empty, out, inner):
        codes = empty(self.experts, out, inner // 2, dtype=torch.uint8)
        scales = empty(self.experts, out, inner // W_GROUP, dtype=torch.uint8)
        for e in range(self.experts):
            w = randn(out, inner, std=inner ** -0.5).to(torch.bfloat16)
            call(tk.tk_cast_fp4, w, tk.TK_DTYPE_BF16, out, inner, W_GROUP, tk.TK_SCALE_UE8M0, codes[e], scales[e])
        return codes, scales

    def route(self):
        """The norm with the residual, the router, and the choice of experts."""
        call(tk.tk_rmsnorm_cast_fp8, self.x, self.residual, tk.TK_DTYPE_BF16, self.norm_weight, self.tokens,
             self.hidden, self.eps, X_GROUP, tk.TK_SCALE_FP32, self.residual, self.y, self.rstd, self.codes, self.scales)
        self.y32.copy_(self.y)
        torch.mm(self.y32, self.router.t(), out=self.logits)
        call(tk.tk_route, self.logits, tk.TK_DTYPE_FP32, self.bias, self.tokens, self.experts, self.k, self.groups,
             self.keep, tk.TK_SCORE_SIGMOID, 1, self.scale, self.idx, self.weight)

    def _product(self, x, scales, slots, weights, out, inner, result):
        call(tk.tk_expert_gemv_fp4, x, scales, tk.TK_DTYPE_FP8, tk.TK_SCALE_FP32, X_GROUP, self.idx, self.tokens,
             self.k, slots, weights[0], weights[1], tk.TK_SCALE_UE8M0, W_GROUP, self.experts, out, inner,
             tk.TK_DTYPE_BF16, result)

    def decode(self):
        """self.out: the block's output for self.x; self.residual becomes the stream with self.x added."""
        self.route()
        rows = self.tokens * self.k
        self._product(self.codes, self.scales, 0, self.gate_up, 2 * self.inter, self.hidden, self.h)
        call(tk.tk_swiglu_cast_fp8, self.h, None, rows, self.inter, X_GROUP, float("inf"), tk.TK_SCALE_FP32, self.act,
             self.act_scales)
        self._product(self.act, self.act_scales, 1, self.down, self.hidden, self.inter, self.z)
        call(tk.tk_moe_reduce, self.z, None, self.pos, self.weight, 1.0, self.tokens, self.k, self.hidden, rows,
             tk.TK_DTYPE_BF16, self.out)

    def capture(self):
        """decode() as a graph; what replays it sets self.x (and self.residual) before."""
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        kept = self.residual.clone()
        with torch.cuda.stream(side):
            self.decode()  # libraries allocate on their first call
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            self.decode()
        self.residual.copy_(kept)
        return graph

    def router_gradients(self, dweight, dstream):
        """After route(): from the gradients of the routing weights [tokens, k]
        (fp32) and of the residual stream [tokens, hidden] (bf16) those of
        self.x (and of the stream before), of the norm's weight and of the
        router's."""
        dlogits = torch.empty_like(self.logits)
        call(tk.tk_route_backward, dweight, self.idx, self.logits, tk.TK_DTYPE_FP32, self.tokens, self.experts, self.k,
             tk.TK_SCORE_SIGMOID, 1, self.scale, dlogits)
        drouter = torch.mm(dlogits.t(), self.y32)
        dy = torch.mm(dlogits, self.router).to(torch.bfloat16)
        dx, dnorm = torch.empty_like(self.x), torch.empty_like(self.norm_weight)
        parts = torch.empty(min(self.tokens, tk.TK_RMSNORM_PARTS), self.hidden, device=dnorm.device)
        call(tk.tk_rmsnorm_backward, dy, self.residual, tk.TK_DTYPE_BF16, self.norm_weight, self.rstd, dstream,
             self.tokens, self.hidden, dx, dnorm, parts)
        return dx, dnorm, drouter


def timed(fn, steps):
    for _ in range(3):
        fn()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(steps):
        fn()
    end.record()
    torch.cuda.synchronize()
    return start.elapsed_time(end) / steps * 1e3


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    for name, value in (("tokens", 1), ("experts", 64), ("k", 8), ("hidden", 7168), ("inter", 2048), ("steps", 50)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    block = MoeBlock(a.tokens, a.hidden, a.inter, a.experts, a.k)
    block.x.normal_()
    block.residual.normal_()
    eager = timed(block.decode, a.steps)
    graph = block.capture()
    replayed = timed(graph.replay, a.steps)
    used = block.idx.unique().numel()
    bytes_ = used * 3 * a.inter * a.hidden * (0.5 + 1 / W_GROUP)
    print(f"{a.tokens} token(s), top-{a.k} of {a.experts} experts, {a.hidden} x {a.inter}: {eager:.1f} us a step, "
          f"{replayed:.1f} us from a graph; weights of {used} experts at {bytes_ / replayed / 1e3:.0f} GB/s")
    dx, dnorm, drouter = block.router_gradients(torch.randn_like(block.weight), torch.randn_like(block.x))
    print("gradients:", ", ".join(f"{n} {tuple(t.shape)} norm {t.float().norm().item():.3g}"
                                  for n, t in (("x", dx), ("norm weight", dnorm), ("router", drouter))))


if __name__ == "__main__":
    main()
