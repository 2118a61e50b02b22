"""The experts of an MoE block in training, around this library's calls: forward
in FP8 with the activations kept in 8 bits, and the backward pass from them.

    python examples/moe_train.py [--tokens 4096] [--experts 64] [--k 8] [--hidden 2048] [--inter 1024] [--steps 10]

prints the time of a forward and a backward pass and what is kept between them."""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import moe_activation_bit_amd as tk  # noqa: E402

GROUP = 128  # columns a scale (UE8M0), of activations and weights
FP8, BF16, FP32, E8 = tk.TK_DTYPE_FP8, tk.TK_DTYPE_BF16, tk.TK_DTYPE_FP32, tk.TK_SCALE_UE8M0


def call(fn, *args):
    rc = fn(*args)
    if rc != tk.TkStatus.TK_OK:
        raise RuntimeError(f"{fn.__name__}: {tk.tk_status_str(rc)}")


class Experts:
    """bf16 weights with their FP8 forms, and buffers for `tokens` tokens at a time."""

    def __init__(self, tokens, hidden, inter, experts, k, clamp=float("inf"), seed=0, device="cuda"):
        self.tokens, self.hidden, self.inter, self.experts, self.k, self.clamp = tokens, hidden, inter, experts, k, clamp
        gen = torch.Generator(device=device).manual_seed(seed)

        def empty(*shape, dtype=torch.bfloat16):
            return torch.empty(shape, dtype=dtype, device=device)

        def weights(out, inner):
            return (torch.randn((experts, out, inner), generator=gen, device=device) * inner ** -0.5).to(torch.bfloat16)

        self.gate_up, self.down = weights(2 * inter, hidden), weights(hidden, inter)
        rows = tokens * k
        self.rows = rows
        self.pos = empty(tokens, k, dtype=torch.int32)
        self.offsets = empty(experts + 1, dtype=torch.int32)
        self.ones = torch.ones((tokens, k), device=device)
        self.h = empty(rows, 2 * inter)
        self.z = empty(rows, hidden)
        self.out = empty(tokens, hidden)
        # what is kept for the backward pass
        self.x8, self.x8s = empty(tokens, hidden, dtype=torch.uint8), empty(tokens, hidden // GROUP, dtype=torch.uint8)
        self.h8, self.h8s = empty(rows, 2 * inter, dtype=torch.uint8), empty(rows, 2 * inter // GROUP, dtype=torch.uint8)
        self.a8, self.a8s = empty(rows, inter, dtype=torch.uint8), empty(rows, inter // GROUP, dtype=torch.uint8)
        # the backward pass's own
        self.dact, self.dh = empty(rows, inter), empty(rows, 2 * inter)
        self.drow = empty(rows, hidden)
        self.drow_weight = empty(rows, dtype=torch.float32)
        self.dx = empty(tokens, hidden)
        self.dgate_up = empty(*self.gate_up.shape, dtype=torch.float32)
        self.ddown = empty(*self.down.shape, dtype=torch.float32)
        self.quantise()

    def quantise(self):
        """The weights' FP8 forms, after each update of the weights."""
        def fp8(w):
            rows, inner = w.shape[0] * w.shape[1], w.shape[2]
            codes = torch.empty(w.shape, dtype=torch.uint8, device=w.device)
            scales = torch.empty((w.shape[0], w.shape[1], inner // GROUP), dtype=torch.uint8, device=w.device)
            call(tk.tk_cast_fp8, w, BF16, rows, inner, GROUP, E8, codes, scales)
            return codes, scales
        self.gate_up8, self.down8 = fp8(self.gate_up), fp8(self.down)

    def _product(self, x, scales, x_rows, index, weights, out, inner, result):
        call(tk.tk_expert_gemm, x, scales, FP8, E8, GROUP, x_rows, index, self.offsets, self.rows, weights[0],
             weights[1], FP8, E8, GROUP, self.experts, out, inner, BF16, result)

    def forward(self, x, topk_idx, topk_weight):
        """x bf16 [tokens, hidden], the routing's indices int32 and weights fp32 [tokens, k] -> [tokens, hidden]."""
        t, n = self.tokens, self.rows
        call(tk.tk_topk_to_pos, topk_idx, t, self.k, self.experts, self.pos, self.offsets)
        # the token and the routing weight of each row; rows past the last one's have none
        slot = torch.where(self.pos < 0, n, self.pos).view(-1).long()
        tokens = torch.arange(t, dtype=torch.int32, device=x.device).repeat_interleave(self.k)
        self.token = torch.full((n + 1,), -1, dtype=torch.int32, device=x.device).scatter_(0, slot, tokens)[:n]
        self.weight = torch.zeros(n + 1, device=x.device).scatter_(0, slot, topk_weight.reshape(-1))[:n]
        call(tk.tk_cast_fp8, x, BF16, t, self.hidden, GROUP, E8, self.x8, self.x8s)
        self._product(self.x8, self.x8s, t, self.token, self.gate_up8, 2 * self.inter, self.hidden, self.h)
        call(tk.tk_swiglu_checkpoint_fp8, self.h, self.weight, n, self.inter, GROUP, self.clamp, E8, self.a8, self.a8s,
             self.h8, self.h8s)
        self._product(self.a8, self.a8s, n, None, self.down8, self.hidden, self.inter, self.z)
        call(tk.tk_moe_reduce, self.z, None, self.pos, self.ones, 1.0, t, self.k, self.hidden, n, BF16, self.out)
        return self.out

    def backward(self, dout, accumulate=False):
        """dout bf16 [tokens, hidden] -> the gradients of x and of the routing weights; those of the weights go to
        self.dgate_up and self.ddown (added to what is there when `accumulate`).  The casts pass gradients on."""
        t, n, e, inter, hidden = self.tokens, self.rows, self.experts, self.inter, self.hidden
        call(tk.tk_expert_gemm_dgrad, dout, t, self.token, self.offsets, n, self.down, e, hidden, inter, BF16, self.dact)
        call(tk.tk_expert_gemm_wgrad, dout, t, self.token, self.a8, self.a8s, FP8, GROUP, n, None, self.offsets, n, e,
             hidden, inter, accumulate, FP32, self.ddown)
        call(tk.tk_swiglu_backward, self.dact, self.h8, self.h8s, FP8, E8, GROUP, self.weight, n, inter, self.clamp,
             self.dh, self.drow_weight, None)
        call(tk.tk_expert_gemm_dgrad, self.dh, n, None, self.offsets, n, self.gate_up, e, 2 * inter, hidden, BF16,
             self.drow)
        call(tk.tk_expert_gemm_wgrad, self.dh, n, None, self.x8, self.x8s, FP8, GROUP, t, self.token, self.offsets, n, e,
             2 * inter, hidden, accumulate, FP32, self.dgate_up)
        call(tk.tk_moe_reduce, self.drow, None, self.pos, self.ones, 1.0, t, self.k, hidden, n, BF16, self.dx)
        dweight = torch.where(self.pos < 0, 0.0, self.drow_weight[self.pos.clamp(min=0).long()])
        return self.dx, dweight


def timed(fn, steps):
    for _ in range(2):
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
    for name, value in (("tokens", 4096), ("experts", 64), ("k", 8), ("hidden", 2048), ("inter", 1024), ("steps", 10)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    block = Experts(a.tokens, a.hidden, a.inter, a.experts, a.k)
    x = torch.randn(a.tokens, a.hidden, device="cuda").to(torch.bfloat16)
    dout = torch.randn(a.tokens, a.hidden, device="cuda").to(torch.bfloat16)
    weight, idx = torch.rand(a.tokens, a.experts, device="cuda").topk(a.k, dim=-1)
    idx = idx.to(torch.int32).contiguous()
    forward = timed(lambda: block.forward(x, idx, weight), a.steps)
    backward = timed(lambda: block.backward(dout), a.steps)
    flops = 2 * block.rows * 3 * a.inter * a.hidden
    kept = sum(t.numel() for t in (block.x8, block.x8s, block.h8, block.h8s, block.a8, block.a8s))
    print(f"{a.tokens} tokens, top-{a.k} of {a.experts} experts, {a.hidden} x {a.inter}: forward {forward:.0f} us "
          f"({flops / forward / 1e6:.0f} TFLOP/s), backward {backward:.0f} us ({2 * flops / backward / 1e6:.0f} TFLOP/s); "
          f"{kept / 2**20:.0f} MiB kept between them")


if __name__ == "__main__":
    main()
