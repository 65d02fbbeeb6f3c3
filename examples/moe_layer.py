"""A routed feed-forward part on ROCmFP2 weights, from residual stream to residual stream.

    python examples/moe_layer.py [--tokens 1] [--width 4096] [--experts 128] [--inner 1536]
                                 [--top-k 8] [--steps 64]

What the attention adds is taken into the stream and normed (rfp2_add_rms_norm), the
router's logits choose each token's experts (rfp2_moe_route), whose gate and up halves are
one product (rfp2_moe_gemv, rfp2_moe_gemv_tokens or rfp2_moe_gemm, by the count of tokens),
the gate's activation goes into int8 (rfp2_quantize_gated_acts), and the down products'
rows come back onto the stream by the router's weights, with the next part's norm in the
same pass (rfp2_moe_combine).  Nothing in a step depends on the host, so it is captured into a
HIP graph once and replayed.  The router's weights are packed like the others here; a
model that keeps them in more bits brings its own product and hands over the logits.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_gemv_amd as rf  # noqa: E402


class MoeLayer:
    """Weights and buffers of one part for `tokens` tokens a step.

    w_router [experts][width], w_gate_up [experts][2 inner][width] (gate rows first) and
    w_down [experts][width][inner] are fp32 and packed to ROCmFP2 here; gain and next_gain
    [width] are those of this part's norm and of the norm that follows."""

    def __init__(self, w_router, w_gate_up, w_down, gain, next_gain, tokens: int, top_k: int,
                 bias=None, score: int = rf.ROUTE_SOFTMAX, groups: int = 1, group_top: int = 1,
                 top_groups: int = 1, renorm: bool = True, scale: float = 1.0,
                 act: int = rf.GATE_SILU, eps: float = 1e-6):
        dev = w_router.device
        self.experts, self.width = w_router.shape
        self.inner, self.tokens, self.top_k = w_down.shape[2], tokens, top_k
        self.gain, self.next_gain, self.eps, self.act = gain, next_gain, eps, act
        self.routing = (bias, score, groups, group_top, top_groups, top_k, renorm, scale)
        self.w_router, self.w_gate_up, self.w_down = (
            self._pack(w.reshape(-1, w.shape[-1])) for w in (w_router, w_gate_up, w_down))

        def f32(*shape):
            return torch.zeros(shape, dtype=torch.float32, device=dev)

        def acts(rows, K):
            return torch.empty((rows, K), dtype=torch.int8, device=dev), f32(rows, K // 32)

        T, S = tokens, tokens * top_k
        self.x, self.add, self.h = f32(T, self.width), f32(T, self.width), f32(T, self.width)
        self.acts_in, self.acts_mid, self.acts_out = (
            acts(T, self.width), acts(S, self.inner), acts(T, self.width))
        self.logits, self.weights = f32(T, self.experts), f32(T, top_k)
        self.ids = torch.zeros(T, top_k, dtype=torch.int32, device=dev)
        self.gate_up, self.down = f32(S, 2 * self.inner), f32(S, self.width)
        self.err = torch.zeros(1, dtype=torch.int32, device=dev)
        self.workspace = torch.empty(
            max(256, rf.rfp2_moe_gemm_workspace_bytes(self.experts, S, 1)), dtype=torch.uint8,
            device=dev)

    @staticmethod
    def _pack(w):
        N, K = w.shape
        packed = torch.empty(N * K // 32 * 10, dtype=torch.uint8, device=w.device)
        rf.rfp2_quantize_weights(w.contiguous(), N, K, packed)
        return packed

    def _routed(self, w, N, K, T, top_k, acts, y):
        """Each of T tokens through its top_k experts."""
        if T <= rf.GEMV_MAX_M and T * top_k <= 64:
            rf.rfp2_moe_gemv_tokens(w, self.experts, N, K, self.ids, T, top_k, *acts, y, self.err)
        else:
            rf.rfp2_moe_gemm(w, self.experts, N, K, self.ids, T, top_k, *acts, y, self.err,
                             self.workspace)

    def step(self):
        """self.x + self.add -> self.h, and the next norm's int8 form in self.acts_out."""
        T, W, I = self.tokens, self.width, self.inner
        rf.rfp2_add_rms_norm(self.x, self.add, T, W, self.gain, self.eps, self.h, None,
                             *self.acts_in)
        product = rf.rfp2_gemv if T <= rf.GEMV_MAX_M else rf.rfp2_gemm_f16
        product(self.w_router, self.experts, W, *self.acts_in, T, self.logits)
        rf.rfp2_moe_route(self.logits, T, self.experts, *self.routing, self.ids, self.weights,
                          self.err)
        self._routed(self.w_gate_up, 2 * I, W, T, self.top_k, self.acts_in, self.gate_up)
        rf.rfp2_quantize_gated_acts(self.gate_up[:, :I], self.gate_up[:, I:], T * self.top_k, I,
                                    self.act, *self.acts_mid)
        # every slot is a token of its own with one expert
        self._routed(self.w_down, W, I, T * self.top_k, 1, self.acts_mid, self.down)
        rf.rfp2_moe_combine(self.h, self.down, self.weights, T, self.top_k, W, self.h,
                            self.next_gain, self.eps, None, *self.acts_out)

    def capture(self) -> torch.cuda.CUDAGraph:
        """The step as a graph."""
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            self.step()
        torch.cuda.current_stream().wait_stream(s)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            self.step()
        return graph


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--tokens", type=int, default=1)
    ap.add_argument("--width", type=int, default=4096)
    ap.add_argument("--experts", type=int, default=128)
    ap.add_argument("--inner", type=int, default=1536)
    ap.add_argument("--top-k", type=int, default=8)
    ap.add_argument("--steps", type=int, default=64)
    a = ap.parse_args()
    torch.manual_seed(0)
    dev = torch.device("cuda:0")
    layer = MoeLayer(0.02 * torch.randn(a.experts, a.width, device=dev),
                     0.02 * torch.randn(a.experts, 2 * a.inner, a.width, device=dev),
                     0.02 * torch.randn(a.experts, a.width, a.inner, device=dev),
                     torch.ones(a.width, device=dev), torch.ones(a.width, device=dev), a.tokens,
                     a.top_k)
    graph = layer.capture()
    layer.x.normal_()
    layer.add.normal_()
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    for _ in range(a.steps):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    assert int(layer.err) == 0
    print(f"{a.tokens} tokens, {a.top_k} of {a.experts} experts of {a.inner} x {a.width}: "
          f"{start.elapsed_time(end) / a.steps * 1e3:.1f} us a step; "
          f"first token's experts {layer.ids[0].tolist()}")


if __name__ == "__main__":
    main()
