"""One attention layer of a decode step on ROCmFP2 weights, token after token.

    python examples/decode_layer.py [--seqs 4] [--context 3000] [--steps 64] [--format i8|f16]

A few sequences (up to eight) decode together: their activations are quantized
and multiplied with the QKV weights (rfp2_quantize_acts, rfp2_gemv), queries and
keys are rotated and keys and values written into the paged cache
(rfp2_rope_kv_write), the new tokens attend over their sequences
(rfp2_paged_attn), and the result goes through the output weights.  Nothing in
a step depends on the host, so it is captured into a HIP graph once and replayed
for every token: positions and lengths are counted up on the GPU.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_gemv_amd as rf  # noqa: E402


class DecodeLayer:
    """Weights, cache and buffers of one layer for `seqs` sequences.

    w_qkv [(heads + 2 kv_heads) * dim][width] and w_out [width][heads * dim] are
    fp32 and packed to ROCmFP2 here."""

    def __init__(self, w_qkv, w_out, heads: int, kv_heads: int, dim: int, seqs: int,
                 max_tokens: int, format: int = rf.KV_I8, page_size: int = 64,
                 rope_base: float = 10000.0):
        dev = w_qkv.device
        self.heads, self.kv_heads, self.dim, self.seqs = heads, kv_heads, dim, seqs
        self.width, self.q_width = w_out.shape[0], heads * dim
        self.rows = w_qkv.shape[0]
        self.w_qkv, self.w_out = self._pack(w_qkv), self._pack(w_out)

        def f32(*shape):
            return torch.empty(shape, dtype=torch.float32, device=dev)

        def acts(K):
            return torch.empty((seqs, K), dtype=torch.int8, device=dev), f32(seqs, K // 32)

        self.x, self.out = torch.zeros(seqs, self.width, device=dev), f32(seqs, self.width)
        self.qkv, self.q, self.attn = f32(seqs, self.rows), f32(seqs, self.q_width), f32(seqs, self.q_width)
        self.acts_in, self.acts_attn = acts(self.width), acts(self.q_width)
        # every sequence gets the pages of its longest context, scattered over the memory
        per = -(-max_tokens // page_size)
        table = torch.randperm(seqs * per, device=dev).to(torch.int32).view(seqs, per)
        self.cache = rf.KvCache.allocate(format, seqs * per, page_size, kv_heads, dim, table)
        self.seq = torch.arange(seqs, dtype=torch.int32, device=dev)
        self.lens = torch.zeros(seqs, dtype=torch.int32, device=dev)
        self.pos = torch.zeros(seqs, dtype=torch.int32, device=dev)
        self.err = torch.zeros(1, dtype=torch.int32, device=dev)
        self.freqs = torch.empty(dim // 2, dtype=torch.float64, device=dev)
        rf.rfp2_rope_freqs(dim, rope_base, 1.0, 0.0, 0.0, 1.0, self.freqs)
        self.workspace = torch.empty(
            rf.rfp2_paged_attn_workspace_bytes(self.cache, seqs, 1, heads), dtype=torch.uint8,
            device=dev)

    @staticmethod
    def _pack(w):
        N, K = w.shape
        packed = torch.empty(N * K // 32 * 10, dtype=torch.uint8, device=w.device)
        rf.rfp2_quantize_weights(w.contiguous(), N, K, packed)
        return packed

    def fill(self, k, v, lens):
        """A prompt's rotated keys and values, [seqs][tokens][kv_heads][dim], of which
        sequence s keeps the first lens[s]."""
        T = k.shape[1]
        at = torch.arange(T, dtype=torch.int32, device=k.device)
        for s, n in enumerate(lens):
            if n:
                rf.rfp2_kv_write(self.cache, k[s], v[s], n, torch.full_like(at, s), at, self.err)
        self.lens.copy_(torch.tensor(lens, dtype=torch.int32))

    def step(self):
        """One token of every sequence: self.x -> self.out."""
        B, D = self.seqs, self.dim
        qw, kw = self.q_width, self.kv_heads * D
        self.pos.copy_(self.lens)
        self.lens.add_(1)
        rf.rfp2_quantize_acts(self.x, B, self.width, *self.acts_in)
        rf.rfp2_gemv(self.w_qkv, self.rows, self.width, *self.acts_in, B, self.qkv)
        q, k, v = self.qkv.split([qw, kw, kw], 1)
        rf.rfp2_rope_kv_write(self.cache, q, k, v, B, self.heads, self.seq, self.pos, self.freqs,
                              D, rf.ROPE_HALF, 1.0, self.q, self.err)
        rf.rfp2_paged_attn(self.cache, self.q, B, 1, self.heads, self.lens, D ** -0.5, self.attn,
                           err=self.err, workspace=self.workspace)
        rf.rfp2_quantize_acts(self.attn, B, qw, *self.acts_attn)
        rf.rfp2_gemv(self.w_out, self.width, qw, *self.acts_attn, B, self.out)

    def capture(self) -> torch.cuda.CUDAGraph:
        """The step as a graph; the lengths are left as they were."""
        lens = self.lens.clone()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            self.step()
        torch.cuda.current_stream().wait_stream(s)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            self.step()
        self.lens.copy_(lens)
        return graph


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--seqs", type=int, default=4)
    ap.add_argument("--context", type=int, default=3000)
    ap.add_argument("--steps", type=int, default=64)
    ap.add_argument("--format", choices=("i8", "f16"), default="i8")
    a = ap.parse_args()
    torch.manual_seed(0)
    dev, heads, kv_heads, dim, width = torch.device("cuda:0"), 32, 8, 128, 4096
    layer = DecodeLayer(0.02 * torch.randn((heads + 2 * kv_heads) * dim, width, device=dev),
                        0.02 * torch.randn(width, heads * dim, device=dev), heads, kv_heads, dim,
                        a.seqs, a.context + a.steps + 1,
                        rf.KV_I8 if a.format == "i8" else rf.KV_F16)
    k, v = torch.randn(2, a.seqs, a.context, kv_heads, dim, device=dev)
    layer.fill(k, v, [a.context - 7 * s for s in range(a.seqs)])
    graph = layer.capture()
    layer.x.normal_()
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    for _ in range(a.steps):
        graph.replay()
        layer.x.copy_(layer.out)          # stands in for the rest of the model
    end.record()
    torch.cuda.synchronize()
    assert int(layer.err) == 0
    print(f"{a.seqs} sequences of {a.context} tokens, {a.format} cache: "
          f"{start.elapsed_time(end) / a.steps * 1e3:.1f} us a layer and step; "
          f"lengths now {layer.lens.tolist()}")


if __name__ == "__main__":
    main()
