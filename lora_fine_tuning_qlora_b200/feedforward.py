"""A transformer's feed-forward block on two int8-LoRA Dense layers, trained
from 8-bit activations.

    Y = down(act(up(X))) + X          (the skip connection is optional)

("Introduce QLoRA-like technique", GPT-2 fine-tuning; keras-llm-light,
"Block-wise gradient checkpointing", for keeping little between forward and
backward.  A gated block, which multiplies two up projections, is not this one.)
The activation, the residual and every checkpoint run in the GEMMs'
epilogues; between the passes the block holds, per token, the codes of X and of
act(Z) (K + N bytes), Z in 8 bits (1.125 N bytes) and a few floats, against 2 K
+ 4 N bytes of bf16 activations:

    forward   up:   Xq, sx, xA; H = act(Z), Z kept in 8 bits
              down: Hq, sh, hA; Y = H W2 + .. + X
    backward  down: dZ = (dY W2^T + ..) * act'(z), dA2 = c H^T G2, dB2, dbias2
              up:   dX = (dZ W1^T + ..) + dY,      dA1 = c X^T G1, dB1, dbias1

``FeedForward`` owns the buffers at M tokens; a step can be captured into a
CUDA graph and replayed.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import qlora


class FeedForward:
    def __init__(self, up: qlora.Layer, down: qlora.Layer, M: int, act: str = "gelu_tanh", skip: bool = True,
                 device="cuda"):
        if up.N != down.K or up.act != down.act:
            raise ValueError("down takes what up gives: the same width and activation dtype")
        if skip and up.K != down.N:
            raise ValueError("a skip connection needs down to give what up takes")
        qlora.act_fn(act)
        dev = torch.device(device)
        self.up, self.down, self.M, self.act, self.skip = up, down, M, act, skip
        dt = up.act

        def buf(*shape, dtype=dt):
            return torch.empty(shape, dtype=dtype, device=dev)

        self.X, self.dY = buf(M, up.K), buf(M, down.N)
        self.X.zero_(), self.dY.zero_()
        self.H, self.Y = buf(M, up.N), buf(M, down.N)          # H is free again after the forward
        self.dZ, self.dX = buf(M, up.N), buf(M, up.K)
        self.keep_up = qlora.Checkpoint.allocate(M, up.K, up.r, dev)
        self.keep_up.zq, self.keep_up.zs = qlora.ckpt_buffers(M, up.N, dev)
        self.keep_down = qlora.Checkpoint.allocate(M, down.K, down.r, dev)
        # one workspace serves both layers: their backward passes run in turn
        need = max(qlora.qlora_ckpt_workspace_bytes(L.desc(), M) for L in (up, down))
        if need == 0:
            raise ValueError("invalid layers or more than 1047552 tokens")
        self.ws = buf(need, dtype=torch.uint8)
        # the trainable gradients in one flat buffer (one all-reduce in data
        # parallel runs): dA, dB, dbias of up, then of down
        sizes = [(L.K, L.r, L.N) for L in (up, down)]
        self.grad_flat = buf(sum(K * r + r * N + N for K, r, N in sizes), dtype=torch.float32)
        self.grads, at = [], 0
        for K, r, N in sizes:
            dA = self.grad_flat[at:at + K * r].view(K, r)
            dB = self.grad_flat[at + K * r:at + K * r + r * N].view(r, N)
            dbias = self.grad_flat[at + K * r + r * N:at + K * r + r * N + N]
            at += K * r + r * N + N
            self.grads.append((dA, dB, dbias))
        self.graph: Optional[torch.cuda.CUDAGraph] = None

    def forward(self, stream=None) -> torch.Tensor:
        """Y of self.X."""
        qlora.forward_act(self.up, self.X, act=self.act, save_z=True, keep=self.keep_up, Y=self.H, stream=stream)
        qlora.forward_act(self.down, self.H, residual=self.X if self.skip else None, keep=self.keep_down, Y=self.Y,
                          stream=stream)
        return self.Y

    def backward(self, stream=None) -> torch.Tensor:
        """dX of self.dY; the parameter gradients into self.grads = [up, down]."""
        qlora.backward_ckpt(self.down, self.keep_down, self.dY, self.ws, act=self.act, z=self.keep_up.z, dX=self.dZ,
                            grads=self.grads[1], stream=stream)
        qlora.backward_ckpt(self.up, self.keep_up, self.dZ, self.ws, add=self.dY if self.skip else None, dX=self.dX,
                            grads=self.grads[0], stream=stream)
        return self.dX

    def step(self, stream=None):
        self.forward(stream)
        self.backward(stream)

    def capture(self, warmup: int = 1):
        """Records one step into a CUDA graph (after `warmup` eager steps)."""
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            for _ in range(warmup):
                self.step()
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            self.step()
        self.graph = g
        return g

    def replay(self):
        assert self.graph is not None
        self.graph.replay()

    def kept_bytes(self) -> int:
        """Bytes that live from the forward to the backward."""
        k, d = self.keep_up, self.keep_down
        return sum(t.numel() * t.element_size() for t in (k.Xq, k.sx, k.xA, k.zq, k.zs, d.Xq, d.sx, d.xA))
