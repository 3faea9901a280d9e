"""Trains one layer of experts on a GPU, from routing to the optimizer step.

    python examples/expert_layer.py [--steps 60] [--bits 8]

Each token goes to the k experts that a router scores highest, every expert multiplies its rows
by its weight, and the results come back weighted by the router's softmax. The goal is a layer
of the same shape with other weights. One step:

    forward   kg_route             tokens into expert order
              kg_dispatch_fp8      their rows as e4m3 codes, one scale per 128 channels
              kg_fprop             rows . w^T per expert
              kg_combine           weighted sum per token
    backward  kg_combine_bwd       gradients of the rows and of the router's weights
              kg_requant, kg_wgrad weight gradients, operands scaled per 128 tokens
              kg_dgrad             row gradients
              kg_combine           ... summed per token (the layer's input gradient)
    update    kg_adamw             all tensors in one launch, states in 8 or 32 bits

Nothing in a step waits for the GPU on the host. (Every slot here has an expert. Slots that are
dropped leave the products fewer rows, and the host has to read how many.)
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import fp8_grouped_gemm_tn_amd as kg  # noqa: E402
from fp8_grouped_gemm_tn_amd import inputs  # noqa: E402


class ExpertLayer:
    """G experts with weights w [G, N, K] (fp32 masters) behind a linear router [G, K]. K and N
    are multiples of 128."""

    def __init__(self, G, K, N, k, bits=8, seed=0, device="cuda"):
        gen = torch.Generator(device).manual_seed(seed)
        self.G, self.K, self.N, self.k = G, K, N, k
        self.w = torch.randn((G, N, K), generator=gen, device=device) * K ** -0.5
        self.router = torch.randn((G, K), generator=gen, device=device) * K ** -0.5
        self.params = [self.w, self.router]
        self.grads = [torch.zeros_like(p) for p in self.params]
        byte = dict(dtype=torch.uint8) if bits == 8 else {}
        state = lambda: [torch.zeros(p.shape, device=device, **byte) for p in self.params]
        scales = lambda: [torch.zeros(-(-p.numel() // 128), device=device) for p in self.params]
        self.table = kg.AdamWTable(self.params, self.grads, state(), state(),
                                   *([scales(), scales()] if bits == 8 else []))
        self.step_count = 0

    def forward(self, x):
        """x bf16 [T, K] -> bf16 [T, N]."""
        T = x.shape[0]
        scores = x.float() @ self.router.t()
        top, idx = scores.topk(self.k, dim=1)
        self.p = torch.softmax(top, dim=1)
        self.idx = idx.to(torch.int32)
        self.ks = torch.empty(self.G, dtype=torch.int32, device=x.device)
        self.pos, _ = kg.kg_route(self.idx, self.ks)
        rows, sa = kg.kg_dispatch_fp8(x, self.pos)
        self.wq, self.sw = inputs.quantize_blocks_128x128(self.w)
        self.x = x
        self.y = torch.empty((T * self.k, self.N), dtype=torch.bfloat16, device=x.device)
        kg.kg_fprop(rows, sa, self.wq, self.sw, self.y, self.ks, kg.KG_FLAG_FP8_MFMA)
        return kg.kg_combine(self.y, self.pos, self.p)

    def backward(self, dout):
        """dout bf16 [T, N] -> the gradient of x, bf16 [T, K]; fills self.grads."""
        T, k, G = self.x.shape[0], self.k, self.G
        dy, dp = kg.kg_combine_bwd(dout, self.y, self.pos, self.p)
        # weight gradients: both operands in fp8 with scales per 128 tokens of an expert
        blocks = T * k // 128 + G  # at least sum(ceil(ks / 128))
        xq, sx = kg.kg_requant(kg.kg_dispatch(self.x, self.pos), None, self.ks, 128,
                               kg.KG_E4M3_F32SCALE, blocks)
        dq, sd = kg.kg_requant(dy, None, self.ks, 128, kg.KG_E4M3_F32SCALE, blocks)
        kg.kg_wgrad(dq, sd, xq, sx, None, self.grads[0], self.ks, 128, kg.KG_E4M3_F32SCALE)
        # row gradients, back to the tokens
        dyq, sdy = inputs.quantize_rows_1x128(dy.float())
        dxp = torch.empty((T * k, self.K), dtype=torch.bfloat16, device=dy.device)
        kg.kg_dgrad(dyq, sdy, self.wq, self.sw, dxp, self.ks, kg.KG_FLAG_FP8_MFMA)
        dx = kg.kg_combine(dxp, self.pos)
        # the router: softmax over the k chosen scores
        dscore = self.p * (dp - (self.p * dp).sum(1, keepdim=True))
        full = torch.zeros((T, G), device=dy.device).scatter_(1, self.idx.long(), dscore)
        torch.mm(full.t(), self.x.float(), out=self.grads[1])
        return dx + (full @ self.router).to(dx.dtype)

    def update(self, lr):
        self.step_count += 1
        kg.kg_adamw(self.table, lr, beta2=0.99, step=self.step_count)


def train(steps=60, bits=8, T=2048, G=8, K=256, N=384, k=2, lr=3e-3, say=None):
    """The losses of `steps` steps towards another layer's outputs."""
    layer, goal = ExpertLayer(G, K, N, k, bits, seed=1), ExpertLayer(G, K, N, k, seed=2)
    goal.router.copy_(layer.router)
    gen = torch.Generator("cuda").manual_seed(3)
    losses = []
    for step in range(steps):
        x = torch.randn((T, K), generator=gen, device="cuda").to(torch.bfloat16)
        want = goal.forward(x).float()
        err = layer.forward(x).float() - want
        losses.append(err.square().mean())
        layer.backward((err * (2 / N)).to(torch.bfloat16))
        layer.update(lr)
        if say and (step % 10 == 0 or step == steps - 1):
            say(f"step {step:4d}  loss {float(losses[-1]):.4f}")
    rc = kg.kg_status()  # what the kernels found (counts that do not add up)
    if rc != kg.KG_OK:
        raise kg.KgError(rc, "expert layer")
    return torch.stack(losses).tolist()


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--bits", type=int, choices=(8, 32), default=8)
    args = ap.parse_args()
    train(args.steps, args.bits, say=print)
