"""Fine-tuning and serving the adapters of several tenants on one MLP block.

A frozen MLP block (two projections around a GELU) carries a low-rank adapter per tenant
on either projection, under a trained read-out.  Every step holds rows of all tenants.
What the backward pass needs of the activations is kept in 8 bits: the inputs of the
three products and the input of the GELU.  After training, the same adapters serve a
decode step, a token per request.

    python examples/adapter_finetune.py [--steps N] [--bf16]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from dense_fp32_gemm_02_gb300 import binding as b   # noqa: E402


class Adapters:
    """A frozen projection W (K, N) and a stack of L low-rank adapters beside it."""

    def __init__(self, K, N, L, R, dtype, g):
        def normal(*shape, scale):
            return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)
        self.W = normal(K, N, scale=K ** -0.5)
        self.A = normal(L, K, R, scale=K ** -0.5)
        self.B = torch.zeros(L, R, N, dtype=dtype, device="cuda")
        self.scale = torch.full((L,), 2.0, device="cuda")

    def forward(self, X, ids, keep):
        """Y, and for a training step what backward() needs: the rank side's sums, and X in 8 bits."""
        Y = torch.empty(X.shape[0], self.W.shape[1], dtype=X.dtype, device="cuda")
        H = torch.empty(X.shape[0], self.A.shape[2], device="cuda") if keep else None
        b.lora_into(X, self.W, self.A, self.B, ids, Y, scale=self.scale, H=H)
        return Y, (H, b.act8_store_into(X, *b.act8_empty(*X.shape))) if keep else None

    def backward(self, dY, kept, ids, rate):
        """dX; the adapters take a gradient step."""
        H, X8 = kept
        dX = torch.empty(dY.shape[0], self.W.shape[0], dtype=dY.dtype, device="cuda")
        dA, dB = torch.empty_like(self.A), torch.empty_like(self.B)
        b.lora_backward_into(dY, X8, self.W, self.A, self.B, ids, H, dX=dX, dA=dA, dB=dB,
                             scale=self.scale)
        self.A -= rate * dA
        self.B -= rate * dB
        return dX


class Model:
    def __init__(self, width=256, hidden=1024, classes=64, tenants=4, rank=16,
                 dtype=torch.float32, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.up = Adapters(width, hidden, tenants, rank, dtype, g)
        self.down = Adapters(hidden, width, tenants, rank, dtype, g)
        self.out = (torch.randn(width, classes, generator=g, device="cuda") * width ** -0.5).to(dtype)
        self.tenants, self.width, self.classes, self.dtype = tenants, width, classes, dtype

    def forward(self, X, ids, keep=False):
        Z, up = self.up.forward(X, ids, keep)
        act = torch.empty_like(Z)
        z8 = b.act8_store_into(Z, *b.act8_empty(*Z.shape), act="gelu", Y=act)
        hidden, down = self.down.forward(act, ids, keep)
        Y = torch.empty(X.shape[0], self.classes, dtype=self.dtype, device="cuda")
        none = torch.empty(0, *self.out.shape[:1], 1, dtype=self.dtype, device="cuda")
        b.lora_into(hidden, self.out, none, none.new_empty(0, 1, self.classes), ids, Y)   # no adapters
        return Y, (up, z8, down, b.act8_store_into(hidden, *b.act8_empty(*hidden.shape))) if keep else None

    def step(self, X, target, ids, rate):
        """One gradient step on the mean squared error; the loss before it, on the device."""
        Y, (up, z8, down, h8) = self.forward(X, ids, keep=True)
        error = Y.float() - target
        dY = (error * (2.0 / error.numel())).to(self.dtype)
        d_out = b.act8_weight_grad_into(*h8, dY, torch.empty_like(self.out))
        d_hidden = dY @ self.out.t()
        d_act = self.down.backward(d_hidden, down, ids, rate)
        dZ = b.act8_grad_into(*z8, d_act, d_act, act="gelu")
        self.up.backward(dZ, up, ids, rate)
        self.out -= rate * d_out
        return (error * error).mean()


def batch(model, requests, length, g):
    """Rows of `requests` sequences, one tenant each, in a row; the last has no adapter."""
    X = torch.randn(requests * length, model.width, generator=g, device="cuda").to(model.dtype)
    ids = torch.randint(0, model.tenants, (requests,), generator=g, device="cuda", dtype=torch.int32)
    ids[-1] = -1
    return X, ids.repeat_interleave(length).contiguous()


def train(model, steps, rate=2.0, requests=12, length=100, seed=1):
    """Fits every tenant to a linear map of its own; the losses."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    maps = torch.randn(model.tenants + 1, model.width, model.classes, generator=g, device="cuda") * model.width ** -0.5
    X, ids = batch(model, requests, length, g)
    target = torch.einsum("mk,mkn->mn", X.float(), maps[ids.long()])
    return [float(model.step(X, target, ids, rate)) for _ in range(steps)], (X, ids)


def main():
    p = argparse.ArgumentParser()
    p.add_argument("--steps", type=int, default=50)
    p.add_argument("--bf16", action="store_true")
    a = p.parse_args()
    model = Model(dtype=torch.bfloat16 if a.bf16 else torch.float32)
    losses, (X, ids) = train(model, a.steps)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {a.steps} steps")
    # a decode step: a token of each request, every one with its own adapter
    rows = torch.arange(0, X.shape[0], 100, device="cuda")
    token, _ = model.forward(X[rows].contiguous(), ids[rows].contiguous())
    whole, _ = model.forward(X, ids)
    print(f"decode step of {len(rows)} requests against the same rows of the prefill: "
          f"largest difference {float((token.float() - whole[rows].float()).abs().max()):.2e}")


if __name__ == "__main__":
    main()
