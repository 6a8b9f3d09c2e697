"""Training and decoding one residual block of ternary linear layers with the
library's operators:

    q, s  = int8 rows of rmsnorm(x) * gain            ternary_rmsnorm_quantize
    u     = gelu(q @ W1 * s * w1 + b1)                ternary_gemm_s8_epilogue
    out   = x + (u as int8 rows) @ W2 * su * w2 + b2  ternary_gemm_s8_epilogue

W1 and W2 are ternary (a master weight's sign where it exceeds half the mean
magnitude, times that mean); gradients go straight through the roundings.  The
backward pass is int8 too: ternary_epilogue_backward and
ternary_rmsnorm_backward around ternary_gemm_s8_dx_scaled and
ternary_gemm_s8_dw_scaled; the gradients are clipped by their global norm
(ternary_clip_grad_norm) before the update.

    python examples/ternary_block.py [--steps 20] [--rows 1782] [--dim 1280] [--hidden 3456]

trains the block to reproduce a fixed random one and then decodes one token.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from ternary_weight_int8_amd import binding as B  # noqa: E402

ACT = "gelu_tanh"


def ternarized(master):
    """The stored codes and the scale of a master weight [N][K]."""
    scale = master.abs().mean()
    w = torch.where(master.abs() > 0.5 * scale, master.sign(), torch.zeros_like(master))
    return B.ternary_pack_weights(w.to(torch.int8)), float(scale)


class Block:
    def __init__(self, dim, hidden, device, seed):
        g = torch.Generator(device=device).manual_seed(seed)
        normal = lambda *s: torch.randn(s, generator=g, device=device)  # noqa: E731
        self.p = {"gain": torch.ones(dim, device=device), "W1": normal(hidden, dim) / dim ** 0.5,
                  "b1": 0.1 * normal(hidden), "W2": normal(dim, hidden) / hidden ** 0.5, "b2": 0.1 * normal(dim)}
        self.dim, self.hidden = dim, hidden
        self.refresh()

    def refresh(self):
        """The stored weights, after the master weights changed."""
        self.W1, self.w1 = ternarized(self.p["W1"])
        self.W2, self.w2 = ternarized(self.p["W2"])

    def forward(self, x, keep=None):
        """x [rows][dim] bfloat16 -> [rows][dim]; `keep`, a dict, takes what backward needs."""
        train = keep is not None
        q, s, h, y, rstd = B.ternary_rmsnorm_quantize(x, self.p["gain"], save=train)
        u, z = B.ternary_gemm_s8_epilogue(q, self.W1, s, self.w1, bias=self.p["b1"], act=ACT, save=train)
        qu, su = B.ternary_quantize_rows(u)
        out, _ = B.ternary_gemm_s8_epilogue(qu, self.W2, su, self.w2, bias=self.p["b2"], residual=h)
        if train:
            keep.update(h=h, y=y, rstd=rstd, u=u, z=z)
        return out

    def backward(self, dout, k):
        """(dx, the parameters' gradients) from out's gradient."""
        bf = torch.bfloat16
        # out = u @ W2 + b2 + h: int8 rows for du, int8 columns for dW2
        _, db2, q, s = B.ternary_epilogue_backward(dout, dout, act="none")
        du = B.ternary_gemm_s8_dx_scaled(q, self.W2, self.hidden, s, self.w2, bf)
        dW2 = self._dw(k["u"], dout)
        dz, db1, q, s = B.ternary_epilogue_backward(du, k["z"], act=ACT)
        dy = B.ternary_gemm_s8_dx_scaled(q, self.W1, self.dim, s, self.w1, bf)
        dW1 = self._dw(k["y"], dz)
        dx, dgain = B.ternary_rmsnorm_backward(dy, k["h"], self.p["gain"], k["rstd"], dH=dout)
        return dx, {"gain": dgain, "W1": dW1, "b1": db1, "W2": dW2, "b2": db2}

    @staticmethod
    def _dw(a, d):
        """d^T @ a as [N][K], the layout of the master weight."""
        qa, sa = B.ternary_quantize_cols(a)
        qd, sd = B.ternary_quantize_cols(d)
        return B.ternary_gemm_s8_dw_scaled(qd, qa, sd, sa, torch.float32)

    def step(self, x, target, lr, max_norm):
        """One training step on the mean squared error; (loss, gradient norm) as device tensors."""
        keep = {}
        out = self.forward(x, keep)
        diff = out.float() - target.float()
        dout = (diff * (2.0 / diff.numel())).to(torch.bfloat16)
        _, grads = self.backward(dout, keep)
        names = list(grads)
        clipped, norm = B.ternary_clip_grad_norm([grads[n] for n in names], max_norm, out=[grads[n] for n in names])
        for n, g in zip(names, clipped):
            self.p[n].sub_(g, alpha=lr)
        self.refresh()
        return diff.square().mean(), norm


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--rows", type=int, default=1782)
    ap.add_argument("--dim", type=int, default=1280)
    ap.add_argument("--hidden", type=int, default=3456)
    ap.add_argument("--lr", type=float, default=1.0)
    a = ap.parse_args(argv)
    dev = torch.device("cuda:0")
    x = torch.randn(a.rows, a.dim, generator=torch.Generator(device=dev).manual_seed(0), device=dev).to(torch.bfloat16)
    target = Block(a.dim, a.hidden, dev, 1).forward(x)
    block = Block(a.dim, a.hidden, dev, 2)
    losses = []
    for i in range(a.steps):
        loss, norm = block.step(x, target, a.lr, 1.0)
        losses.append(float(loss))
        print(f"step {i:3d}  loss {losses[-1]:.4f}  gradient norm {float(norm):.4f}", flush=True)
    one = block.forward(x[:1].contiguous())
    print(f"one token: {a.dim} values, rms {float(one.float().square().mean().sqrt()):.3f}", flush=True)
    return losses, one, block, x


if __name__ == "__main__":
    main()
