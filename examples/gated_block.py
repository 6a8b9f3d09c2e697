"""Training and decoding one gated block of ternary layers under a layer norm,
with an 8-bit head, with the library's operators:

    q, s    = int8 rows of layernorm(x) * gain + beta       ternary_layernorm_quantize
    u       = silu(q @ Wg * s * wg + bg) * (q @ Wu * s * wu + bu)   ternary_gemm_s8_gated
    h       = x + (u as int8 rows) @ Wd * su * wd           ternary_gemm_s8_epilogue
    logits  = (h as int8 rows) @ W8 * sh * w8[channel] + b8     ternary_gemm_s8s8_epilogue

Wg, Wu and Wd are ternary, W8 is int8 with a scale a channel; gradients go
straight through the roundings.  The gate's and the up projection's codes are
one stored matrix, so the backward pass takes one ternary_gemm_s8_dx_scaled call
for both, on the int8 rows of ternary_gated_backward, and one
ternary_gemm_s8_dw_scaled call; the head's input gradient is
ternary_gemm_s8s8_epilogue again, on the transposed weights.

    python examples/gated_block.py [--steps 10] [--rows 1782] [--dim 1280] [--hidden 3456] [--vocab 16384]

trains the block to name, for random vectors, the classes of a fixed random block
and then decodes one token.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from ternary_block import ternarized  # noqa: E402
from ternary_weight_int8_amd import binding as B  # noqa: E402

ACT = "silu"


class Block:
    def __init__(self, dim, hidden, vocab, device, seed):
        g = torch.Generator(device=device).manual_seed(seed)
        normal = lambda *s: torch.randn(s, generator=g, device=device)  # noqa: E731
        self.p = {"gain": torch.ones(dim, device=device), "beta": 0.1 * normal(dim), "Wg": normal(hidden, dim) / dim ** 0.5,
                  "Wu": normal(hidden, dim) / dim ** 0.5, "bgu": 0.1 * normal(2 * hidden),
                  "Wd": normal(dim, hidden) / hidden ** 0.5, "W8": normal(vocab, dim) / dim ** 0.5, "b8": 0.1 * normal(vocab)}
        self.dim, self.hidden, self.vocab = dim, hidden, vocab
        self.refresh()

    def refresh(self):
        """The stored weights, after the master weights changed."""
        (g, self.wg), (u, self.wu) = ternarized(self.p["Wg"]), ternarized(self.p["Wu"])
        self.Wgu = torch.cat((g, u))
        self.Wd, self.wd = ternarized(self.p["Wd"])
        self.W8, self.w8 = B.ternary_quantize_rows(self.p["W8"])
        self.W8t, self.w8t = B.ternary_quantize_rows(self.p["W8"].t().contiguous())

    def forward(self, x, keep=None):
        """x [rows][dim] bfloat16 -> logits float32 [rows][vocab]; `keep`, a dict, takes what backward needs."""
        train = keep is not None
        q, s, h0, y, mean, rstd = B.ternary_layernorm_quantize(x, self.p["gain"], self.p["beta"], save=train)
        u, z = B.ternary_gemm_s8_gated(q, self.Wgu, s, self.wg, self.wu, bias=self.p["bgu"], act=ACT, save=train)
        qu, su = B.ternary_quantize_rows(u)
        h, _ = B.ternary_gemm_s8_epilogue(qu, self.Wd, su, self.wd, residual=h0)
        qh, sh = B.ternary_quantize_rows(h)
        logits, _ = B.ternary_gemm_s8s8_epilogue(qh, self.W8, sh, self.w8, bias=self.p["b8"], out_dtype=torch.float32)
        if train:
            keep.update(h0=h0, y=y, mean=mean, rstd=rstd, u=u, z=z, h=h)
        return logits

    def backward(self, dlogits, k):
        """(dx, the parameters' gradients) from the gradient of the logits (bfloat16)."""
        bf = torch.bfloat16
        q, s = B.ternary_quantize_rows(dlogits)
        dh, _ = B.ternary_gemm_s8s8_epilogue(q, self.W8t, s, self.w8t, out_dtype=bf)
        grads = {"W8": self._dw(k["h"], dlogits), "b8": dlogits.float().sum(0), "Wd": self._dw(k["u"], dh)}
        q, s = B.ternary_quantize_rows(dh)
        du = B.ternary_gemm_s8_dx_scaled(q, self.Wd, self.hidden, s, self.wd, bf)
        dz, grads["bgu"], q, s = B.ternary_gated_backward(du, k["z"], self.wg, self.wu, act=ACT)
        dy = B.ternary_gemm_s8_dx_scaled(q, self.Wgu, self.dim, s, 1.0, bf)
        grads["Wg"], grads["Wu"] = self._dw(k["y"], dz).chunk(2)
        dx, grads["gain"], grads["beta"] = B.ternary_layernorm_backward(dy, k["h0"], self.p["gain"], k["mean"], k["rstd"],
                                                                        dH=dh)
        return dx, grads

    @staticmethod
    def _dw(a, d):
        """d^T @ a as [N][K], the layout of the master weight."""
        qa, sa = B.ternary_quantize_cols(a)
        qd, sd = B.ternary_quantize_cols(d)
        return B.ternary_gemm_s8_dw_scaled(qd, qa, sd, sa, torch.float32)

    def step(self, x, target, lr, max_norm):
        """One training step on the cross entropy; (loss, gradient norm) as device tensors."""
        keep = {}
        logits = self.forward(x, keep)
        logp = torch.log_softmax(logits, 1)
        loss = -logp.gather(1, target[:, None]).mean()
        d = logp.exp()
        d.scatter_add_(1, target[:, None], torch.full_like(logits[:, :1], -1.0))
        _, grads = self.backward((d / len(x)).to(torch.bfloat16), keep)
        names = list(grads)
        flat = [grads[n].contiguous() for n in names]
        clipped, norm = B.ternary_clip_grad_norm(flat, max_norm, out=flat)
        for n, g in zip(names, clipped):
            self.p[n].sub_(g, alpha=lr)
        self.refresh()
        return loss, norm


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=10)
    ap.add_argument("--rows", type=int, default=1782)
    ap.add_argument("--dim", type=int, default=1280)
    ap.add_argument("--hidden", type=int, default=3456)
    ap.add_argument("--vocab", type=int, default=16384)
    ap.add_argument("--lr", type=float, default=1.0)
    a = ap.parse_args(argv)
    dev = torch.device("cuda:0")
    x = torch.randn(a.rows, a.dim, generator=torch.Generator(device=dev).manual_seed(0), device=dev).to(torch.bfloat16)
    target = Block(a.dim, a.hidden, a.vocab, dev, 1).forward(x).argmax(1)
    block = Block(a.dim, a.hidden, a.vocab, dev, 2)
    losses = []
    for i in range(a.steps):
        loss, norm = block.step(x, target, a.lr, 1.0)
        losses.append(float(loss))
        print(f"step {i:3d}  loss {losses[-1]:.4f}  gradient norm {float(norm):.4f}", flush=True)
    one = block.forward(x[:1].contiguous())
    print(f"one token: class {int(one.argmax())} of {a.vocab}", flush=True)
    return losses, one, block, x


if __name__ == "__main__":
    main()
