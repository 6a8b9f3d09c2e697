"""The operators together: the example block trains, decodes one token as in a
batch, and its gradients are those of the same block in 64 bits."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))
import block_ref as ref  # noqa: E402
import ternary_block as example  # noqa: E402

pytestmark = pytest.mark.gpu


def test_block_trains_and_decodes():
    print("example block", flush=True)
    losses, one, block, x = example.main(["--steps", "12", "--rows", "300", "--dim", "256", "--hidden", "512"])
    assert losses[-1] < 0.8 * losses[0], losses
    # a token alone takes other kernels than the batch, with the same formulas
    batch = block.forward(x)[:1].float()
    assert float((one.float() - batch).abs().max()) <= 2.0 ** -6 * float(batch.abs().max())


def test_block_gradients():
    """Against autograd in 64 bits of the block without its int8 roundings: these are half a step of 1/127 of each
    row's (column's) largest value, independent from element to element, so the gradients agree to a few per cent."""
    print("example block gradients", flush=True)
    dev = torch.device("cuda:0")
    g = torch.Generator(device=dev).manual_seed(3)
    block = example.Block(256, 512, dev, 2)
    x = torch.randn(300, 256, generator=g, device=dev).to(torch.bfloat16)
    dout = (torch.randn(300, 256, generator=g, device=dev) * 1e-2).to(torch.bfloat16)
    keep = {}
    block.forward(x, keep)
    dx, grads = block.backward(dout, keep)
    v = {n: t.double().clone().requires_grad_() for n, t in block.p.items()}
    xd = x.double().clone().requires_grad_()
    W1 = ref.unpack(block.W1) * block.w1 + v["W1"] - v["W1"].detach()      # straight through
    W2 = ref.unpack(block.W2) * block.w2 + v["W2"] - v["W2"].detach()
    y = xd * (xd.square().mean(1, keepdim=True) + 1e-6).rsqrt() * v["gain"]
    z = y @ W1.t() + v["b1"]
    out = torch.nn.functional.gelu(z, approximate="tanh") @ W2.t() + v["b2"] + xd
    out.backward(dout.double())
    for name, got, want in [("x", dx, xd.grad)] + [(n, grads[n], v[n].grad) for n in grads]:
        err = float((got.double() - want).norm() / want.norm())
        print(f"{name}: {err:.4f}", flush=True)
        assert err < 0.05, name
