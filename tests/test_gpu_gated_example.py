"""The operators together: the gated example block trains, decodes a token as in
a batch, and its gradients are those of the same block in 64 bits; a training
step captured into a graph is the eager one; calls on other streams."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))
import block_ref as ref  # noqa: E402
import gated_block as example  # noqa: E402
from ternary_weight_int8_amd import binding as B  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def test_block_runs_and_decodes():
    print("gated example block", flush=True)
    losses, one, block, x = example.main(["--steps", "3", "--rows", "300", "--dim", "256", "--hidden", "512", "--vocab", "1000"])
    assert len(losses) == 3 and all(v == v for v in losses)
    # a token alone takes other kernels than the batch.  The norm adds its row up in another order, so a value on
    # the border of two int8 steps may go either way: one step of 1/127 of a row's largest value, in a few of them
    batch = block.forward(x)[:1]
    assert float((one - batch).abs().max()) <= 2.0 ** -6 * float(batch.abs().max())


def test_block_gradients():
    """Against autograd in 64 bits of the block without its int8 roundings.  One of them is at most half a step of
    1/127 of its row's (column's) largest value, independent from element to element: of rows whose largest value is
    seven times their root mean square, 7 / 127 / sqrt(12) = 1.6% of the norm.  A gradient here passes at most nine of
    them, forward and backward, 4.8% when they add up as independent errors do; bfloat16's 2^-9 are lost in that."""
    print("gated example block gradients", flush=True)
    g = torch.Generator(device=DEV).manual_seed(3)
    block = example.Block(256, 512, 300, DEV, 2)
    x = torch.randn(400, 256, generator=g, device=DEV).to(torch.bfloat16)
    dout = (torch.randn(400, 300, generator=g, device=DEV) * 1e-2).to(torch.bfloat16)
    keep = {}
    block.forward(x, keep)
    dx, grads = block.backward(dout, keep)
    v = {n: t.double().clone().requires_grad_() for n, t in block.p.items()}
    xd = x.double().clone().requires_grad_()
    through = lambda stored, n: stored + v[n] - v[n].detach()  # noqa: E731
    W = ref.unpack(block.Wgu)
    Wg, Wu = through(W[:512] * block.wg, "Wg"), through(W[512:] * block.wu, "Wu")
    Wd = through(ref.unpack(block.Wd) * block.wd, "Wd")
    W8 = through(block.W8.double() * block.w8.double()[:, None], "W8")
    d = xd - xd.mean(1, keepdim=True)
    y = d * (d.square().mean(1, keepdim=True) + 1e-5).rsqrt() * v["gain"] + v["beta"]
    u = torch.nn.functional.silu(y @ Wg.t() + v["bgu"][:512]) * (y @ Wu.t() + v["bgu"][512:])
    h = xd + u @ Wd.t()
    (h @ W8.t() + v["b8"]).backward(dout.double())
    for name, got, want in [("x", dx, xd.grad)] + [(n, grads[n], v[n].grad) for n in grads]:
        err = float((got.double() - want).norm() / want.norm())
        print(f"{name}: {err:.4f}", flush=True)
        assert err < 0.05, name


@pytest.mark.parametrize("rows", [5, 300])
def test_step_in_a_graph(rows):
    """Forward and backward captured and replayed on other inputs, with eager work between the replays.  The column
    quantizer's and the weights' calls are the framework's older ones and stay outside."""
    print(f"graph of {rows} rows", flush=True)
    g = torch.Generator(device=DEV).manual_seed(5)
    block = example.Block(256, 320, 200, DEV, 2)
    xs = [torch.randn(rows, 256, generator=g, device=DEV).to(torch.bfloat16) for _ in range(3)]
    dus = [(torch.randn(rows, 320, generator=g, device=DEV) * 1e-3).to(torch.bfloat16) for _ in range(3)]

    def work(x, du):
        q, s, h, y, mean, rstd = B.ternary_layernorm_quantize(x, block.p["gain"], block.p["beta"], residual=x, save=True)
        u, z = B.ternary_gemm_s8_gated(q, block.Wgu, s, block.wg, block.wu, bias=block.p["bgu"], save=True)
        l, _ = B.ternary_gemm_s8s8_epilogue(q, block.W8, s, block.w8, bias=block.p["b8"], act="gelu_tanh")
        dz, db, qz, sz = B.ternary_gated_backward(du, z, block.wg, block.wu)
        dx, dg, dbeta = B.ternary_layernorm_backward(y, h, block.p["gain"], mean, rstd, dH=x)
        return q, s, h, y, mean, rstd, u, z, l, dz, db, qz, sz, dx, dg, dbeta

    want = [[t.clone() for t in work(x, du)] for x, du in zip(xs, dus)]
    x, du = xs[0].clone(), dus[0].clone()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        work(x, du)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = work(x, du)
    for i in (1, 0, 2, 1):
        x.copy_(xs[i])
        du.copy_(dus[i])
        graph.replay()
        work(xs[2], dus[2])                   # eager calls while the graph runs
        torch.cuda.synchronize()
        for a, b in zip(out, want[i]):
            assert torch.equal(a, b), i


def test_two_streams_at_once():
    """Calls on two streams, outputs and workspaces made by the calls themselves, against one after the other."""
    print("two streams", flush=True)
    g = torch.Generator(device=DEV).manual_seed(6)
    A = torch.randint(-128, 128, (900, 260), generator=g, device=DEV, dtype=torch.int8)
    W = torch.randint(0, 256, (1000, 65), generator=g, device=DEV, dtype=torch.uint8)
    W8 = torch.randint(-128, 128, (700, 260), generator=g, device=DEV, dtype=torch.int8)
    rs = torch.rand(900, generator=g, device=DEV) * 1e-3
    dY = torch.randn(900, 500, generator=g, device=DEV).to(torch.bfloat16)
    H = torch.randn(900, 500, generator=g, device=DEV).to(torch.bfloat16)
    gain, mean = torch.rand(500, generator=g, device=DEV), torch.zeros(900, device=DEV)

    def work(s):
        Y, Z = B.ternary_gemm_s8_gated(A, W, rs, 0.5, 0.25, save=True, stream=s)
        L, _ = B.ternary_gemm_s8s8_epilogue(A, W8, rs, stream=s)
        out = [Y, Z, L, *B.ternary_gated_backward(dY, Z, 0.5, 0.25, stream=s)]
        return out + list(B.ternary_layernorm_backward(dY, H, gain, mean, rs, stream=s))

    want = work(None)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [work(s) for _ in range(4) for s in streams]
    torch.cuda.synchronize()
    for out in got:
        for a, b in zip(out, want):
            assert torch.equal(a, b)
