"""The operators together: the example's residual blocks against 64-bit autograd (needs a GB300)."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("fp8_residual_blocks", os.path.join(ROOT, "examples", "fp8_residual_blocks.py"))
    m = importlib.util.module_from_spec(spec)
    import sys
    sys.modules[spec.name] = m       # dataclasses look their module up
    spec.loader.exec_module(m)
    return m


def matrices(w):
    G, N, K = w.codes.shape
    s = w.scales.double().repeat_interleave(128, 1)[:, :N].repeat_interleave(128, 2)[:, :, :K]
    return w.codes.view(torch.float8_e4m3fn).double() * s


def reference(blocks, x, padding):
    """The blocks in 64 bits with the same matrices and picks, without any rounding of activations."""
    rms = lambda v, w: v * (v.square().mean(1, keepdim=True) + 1e-6).rsqrt() * w  # noqa: E731
    for b in blocks:
        n = rms(x, b["w_in"])
        logits = n @ b["router"].t()
        ids = b["ids"].clamp_min(0).long()
        w = torch.softmax(logits.gather(1, ids), 1)
        gu = torch.einsum("th,tknh->tkn", n, b["gate_up"][ids])
        g, u = gu.chunk(2, dim=2)
        ys = torch.einsum("tki,tkhi->tkh", torch.nn.functional.silu(g) * u, b["down"][ids])
        y = torch.where(padding[:, None], 0.0, (w[..., None] * ys).sum(1))
        x = x + b["gate"] * rms(y, b["w_out"])
    return x


def off(a, b):
    return float((a.double() - b).norm() / b.norm())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_blocks_against_autograd(cuda_lib, example, dtype):
    """A chain of at most six e4m3 roundings of rows (2^-4 of an element at most, a quarter of that in
    the mean) and as many of bf16 lies between a value and its 64-bit form."""
    T, H = 96, 256
    blocks = example.make_blocks(2, T, H, inner=128, E=8, k=2, seed=3)
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    x = torch.randn(T, H, generator=g, device="cuda").to(dtype)
    dout = torch.randn(T, H, generator=g, device="cuda").to(dtype)
    padding = torch.arange(T, device="cuda") % 13 == 4
    out, trace = example.forward(blocks, x, padding)
    ids = [b.saved["ids"].clone() for b in blocks]
    grads, dx = example.backward(blocks, trace, dout)
    names = ("router", "w_in", "w_out", "gate")
    ref_blocks = []
    for b, i in zip(blocks, ids):
        d = {n: getattr(b, n).double().requires_grad_(True) for n in names}
        ref_blocks.append(dict(d, ids=i, gate_up=matrices(b.gate_up), down=matrices(b.down)))
    x64 = x.double().requires_grad_(True)
    ref = reference(ref_blocks, x64, padding)
    ref.backward(dout.double())
    bound = 6 * (2.0 ** -4 / 4 + 2.0 ** -8)
    assert off(out, ref.detach()) < bound
    assert off(dx, x64.grad) < bound
    for got, want in zip(grads, ref_blocks):
        assert sorted(got) == sorted(names)
        for n in names:
            # a router's gradient is a difference of nearly equal weights' gradients
            assert off(got[n], want[n].grad) < (3 * bound if n == "router" else bound), n
    # tokens without experts pass the residual stream through
    assert torch.equal(out[padding], x[padding])


def test_training_lowers_the_loss(cuda_lib, example):
    T, H = 256, 256
    blocks, teacher = (example.make_blocks(2, T, H, inner=128, E=16, k=2) for _ in range(2))
    for b in teacher:
        b.gate.mul_(0.5).add_(0.5)
    x = torch.randn(T, H, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    padding = torch.zeros(T, dtype=torch.bool, device="cuda")
    target = example.forward(teacher, x, padding)[0].float()
    losses = example.train(blocks, x, target, padding, steps=12)
    assert losses[-1] < 0.5 * losses[0]
