"""The example layer's step (examples/moe_layer.py) against automatic
differentiation of the whole layer in 64 bits on the CPU, at the choice the
layer made (GPU).

Tolerance, normwise: between the input and a gradient at most five tensors are
rounded to bf16 (unit roundoff 2^-8): the router's logits or the rows of C, the
activation, the output's or D's rows, the products with the weights, the sum of
a token's rows.  Their errors are independent and at most 2^-8 each, normwise:
sqrt(5) 2^-8 = 8.7e-3, and 1.2e-2 with the logits' effect on the weights of the
choice (|d w| <= |d logit| / 2, logits of size 3).
"""
import importlib.util
import os

import pytest
import torch

from tests.parity_util import normwise, say

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TOL = 1.2e-2


def example():
    path = os.path.join(ROOT, "examples", "moe_layer.py")
    spec = importlib.util.spec_from_file_location("moe_layer_example", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def reference(layer, x, dout, weight):
    """(out, balance, dx, [router, w1, w2 gradients]) in float64."""
    H, I, E, k = layer.H, layer.I, layer.E, layer.k
    x = x.double().cpu().requires_grad_(True)
    router, w1, w2 = (w.double().cpu().requires_grad_(True) for w in (layer.router, layer.w1, layer.w2))
    ids = layer.ids.long().cpu()
    logits = x @ router.t()
    w = torch.softmax(logits.gather(1, ids), 1)
    p = torch.softmax(logits, 1)
    counts = torch.bincount(ids.flatten(), minlength=E).double()
    T = x.shape[0]
    balance = E / (k * T * T) * (counts * p.sum(0)).sum()
    out = torch.zeros(T, H, dtype=torch.float64)
    for e in range(E):
        t, j = (ids == e).nonzero(as_tuple=True)
        pair = (x[t] @ w1[e]).view(-1, I // 32, 2, 32)
        act = (pair[:, :, 0] * torch.nn.functional.silu(pair[:, :, 1])).reshape(-1, I) * w[t, j][:, None]
        out = out.index_add(0, t, act @ w2[e])
    total = (out * dout.double().cpu()).sum() + weight * balance[None].sum()
    grads = torch.autograd.grad(total, (x, router, w1, w2))
    return out.detach(), float(balance), grads[0], grads[1:]


@pytest.mark.parametrize("T,H,I,E,k", [(300, 128, 64, 6, 2), (1, 128, 64, 4, 2), (700, 256, 96 * 2, 12, 3)])
def test_step(T, H, I, E, k):
    say("moe layer", T, H, I, E, k)
    layer = example().MoELayer(H, I, E, k, seed=T)
    g = torch.Generator(device="cuda").manual_seed(7)
    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    dout = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    out, balance = layer.forward(x)
    dx = layer.backward(dout, 0.5)
    torch.cuda.synchronize()
    want, loss, want_dx, want_w = reference(layer, x, dout, 0.5)
    err = {"out": normwise(out.float().cpu(), want), "dx": normwise(dx.float().cpu(), want_dx)}
    for name, got, ref in zip(("router", "w1", "w2"), layer.grads, want_w):
        err[name] = normwise(got.float().cpu(), ref)
    say("  ", {n: f"{v:.2e}" for n, v in err.items()}, f"balance {float(balance):.5f} ref {loss:.5f}")
    assert max(err.values()) <= TOL, err
    assert abs(float(balance) - loss) <= TOL * loss
    before = [d.double() for d in layer.grads]
    norm = layer.clip(0.25)
    ref = sum(float(d.square().sum()) for d in before) ** 0.5
    assert abs(float(norm[0]) - ref) <= 1e-6 * ref
    after = sum(float(d.double().square().sum()) for d in layer.grads) ** 0.5
    assert abs(after - min(ref, 0.25)) <= 2.0 ** -8 * 0.25


def test_the_example_learns(capsys):
    example().main(steps=3, tokens=512, hidden=256, inner=128, experts=8, top_k=2)
    losses = [float(line.split("loss ")[1].split(",")[0]) for line in capsys.readouterr().out.splitlines()]
    assert len(losses) == 3 and losses[2] < losses[0]
