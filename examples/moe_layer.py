"""One training step of a mixture-of-experts layer on the library's calls.

The layer: a linear router, top-k experts, SwiGLU experts (x W1, silu(gate) *
input times the choice's weight, then W2), the balance loss.  A step runs

  forward   gg_route   logits -> experts, weights, counts, balance loss
            gg_plan, gg_permute   tokens -> rows sorted by expert, padded to 256
            (the two forward products: torch, expert by expert)
            gg_glu       the activation between them
            gg_combine   rows -> tokens
  backward  gg_permute   the output's gradient -> rows
            gg_dglu      through W2 and the activation; the weights' gradient
            gg_wgrad     of W2 and of W1
            (the product with W1: torch, expert by expert)
            gg_combine   rows -> the input's gradient
            gg_route_bwd the logits' gradient, from the weights' and the loss's
  update    gg_grad_norm, gg_grad_clip over the three weights' gradients

Mx4Experts is the trained layer for inference, its weights in 4 bits:

  a batch   gg_plan, gg_permute   tokens -> rows sorted by expert
            gg_mx4_quant, gg_gemm_mx4, gg_glu, gg_mx4_quant, gg_gemm_mx4
            gg_combine   rows -> tokens, weighted
  a few     gg_moe_few   up to 64 tokens, in one call

Run it (on an MI355X) for a few steps of gradient descent on random data, and
the trained layer in 4 bits:
    python examples/moe_layer.py
"""
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from moe_grouped_gemm_offset_amd import binding as gg  # noqa: E402


class MoELayer:
    """Weights in bf16: router (E, H), w1 (E, H, 2I) with its columns in
    32-wide blocks, input and gate in turn, w2 (E, I, H)."""

    def __init__(self, hidden, inner, experts, top_k, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        self.H, self.I, self.E, self.k = hidden, inner, experts, top_k
        self.dev = torch.device(device)

        def weights(*shape, fan):
            return (torch.randn(*shape, generator=g, device=device) * fan ** -0.5).bfloat16()

        self.router = weights(experts, hidden, fan=hidden)
        self.w1 = weights(experts, hidden, 2 * inner, fan=hidden)
        self.w2 = weights(experts, inner, hidden, fan=inner)
        self.grads = [torch.empty_like(w) for w in (self.router, self.w1, self.w2)]
        self.table = gg.grad_table(self.grads)
        self.ones = torch.ones(experts, device=device)

    def _int(self, *shape):
        return torch.empty(*shape, dtype=torch.int32, device=self.dev)

    def _products(self, rows, weights, out):
        """out[g] = rows[g] @ weights[g] for every group's rows."""
        begin = 0
        for e, end in enumerate(self.ends_host):
            if end > begin:
                torch.mm(rows[begin:end], weights[e], out=out[begin:end])
            begin = end

    def route(self, x):
        """The choices of x's tokens (self.ids), their weights and the balance loss."""
        T, E, k = x.shape[0], self.E, self.k
        self.x = x
        self.logits = (x @ self.router.t()).float()
        self.ids, self.counts, self.routed = self._int(T, k), self._int(E), self._int(1)
        prob, balance = torch.empty(T, k, device=self.dev), torch.empty(1, device=self.dev)
        gg.gg_route(self.logits, self.ids, prob, self.counts, self.routed, balance,
                    flags=gg.GG_FLAG_NORMALIZE)
        return prob, balance

    def forward(self, x):
        T, E, k = x.shape[0], self.E, self.k
        prob, balance = self.route(x)

        m = gg.gg_plan_max_rows(T, k, E)
        self.kept, self.ends, self.row_of = self._int(E), self._int(E), self._int(T, k)
        prob_rows = torch.empty(m, device=self.dev)
        gg.gg_plan(self.ids, self.kept, self.ends, self.row_of, m, prob=prob, prob_rows=prob_rows)
        x_rows = torch.empty(m, self.H, dtype=x.dtype, device=self.dev)
        gg.gg_permute(x, self.row_of, self.kept, self.ends, x_rows)

        # the rows in use (the forward products here are cut on the host)
        self.ends_host = self.ends.tolist()
        n = self.rows = self.ends_host[-1]
        self.x_rows, self.prob_rows = x_rows[:n], prob_rows[:n]
        self.c = torch.empty(n, 2 * self.I, dtype=x.dtype, device=self.dev)
        self._products(self.x_rows, self.w1, self.c)
        self.act = torch.empty(n, self.I, dtype=x.dtype, device=self.dev)
        gg.gg_glu(self.c, self.act, prob=self.prob_rows)
        y_rows = torch.empty(n, self.H, dtype=x.dtype, device=self.dev)
        self._products(self.act, self.w2, y_rows)
        out = torch.empty_like(x)
        gg.gg_combine(y_rows, self.row_of, out)
        return out, balance

    def backward(self, dout, balance_weight):
        """The input's gradient; the weights' go to self.grads."""
        n, d_router, d_w1, d_w2 = self.rows, *self.grads
        dy_rows = torch.empty(n, self.H, dtype=dout.dtype, device=self.dev)
        gg.gg_permute(dout, self.row_of, self.kept, self.ends, dy_rows)
        d_rows = torch.empty(n, 2 * self.I, dtype=dout.dtype, device=self.dev)
        dprob = torch.zeros(n, device=self.dev)
        gg.gg_dglu(dy_rows, self.w2, None, gg.GG_MAJOR_K, self.I, self.c, self.ends, self.ones, self.ones,
                   self.prob_rows, d_rows, dprob)
        gg.gg_wgrad(self.act, gg.GG_MAJOR_M, dy_rows, gg.GG_MAJOR_N, self.ends, n, self.I, self.H,
                    wgrad_dense=d_w2)
        gg.gg_wgrad(self.x_rows, gg.GG_MAJOR_M, d_rows, gg.GG_MAJOR_N, self.ends, n, self.H, 2 * self.I,
                    wgrad_dense=d_w1)
        dx_rows = torch.empty(n, self.H, dtype=dout.dtype, device=self.dev)
        self._products(d_rows, self.w1.transpose(1, 2), dx_rows)
        dx = torch.empty_like(dout)
        gg.gg_combine(dx_rows, self.row_of, dx)

        d_logits = torch.empty_like(self.logits)
        gg.gg_route_bwd(self.logits, self.ids, self.counts, self.routed, dprob, d_logits,
                        row_of=self.row_of, dbalance=torch.full((1,), balance_weight, device=self.dev),
                        flags=gg.GG_FLAG_NORMALIZE)
        d_router.copy_(d_logits.t() @ self.x.float())
        return dx + (d_logits @ self.router.float()).to(dx.dtype)

    def clip(self, max_norm):
        """Scales self.grads to a norm of at most max_norm; (norm, factor)."""
        sumsq = torch.empty(1, dtype=torch.float64, device=self.dev)
        norm = torch.empty(2, device=self.dev)
        gg.gg_grad_norm(*self.table, sumsq)
        gg.gg_grad_clip(*self.table, sumsq, max_norm, norm)
        return norm


class Mx4Experts:
    """A layer's experts for inference, weights in MXFP4 with the reduction axis
    along the rows: w1 (E, 2I, H), w2 (E, H, I)."""

    def __init__(self, layer):
        self.H, self.I, self.E, self.dev = layer.H, layer.I, layer.E, layer.dev
        self.w1, self.sf1 = self._rows(layer.w1.transpose(1, 2).reshape(-1, self.H), (self.E, 2 * self.I, self.H))
        self.w2, self.sf2 = self._rows(layer.w2.transpose(1, 2).reshape(-1, self.I), (self.E, self.H, self.I))

    def _rows(self, x, shape=None, end=None):
        """The MXFP4 codes and scales of x's rows up to `end`."""
        n, width = x.shape
        codes = torch.empty(n, width // 2, dtype=torch.uint8, device=self.dev)
        scales = torch.empty(n, width // 32, dtype=torch.uint8, device=self.dev)
        gg.gg_mx4_quant(x, codes, scales, end=end)
        if shape is None:
            return codes, scales
        return codes.view(*shape[:2], shape[2] // 2), scales.view(*shape[:2], shape[2] // 32)

    def __call__(self, x, ids, prob):
        """The experts' weighted sum for x's tokens with these choices."""
        if x.shape[0] > 64:
            return self.batch(x, ids, prob)
        y = torch.empty_like(x)
        gg.gg_moe_few(x, ids, prob, self.w1, self.w2, y, sf1=self.sf1, sf2=self.sf2)
        return y

    def batch(self, x, ids, prob):
        """The same with activations in MXFP4 too, for any number of tokens, H and I
        multiples of 128.  The buffers hold all the rows that the choices can need;
        nothing is read back: the calls take the rows in use from the last end."""
        (T, k), E = ids.shape, self.E
        i32 = dict(dtype=torch.int32, device=self.dev)
        m = gg.gg_plan_max_rows(T, k, E, granule=1)
        counts, self.ends, self.row_of = torch.empty(E, **i32), torch.empty(E, **i32), torch.empty(T, k, **i32)
        gg.gg_plan(ids, counts, self.ends, self.row_of, m, granule=1)
        bf16 = dict(dtype=torch.bfloat16, device=self.dev)
        self.x_rows = torch.empty(m, self.H, **bf16)
        gg.gg_permute(x, self.row_of, counts, self.ends, self.x_rows)
        end = self.ends[-1:]
        self.a = self._rows(self.x_rows, end=end)
        self.c = torch.empty(m, 2 * self.I, **bf16)
        gg.gg_gemm_mx4(*self.a, self.w1, self.sf1, self.ends, self.c)
        self.act = torch.empty(m, self.I, **bf16)
        gg.gg_glu(self.c, self.act, end=end)
        self.h = self._rows(self.act, end=end)
        self.y_rows = torch.empty(m, self.H, **bf16)
        gg.gg_gemm_mx4(*self.h, self.w2, self.sf2, self.ends, self.y_rows)
        y = torch.empty_like(x)
        gg.gg_combine(self.y_rows, self.row_of, y, weights=prob)
        return y


def main(steps=5, tokens=4096, hidden=1024, inner=512, experts=16, top_k=2):
    layer = MoELayer(hidden, inner, experts, top_k)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(tokens, hidden, generator=g, device="cuda").bfloat16()
    target = torch.randn(tokens, hidden, generator=g, device="cuda").bfloat16()
    for step in range(steps):
        out, balance = layer.forward(x)
        err = out.float() - target.float()
        layer.backward((err * (2.0 / err.numel())).bfloat16(), balance_weight=0.01)
        norm = layer.clip(max_norm=0.01)
        for w, d in zip((layer.router, layer.w1, layer.w2), layer.grads):
            w.sub_(20.0 * d)
        print(f"step {step}: loss {float(err.square().mean()):.4f}, balance {float(balance):.4f}, "
              f"gradient norm {float(norm[0]):.5f}, factor {float(norm[1]):.3f}", flush=True)
    return layer, x


def in_4_bits(layer, x, few=16):
    """How far 4-bit experts take the layer's output, for a few tokens and all."""
    experts = Mx4Experts(layer)
    for n in (few, x.shape[0]):
        out, _ = layer.forward(x[:n])
        prob, _ = layer.route(x[:n])
        y = experts(x[:n], layer.ids, prob)
        off = float((y.float() - out.float()).norm() / out.float().norm())
        print(f"{n} tokens with the experts in 4 bits: {off:.3f} of the output's norm away", flush=True)


if __name__ == "__main__":
    in_4_bits(*main())
