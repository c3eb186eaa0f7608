"""The 4-bit calls as a program runs them together (GPU): the example layer's
experts (examples/moe_layer.py) for a batch and for a few tokens, stage by stage
against 64 bits; captured into HIP graphs, two at a time; on a side stream.

Each stage is checked on what the stage before it gave, so a code that a rounding
moved does not count against the next.  Quantised rows are exact.  A product
of k values (exact in fp32 but for its sum, (k + 2) 2^-24 of the sum of the
magnitudes) and an activation (10 2^-24 of itself) are rounded to bf16, half a
step: 2^-8; so is a token's sum of rows, after (k + 1) 2^-24 of its terms.  A
layer's call for a few tokens: tests/test_moe_few.py."""
import pytest
import torch

from moe_grouped_gemm_offset_amd import binding as B
from tests import mx4_util as mx
from tests import test_moe_few as few
from tests.parity_util import say
from tests.test_moe_layer import example

pytestmark = pytest.mark.gpu

U, HALF = 2.0 ** -24, 2.0 ** -8


def layer_and_experts(H=256, I=96, E=6, k=2, seed=3):
    mod = example()
    layer = mod.MoELayer(H, I, E, k, seed=seed)
    return layer, mod.Mx4Experts(layer)


def tokens(T, H, seed=0):
    return torch.randn(T, H, generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()


def near(got, want, tol):
    got, tol = got.double().cpu(), tol + HALF * (want.abs() + tol)
    assert ((got - want).abs() <= tol).all(), float(((got - want).abs() / tol).max())


def product(a, b, ends):
    """(result, tolerance before rounding) of quantised rows times the experts'."""
    a = mx.values(*(t.cpu() for t in a))
    n = int(ends[-1])
    d, mag, at = torch.zeros(n, b[0].shape[1], dtype=torch.float64), torch.zeros(n, b[0].shape[1], dtype=torch.float64), 0
    for e, end in enumerate(ends.tolist()):
        w = mx.values(b[0][e].cpu(), b[1][e].cpu())
        d[at:end], mag[at:end] = a[at:end] @ w.T, a[at:end].abs() @ w.abs().T
        at = end
    return d, (a.shape[1] + 2) * U * mag


@pytest.mark.parametrize("T,H,I", [(1, 128, 128), (65, 256, 128), (300, 384, 256), (1500, 256, 256)])
def test_batch(T, H, I):
    layer, experts = layer_and_experts(H, I)
    x = tokens(T, H)
    prob, _ = layer.route(x)
    ids = layer.ids.clone()
    ids[::5, 0] = -1                                         # dropped choices, and tokens without any
    ids[::10] = -1
    y = experts.batch(x, ids, prob)
    ends, n = experts.ends.cpu(), int(experts.ends[-1])
    say("batch", T, H, I, "rows", n)
    for codes, rows in ((experts.a, experts.x_rows), (experts.h, experts.act)):
        want_c, want_s = mx.quantise(rows[:n].cpu())
        assert torch.equal(codes[0][:n].cpu(), want_c) and torch.equal(codes[1][:n].cpu(), want_s)
    near(experts.c[:n], *product([t[:n] for t in experts.a], (experts.w1, experts.sf1), ends))
    c = experts.c[:n].double().cpu().reshape(n, I // 32, 2, 32)
    act = (c[:, :, 1] * torch.sigmoid(c[:, :, 1]) * c[:, :, 0]).reshape(n, I)
    near(experts.act[:n], act, 10 * U * act.abs() + 2.0 ** -126 * 1e3)
    near(experts.y_rows[:n], *product([t[:n] for t in experts.h], (experts.w2, experts.sf2), ends))
    row = experts.row_of.cpu().long()
    term = experts.y_rows.double().cpu()[row.clamp_min(0)] * (prob.cpu().double() * (row >= 0))[:, :, None]
    term = torch.where((row >= 0)[:, :, None], term, 0.0)
    near(y, term.sum(1), 3 * U * term.abs().sum(1))
    assert not y[::10].any()


@pytest.mark.parametrize("T", [1, 3, 64])
def test_few(T):
    layer, experts = layer_and_experts()
    x = tokens(T, 256)
    prob, _ = layer.route(x)
    y = experts(x, layer.ids, prob)
    s = dict(T=T, E=6, k=2, H=256, I=96, mx4=True, x=x.cpu(), ids=layer.ids.cpu(), prob=prob.cpu(), bias1=None, bias2=None,
             **{n: getattr(experts, n).cpu() for n in ("w1", "sf1", "w2", "sf2")})
    few.check(s, y.cpu(), torch.bfloat16)


class Calls:
    """Every call of this group on buffers allocated once."""

    def __init__(self, T, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.H, self.I, self.E, self.k = H, I, E, k = 256, 128, 5, 2

        def normal(*s):
            return torch.randn(*s, generator=g, device="cuda")

        def quantised(*shape):
            c = torch.zeros(shape[0] * shape[1], shape[2] // 2, dtype=torch.uint8, device="cuda")
            s = torch.zeros(shape[0] * shape[1], shape[2] // 32, dtype=torch.uint8, device="cuda")
            B.gg_mx4_quant(normal(shape[0] * shape[1], shape[2]) * shape[2] ** -0.5, c, s)
            return c.view(*shape[:2], -1), s.view(*shape[:2], -1)

        self.w1, self.sf1 = quantised(E, 2 * I, H)
        self.w2, self.sf2 = quantised(E, H, I)
        self.x = normal(T, H).bfloat16()
        self.ids = torch.rand(T, E, generator=g, device="cuda").topk(k, 1).indices.int()
        self.prob = torch.softmax(normal(T, k), 1)
        sizes = torch.tensor([T // 3, 0, T // 2, T - T // 3 - T // 2, 0]).cumsum(0).int().cuda()
        self.ends = sizes
        u8 = dict(dtype=torch.uint8, device="cuda")
        self.out = dict(a=torch.zeros(T, H // 2, **u8), sa=torch.zeros(T, H // 32, **u8), c=torch.zeros(T, 2 * I, device="cuda"),
                        h=torch.zeros(T, I, device="cuda").half(), back=torch.zeros(T, H, device="cuda"),
                        y=torch.zeros(min(T, 64), H, device="cuda"))
        self.ws = [torch.full((n,), 255, **u8) for n in (B.gg_gemm_mx4_workspace_size(),
                                                         B.gg_moe_few_workspace_size(min(T, 64), k, H, I))]

    def call(self, stream=None, own=True):
        o, ws, n = self.out, self.ws if own else (None, None), min(self.x.shape[0], 64)
        B.gg_mx4_quant(self.x, o["a"], o["sa"], stream=stream)
        B.gg_gemm_mx4(o["a"], o["sa"], self.w1, self.sf1, self.ends, o["c"], workspace=ws[0], stream=stream)
        B.gg_glu(o["c"], o["h"], act=B.GG_DSITUGLU, stream=stream)
        B.gg_mx4_dequant(o["a"], o["sa"], o["back"], stream=stream)
        B.gg_moe_few(self.x[:n], self.ids[:n], self.prob[:n], self.w1, self.w2, o["y"], sf1=self.sf1, sf2=self.sf2,
                     workspace=ws[1], stream=stream)

    def results(self):
        return [t.clone() for t in self.out.values()]

    def spoil(self, r):
        for t in self.out.values():
            t.fill_(91 if t.dtype == torch.uint8 else float("nan"))
        for w in self.ws:
            w.fill_(170 + r)


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("T", [2, 7, 50, 2000])
def test_graph_replays(T):
    """Two graphs of their own buffers, captured once and replayed in turn with
    eager work in between: every replay equals the eager call bit for bit."""
    both = [Calls(T, 1), Calls(T, 2)]
    want, graphs = [], []
    for c in both:
        c.call()
        torch.cuda.synchronize()
        want.append(c.results())
    for c in both:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.call()
        graphs.append(g)
    for r in range(3):
        for c in both:
            c.spoil(r)
        (torch.randn(1 << 18, device="cuda") * 2.0).sum().item()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        say("replay", T, r)
        for c, w in zip(both, want):
            assert same(c.results(), w), f"replay {r} differs from the eager call"


def test_side_stream():
    """On a side stream, workspaces left to the binding and dropped at once."""
    c = Calls(1000, 4)
    c.call()
    torch.cuda.synchronize()
    want = c.results()
    c.spoil(0)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    c.call(stream=side, own=False)
    junk = [torch.full((1 << 16,), 77, dtype=torch.uint8, device="cuda") for _ in range(20)]
    side.synchronize()
    assert same(c.results(), want) and len(junk) == 20


def test_two_streams_at_once():
    """Two calls at a time, each with its own workspace."""
    c = [Calls(1500, 5), Calls(1500, 6)]
    want = []
    for x in c:
        x.call()
        torch.cuda.synchronize()
        want.append(x.results())
        x.spoil(0)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(4):
        for x, s in zip(c, streams):
            x.call(stream=s)
    torch.cuda.synchronize()
    assert all(same(x.results(), w) for x, w in zip(c, want))


def test_the_example_runs(capsys):
    layer, _ = layer_and_experts(I=128)
    example().in_4_bits(layer, tokens(200, 256))
    out = capsys.readouterr().out.splitlines()
    assert [line.split()[0] for line in out] == ["16", "200"]
