"""The router, dispatch/combine and clipping entry points as a program calls
them (GPU): captured into a HIP graph, on a side stream with the workspace
left to the binding, on buffers past 2^32 bytes; and together, as the backward
of a mixture-of-experts layer around the grouped GEMMs.
"""
import pytest
import torch

from moe_grouped_gemm_offset_amd import binding as B
from tests.parity_util import say

pytestmark = pytest.mark.gpu


class Step:
    """Routing, its loss, the dispatched rows, their weighted sum and both
    gradients, then the clipping of what came out: buffers allocated once."""

    def __init__(self, T=700, E=24, k=3, H=384, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape):
            return torch.randn(*shape, generator=g, device="cuda")

        self.k, self.E = k, E
        self.logits = normal(T, E)
        self.x = normal(T, H).bfloat16()
        self.dout = normal(T, H).bfloat16()
        m = self.m = B.gg_plan_max_rows(T, k, E)
        i32 = dict(dtype=torch.int32, device="cuda")
        self.ids, self.row_of = torch.zeros(T, k, **i32), torch.zeros(T, k, **i32)
        self.counts, self.rows_e, self.ends = (torch.zeros(E, **i32) for _ in range(3))
        self.routed = torch.zeros(1, **i32)
        f = dict(device="cuda")
        self.prob, self.dprob = torch.zeros(T, k, **f), torch.zeros(T, k, **f)
        self.prob_rows, self.balance = torch.zeros(m, **f), torch.zeros(1, **f)
        self.dbalance = torch.full((1,), 0.1, **f)
        self.x_rows = torch.zeros(m, H, dtype=torch.bfloat16, **f)
        self.dy_rows = torch.zeros_like(self.x_rows)
        self.out, self.dx = torch.zeros_like(self.x), torch.zeros_like(self.x)
        self.dlogits = torch.zeros(T, E, **f)
        self.clipped = [torch.zeros_like(self.dlogits), torch.zeros_like(self.dx)]
        self.table = B.grad_table([self.dlogits, self.dx])
        self.out_ptrs = B.grad_table(self.clipped)[0]
        self.sumsq = torch.zeros(1, dtype=torch.float64, **f)
        self.norm = torch.zeros(2, **f)

    def call(self, stream=None, ws=(None, None, None)):
        kw = dict(stream=stream)
        w = [B.gg_route(self.logits, self.ids, self.prob, self.counts, self.routed, self.balance,
                        score=B.GG_SIGMOID, flags=B.GG_FLAG_NORMALIZE, workspace=ws[0], **kw)]
        w.append(B.gg_plan(self.ids, self.rows_e, self.ends, self.row_of, self.m, prob=self.prob,
                           prob_rows=self.prob_rows, workspace=ws[1], **kw))
        B.gg_permute(self.x, self.row_of, self.rows_e, self.ends, self.x_rows, **kw)
        B.gg_combine(self.x_rows, self.row_of, self.out, weights=self.prob, **kw)
        B.gg_combine_bwd(self.dout, self.x_rows, self.row_of, self.prob, self.rows_e, self.ends,
                         self.dy_rows, self.dprob, **kw)
        B.gg_combine(self.dy_rows, self.row_of, self.dx, **kw)
        B.gg_route_bwd(self.logits, self.ids, self.counts, self.routed, self.dprob, self.dlogits,
                       dbalance=self.dbalance, score=B.GG_SIGMOID, flags=B.GG_FLAG_NORMALIZE, **kw)
        w.append(B.gg_grad_norm(*self.table, self.sumsq, workspace=ws[2], **kw))
        B.gg_grad_clip(*self.table, self.sumsq, 0.5, self.norm, out_ptrs=self.out_ptrs, **kw)
        return w

    def results(self):
        end = int(self.ends[-1])
        return [t.clone() for t in (self.ids, self.prob, self.counts, self.routed, self.balance,
                                    self.ends, self.row_of, self.prob_rows[:end], self.x_rows[:end],
                                    self.out, self.dy_rows[:end], self.dprob, self.dx, self.dlogits,
                                    self.norm, *self.clipped)]

    def spoil(self):
        for t in (self.ids, self.counts, self.rows_e, self.ends, self.row_of, self.routed):
            t.fill_(-3)
        for t in (self.prob, self.balance, self.prob_rows, self.x_rows, self.out, self.dy_rows, self.dprob,
                  self.dx, self.dlogits, self.norm, self.sumsq, *self.clipped):
            t.fill_(float("nan"))


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("T", [40, 700, 5000])
def test_graph_replays(T):
    """Captured once, replayed with eager work in between: every replay equals
    the eager call bit for bit, with spoilt outputs and workspaces."""
    s = Step(T=T)
    ws = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in (
        B.gg_route_workspace_size(T, s.E), B.gg_plan_workspace_size(T, s.E), B.gg_grad_workspace_size())]
    s.call(ws=ws)
    torch.cuda.synchronize()
    want = s.results()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.call(ws=ws)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.call(ws=ws)
    for r in range(3):
        s.spoil()
        for w in ws:
            w.fill_(170 + r)
        (torch.randn(1 << 18, device="cuda") * 2.0).sum().item()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        say("replay", T, r)
        assert same(s.results(), want), f"replay {r} differs from the eager call"


def test_side_stream():
    """Queued on a side stream, workspaces left to the binding and dropped at
    once: a block of theirs is not handed to the current stream, and the
    results equal the current stream's."""
    s = Step(T=3000)
    s.call()
    torch.cuda.synchronize()
    want = s.results()
    s.spoil()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ws = s.call(stream=side)
    taken = [(w.data_ptr(), w.numel()) for w in ws]
    del ws
    for ptr, n in taken:
        assert torch.empty(n, dtype=torch.uint8, device="cuda").data_ptr() != ptr
    side.synchronize()
    assert same(s.results(), want)


def test_workspaces_hold_nothing_between_calls():
    """A workspace used by another size, another operator, or filled with
    anything gives the same results."""
    big, small = Step(T=6000, E=200, seed=1), Step(T=90, E=7, seed=2)
    want = []
    for s in (big, small):
        s.call()
        torch.cuda.synchronize()
        want.append(s.results())
    ws = torch.full((1 << 22,), 213, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        for s, w in ((small, want[1]), (big, want[0])):
            s.spoil()
            s.call(ws=(ws, ws, ws))
            torch.cuda.synchronize()
            assert same(s.results(), w)


@pytest.mark.parametrize("T", [3, 3000])
def test_error_word_is_each_calls_own(T):
    """gg_device_error after a call reads that call's word: 0 after the router
    and the norm, which set none, on a workspace never written before, and on
    one where gg_plan has left its flags."""
    s = Step(T=T)
    bad = s.ids.clone().fill_(9999)
    for fill in (255, None):
        ws = torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda")
        for call in (
                lambda: B.gg_route(s.logits, s.ids, s.prob, s.counts, s.routed, s.balance, workspace=ws),
                lambda: B.gg_grad_norm(*s.table, s.sumsq, workspace=ws),
                lambda: B.gg_grad_norm(*B.grad_table([s.norm]), s.sumsq, workspace=ws),
                lambda: B.gg_grad_norm(*B.grad_table([]), s.sumsq, workspace=ws)):
            if fill is None:
                B.gg_plan(bad, s.rows_e, s.ends, s.row_of, s.m, workspace=ws)
                assert B.gg_device_error(ws) == B.GG_DEVERR_IDS
            else:
                ws.fill_(fill)
            call()
            assert B.gg_device_error(ws) == 0


def test_the_most_tokens():
    """2^23 tokens: the largest grids and the largest indices of a token."""
    T, E, H = 1 << 23, 8, 3
    g = torch.Generator(device="cuda").manual_seed(3)
    logits = torch.randn(T, E, generator=g, device="cuda").bfloat16()
    i32 = dict(dtype=torch.int32, device="cuda")
    ids, row_of = torch.empty(T, 1, **i32), torch.empty(T, 1, **i32)
    counts, kept, ends, routed = (torch.empty(n, **i32) for n in (E, E, E, 1))
    prob, balance = torch.empty(T, 1, device="cuda"), torch.empty(1, device="cuda")
    say("most tokens: route")
    B.gg_route(logits, ids, prob, counts, routed, balance)
    torch.cuda.synchronize()
    p = torch.softmax(logits.double(), 1)
    first = logits.float().sort(dim=1, descending=True, stable=True).indices[:, :1]
    assert torch.equal(ids.long(), first)
    want = torch.bincount(first.flatten(), minlength=E)
    assert torch.equal(counts.long(), want) and int(routed) == T
    assert bool(((prob.double() - p.gather(1, first)).abs() <= 128 * 2.0 ** -24).all())
    # (a group of lanes sums T / (768 * 64) = 171 tokens in fp32)
    loss = float(E * (want / T * (p.sum(0) / T)).sum())
    assert abs(float(balance) - loss) <= (128 + 171) * 2.0 ** -24 * loss
    say("most tokens: plan")
    m = B.gg_plan_max_rows(T, 1, E)
    B.gg_plan(ids, kept, ends, row_of, m)
    torch.cuda.synchronize()
    assert torch.equal(kept, counts)
    flat = ids.flatten().long()
    begin = ends.long() - (want + 255) // 256 * 256
    order = flat.argsort(stable=True)
    rows = torch.empty_like(flat)
    rows[order] = begin[flat[order]] + torch.arange(T, device="cuda") - (want.cumsum(0) - want)[flat[order]]
    assert torch.equal(row_of.flatten().long(), rows)
    say("most tokens: rows")
    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    x_rows = torch.full((m, H), 7.0, dtype=torch.bfloat16, device="cuda")
    B.gg_permute(x, row_of, kept, ends, x_rows)
    out, dw = torch.empty_like(x), torch.empty(T, 1, device="cuda")
    dy = torch.full((m, H), 7.0, dtype=torch.bfloat16, device="cuda")
    B.gg_combine(x_rows, row_of, out)
    B.gg_combine_bwd(x, x_rows, row_of, torch.ones_like(prob), kept, ends, dy, dw)
    torch.cuda.synchronize()
    assert torch.equal(x_rows[rows], x) and torch.equal(out, x)
    assert torch.equal(dy, x_rows) and bool((x_rows[int(ends[-1]):] == 7.0).all())
    norm = x.double().square().sum(1, keepdim=True)
    assert bool(((dw.double() - norm).abs() <= 32 * 2.0 ** -24 * norm).all())
    say("most tokens: route_bwd")
    d = torch.empty_like(logits)
    B.gg_route_bwd(logits, ids, counts, routed, prob, d)
    torch.cuda.synchronize()
    w = p.gather(1, first) * prob.double()
    want = torch.zeros_like(p).scatter_(1, first, w) - p * w
    size = torch.zeros_like(p).scatter_(1, first, w) + p * w
    assert bool(((d.double() - want).abs() <= 160 * 2.0 ** -24 * size + 2.0 ** -8 * 1.01 * want.abs()).all())


def test_logits_past_32_bits():
    """Rows of logits at a pitch that takes the last ones past 2^32 bytes and
    2^31 elements: the same bits as of the rows put together."""
    T, E, k = 300_000, 40, 3
    wide = torch.empty(T, 8192, dtype=torch.bfloat16, device="cuda")
    x = wide[:, 17:17 + E]
    x.copy_(torch.randn(T, E, generator=torch.Generator(device="cuda").manual_seed(4), device="cuda"))
    i32 = dict(dtype=torch.int32, device="cuda")
    got = []
    for logits in (x, x.contiguous()):
        o = [torch.full((T, k), -7, **i32), torch.zeros(T, k, device="cuda"), torch.zeros(E, **i32),
             torch.zeros(1, **i32), torch.zeros(1, device="cuda"), torch.zeros(T, E, dtype=x.dtype, device="cuda")]
        say("logits past 32 bits", logits.stride())
        B.gg_route(logits, *o[:5])
        B.gg_route_bwd(logits, o[0], o[2], o[3], o[1], o[5], dbalance=torch.ones(1, device="cuda"))
        torch.cuda.synchronize()
        got.append(o)
    assert same(*got) and int(got[0][3]) == T
    top = x[-1].float().sort(descending=True, stable=True).indices[:k]
    assert torch.equal(got[0][0][-1].long(), top)


def test_rows_past_32_bits():
    """Expert rows past 2^32 bytes from the first, and past 2^31 elements."""
    H, T, k = 8192, 6, 2
    m = 280_000                                        # 280000 * 8192 elements of bf16: 4.6 GB
    rows = torch.empty(m, H, dtype=torch.bfloat16, device="cuda")
    dy = torch.empty(m, H, dtype=torch.bfloat16, device="cuda")
    x = torch.randn(T, H, device="cuda").bfloat16()
    row_of = torch.tensor([[m - 1, 0], [m - 2, 1], [m - 3, 2], [270_000, 3], [262_144, 4], [262_143, 5]],
                          dtype=torch.int32, device="cuda")
    counts = torch.tensor([6, m - 6 - 256], dtype=torch.int32, device="cuda")
    ends = torch.tensor([6, m], dtype=torch.int32, device="cuda")      # 256 rows of padding at the end
    pad = torch.arange(m - 256, m, device="cuda")
    B.gg_permute(x, row_of, counts, ends, rows)
    w = torch.rand(T, k, device="cuda")
    out = torch.zeros_like(x)
    torch.cuda.synchronize()
    say("rows past 32 bits: permute")
    # (rows m-1, m-2, m-3 are padding too, by these counts: either value may stand there)
    assert torch.equal(rows[row_of[3:].flatten().long()].view(3, k, H), x[3:, None].expand(3, k, H))
    hidden = [int(r) for r in pad.tolist() if r < m - 3]
    assert bool((rows[hidden] == 0).all())
    rows[row_of.flatten().long()] = x.repeat_interleave(k, 0)
    B.gg_combine(rows, row_of, out, weights=w)
    dw = torch.zeros(T, k, device="cuda")
    B.gg_combine_bwd(x, rows, row_of, w, torch.tensor([6, m - 6], dtype=torch.int32, device="cuda"), ends, dy,
                     dw)
    torch.cuda.synchronize()
    say("rows past 32 bits: combine")
    want = x.double() * w.double().sum(1, keepdim=True)
    assert bool(((out.double() - want).abs() <= 2 ** -8 * 1.01 * want.abs()).all())
    want = w.double()[:, :, None] * x.double()[:, None]
    got = dy[row_of.flatten().long()].double().view(T, k, H)
    assert bool(((got - want).abs() <= 2 ** -8 * 1.01 * want.abs()).all())
    norm = x.double().square().sum(1, keepdim=True).expand(T, k)
    assert bool(((dw.double() - norm).abs() <= 64 * 2.0 ** -24 * norm).all())


def test_clip_past_32_bits():
    """Tensors of more than 2^32 bytes together and one of 2^31 elements and
    more: the ends of both are reached."""
    n = (1 << 31) + 4096 + 3
    big = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    tail = torch.zeros(1000, dtype=torch.float32, device="cuda")
    big[0], big[-1], big[1 << 31], tail[-1] = 3.0, 4.0, 12.0, 84.0
    ptrs, ends, dtypes, total = B.grad_table([big, tail])
    sumsq, norm = torch.zeros(1, dtype=torch.float64, device="cuda"), torch.zeros(2, device="cuda")
    B.gg_grad_norm(ptrs, ends, dtypes, total, sumsq)
    B.gg_grad_clip(ptrs, ends, dtypes, total, sumsq, 42.5, norm, eps=0.0)
    torch.cuda.synchronize()
    assert float(sumsq) == 85.0 ** 2 and norm.tolist() == [85.0, 0.5]
    assert [float(v) for v in (big[0], big[-1], big[1 << 31], tail[-1])] == [1.5, 2.0, 6.0, 42.0]
