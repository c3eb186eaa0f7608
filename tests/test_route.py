"""gg_route and gg_route_bwd against a plain implementation in 64 bits (GPU),
and their refusals (CPU).

Tolerances, from the arithmetic.  The kernels work in fp32 (unit roundoff
u = 2^-24).  A score is an exp of an argument |a| <= 40 here, scaled by log2(e)
in fp32 (relative error of the result: |a| log2(e) u + 2 u, under 64 u for the
scores that matter), divided by a sum of up to 1024 of them (added pairwise
over lanes, 16 in a row: 32 u): 128 u = 7.6e-6 relative to the row's largest
weight.  The loss is a sum of such terms: the same bound, relative.  A
gradient is a difference of products of at most four such factors: 512 u =
3.1e-5 times the largest magnitude its terms can reach; 16-bit outputs add
half an ulp (2^-8 bf16, 2^-11 fp16) of the value, fp16 also half of its
smallest subnormal, 2^-25.
"""
import math

import pytest
import torch

from moe_grouped_gemm_offset_amd import binding as B
from tests.parity_util import say

INF = float("inf")
U = 2.0 ** -24
TINY = 1e-20
HALF_ULP = {torch.float32: U, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
FLOOR = {torch.float32: 0.0, torch.bfloat16: 0.0, torch.float16: 2.0 ** -25}


# --------------------------------------------------------------------------
# the definition, in 64 bits on the CPU
# --------------------------------------------------------------------------

def ref_scores(x, softmax):
    """(scores, balance probabilities), 0 in rows without a finite logit."""
    if softmax:
        top = x.max(1, keepdim=True).values
        e = torch.exp(x - torch.where(top == -INF, torch.zeros_like(top), top))
        s = e.sum(1, keepdim=True)
        p = torch.where(s == 0, torch.zeros_like(e), e / torch.where(s == 0, torch.ones_like(s), s))
        return p, p
    a = torch.sigmoid(x)
    return a, a / (a.sum(1, keepdim=True) + TINY)


def ref_route(logits, bias, k, softmax, normalize, scale, ids=None):
    """A dict of the outputs; with ids given, differentiable in `logits`
    (float64) at that choice."""
    T, E = logits.shape
    x = logits
    if ids is None:
        key = x.float() + (0.0 if bias is None else bias)
        ids = torch.full((T, k), -1, dtype=torch.int64)
        for t in range(T):
            # NaN first, then by value; ties and equal zeros to the lower index
            order = sorted((e for e in range(E) if not (x[t, e] == -INF or key[t, e] == -INF)),
                           key=lambda e: (0, 0.0, e) if math.isnan(key[t, e]) else (1, -float(key[t, e]), e))
            for j, e in enumerate(order[:k]):
                ids[t, j] = e
    there = ids >= 0
    a, p = ref_scores(x, softmax)
    at = ids.clamp_min(0)
    if softmax and normalize:
        v = torch.where(there, x.gather(1, at), torch.full_like(x[:, :1], -INF))
        w = ref_scores(v, True)[0]
    else:
        w = torch.where(there, a.gather(1, at), torch.zeros_like(x[:, :1]))
        if normalize:
            w = w / (w.sum(1, keepdim=True) + TINY)
    counts = torch.zeros(E, dtype=torch.int64)
    counts.index_add_(0, at.flatten(), there.flatten().long())
    n = int(there[:, 0].sum()) if T else 0
    p = torch.where(there[:, :1], p, torch.zeros_like(p))      # the loss is over the tokens with a choice
    loss = E / (k * max(n, 1) ** 2) * (counts.double() * p.sum(0)).sum()
    return dict(ids=ids, prob=scale * w, counts=counts, routed=n, balance=loss)


def make_logits(T, E, dtype, seed, masked=0.0, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    x = spread * torch.randn(T, E, generator=g)
    if masked:
        x[torch.rand(T, E, generator=g) < masked] = -INF
        x[torch.rand(T, generator=g) < masked] = -INF
    return x.to(dtype)


def run_route(x, k, bias=None, score=B.GG_SOFTMAX, normalize=False, scale=1.0, balance=True, **kw):
    T, E = x.shape
    dev = x.device
    o = dict(ids=torch.full((T, k), -7, dtype=torch.int32, device=dev),
             prob=torch.full((T, k), float("nan"), device=dev),
             counts=torch.full((E,), -7, dtype=torch.int32, device=dev),
             routed=torch.full((1,), -7, dtype=torch.int32, device=dev),
             balance=torch.full((1,), float("nan"), device=dev) if balance else None)
    B.gg_route(x, o["ids"], o["prob"], o["counts"], o["routed"], o["balance"], bias=bias, score=score,
               scale=scale, flags=B.GG_FLAG_NORMALIZE if normalize else 0, **kw)
    torch.cuda.synchronize()
    return o


def check_route(x, k, bias, score, normalize, scale):
    o = run_route(x.cuda(), k, None if bias is None else bias.cuda(), score, normalize, scale)
    r = ref_route(x.double(), bias, k, score == B.GG_SOFTMAX, normalize, scale)
    assert torch.equal(o["ids"].cpu().long(), r["ids"])
    assert torch.equal(o["counts"].cpu().long(), r["counts"])
    assert int(o["routed"]) == r["routed"]
    err = (o["prob"].cpu().double() - r["prob"]).abs()
    tol = 128 * U * abs(scale) * torch.ones_like(err)
    say(f"  prob: worst {float(err.max()) if err.numel() else 0:.2e} of {128 * U * abs(scale):.2e}")
    assert bool((err <= tol).all())
    loss = float(r["balance"])
    say(f"  balance {float(o['balance']):.6f} ref {loss:.6f}")
    assert abs(float(o["balance"]) - loss) <= 128 * U * abs(loss)


SHAPES = [(1, 1, 1), (1, 8, 8), (3, 7, 2), (5, 64, 6), (33, 65, 3), (64, 61, 32), (70, 128, 8),
          (17, 129, 5), (130, 256, 8), (9, 257, 32), (40, 512, 10), (21, 513, 4), (12, 1000, 16),
          (6, 1024, 32)]


@pytest.mark.gpu
@pytest.mark.parametrize("score", [B.GG_SOFTMAX, B.GG_SIGMOID])
@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_route(dtype, normalize, score):
    for i, (T, E, k) in enumerate(SHAPES):
        say("route", T, E, k, dtype, normalize, score)
        bias = 0.3 * torch.randn(E, generator=torch.Generator().manual_seed(i)) if i % 2 else None
        check_route(make_logits(T, E, dtype, 10 + i, masked=0.3 if i % 3 else 0.0), k, bias, score,
                    normalize, 2.5 if i % 2 else 1.0)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [0, 1, 31, 32, 33, 63, 64, 65, 257, 2100])
def test_route_lengths(T):
    """Block and wave boundaries, and several blocks joined."""
    say("route lengths", T)
    check_route(make_logits(T, 96, torch.float32, T, masked=0.1), 4, None, B.GG_SIGMOID, True, 1.0)


@pytest.mark.gpu
def test_route_ties_zeros_and_masks():
    """Equal logits go by index; -0 equals +0; rows with fewer live experts
    than top_k, with none, and of the type's lowest values."""
    for dtype in (torch.bfloat16, torch.float16, torch.float32):
        low = torch.finfo(dtype).min
        E, k = 70, 5
        x = torch.zeros(8, E, dtype=dtype)
        x[0, ::2] = -0.0
        x[1] = 1.0
        x[1, 69] = 2.0
        x[2] = -INF
        x[3] = -INF
        x[3, 68], x[3, 3] = low, low
        x[4] = low
        x[5] = -INF
        x[5, 66] = 0.5
        x[6] = low
        x[6, 40:43] = torch.tensor([3.0, 3.0, -3.0])
        x[7] = torch.arange(E).flip(0).to(dtype) / 64 - 90
        for score in (B.GG_SOFTMAX, B.GG_SIGMOID):
            for normalize in (False, True):
                say("route ties", dtype, score, normalize)
                check_route(x, k, None, score, normalize, 1.0)


@pytest.mark.gpu
def test_route_bias_only_chooses():
    """A bias moves the choice, not the weights; -inf takes an expert out; the
    weights over a choice far below the row's top stay finite."""
    x = torch.tensor([[200.0, 1.0, 0.5, -1.0], [0.0, 0.0, 0.0, 0.0]])
    bias = torch.tensor([-INF, 0.0, 0.0, 5.0])
    for score in (B.GG_SOFTMAX, B.GG_SIGMOID):
        for normalize in (False, True):
            say("route bias", score, normalize)
            check_route(x, 3, bias, score, normalize, 1.0)


@pytest.mark.gpu
def test_route_bias_takes_every_choice():
    """A token whose bias leaves it no choice takes no part in the loss, though
    its logits are finite, nor has it a gradient."""
    x = torch.randn(9, 20, generator=torch.Generator().manual_seed(2))
    x[3:6, 15:] = -INF
    bias = torch.zeros(20)
    bias[:15] = -INF
    for score in (B.GG_SOFTMAX, B.GG_SIGMOID):
        say("route bias takes all", score)
        check_route(x, 4, bias, score, False, 1.0)
        o = run_route(x.cuda(), 4, bias.cuda(), score)
        assert int(o["routed"]) == 6 and bool((o["ids"][3:6] == -1).all())
        d = run_bwd(x.cuda(), o["ids"], o["counts"], o["routed"], torch.ones(9, 4).cuda(), score, False, 1.0,
                    dbalance=torch.ones(1).cuda())
        assert bool((d[3:6] == 0).all()) and bool((d[:3].abs().sum(1) > 0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_route_nan_with_its_sign_set(dtype):
    """A NaN is chosen first whatever its sign (an invalid operation gives
    either, by the machine), also beside a bias and in a row of -inf."""
    size = torch.empty(0, dtype=dtype).element_size()
    x = torch.randn(6, 61, generator=torch.Generator().manual_seed(4)).to(dtype)
    x[2:4] = -INF
    bits = {torch.bfloat16: -0x40, torch.float16: -0x200, torch.float32: -0x400000}[dtype]    # 0xFFC0, 0xFE00
    raw = x.view(torch.int16 if size == 2 else torch.int32)
    raw[1, 60] = raw[2, 7] = raw[2, 30] = raw[4, 0] = bits
    assert bool(torch.isnan(x[1, 60])) and int(raw[1, 60]) < 0
    for bias in (None, torch.randn(61, generator=torch.Generator().manual_seed(5))):
        o = run_route(x.cuda(), 4, bias=None if bias is None else bias.cuda())
        r = ref_route(x.double(), bias, 4, True, False, 1.0)
        assert torch.equal(o["ids"].cpu().long(), r["ids"])
        assert int(o["ids"][1, 0]) == 60 and o["ids"][2].tolist() == [7, 30, -1, -1]
        assert int(o["routed"]) == r["routed"] == 5
        assert torch.equal(o["counts"].cpu().long(), r["counts"])
        nan = torch.isnan(o["prob"].cpu())
        assert torch.equal(nan, torch.isnan(r["prob"]))
        assert bool(nan[1].all()) and bool(nan[2, :2].all()) and not bool(nan[[0, 3, 5]].any())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_route_bias_of_minus_infinity(dtype):
    """An expert whose bias is -inf is never chosen, whatever its logit."""
    bias = torch.zeros(61)
    bias[33] = -INF
    y = torch.randn(4, 61, generator=torch.Generator().manual_seed(6)).to(dtype)
    y[1, 33], y[2, 33], y[3, 33] = INF, float("nan"), -INF
    y[2, 5] = INF
    o = run_route(y.cuda(), 3, bias=bias.cuda())
    masked = y.clone()
    masked[:, 33] = -INF
    r = ref_route(masked.double(), None, 3, True, False, 1.0)
    assert torch.equal(o["ids"].cpu().long(), r["ids"]) and int(o["ids"][2, 0]) == 5
    assert torch.equal(o["counts"].cpu().long(), r["counts"]) and int(o["routed"]) == 4


@pytest.mark.gpu
@pytest.mark.parametrize("T", [5, 3000])
@pytest.mark.parametrize("score", [B.GG_SOFTMAX, B.GG_SIGMOID])
def test_route_loss_leaves_out_tokens_without_a_choice(score, T):
    """A token whose only logits above -inf are NaN or +inf, at an expert that a
    bias of -inf takes out, has no choice: the loss is that of the others, and
    0 where no token has one."""
    x = make_logits(T, 20, torch.float32, 91)
    bias = torch.zeros(20)
    bias[7] = -INF
    x[1:4] = -INF
    x[1, 7], x[2, 7] = float("nan"), INF
    y = x.clone()
    y[1:4] = -INF
    o = run_route(x.cuda(), 3, bias.cuda(), score)
    r = ref_route(y.double(), bias, 3, score == B.GG_SOFTMAX, False, 1.0)
    assert torch.equal(o["ids"].cpu().long(), r["ids"])
    assert int(o["routed"]) == r["routed"] == T - 3
    say("loss", float(o["balance"]), float(r["balance"]))
    assert abs(float(o["balance"]) - float(r["balance"])) <= 128 * U * float(r["balance"])
    o = run_route(x[1:4].cuda(), 3, bias.cuda(), score)
    assert int(o["routed"]) == 0 and float(o["balance"]) == 0.0


@pytest.mark.gpu
def test_route_nan_and_inf():
    """NaN and +inf logits: valid, distinct ids (NaN above +inf), NaN where
    the formulas give it, other tokens untouched."""
    x = torch.randn(4, 64, generator=torch.Generator().manual_seed(3))
    x[1, 10], x[1, 5], x[2, 7] = float("nan"), INF, INF
    o = run_route(x.cuda(), 4)
    r = ref_route(x.double(), None, 4, True, False, 1.0)
    assert torch.equal(o["ids"].cpu().long(), r["ids"])
    assert o["ids"][1, :2].tolist() == [10, 5] and int(o["ids"][2, 0]) == 7
    prob = o["prob"].cpu().double()
    assert bool(torch.isnan(prob[1]).all()) and bool(torch.isnan(o["balance"]).all())
    keep = [0, 3]
    assert float((prob[keep] - r["prob"][keep]).abs().max()) <= 128 * U
    s = run_route(x.cuda(), 4, score=B.GG_SIGMOID)
    assert math.isnan(float(s["prob"][1, 0])) and float(s["prob"][1, 1]) == 1.0


@pytest.mark.gpu
def test_route_pitch_and_no_balance():
    """Rows at a pitch and an odd start; without the loss the rest is the
    same, bit for bit."""
    for dtype in (torch.bfloat16, torch.float32):
        wide = make_logits(50, 301, dtype, 5).cuda()
        x = wide[:, 3:3 + 133]
        a = run_route(x, 6, score=B.GG_SIGMOID, normalize=True)
        b = run_route(x.contiguous(), 6, score=B.GG_SIGMOID, normalize=True, balance=False)
        for n in ("ids", "prob", "counts", "routed"):
            assert torch.equal(a[n], b[n]), n


@pytest.mark.gpu
def test_route_repeats_bit_for_bit():
    x = make_logits(5000, 160, torch.bfloat16, 8).cuda()
    a = run_route(x, 8)
    for _ in range(3):
        b = run_route(x, 8)
        for n in a:
            assert torch.equal(a[n], b[n]), n


# --------------------------------------------------------------------------
# the gradient
# --------------------------------------------------------------------------

def run_bwd(x, ids, counts, routed, dprob, score, normalize, scale, row_of=None, dbalance=None):
    d = torch.full(x.shape, float("nan"), dtype=x.dtype, device=x.device)
    B.gg_route_bwd(x, ids, counts, routed, dprob, d, row_of=row_of, dbalance=dbalance, score=score,
                   scale=scale, flags=B.GG_FLAG_NORMALIZE if normalize else 0)
    torch.cuda.synchronize()
    return d


def ref_bwd(x, ids, k, softmax, normalize, scale, g, db):
    """The formula's gradient by automatic differentiation in 64 bits."""
    live = (x > -INF)
    v = torch.where(live, x.double(), torch.zeros_like(x.double())).requires_grad_(True)
    # a masked logit takes part as -inf and has no gradient
    z = torch.where(live, v, torch.full_like(v, -INF))
    some = live.any(1)
    z = torch.where(some[:, None], z, torch.zeros_like(z))
    r = ref_route(z, None, k, softmax, normalize, scale, ids=torch.where(some[:, None], ids, -1))
    a, p = ref_scores(z, softmax)
    n = max(int((ids[:, 0] >= 0).sum()), 1)
    counts = r["counts"].double()
    loss = x.shape[1] / (k * n * n) * (counts * (p * some[:, None]).sum(0)).sum()
    total = (torch.where(ids >= 0, r["prob"] * g, torch.zeros_like(g))).sum() + db * loss
    (d,) = torch.autograd.grad(total, v)
    d = torch.where(live & some[:, None], torch.nan_to_num(d, nan=0.0), torch.zeros_like(d))
    return torch.where((ids[:, :1] >= 0), d, torch.zeros_like(d))


def check_bwd(T, E, k, dtype, score, normalize, scale, masked, seed, rows=False):
    softmax = score == B.GG_SOFTMAX
    x = make_logits(T, E, dtype, seed, masked)
    f = ref_route(x.double(), None, k, softmax, normalize, scale)
    gen = torch.Generator().manual_seed(seed + 1)
    g = torch.randn(T, k, generator=gen)
    db = 0.7
    ids = f["ids"].to(torch.int32).cuda()
    counts = f["counts"].to(torch.int32).cuda()
    routed = torch.tensor([f["routed"]], dtype=torch.int32).cuda()
    row_of, dprob = None, g
    if rows:
        m = T * k + 5
        row_of = torch.randperm(m, generator=gen)[: T * k].reshape(T, k).to(torch.int32)
        row_of[torch.rand(T, k, generator=gen) < 0.2] = -1
        dprob = torch.full((m,), 1e30)
        dprob[row_of[row_of >= 0].long()] = g[row_of >= 0]
        g = torch.where(row_of >= 0, g, torch.zeros_like(g))
        row_of = row_of.cuda()
    d = run_bwd(x.cuda(), ids, counts, routed, dprob.cuda(), score, normalize, scale, row_of,
                torch.tensor([db]).cuda())
    want = ref_bwd(x, f["ids"], k, softmax, normalize, scale, g.double(), db)
    # the largest magnitude of a term: scale |g| through weights of at most 1
    # (k of them in the mean), or the balance loss's E max(counts) / (k n^2)
    n = max(f["routed"], 1)
    size = abs(scale) * float(g.abs().max() if g.numel() else 0) * 2 + \
        db * E * float(f["counts"].max() if E else 0) / (k * n * n) * 2
    tol = 512 * U * size + (HALF_ULP[dtype] + U) * want.abs() + FLOOR[dtype]
    err = (d.cpu().double() - want).abs()
    say(f"  dlogits: worst {float((err / tol).max()) if err.numel() else 0:.3f} of the tolerance")
    assert not bool(torch.isnan(d).any())
    assert bool((err <= tol).all())
    none = f["ids"][:, 0] < 0
    assert bool((d.cpu()[none] == 0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("score", [B.GG_SOFTMAX, B.GG_SIGMOID])
@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_route_bwd(dtype, normalize, score):
    for i, (T, E, k) in enumerate(SHAPES):
        say("route_bwd", T, E, k, dtype, normalize, score)
        check_bwd(T, E, k, dtype, score, normalize, 2.5 if i % 2 else 1.0, 0.3 if i % 3 else 0.0, 40 + i,
                  rows=bool(i % 2))


@pytest.mark.gpu
@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("score", [B.GG_SOFTMAX, B.GG_SIGMOID])
def test_route_bwd_differences(score, normalize):
    """Against central differences of the 64-bit forward at the kernel's own
    choice; a difference of step h = 1e-4 is off by h^2 / 6 times the third
    derivative (under 100 here): 2e-7, besides the gradient's tolerance."""
    T, E, k, scale, db = 3, 12, 4, 1.5, 0.4
    softmax = score == B.GG_SOFTMAX
    x = make_logits(T, E, torch.float32, 77, spread=1.0)
    f = ref_route(x.double(), None, k, softmax, normalize, scale)
    g = torch.randn(T, k, generator=torch.Generator().manual_seed(78))
    d = run_bwd(x.cuda(), f["ids"].to(torch.int32).cuda(), f["counts"].to(torch.int32).cuda(),
                torch.tensor([f["routed"]], dtype=torch.int32).cuda(), g.cuda(), score, normalize, scale,
                None, torch.tensor([db]).cuda()).cpu().double()

    def total(z):
        r = ref_route(z, None, k, softmax, normalize, scale, ids=f["ids"])
        return float((r["prob"] * g.double()).sum() + db * r["balance"])

    h = 1e-4
    for t in range(T):
        for e in range(E):
            z = x.double().clone()
            z[t, e] += h
            up = total(z)
            z[t, e] -= 2 * h
            slope = (up - total(z)) / (2 * h)
            assert abs(slope - float(d[t, e])) <= 2e-7 + 512 * U * 20, (t, e)


@pytest.mark.gpu
def test_route_bwd_without_balance_and_extremes():
    """No balance gradient; logits that underflow every sigmoid; an id past the
    experts is no choice."""
    x = torch.full((2, 40), -200.0)
    x[1] = torch.linspace(-3, 3, 40)
    ids = torch.tensor([[0, 1], [39, 1000]], dtype=torch.int32)
    counts = torch.ones(40, dtype=torch.int32)
    routed = torch.tensor([2], dtype=torch.int32)
    g = torch.ones(2, 2)
    for score in (B.GG_SOFTMAX, B.GG_SIGMOID):
        for normalize in (False, True):
            d = run_bwd(x.cuda(), ids.cuda(), counts.cuda(), routed.cuda(), g.cuda(), score, normalize, 1.0)
            want = ref_bwd(x, torch.where(ids < 40, ids, -1).long(), 2, score == B.GG_SOFTMAX, normalize,
                           1.0, g.double(), 0.0)
            assert float((d.cpu().double() - want).abs().max()) <= 512 * U * 2


def ref_bwd_terms(x, ids, softmax, normalize, scale, g, db):
    """(gradient, the magnitudes of the terms it is the sum of) by the formulas,
    in 64 bits and without cancellation in a sigmoid's slope.  Rows with a
    choice, logits without NaN or +inf."""
    T, E = x.shape
    k = ids.shape[1]
    x = x.double()
    there, at = ids >= 0, ids.clamp_min(0)
    any_ = there[:, :1]
    n = max(int(there[:, 0].sum()), 1)
    counts = torch.bincount(at[there], minlength=E).double()
    G = torch.where(there, scale * g.double(), torch.zeros(1).double())
    a, p = ref_scores(x, softmax)
    c = (db * E / (k * n * n) * counts).expand(T, E)
    pc = (p * c).sum(1, keepdim=True)

    def place(v):
        return torch.zeros(T, E, dtype=torch.float64).scatter_add_(1, at, torch.where(there, v, torch.zeros_like(v)))

    if softmax:
        if normalize:
            q = ref_scores(torch.where(there, x.gather(1, at), torch.full_like(x[:, :1], -INF)), True)[0]
            d = place(q * (G - (q * G).sum(1, keepdim=True)))
            size = place(q * (G.abs() + (q * G.abs()).sum(1, keepdim=True)))
        else:
            d, size = p * (place(G) - (p * place(G)).sum(1, keepdim=True)), \
                p * (place(G.abs()) + (p * place(G.abs())).sum(1, keepdim=True))
        d, size = d + p * (c - pc), size + p * (c + pc)
    else:
        e = torch.exp(-x.abs())
        slope = e / (1 + e) ** 2
        total = a.sum(1, keepdim=True) + TINY
        d, size = (c - pc) / total, (c + pc) / total
        if normalize:
            s = torch.where(there, a.gather(1, at), torch.zeros_like(x[:, :1]))
            chosen = s.sum(1, keepdim=True) + TINY
            d = d + place((G - (s * G).sum(1, keepdim=True) / chosen) / chosen)
            size = size + place((G.abs() + (s * G.abs()).sum(1, keepdim=True) / chosen) / chosen)
        else:
            d, size = d + place(G), size + place(G.abs())
        d, size = d * slope, size * slope
    zero = torch.zeros_like(d)
    return torch.where(any_, d, zero), torch.where(any_, size, zero)


def check_bwd_terms(x, k, score, normalize, g, db, scale=1.5):
    """Every element within its own terms' error.  In fp32, with u = 2^-24: an
    exponential 4 u, and |a| u of its argument a (softmax's x - top is rounded);
    a row's sum of up to 1024 positive terms 24 u (16 in a row, 6 joins); the
    quotient 2 u; a probability 30 u; the mean of c or G over them 60 u; the
    difference and the factor in front 40 u: 130 u, and |a| u, of the terms."""
    softmax = score == B.GG_SOFTMAX
    f = ref_route(x.double(), None, k, softmax, normalize, scale)
    dev = dict(device="cuda")
    d = run_bwd(x.cuda(), f["ids"].to(torch.int32).cuda(), f["counts"].to(torch.int32).cuda(),
                torch.tensor([f["routed"]], dtype=torch.int32, **dev), g.cuda(), score, normalize, scale, None,
                torch.tensor([db], **dev))
    want, size = ref_bwd_terms(x, f["ids"], softmax, normalize, scale, g, db)
    arg = (x.double() - x.double().max(1, keepdim=True).values).abs() if softmax else torch.zeros(1).double()
    arg = torch.where(arg.isfinite(), arg, torch.zeros(1).double())
    # (fp32 holds nothing below 2^-126 to its full precision)
    tol = (130 + arg) * U * size + (HALF_ULP[x.dtype] + U) * want.abs() + FLOOR[x.dtype] + 2.0 ** -120
    err = (d.cpu().double() - want).abs()
    say(f"  dlogits: worst {float((err / tol).max()):.3f} of the terms' tolerance")
    assert bool((err <= tol).all())


@pytest.mark.gpu
@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("db", [0.0, 0.7])
def test_route_bwd_saturated_sigmoids(db, sign, normalize):
    """The slope of a sigmoid far from 0, on either side: not 1 minus what
    rounds to 1."""
    say("saturated", db, sign, normalize)
    gen = torch.Generator().manual_seed(8)
    x = sign * (8 + 17 * torch.rand(40, 61, generator=gen))
    check_bwd_terms(x, 5, B.GG_SIGMOID, normalize, torch.randn(40, 5, generator=gen), db)


@pytest.mark.gpu
@pytest.mark.parametrize("score", [B.GG_SOFTMAX, B.GG_SIGMOID])
@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("bad", [float("nan"), INF])
def test_route_bwd_of_a_masked_nan(bad, normalize, score):
    """An expert that a bias of -inf took out, with a logit of NaN or +inf.
    Without the balance loss only the chosen experts' weights have a
    gradient: the row's is that of a row where the expert is masked, 0 for the
    expert itself.  Plain softmax weights are over all experts: NaN there."""
    softmax = score == B.GG_SOFTMAX
    x = make_logits(6, 61, torch.float32, 17)
    y = x.clone()
    x[2, 33] = x[4, 9] = bad
    y[2, 33] = y[4, 9] = -INF
    f = ref_route(y.double(), None, 4, softmax, normalize, 1.0)
    g = torch.randn(6, 4, generator=torch.Generator().manual_seed(18))
    args = (f["ids"].to(torch.int32).cuda(), f["counts"].to(torch.int32).cuda(),
            torch.tensor([6], dtype=torch.int32).cuda(), g.cuda(), score, normalize, 1.0)
    d = run_bwd(x.cuda(), *args).cpu().double()
    want = ref_bwd(y, f["ids"], 4, softmax, normalize, 1.0, g.double(), 0.0)
    rows = [0, 1, 3, 5] if softmax and not normalize else list(range(6))
    assert float((d[rows] - want[rows]).abs().max()) <= 512 * U * 2 * float(g.abs().max())
    if softmax and not normalize:
        assert bool(torch.isnan(d[[2, 4]]).all())
    # the balance loss is over all experts' probabilities: its gradient's rows
    # are NaN where the formula's are, and no others
    d = run_bwd(x.cuda(), *args, dbalance=torch.ones(1).cuda()).cpu()
    assert not bool(torch.isnan(d[[0, 1, 3, 5]]).any())
    if bad != bad:
        assert bool(torch.isnan(d[[2, 4]]).all())


@pytest.mark.gpu
@pytest.mark.parametrize("score", [B.GG_SOFTMAX, B.GG_SIGMOID])
@pytest.mark.parametrize("normalize", [False, True])
def test_route_weights_to_their_own_size(normalize, score):
    """Every weight to fp32's precision of its own, far from 0 as well.  In u =
    2^-24, for logits in steps of 1/8 (x - top is exact): an exponential 4, a
    sigmoid's sum and quotient 2, the sum of six chosen ones 3 more, the last
    quotient and products 3: 18 of the weight itself."""
    softmax = score == B.GG_SOFTMAX
    gen = torch.Generator().manual_seed(55)
    x = -(25 * 8 + torch.randint(0, 20 * 8, (4000, 8), generator=gen)).float() / 8
    if softmax:
        x[:, 0] = -1.0
    r = ref_route(x.double(), None, 6, softmax, normalize, 2.0)
    o = run_route(x.cuda(), 6, None, score, normalize, 2.0)
    assert torch.equal(o["ids"].cpu().long(), r["ids"])
    err = (o["prob"].cpu().double() - r["prob"]).abs() / r["prob"]
    say(f"  weights: rms {float(err.square().mean().sqrt()) / U:.2f} u, worst {float(err.max()) / U:.2f} u")
    assert float(err.max()) <= 18 * U


@pytest.mark.gpu
@pytest.mark.parametrize("score", [B.GG_SOFTMAX, B.GG_SIGMOID])
@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("db", [0.0, 0.7])
def test_route_bwd_to_its_terms(db, normalize, score):
    """Every element of the gradient within its own terms' error, the balance
    loss's alone (dprob 0) too."""
    for i, (T, E, k) in enumerate(SHAPES):
        gen = torch.Generator().manual_seed(300 + i)
        g = torch.randn(T, k, generator=gen) * (i % 2 if db else 1)
        say("bwd terms", T, E, k, normalize, score, db)
        for dtype in (torch.float32, torch.bfloat16):
            check_bwd_terms(make_logits(T, E, dtype, 310 + i, masked=0.3 if i % 3 == 0 else 0.0, spread=4.0), k,
                            score, normalize, g, db)


# --------------------------------------------------------------------------
# many tokens: several blocks joined, several passes of a block
# --------------------------------------------------------------------------

def check_route_many(T, E, k, dtype, score, masked=0.02):
    """check_route with a choice by a stable sort (finite or -inf logits)."""
    x = make_logits(T, E, dtype, T, masked=masked)
    key = x.float().sort(dim=1, descending=True, stable=True)
    ids = torch.where(key.values[:, :k] > -INF, key.indices[:, :k], -1)
    o = run_route(x.cuda(), k, None, score, True, 2.5)
    r = ref_route(x.double(), None, k, score == B.GG_SOFTMAX, True, 2.5, ids=ids)
    assert torch.equal(o["ids"].cpu().long(), ids)
    assert torch.equal(o["counts"].cpu().long(), r["counts"])
    assert int(o["routed"]) == r["routed"]
    assert float((o["prob"].cpu().double() - r["prob"]).abs().max()) <= 128 * U * 2.5
    loss = float(r["balance"])
    say(f"  balance {float(o['balance']):.7f} ref {loss:.7f}")
    # (the tokens that a group of lanes sums in fp32: T over 768 blocks of 8)
    assert abs(float(o["balance"]) - loss) <= (128 + T / 6144) * U * loss


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1537, 3100, 4700, 6144, 6145, 7000, 13000])
def test_route_joins_every_block(T):
    """8 tokens a block at 1024 experts: 193 to 768 blocks, one to four
    quarters of the join, then a second and a third pass of the blocks."""
    say("route many", T)
    check_route_many(T, 1024, 4, torch.float32, B.GG_SOFTMAX)
    check_route_many(T, 1001, 6, torch.bfloat16, B.GG_SIGMOID)


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k", [(100_000, 64, 2), (49_500, 61, 8), (26_000, 256, 8), (13_001, 300, 4)])
def test_route_passes(T, E, k):
    """Several passes of the blocks in the other layouts."""
    say("route passes", T, E, k)
    check_route_many(T, E, k, torch.float16, B.GG_SOFTMAX)
    check_route_many(T, E, k, torch.float32, B.GG_SIGMOID)


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k", [(9000, 1024, 4), (17_001, 500, 3), (33_000, 256, 8), (33_000, 97, 2),
                                   (66_000, 61, 2)])
def test_route_bwd_passes(T, E, k):
    """More tokens than 2048 blocks take in one pass."""
    for score in (B.GG_SOFTMAX, B.GG_SIGMOID):
        say("route_bwd passes", T, E, k, score)
        for normalize, db in ((True, 0.7 * T), (False, 0.0)):
            x = make_logits(T, E, torch.float32, T)
            key = x.sort(dim=1, descending=True, stable=True)
            ids = key.indices[:, :k]
            counts = torch.bincount(ids.flatten(), minlength=E)
            g = torch.randn(T, k, generator=torch.Generator().manual_seed(T))
            d = run_bwd(x.cuda(), ids.to(torch.int32).cuda(), counts.to(torch.int32).cuda(),
                        torch.tensor([T], dtype=torch.int32).cuda(), g.cuda(), score, normalize, 1.5, None,
                        torch.tensor([db]).cuda())
            want, size = ref_bwd_terms(x, ids, score == B.GG_SOFTMAX, normalize, 1.5, g, db)
            # (the terms' error of check_bwd_terms, arguments below 30)
            tol = 160 * U * size + 2.0 ** -120
            assert bool(((d.cpu().double() - want).abs() <= tol).all())


# --------------------------------------------------------------------------
# refusals, on the host (no GPU)
# --------------------------------------------------------------------------

P, WS = 1 << 20, 1 << 24
NULL, SHAPE, DTYPE, LAYOUT, ALIGN, MODE, WORKSPACE, UNSUPPORTED, VALUE = 1, 2, 3, 4, 5, 6, 7, 8, 12


def c_route(**kw):
    a = dict(logits=P, dtype=0, ld=64, T=16, E=64, bias=None, k=4, score=0, scale=1.0, flags=0, ids=P,
             prob=P, counts=P, routed=P, balance=P, ws=WS, wsb=1 << 20)
    a.update(kw)
    return B.load_library().gg_route(a["logits"], a["dtype"], a["ld"], a["T"], a["E"], a["bias"], a["k"],
                                     a["score"], a["scale"], a["flags"], a["ids"], a["prob"], a["counts"],
                                     a["routed"], a["balance"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(logits=None), NULL), (dict(ids=None), NULL), (dict(prob=None), NULL),
    (dict(counts=None), NULL), (dict(routed=None), NULL), (dict(ws=None), NULL),
    (dict(dtype=3), DTYPE), (dict(E=0), SHAPE), (dict(E=1025, ld=2000), SHAPE), (dict(T=-1), SHAPE),
    (dict(T=(1 << 23) + 1), UNSUPPORTED), (dict(k=0), SHAPE), (dict(k=33), UNSUPPORTED),
    (dict(E=3, k=4), SHAPE), (dict(ld=63), LAYOUT), (dict(score=2), MODE), (dict(flags=4), MODE),
    (dict(scale=float("inf")), VALUE), (dict(scale=float("nan")), VALUE), (dict(logits=P + 1), ALIGN),
    (dict(ids=P + 2), ALIGN), (dict(balance=P + 1), ALIGN), (dict(ws=WS + 8), ALIGN),
    (dict(wsb=16), WORKSPACE),
])
def test_route_rejects(kw, status):
    assert c_route(**kw) == status
    assert B.gg_last_error() != ""


def c_bwd(**kw):
    a = dict(logits=P, dtype=0, ld=64, T=16, E=64, k=4, score=0, scale=1.0, flags=0, ids=P, counts=P,
             routed=P, dprob=P, row_of=None, m=0, db=None, dl=P)
    a.update(kw)
    return B.load_library().gg_route_bwd(a["logits"], a["dtype"], a["ld"], a["T"], a["E"], a["k"],
                                         a["score"], a["scale"], a["flags"], a["ids"], a["counts"],
                                         a["routed"], a["dprob"], a["row_of"], a["m"], a["db"], a["dl"],
                                         None)


@pytest.mark.parametrize("kw,status", [
    (dict(ids=None), NULL), (dict(counts=None), NULL), (dict(routed=None), NULL), (dict(dprob=None), NULL),
    (dict(dl=None), NULL), (dict(dl=P + 1), ALIGN), (dict(dprob=P + 2), ALIGN), (dict(db=P + 2), ALIGN),
    (dict(row_of=P, m=-1), SHAPE), (dict(row_of=P, m=1 << 31), SHAPE), (dict(dtype=4), DTYPE),
    (dict(flags=64 + 1), MODE), (dict(k=65), UNSUPPORTED), (dict(ld=1), LAYOUT),
])
def test_route_bwd_rejects(kw, status):
    assert c_bwd(**kw) == status


def test_binding_rejects():
    """The binding checks types, shapes and layouts before the call."""
    x = torch.zeros(4, 8)
    i32, f32 = torch.int32, torch.float32
    good = dict(ids=torch.zeros(4, 2, dtype=i32), prob=torch.zeros(4, 2), counts=torch.zeros(8, dtype=i32),
                routed=torch.zeros(1, dtype=i32))
    bad = [dict(ids=torch.zeros(4, 2, dtype=torch.int64)), dict(prob=torch.zeros(4, 3)),
           dict(counts=torch.zeros(7, dtype=i32)), dict(routed=torch.zeros(1, dtype=f32)),
           dict(prob=torch.zeros(2, 4).t()), dict(balance=torch.zeros(2)), dict(bias=torch.zeros(9))]
    for b in bad:
        with pytest.raises(B.GGError):
            B.gg_route(x, workspace=torch.zeros(1 << 16, dtype=torch.uint8), **{**good, **b})
    with pytest.raises(B.GGError):
        B.gg_route(torch.zeros(8, 4).t(), workspace=torch.zeros(1 << 16, dtype=torch.uint8), **good)
    with pytest.raises(B.GGError):
        B.gg_route(x.double(), workspace=torch.zeros(1 << 16, dtype=torch.uint8), **good)
