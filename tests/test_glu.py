"""gg_glu against the formulas in 64 bits (GPU), its agreement with gg_dglu's
gradient, and its refusals (CPU).

Tolerance, in units u = 2^-24 of the result: a sigmoid is good to 6, each of
the three products that follow adds 1 (SwiGLU: 9, with second orders 10).
GeGLU's argument alpha gc is rounded once, which moves the sigmoid by up to
|alpha gc| u of itself, and uc + offset once: 11 + |alpha gc|.  SiTU-GLU has
two tanh of 2 ulp (4 u), each of a rounded quotient (1 u: x tanh'(x) <= tanh x)
and a product (1 u): 10 + 2 * 6 = 22, taken as 24.  Below 2^-126 a sigmoid is
off by up to that much itself.  Then half a step of the output's type, and of
its subnormals."""
import pytest
import torch

from moe_grouped_gemm_offset_amd import binding as B
from tests.parity_util import say

DTYPES = [torch.bfloat16, torch.float16, torch.float32]
U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
FLOOR = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}
ACTS = [B.GG_DSWIGLU, B.GG_DGEGLU, B.GG_DSITUGLU]
P = 1 << 20


def split(c, gate_first=False):
    rows, n = c.shape[0], c.shape[1] // 2
    pair = c.double().reshape(rows, n // 32, 2, 32)
    u, g = (pair[:, :, 1], pair[:, :, 0]) if gate_first else (pair[:, :, 0], pair[:, :, 1])
    return u.reshape(rows, n), g.reshape(rows, n)


def formula(u, g, act, alpha=1.702, lo=-7.0, hi=7.0, off=1.0, b1=4.0, b2=25.0):
    """(activation, its error in u of itself, an absolute one)."""
    if act == B.GG_DSWIGLU:
        return g * torch.sigmoid(g) * u, 10.0, (g * u).abs() * 2.0 ** -126
    if act == B.GG_DGEGLU:
        gc, uc = g.clamp(max=hi), u.clamp(lo, hi)
        # (constants as the call holds them)
        alpha = float(torch.tensor(alpha, dtype=torch.float32))
        return (gc * torch.sigmoid(alpha * gc) * (uc + off), 11.0 + (alpha * gc).abs(),
                (gc * (uc + off)).abs() * 2.0 ** -126)
    t = b1 * torch.tanh(g / b1) * torch.sigmoid(g) * b2 * torch.tanh(u / b2)
    return t, 24.0, b1 * b2 * 2.0 ** -126


def check(got, c, act, prob, dtype, gate_first=False, **kw):
    u, g = split(c, gate_first)
    y, rel, floor = formula(u, g, act, **kw)
    w = 1.0 if prob is None else prob.double()[:, None]
    y, floor = y * w, floor * abs(w)
    fits = y.abs() <= torch.finfo(dtype).max * (1 - HALF[dtype])
    tol = (rel * U + HALF[dtype]) * y.abs() + floor + FLOOR[dtype]
    err = (got.double() - y).abs()
    bad = fits & ~(err <= tol)
    assert not bad.any(), (y[bad][:4], got[bad][:4])
    return float((err / tol)[fits].max()) if fits.any() else 0.0


@pytest.mark.gpu
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("c_dtype", DTYPES, ids=str)
@pytest.mark.parametrize("y_dtype", DTYPES, ids=str)
def test_glu(act, c_dtype, y_dtype):
    for i, (rows, n, pc, py, prob, first) in enumerate([
            (1, 32, 0, 0, True, False), (3, 64, 5, 3, False, True), (130, 1536, 0, 0, True, False),
            (77, 2080, 1, 7, True, True), (9, 8224, 0, 0, False, False), (1100, 32, 0, 1, True, False)]):
        g = torch.Generator().manual_seed(i + 10 * act)
        c = (3.0 * torch.randn(rows, 2 * n + pc, generator=g)).to(c_dtype)[:, :2 * n]
        c[:, ::7] *= 8                                       # past the clamps, deep into the tails
        w = torch.rand(rows, generator=g) if prob else None
        dev = torch.zeros(rows * (2 * n + pc) + 1, dtype=c_dtype, device="cuda")[1:].as_strided(c.shape, (2 * n + pc, 1))
        dev.copy_(c)
        y = torch.full((rows, n + py), 9.0, dtype=y_dtype, device="cuda")
        B.gg_glu(dev, y[:, :n], prob=None if w is None else w.cuda(), act=act,
                 flags=B.GG_FLAG_GATE_FIRST if first else 0)
        used = check(y[:, :n].cpu(), c, act, w, y_dtype, first)
        assert (y[:, n:] == 9.0).all()
        say("glu", act, c_dtype, y_dtype, rows, n, f"{used:.2f} of the tolerance")


@pytest.mark.gpu
@pytest.mark.parametrize("act", ACTS)
def test_constants_and_specials(act):
    """Other constants; NaNs and infinities give what the formula gives."""
    kw = dict(geglu_alpha=1.1, clamp_min=-2.0, clamp_max=3.0, linear_offset=0.25, situ_beta1=1.5, situ_beta2=9.0)
    g = torch.Generator().manual_seed(1)
    c = 4 * torch.randn(64, 128, generator=g)
    y = torch.zeros(64, 64, device="cuda")
    B.gg_glu(c.cuda(), y, act=act, **kw)
    check(y.cpu(), c, act, None, torch.float32, alpha=1.1, lo=-2.0, hi=3.0, off=0.25, b1=1.5, b2=9.0)
    odd = torch.tensor([float("nan"), float("inf"), -float("inf"), 0.0, -0.0, 1.0, -200.0, 3e38])
    u, v = torch.meshgrid(odd, odd, indexing="ij")
    c = torch.stack([u.reshape(2, 32), v.reshape(2, 32)], 1).reshape(1, 128).float()
    y = torch.zeros(1, 64, device="cuda")
    B.gg_glu(c.cuda(), y, act=act, **kw)
    uu, gg = split(c)
    want = formula(uu, gg, act, 1.1, -2.0, 3.0, 0.25, 1.5, 9.0)[0]
    got = y.cpu().double()
    assert torch.isnan(got[torch.isnan(uu) | torch.isnan(gg)]).all()
    # (elsewhere: a NaN of the formula is an infinity times a sigmoid that is 0)
    ok = ~torch.isnan(want) & (want.abs() < 3e38)
    assert (((got - want).abs() <= 40 * U * want.abs() + 1e-35) | ~ok).all()


@pytest.mark.gpu
@pytest.mark.parametrize("act", [B.GG_DSWIGLU, B.GG_DGEGLU])
def test_dglu_is_its_gradient(act):
    """gg_dglu's D at beta 1, with R = 1, against central differences of gg_glu's
    fp32 result: step 2^-7, truncation below 2^-14 |f'''| / 6 (at most 2 here,
    |input| <= 8: 1.6e-4) and 2 * 24 u |y| / 2^-6 (|y| <= 40: 7e-3); D in fp32."""
    n, rows = 32, 256
    g = torch.Generator().manual_seed(2)
    c = torch.randn(rows, 2 * n, generator=g).clamp(-4, 4).cuda()
    prob = (0.5 + torch.rand(rows, generator=g)).cuda()
    a = torch.zeros(rows, 64, dtype=torch.bfloat16, device="cuda")
    a[:, 0] = 1.0
    b = torch.zeros(1, n, 64, dtype=torch.bfloat16, device="cuda")
    b[:, :, 0] = 1.0                                         # R = 1 everywhere
    one = torch.ones(1, device="cuda")
    d = torch.zeros(rows, 2 * n, device="cuda")
    dprob = torch.zeros(rows, device="cuda")
    B.gg_dglu(a, b, None, B.GG_MAJOR_K, n, c, torch.tensor([rows], dtype=torch.int32, device="cuda"), one, one, prob, d,
              dprob, act=act, flags=B.GG_FLAG_GEGLU_MASK_FILTER if act == B.GG_DGEGLU else 0)

    def f(c, w):
        y = torch.zeros(rows, n, device="cuda")
        B.gg_glu(c, y, prob=w, act=act)
        return y.double()

    step = 2.0 ** -7
    for block, name in ((0, "input"), (1, "gate")):
        move = torch.zeros(1, 2 * n, device="cuda")
        move[:, 32 * block:32 * block + 32] = step
        slope = (f(c + move, prob) - f(c - move, prob)) / (2 * step)
        got = d[:, 32 * block:32 * block + 32].double()
        assert (slope - got).abs().max() <= 7.2e-3, name
    want = f(c, torch.ones_like(prob)).sum(1)
    assert (want - dprob.double()).abs().max() <= 1e-3 * want.abs().max()


@pytest.mark.gpu
@pytest.mark.parametrize("rows,end", [(0, None), (6, 0), (6, -1), (6, 4), (6, 7)])
def test_rows_behind_the_end(rows, end):
    c = torch.randn(rows, 64, generator=torch.Generator().manual_seed(0))
    y = torch.full((rows, 32), 5.0, device="cuda")
    B.gg_glu(c.cuda(), y, end=None if end is None else torch.tensor([end], dtype=torch.int32, device="cuda"))
    n = rows if end is None else max(0, min(rows, end))
    check(y[:n].cpu(), c[:n], B.GG_DSWIGLU, None, torch.float32)
    assert (y[n:] == 5.0).all()


@pytest.mark.gpu
def test_past_4_gib():
    rows, n = (1 << 26) + 5, 32
    c = torch.zeros(rows, 2 * n, dtype=torch.bfloat16, device="cuda")
    tail = torch.randn(500, 2 * n, generator=torch.Generator().manual_seed(0)).bfloat16()
    c[-500:] = tail.cuda()
    y = torch.full((rows, n), 3.0, dtype=torch.bfloat16, device="cuda")
    B.gg_glu(c, y)
    check(y[-500:].cpu(), tail, B.GG_DSWIGLU, None, torch.bfloat16)
    assert not y[:-500].any()


# --------------------------------------------------------------------------
# refusals (CPU)
# --------------------------------------------------------------------------

def c_glu(**kw):
    a = dict(c=P, cd=B.GG_BF16, ldc=128, prob=None, rows=4, n=64, y=P, yd=B.GG_BF16, ldy=64, act=0, alpha=1.7, lo=-7.0,
             hi=7.0, off=1.0, b1=4.0, b2=25.0, flags=0, end=None)
    a.update(kw)
    return B.load_library().gg_glu(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(cd=B.GG_F8E4M3), 3), (dict(yd=B.GG_MXFP4), 3), (dict(rows=-1), 2), (dict(n=40), 2), (dict(n=0), 2),
    (dict(rows=1 << 31), 8), (dict(n=1 << 21, ldc=1 << 22, ldy=1 << 21), 8), (dict(ldc=127), 4), (dict(ldy=63), 4),
    (dict(act=3), 6), (dict(act=-1), 6), (dict(flags=2), 6), (dict(act=1, alpha=float("nan")), 12),
    (dict(act=1, lo=1.0, hi=0.0), 12), (dict(act=1, hi=float("nan")), 12), (dict(act=2, b1=0.0), 12),
    (dict(act=2, b2=float("inf")), 12), (dict(c=None), 1), (dict(y=None), 1), (dict(c=P + 1), 5), (dict(y=P + 1), 5),
    (dict(prob=P + 2), 5), (dict(end=P + 1), 5)])
def test_refused(kw, status):
    assert c_glu(**kw) == status
    assert B.gg_last_error()


def test_binding_refuses():
    c, y = torch.zeros(4, 128), torch.zeros(4, 64)
    for bad in [dict(c=c.double()), dict(y=y.int()), dict(y=y[:3]), dict(y=y[:, :32]), dict(prob=torch.zeros(3)),
                dict(prob=torch.zeros(4).double()), dict(c=c.t()), {}]:
        a = dict(c=c, y=y, prob=None)
        a.update(bad)
        with pytest.raises(B.GGError):
            B.gg_glu(a["c"], a["y"], prob=a["prob"])
