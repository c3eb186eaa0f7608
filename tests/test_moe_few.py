"""gg_moe_few against the layer in 64 bits (GPU), and its refusals (CPU).

Tolerance, element by element, u = 2^-24.  A sum of n products that are exact in
fp32 (bf16 by bf16) is off by at most n u of the sum of their magnitudes; the
waves' eight parts and a bias add 9 roundings, so a pre-activation c is off by
dc = (H + 9) u (sum |w1 x| + |bias1|).  The activation passes that on by its
slopes (taken by central differences of the 64-bit formula) and adds 24 u of
itself (the largest of the three, tests/test_glu.py; 11 + |alpha gc| u <= 24 u
at the clamp of 7 and alpha 1.702), the product with prob u; the two bf16 parts
of h leave 2^-16 of it at most (a bf16 rounding is 2^-8 of the value, of what is
left 2^-8 again), and 2^-133 where the second is subnormal.  So h is off by
dh = |prob| (|act_g| dc_g + |act_u| dc_u) + (2^-16 + 26 u) |h| + 2^-133, and y by
sum |w2| dh + (2 I + 10 + k) u (sum |w2 h| + sum |prob bias2|), then half a step
of its type (and of fp16's subnormals)."""
import pytest
import torch

from moe_grouped_gemm_offset_amd import binding as B
from tests import mx4_util as mx
from tests.parity_util import say

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
FLOOR = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}
P = 1 << 20


def act64(u, g, act):
    if act == B.GG_DSWIGLU:
        return g * torch.sigmoid(g) * u
    if act == B.GG_DGEGLU:
        gc = g.clamp(max=7.0)
        return gc * torch.sigmoid(1.702 * gc) * (u.clamp(-7.0, 7.0) + 1.0)
    return 4.0 * torch.tanh(g / 4.0) * torch.sigmoid(g) * 25.0 * torch.tanh(u / 25.0)


def case(T, E, k, H, I, mx4, bias=False, seed=0, masked=0.0):
    g = torch.Generator().manual_seed(seed)
    s = dict(T=T, E=E, k=k, H=H, I=I, mx4=mx4)
    s["x"] = torch.randn(T, H, generator=g).bfloat16()
    s["ids"] = torch.rand(T, max(E, k), generator=g).argsort(1)[:, :k].to(torch.int32) % E
    s["ids"][torch.rand(T, k, generator=g) < masked] = -1
    s["prob"] = torch.rand(T, k, generator=g)
    if mx4:
        for w, sf, shape, fan in (("w1", "sf1", (E, 2 * I, H), H), ("w2", "sf2", (E, H, I), I)):
            c, q = mx.quantise(torch.randn(shape[0] * shape[1], shape[2], generator=g) * fan ** -0.5)
            s[w], s[sf] = c.reshape(*shape[:2], -1), q.reshape(*shape[:2], -1)
    else:
        s["w1"] = (torch.randn(E, 2 * I, H, generator=g) * H ** -0.5).bfloat16()
        s["w2"] = (torch.randn(E, H, I, generator=g) * I ** -0.5).bfloat16()
        s["sf1"] = s["sf2"] = None
    s["bias1"] = 0.3 * torch.randn(E, 2 * I, generator=g) if bias else None
    s["bias2"] = 0.3 * torch.randn(E, H, generator=g) if bias else None
    return s


def weights(s, w, sf, e):
    return mx.values(s[w][e], s[sf][e]) if s["mx4"] else s[w][e].double()


def want(s, act, gate_first=False):
    """(y, its tolerance before the rounding to its type) in float64."""
    T, H, I = s["T"], s["H"], s["I"]
    y, tol = torch.zeros(T, H, dtype=torch.float64), torch.zeros(T, H, dtype=torch.float64)
    mag = torch.zeros(T, H, dtype=torch.float64)
    for e in sorted({int(i) for i in s["ids"].flatten() if 0 <= int(i) < s["E"]}):
        t, j = (s["ids"] == e).nonzero(as_tuple=True)
        x, pr = s["x"][t].double(), s["prob"][t, j].double()[:, None]
        w1, w2 = weights(s, "w1", "sf1", e), weights(s, "w2", "sf2", e)
        b1 = torch.zeros(2 * I, dtype=torch.float64) if s["bias1"] is None else s["bias1"][e].double()
        b2 = torch.zeros(H, dtype=torch.float64) if s["bias2"] is None else s["bias2"][e].double()
        c = (x @ w1.T + b1).reshape(-1, I // 32, 2, 32)
        dc = ((H + 9) * U * (x.abs() @ w1.abs().T + b1.abs())).reshape(-1, I // 32, 2, 32)
        a, b = (1, 0) if gate_first else (0, 1)
        u, g = c[:, :, a].reshape(-1, I), c[:, :, b].reshape(-1, I)
        du, dg = dc[:, :, a].reshape(-1, I), dc[:, :, b].reshape(-1, I)
        v, st = act64(u, g, act), 2.0 ** -20
        sg = (act64(u, g + st, act) - act64(u, g - st, act)).abs() / (2 * st)
        su = (act64(u + st, g, act) - act64(u - st, g, act)).abs() / (2 * st)
        h = pr * v
        dh = pr.abs() * (sg * dg + su * du) + (2.0 ** -16 + 26 * U) * h.abs() + 2.0 ** -133
        y.index_add_(0, t, h @ w2.T + pr * b2)
        tol.index_add_(0, t, dh @ w2.abs().T)
        mag.index_add_(0, t, h.abs() @ w2.abs().T + (pr * b2).abs())
    return y, tol + (2 * I + 10 + s["k"]) * U * mag


def run(s, dtype=torch.float32, act=B.GG_DSWIGLU, gate_first=False, px=0, py=0, fill=55.0, workspace=None):
    T, H = s["T"], s["H"]
    x = torch.zeros(T, H + px, dtype=torch.bfloat16, device="cuda")[:, :H]
    x.copy_(s["x"])
    y = torch.full((T, H + py), fill, dtype=dtype, device="cuda")
    dev = {n: None if s[n] is None else s[n].cuda() for n in ("sf1", "sf2", "bias1", "bias2")}
    B.gg_moe_few(x, s["ids"].cuda(), s["prob"].cuda(), s["w1"].cuda(), s["w2"].cuda(), y[:, :H], act=act,
                 flags=B.GG_FLAG_GATE_FIRST if gate_first else 0, workspace=workspace, **dev)
    assert (y[:, H:] == fill).all()
    return y[:, :H].cpu()


def check(s, got, dtype, act=B.GG_DSWIGLU, gate_first=False):
    y, tol = want(s, act, gate_first)
    tol = tol + HALF[dtype] * (y.abs() + tol) + FLOOR[dtype]
    err = (got.double() - y).abs()
    assert (err <= tol).all(), (float((err / tol).max()), y[err > tol][:4], got[err > tol][:4])
    return float((err / tol).max()) if y.numel() else 0.0


# widths of less than a wave's chunk, of whole ones and of parts; one token to
# 64; columns of one block of 16 to several passes
SHAPES = [(1, 1, 1, 32, 32), (1, 64, 8, 256, 128), (2, 8, 2, 2048, 96), (3, 5, 3, 544, 288), (16, 4, 2, 96, 64),
          (17, 3, 2, 320, 160), (33, 2, 1, 64, 544), (64, 1, 1, 288, 96), (64, 40, 6, 512, 64), (64, 2, 2, 160, 320),
          (9, 1024, 32, 64, 32), (64, 1024, 32, 32, 32), (5, 3, 7, 128, 64), (64, 16, 8, 2112, 1120),
          (40, 64, 2, 512, 256), (13, 20, 3, 1056, 2080), (6, 4, 9, 2048, 544)]
DTYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.mark.gpu
@pytest.mark.parametrize("mx4", [False, True], ids=["bf16", "mx4"])
@pytest.mark.parametrize("T,E,k,H,I", SHAPES)
def test_layer(T, E, k, H, I, mx4):
    i = SHAPES.index((T, E, k, H, I))
    act, dtype, first = i % 3, DTYPES[i // 2 % 3], i % 2 == 1
    s = case(T, E, k, H, I, mx4, bias=i % 2 == 0, seed=i, masked=(0.0, 0.3)[i % 4 == 3])
    say("moe_few", T, E, k, H, I, mx4, act, dtype)
    got = run(s, dtype, act, first, px=8 * (i % 3), py=(0, 3, 5)[i % 3])
    say(f"  {check(s, got, dtype, act, first):.3f} of the tolerance")


@pytest.mark.gpu
@pytest.mark.parametrize("mx4", [False, True], ids=["bf16", "mx4"])
@pytest.mark.parametrize("act", [0, 1, 2])
@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_types(mx4, act, dtype):
    s = case(7, 6, 2, 480, 224, mx4, bias=True, seed=act, masked=0.2)
    check(s, run(s, dtype, act), dtype, act)


@pytest.mark.gpu
def test_ids_that_are_no_choice():
    """-1, past the experts, negative: no choice, whatever their prob; a token
    without any is 0; a token that chose an expert twice has it twice."""
    s = case(6, 4, 3, 64, 32, False, bias=True)
    s["ids"] = torch.tensor([[-1, -1, -1], [4, 2 ** 31 - 1, -2 ** 31], [1, -1, 1], [3, 3, 3], [0, 9, 2], [2, -7, -1]],
                            dtype=torch.int32)
    s["prob"][(s["ids"] < 0) | (s["ids"] > 3)] = float("nan")
    got = run(s)
    assert (got[:2] == 0).all()
    s["prob"] = torch.nan_to_num(s["prob"])
    check(s, got, torch.float32)
    s["ids"].fill_(-1)
    assert (run(s) == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("mx4", [False, True], ids=["bf16", "mx4"])
def test_a_nan_stays_in_its_token(mx4):
    """A NaN or infinity in a token, or in an expert that others did not choose
    (bias, weight scale), reaches no other token; also past odd widths."""
    s = case(20, 3, 1, 288, 96, mx4, bias=True, seed=3)
    s["ids"] = (torch.arange(20, dtype=torch.int32) % 2).reshape(-1, 1)
    s["ids"][5] = 2
    clean = run(s)
    s["x"][7, 0] = float("nan")
    s["x"][8, -1] = float("inf")
    s["bias1"][2, 1] = float("nan")
    if mx4:
        s["sf2"][2, 3, 0] = 255
    got = run(s)
    rest = torch.ones(20, dtype=torch.bool)
    rest[[5, 7, 8]] = False
    assert torch.equal(got[rest], clean[rest])
    assert torch.isnan(got[[5, 7, 8]]).any(1).all()


@pytest.mark.gpu
def test_no_tokens():
    s = case(1, 4, 2, 64, 32, False)
    y = torch.zeros(0, 64, device="cuda")
    B.gg_moe_few(s["x"].cuda()[:0], s["ids"].cuda()[:0], s["prob"].cuda()[:0], s["w1"].cuda(), s["w2"].cuda(), y)


@pytest.mark.gpu
@pytest.mark.parametrize("mx4", [False, True], ids=["bf16", "mx4"])
def test_equal_calls_give_equal_bits(mx4):
    """Also with a spoilt workspace, and at other places of a token's batch."""
    s = case(40, 9, 4, 608, 352, mx4, bias=True, seed=8)
    ws = torch.full((B.gg_moe_few_workspace_size(40, 4, 608, 352),), 255, dtype=torch.uint8, device="cuda")
    a = run(s, workspace=ws)
    ws.fill_(127)
    assert torch.equal(a, run(s, workspace=ws))
    assert torch.equal(a, run(s))
    p = torch.randperm(40, generator=torch.Generator().manual_seed(0))
    s2 = dict(s, x=s["x"][p], ids=s["ids"][p], prob=s["prob"][p])
    assert torch.equal(a[p], run(s2))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [2, 24])
def test_past_4_gib(T):
    """The last expert's weights lie past 2^32 bytes."""
    E, H, I = 40, 8192, 4096
    s = case(T, 1, 1, H, I, False)
    w1 = torch.zeros(E, 2 * I, H, dtype=torch.bfloat16, device="cuda")
    w2 = torch.zeros(E, H, I, dtype=torch.bfloat16, device="cuda")
    w1[-1], w2[-1] = s["w1"][0].cuda(), s["w2"][0].cuda()
    y = torch.zeros(T, H, device="cuda")
    B.gg_moe_few(s["x"].cuda(), torch.full((T, 1), E - 1, dtype=torch.int32, device="cuda"), s["prob"].cuda(), w1, w2, y)
    check(s, y.cpu(), torch.float32)


# --------------------------------------------------------------------------
# refusals (CPU)
# --------------------------------------------------------------------------

def c_few(**kw):
    a = dict(x=P, ldx=64, T=4, H=64, ids=P, prob=P, k=2, E=4, w1=P, sf1=None, b1=None, w2=P, sf2=None, b2=None,
             wd=B.GG_BF16, I=32, y=P, yd=B.GG_BF16, ldy=64, act=0, alpha=1.7, lo=-7.0, hi=7.0, off=1.0, be1=4.0, be2=25.0,
             flags=0, ws=P, nb=1 << 20)
    a.update(kw)
    return B.load_library().gg_moe_few(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(wd=B.GG_F16), 3), (dict(wd=B.GG_F8E4M3), 3), (dict(yd=B.GG_MXFP4), 3), (dict(T=-1), 2), (dict(T=65), 8),
    (dict(k=0), 2), (dict(k=33), 8), (dict(E=0), 2), (dict(E=1025), 2), (dict(H=48), 2), (dict(H=0), 2), (dict(I=31), 2),
    (dict(H=1 << 17, ldx=1 << 17, ldy=1 << 17), 8), (dict(I=1 << 17), 8), (dict(ldx=63), 4), (dict(ldx=68), 4),
    (dict(ldx=1 << 24), 4), (dict(ldy=63), 4), (dict(x=None), 1), (dict(ids=None), 1), (dict(prob=None), 1),
    (dict(w1=None), 1), (dict(w2=None), 1), (dict(y=None), 1), (dict(wd=B.GG_MXFP4, sf1=P), 1), (dict(sf1=P), 6),
    (dict(x=P + 8), 5), (dict(w1=P + 8), 5), (dict(w2=P + 4), 5), (dict(ids=P + 2), 5), (dict(b1=P + 2), 5),
    (dict(b2=P + 1), 5), (dict(y=P + 1), 5), (dict(act=3), 6), (dict(flags=4), 6), (dict(act=1, lo=2.0, hi=1.0), 12),
    (dict(act=2, be1=-1.0), 12), (dict(ws=None), 1), (dict(ws=P + 64), 5), (dict(nb=256), 7)])
def test_refused(kw, status):
    assert c_few(**kw) == status
    assert B.gg_last_error()


def test_workspace_size():
    assert B.gg_moe_few_workspace_size(3, 2, 64, 32) == -(-(256 + 6 * 32 * 6 + 6 * 64 * 4) // 256) * 256
    for bad in [(65, 1, 64, 32), (-1, 1, 64, 32), (1, 0, 64, 32), (1, 33, 64, 32), (1, 1, 1 << 17, 32), (1, 1, 64, 0)]:
        assert B.gg_moe_few_workspace_size(*bad) == 0


def test_binding_refuses():
    s = case(3, 4, 2, 64, 32, False)
    good = dict(x=s["x"], ids=s["ids"], prob=s["prob"], w1=s["w1"], w2=s["w2"], y=torch.zeros(3, 64))
    for bad in [dict(x=s["x"].half()), dict(ids=s["ids"].long()), dict(ids=s["ids"][:2]), dict(prob=s["prob"][:, :1]),
                dict(w1=s["w1"][0]), dict(w1=s["w1"][:, :, :32]), dict(w2=s["w2"].transpose(1, 2)), dict(w2=s["w2"].half()),
                dict(w1=s["w1"].float()), dict(y=torch.zeros(3, 32)), dict(y=torch.zeros(2, 64)),
                dict(sf1=torch.zeros(4, 64, 2)), dict(bias1=torch.zeros(4, 63)), dict(bias2=torch.zeros(4, 64).double()), {}]:
        a = dict(good)
        a.update(bad)
        with pytest.raises(B.GGError):
            B.gg_moe_few(**a)


# One to 8 tokens whose choices are few for the experts: 1 to 8 choices, widths of
# less than a piece of 512 (MXFP4) or 128 (bf16) values, of whole ones and of parts;
# rows of one wave, of several blocks, of blocks that are not full.  (Sums: a
# choice's I terms, then at most 8 waves times 3 parts, within 2 I + 10 roundings.)
APART = [(1, 8, 1, 32, 32), (1, 1, 1, 160, 1056), (2, 6, 3, 96, 544), (4, 32, 8, 256, 96), (3, 15, 5, 1056, 32),
         (1, 64, 7, 544, 288), (4, 9, 2, 64, 1184), (8, 64, 4, 128, 160), (7, 64, 4, 512, 512), (1, 12, 8, 2080, 2080)]


@pytest.mark.gpu
@pytest.mark.parametrize("mx4", [False, True], ids=["bf16", "mx4"])
@pytest.mark.parametrize("T,E,k,H,I", APART)
def test_choices_apart(T, E, k, H, I, mx4):
    i = APART.index((T, E, k, H, I))
    act, dtype, first = i % 3, DTYPES[(i + 1) // 2 % 3], i % 2 == 0
    s = case(T, E, k, H, I, mx4, bias=i % 2 == 1, seed=50 + i, masked=(0.0, 0.3)[i % 3 == 1])
    say("moe_few", T, E, k, H, I, mx4, act, dtype)
    got = run(s, dtype, act, first, px=8 * (i % 3), py=(0, 3, 5)[i % 3])
    say(f"  {check(s, got, dtype, act, first):.3f} of the tolerance")


@pytest.mark.gpu
@pytest.mark.parametrize("mx4", [False, True], ids=["bf16", "mx4"])
def test_choices_apart_stay_apart(mx4):
    """Ids that are no choice, an expert chosen twice, NaN and infinity in a token
    or an expert, a spoilt workspace, and tokens in another order."""
    s = case(4, 32, 3, 288, 352, mx4, bias=True, seed=77)
    s["ids"] = torch.tensor([[-1, 32, 2 ** 31 - 1], [5, 5, -1], [31, 0, 7], [-2 ** 31, 2, 7]], dtype=torch.int32)
    s["prob"][(s["ids"] < 0) | (s["ids"] > 31)] = float("nan")
    ws = torch.full((B.gg_moe_few_workspace_size(4, 3, 288, 352),), 255, dtype=torch.uint8, device="cuda")
    got = run(s, workspace=ws)
    assert (got[0] == 0).all() and torch.equal(got, run(s))
    p = torch.tensor([2, 0, 3, 1])
    assert torch.equal(got[p], run(dict(s, x=s["x"][p], ids=s["ids"][p], prob=s["prob"][p])))
    check(dict(s, prob=torch.nan_to_num(s["prob"])), got, torch.float32)
    s["x"][3, 287] = float("inf")
    s["bias1"][5, 1] = float("nan")
    if mx4:
        s["sf2"][31, 3, 0] = 255
        s["sf1"][6, 0, 0] = 255                              # not chosen: its neighbour 5 ends before it
    bad = run(s)
    assert (bad[0] == 0).all() and torch.isnan(bad[1]).any() and not torch.isfinite(bad[3]).all()
    assert torch.isnan(bad[2, 3]) == mx4
    rest = torch.arange(288) != 3
    assert torch.equal(bad[2][rest], got[2][rest])


# --------------------------------------------------------------------------
# h at the edges of what its bf16 parts hold
# --------------------------------------------------------------------------

# choices apart, and two tokens more than the experts allow
EDGE = [(4, 8), (5, 2)]


def edge_case(T, E, mx4, w2, prob, odd=None):
    """H = I = 32, x = 0 and biases that make act = 32 sigmoid(32) 2^-5 = 1 (in fp32
    and to 2^-46 in 64 bits) of every h; w2 everywhere; row 3 of w2 instead all 0
    but its first, `odd`."""
    s = dict(T=T, E=E, k=1, H=32, I=32, mx4=mx4, x=torch.zeros(T, 32).bfloat16(), bias2=None)
    s["ids"] = (torch.arange(T, dtype=torch.int32) % E).reshape(T, 1)
    s["prob"] = torch.tensor(prob[:T]).float().reshape(T, 1)
    s["bias1"] = torch.cat([torch.full((E, 32), 2.0 ** -5), torch.full((E, 32), 32.0)], 1)
    w = torch.full((E, 32, 32), w2, dtype=torch.float64)
    if odd is not None:
        w[:, 3] = 0.0
        w[:, 3, 0] = odd
    if not mx4:
        s["w1"], s["w2"] = torch.zeros(E, 64, 32).bfloat16(), w.bfloat16()
        s["sf1"] = s["sf2"] = None
    else:
        s["w1"], s["sf1"] = torch.zeros(E, 64, 16, dtype=torch.uint8), torch.full((E, 64, 1), 127, dtype=torch.uint8)
        c, q = mx.quantise(torch.where(w.isinf(), 0.0, w).reshape(-1, 32))
        s["w2"], s["sf2"] = c.reshape(E, 32, 16), q.reshape(E, 32, 1)
        if odd is not None:                                  # 6 * 2^127: past bf16's largest
            s["w2"][:, 3, 0], s["sf2"][:, 3] = 7 if odd > 0 else 15, 254
    return s


@pytest.mark.gpu
@pytest.mark.parametrize("mx4", [False, True], ids=["bf16", "mx4"])
@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("T,E", EDGE)
def test_h_past_the_largest_bf16(T, E, dtype, mx4):
    """A finite h between bf16's largest number and fp32's stays finite: y is 32
    2^-120 h.  Errors: the activation 10 u and the product with prob u of h, its
    parts 2^-16 (fp32 y: 2^-24), 32 terms in two or three parts 96 u; then the
    rounding of y."""
    s = edge_case(T, E, mx4, 2.0 ** -120, [3.4e38, -3.4e38, 3.395e38, 3.4028e38, 3.3895e38])
    y = 32 * 2.0 ** -120 * s["prob"].double().expand(T, 32)
    tol = ((2.0 ** -24 if dtype == torch.float32 else 2.0 ** -16) + 107 * U + HALF[dtype]) * y.abs()
    assert ((run(s, dtype).double() - y).abs() <= tol).all()


@pytest.mark.gpu
@pytest.mark.parametrize("mx4", [False, True], ids=["bf16", "mx4"])
@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("T,E", EDGE)
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_infinite_weights(T, E, dtype, mx4, sign):
    """An infinite weight (of MXFP4: a value past bf16's largest) times h is an
    infinity of the product's sign, whatever is left of h after its first part
    (nothing of 1 and 2, something of either sign of 0.3 and 0.7); a NaN where h
    is 0.  The other rows of y are untouched."""
    s = edge_case(T, E, mx4, 0.5, [1.0, 0.3, -0.7, 0.0, 2.0], odd=sign * float("inf"))
    got = run(s, dtype)
    want3 = s["prob"][:, 0].double() * sign * float("inf")
    assert torch.equal(torch.isnan(got[:, 3]), torch.isnan(want3)) and torch.isnan(want3).sum() == 1
    ok = ~torch.isnan(want3)
    assert torch.equal(got[:, 3].double()[ok], want3[ok])
    rest = torch.arange(32) != 3
    y = 16 * s["prob"].double().expand(T, 31)
    assert ((got[:, rest].double() - y).abs() <= (2.0 ** -16 + 107 * U + HALF[dtype]) * y.abs()).all()


@pytest.mark.gpu
def test_no_tokens_clear_the_error_word():
    """As every call on a workspace does."""
    s = case(1, 4, 2, 64, 32, False)
    ws = torch.full((B.gg_moe_few_workspace_size(0, 2, 64, 32),), 255, dtype=torch.uint8, device="cuda")
    y = torch.zeros(0, 64, device="cuda")
    used = B.gg_moe_few(s["x"].cuda()[:0], s["ids"].cuda()[:0], s["prob"].cuda()[:0], s["w1"].cuda(), s["w2"].cuda(), y,
                        workspace=ws)
    assert B.gg_device_error(used) == 0 and (ws[4:] == 255).all()


# --------------------------------------------------------------------------
# every shape of a block (GG_LOG reports both passes)
# --------------------------------------------------------------------------

def logged(capfd, monkeypatch, call):
    """(the call's result, the report's kernels)."""
    capfd.readouterr()
    monkeypatch.setenv("GG_LOG", "1")
    got = call()
    monkeypatch.setenv("GG_LOG", "0")
    lines = [line for line in capfd.readouterr().err.splitlines() if line.startswith("[gg] gg_moe_few ")]
    return got, [line.split(": ", 1)[1] for line in lines]


def few_lines(s, dtype, first, second, active):
    """What the report says of blocks of (waves, parts of K): a wave's rows are 32,
    16 columns (eight waves: 32) are shared by the parts of K, and by those of h."""
    name, h = "mxfp4" if s["mx4"] else "bf16", 3 if dtype == torch.float32 else 2
    lines = []
    for (waves, wk), units, parts, what in ((first, s["I"] // 16, 1, "first, K in {}>"),
                                            (second, s["H"] // 32, h, "second, K in {}, h in %d>, few_sum_kernel" % h)):
        rows = waves // wk
        cols = (32 if waves == 8 else 16) // wk // parts
        lines.append(f"few_kernel<{name}, {what.format(wk)}, tile {32 * rows}x{cols}, {waves} waves, "
                     f"grid {-(-units // rows) * active}")
    return lines


# T, E, k, H, I; (waves, parts of K) of the first pass, of the second for a 16-bit
# and an fp32 y, with bf16 weights and with MXFP4 ones: all nine shapes in both
# passes, the second with two and three parts of h, on a device of 256 CUs.  Widths
# that end within a piece, tokens without a choice, more choices of an expert than
# a pass takes.
BLOCKS = [
    ((1, 1, 9, 1056, 2144), (4, 4), (4, 4), (4, 4), (4, 2), (4, 4), (4, 4)),
    ((2, 1, 2, 2080, 2176), (4, 4), (4, 4), (4, 2), (4, 4), (4, 4), (4, 2)),
    ((1, 1, 5, 1952, 672), (4, 4), (4, 2), (4, 2), (4, 4), (4, 2), (4, 2)),
    ((2, 3, 3, 672, 736), (4, 2), (4, 2), (4, 2), (4, 2), (4, 2), (4, 2)),
    ((21, 16, 2, 2080, 96), (4, 2), (2, 1), (8, 1), (4, 2), (4, 1), (8, 1)),
    ((45, 16, 4, 64, 1056), (8, 1), (2, 1), (2, 1), (8, 1), (2, 1), (2, 1)),
    ((24, 32, 7, 1056, 64), (2, 1), (8, 1), (8, 1), (2, 1), (8, 1), (8, 1)),
    ((5, 5, 1, 3232, 96), (4, 4), (2, 1), (2, 1), (4, 4), (4, 1), (4, 1)),
    ((40, 64, 2, 512, 256), (2, 1), (2, 1), (2, 1), (4, 1), (4, 1), (4, 1)),
]


@pytest.mark.gpu
@pytest.mark.parametrize("mx4", [False, True], ids=["bf16", "mx4"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("case_at", range(len(BLOCKS)))
def test_block_shapes(case_at, dtype, mx4, capfd, monkeypatch):
    shape, *ways = BLOCKS[case_at]
    first, *second = ways[3 * mx4:][:3]
    T, E, k, _, _ = shape
    i = case_at
    s = case(*shape, mx4, bias=i % 2 == 0, seed=100 + i, masked=0.1 if T > 4 else 0.0)
    say("moe_few blocks", *shape, mx4, dtype)
    got, lines = logged(capfd, monkeypatch, lambda: run(s, dtype, i % 3, i % 2 == 1, px=8 * (i % 2), py=i % 4))
    if torch.cuda.get_device_properties(0).multi_processor_count == 256:
        assert lines == few_lines(s, dtype, first, second[dtype == torch.float32], min(T * k, E))
    say(f"  {check(s, got, dtype, i % 3, i % 2 == 1):.3f} of the tolerance")


# T, E, k, H, I; parts of K of the first pass, of the second (choices apart)
LONE = [((1, 8, 1, 32, 32), 4, 8), ((2, 6, 3, 96, 544), 4, 2), ((4, 32, 8, 256, 96), 4, 1), ((4, 9, 2, 64, 1184), 1, 4),
        ((8, 64, 4, 128, 160), 2, 2), ((1, 12, 8, 2080, 2080), 1, 1)]


@pytest.mark.gpu
@pytest.mark.parametrize("mx4", [False, True], ids=["bf16", "mx4"])
@pytest.mark.parametrize("dtype", [torch.float16, torch.float32], ids=str)
@pytest.mark.parametrize("case_at", range(len(LONE)))
def test_lone_shapes(case_at, dtype, mx4, capfd, monkeypatch):
    shape, wk1, wk2 = LONE[case_at]
    T, _, k, H, I = shape
    s = case(*shape, mx4, bias=case_at % 2 == 1, seed=120 + case_at)
    say("moe_few lone", *shape, mx4, dtype)
    got, lines = logged(capfd, monkeypatch, lambda: run(s, dtype))
    name, h = "mxfp4" if mx4 else "bf16", 3 if dtype == torch.float32 else 2
    if torch.cuda.get_device_properties(0).multi_processor_count == 256:
        assert lines == [f"lone_first_kernel<{name}, K in {wk1}>, tile {128 // wk1}x1, 4 waves, "
                         f"grid {(I // 16 * wk1 + 3) // 4 * T * k}",
                         f"lone_second_kernel<{name}, K in {wk2}, h in {h}>, tile 16x{k}, 8 waves, grid {H // 16 * T}"]
    check(s, got, dtype)


# --------------------------------------------------------------------------
# the third part of h
# --------------------------------------------------------------------------

PRECISE = [b[0] for b in BLOCKS] + [l[0] for l in LONE]


@pytest.mark.gpu
@pytest.mark.parametrize("mx4", [False, True], ids=["bf16", "mx4"])
@pytest.mark.parametrize("T,E,k,H,I", PRECISE)
def test_h_of_an_fp32_result(T, E, k, H, I, mx4):
    """An fp32 y has 24 bits of h.  x has one value a token and w2 one +-1 a row, so
    both products are exact: h is off by 10 u of SwiGLU and u of prob, its three parts
    by u (2^-24), their sum by 2 u, the choices' by k u of the magnitudes; then the
    rounding of y is in these.  (Two parts alone are off by up to 256 u.)"""
    s = case(T, E, k, H, I, mx4, seed=200 + T + H)
    g = torch.Generator().manual_seed(9)
    s["x"].zero_()
    s["x"][torch.arange(T), torch.randint(0, H, (T,), generator=g)] = (3 * torch.randn(T, generator=g)).bfloat16()
    if mx4:
        s["w1"], s["sf1"] = mx.random_mx4(g, (E, 2 * I, H), 125, 127)
    else:
        s["w1"] = torch.randn(E, 2 * I, H, generator=g).bfloat16()
    w2 = torch.zeros(E, H, I)
    at = (torch.arange(H) * 7 % I).expand(E, H) + 3 * torch.arange(E)[:, None]
    w2.scatter_(2, (at % I)[:, :, None], torch.where(torch.rand(E, H, 1, generator=g) < 0.5, -1.0, 1.0))
    if mx4:
        code = torch.where(w2 == 0, 0, torch.where(w2 > 0, 2, 10)).to(torch.uint8).reshape(E, H, I // 2, 2)
        s["w2"] = code[..., 0] | code[..., 1] << 4
        s["sf2"] = torch.full((E, H, I // 32), 127, dtype=torch.uint8)
    else:
        s["w2"] = w2.bfloat16()
    say("moe_few precise", T, E, k, H, I, mx4)
    got = run(s)
    y, mag = torch.zeros(T, H, dtype=torch.float64), torch.zeros(T, H, dtype=torch.float64)
    for t in range(T):
        for j in range(k):
            e = int(s["ids"][t, j])
            c = (weights(s, "w1", "sf1", e) @ s["x"][t].double()).reshape(I // 32, 2, 32)
            h = float(s["prob"][t, j]) * act64(c[:, 0].reshape(I), c[:, 1].reshape(I), B.GG_DSWIGLU)
            term = w2[e].double() @ h
            y[t] += term
            mag[t] += term.abs()
    tol = (14 + k) * U * mag + 2.0 ** -120
    err = (got.double() - y).abs()
    say(f"  {float((err / tol).max()):.3f} of the tolerance")
    assert (err <= tol).all(), float((err / tol).max())
