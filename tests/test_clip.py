"""gg_grad_norm and gg_grad_clip against plain 64-bit sums (GPU), and their
refusals (CPU).

Tolerances, from the arithmetic: the squares are exact in fp64 (24-bit factors)
and summed in fp64: off by at most n 2^-53 relative.  The norm is rounded once
to fp32 (2^-24); the factor is rounded once; a scaled value is one fp32
product rounded once more to its type: 2^-24 + 2^-24 relative for the fp32
factor and product, then half an ulp (2^-8 bf16, 2^-11 fp16 and half of fp16's
smallest subnormal, 2^-25; fp32's 2^-150).
"""
import math

import pytest
import torch

from moe_grouped_gemm_offset_amd import binding as B
from tests.parity_util import say

U = 2.0 ** -24
HALF_ULP = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
FLOOR = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}
KINDS = [torch.bfloat16, torch.float32, torch.float16]


def run(tensors, max_norm, eps=1e-6, outs=None, accumulate=None):
    ptrs, ends, dtypes, total = B.grad_table(tensors)
    sumsq = torch.full((1,), float("nan") if accumulate is None else accumulate, dtype=torch.float64,
                       device="cuda")
    norm = torch.full((2,), float("nan"), device="cuda")
    B.gg_grad_norm(ptrs, ends, dtypes, total, sumsq, accumulate=accumulate is not None)
    out_ptrs = None if outs is None else B.grad_table(outs)[0]
    B.gg_grad_clip(ptrs, ends, dtypes, total, sumsq, max_norm, norm, eps=eps, out_ptrs=out_ptrs)
    torch.cuda.synchronize()
    return float(sumsq), norm.cpu()


def check(tensors, max_norm, in_place, extra=0.0):
    before = [t.cpu().double() for t in tensors]
    outs = None if in_place else [torch.full_like(t, 5.0) for t in tensors]
    want = sum(float(t.square().sum()) for t in before) + extra
    sumsq, norm = run(tensors, max_norm, outs=outs, accumulate=extra if extra else None)
    n = sum(t.numel() for t in tensors)
    assert abs(sumsq - want) <= (n + 4) * 2.0 ** -52 * want
    ref = math.sqrt(want)
    assert abs(float(norm[0]) - ref) <= 2 * U * ref
    factor = min(1.0, max_norm / (ref + 1e-6))
    assert abs(float(norm[1]) - factor) <= 2 * U * factor
    for i, (b, t) in enumerate(zip(before, tensors if in_place else outs)):
        got = t.cpu().double()
        tol = (HALF_ULP[t.dtype] * (1 + 2 ** -7) + 4 * U) * b.abs() * factor + FLOOR[t.dtype]
        assert bool(((got - b * factor).abs() <= tol).all()), i
        if not in_place:
            assert torch.equal(tensors[i].cpu().double(), b), "the input changed"


def make(sizes, seed, std=1.0, kinds=KINDS):
    g = torch.Generator().manual_seed(seed)
    return [(std * torch.randn(n, generator=g)).to(kinds[i % len(kinds)]).cuda() for i, n in enumerate(sizes)]


SIZES = {"one": [1], "empty": [0], "none": [], "odd": [1, 0, 7, 0, 0, 2049, 3, 5000, 1, 0],
         "vector": [8, 4, 8, 2048, 2048, 2048], "large": [40000, 3, 123457, 2048 * 9],
         "many": [(i * 37) % 211 for i in range(700)], "blocks": [5_000_011, 2, 700_001]}


@pytest.mark.gpu
@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("name", list(SIZES))
def test_clip(name, in_place):
    say("clip", name, in_place)
    t = make(SIZES[name], 3)
    if name == "none":
        sumsq, norm = run(t, 1.0)
        assert sumsq == 0.0 and norm.tolist() == [0.0, 1.0]
        return
    check(t, 0.75, in_place)


@pytest.mark.gpu
@pytest.mark.parametrize("in_place", [True, False])
def test_clip_below_the_limit_keeps_the_bits(in_place):
    """A factor of 1 leaves every bit, NaN payloads of other tensors apart."""
    t = make([1000, 33], 4)
    keep = [x.clone() for x in t]
    outs = None if in_place else [torch.zeros_like(x) for x in t]
    _, norm = run(t, 1e9, outs=outs)
    assert float(norm[1]) == 1.0
    for a, b in zip(keep, t if in_place else outs):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_clip_unaligned_and_accumulated():
    """Views at odd elements of one buffer, results packed end to end in
    another; sums of two tables added up."""
    for dt in KINDS:
        flat = make([9000], 5, kinds=[dt])[0]
        tensors = [flat[1:778], flat[778:779], flat[801:5002], flat[5003:9000]]
        out = torch.zeros(sum(t.numel() for t in tensors), dtype=dt, device="cuda")
        outs, at = [], 0
        for t in tensors:
            outs.append(out[at:at + t.numel()])
            at += t.numel()
        before = [t.cpu().double() for t in tensors]
        want = sum(float(b.square().sum()) for b in before) + 2.5
        sumsq, norm = run(tensors, 1.0, outs=outs, accumulate=2.5)
        assert abs(sumsq - want) <= 1e-12 * want
        f = 1.0 / (math.sqrt(want) + 1e-6)
        for b, o in zip(before, outs):
            tol = (HALF_ULP[dt] * (1 + 2 ** -7) + 4 * U) * b.abs() * f + FLOOR[dt]
            assert bool(((o.cpu().double() - b * f).abs() <= tol).all())
        check(tensors, 1.0, True, extra=1.0)
        # what lies between and around the views is untouched
        assert torch.equal(flat[779:801], make([9000], 5, kinds=[dt])[0][779:801])


@pytest.mark.gpu
def test_clip_extremes():
    """Squares far outside fp32's range; a norm of infinity or NaN follows the
    formula; max_norm 0 clears."""
    big = torch.full((3000,), 1e30, device="cuda")
    small = torch.full((100,), 1e-30, device="cuda")
    _, norm = run([big, small], 1.0)
    ref = math.sqrt(3000 * float(torch.tensor(1e30)) ** 2)
    assert abs(float(norm[0]) - ref) <= 2 * U * ref
    assert abs(float(big[0]) - 1 / math.sqrt(3000)) <= 4 * U
    tiny = torch.full((64,), 2.0 ** -140, device="cuda")
    _, norm = run([tiny], 1.0, eps=0.0)
    assert float(norm[0]) == 8 * 2.0 ** -140 and float(norm[1]) == 1.0
    for bad in (float("nan"), float("inf")):
        t = make([50, 40], 9)
        t[0][7] = bad
        outs = [torch.zeros_like(x) for x in t]
        _, norm = run(t, 1.0, outs=outs)
        if math.isnan(bad):
            assert torch.isnan(norm).all() and all(bool(torch.isnan(o).all()) for o in outs)
        else:
            assert float(norm[0]) == bad and float(norm[1]) == 0.0
            assert bool(torch.isnan(outs[0][7])) and float(outs[1].abs().max()) == 0.0
    z = make([77], 10)
    _, norm = run(z, 0.0)
    assert float(norm[1]) == 0.0 and float(z[0].abs().max()) == 0.0


@pytest.mark.gpu
def test_norm_repeats_bit_for_bit():
    t = make([3_000_001, 17, 900_000], 12)
    a = run([x.clone() for x in t], 1.0)
    for _ in range(3):
        b = run([x.clone() for x in t], 1.0)
        assert a[0] == b[0] and torch.equal(a[1], b[1])


@pytest.mark.gpu
def test_clip_where_the_quotient_is_undefined():
    """A limit that the norm does not pass leaves every bit: 0 / 0 (no norm, no
    limit, no eps) and infinity / infinity (no limit asked for) as well.  Only a
    norm that is NaN gives a factor that is NaN."""
    for in_place in (True, False):
        z = [torch.zeros(900, device="cuda"), torch.zeros(5, device="cuda").bfloat16()]
        outs = None if in_place else [torch.full_like(t, 7.0) for t in z]
        _, norm = run(z, 0.0, eps=0.0, outs=outs)
        assert norm.tolist() == [0.0, 1.0]
        assert all(bool((t == 0).all()) for t in (z if in_place else outs))
        t = make([50, 40], 9)
        t[0][7] = float("inf")
        keep = [x.clone() for x in t]
        outs = None if in_place else [torch.zeros_like(x) for x in t]
        _, norm = run(t, float("inf"), outs=outs)
        assert norm.tolist() == [float("inf"), 1.0]
        for a, b in zip(keep, t if in_place else outs):
            assert torch.equal(a, b)
        t[1][3] = float("nan")
        _, norm = run(t, float("inf"), outs=outs)
        assert bool(torch.isnan(norm).all())


# --------------------------------------------------------------------------
# refusals, on the host (no GPU)
# --------------------------------------------------------------------------

P, WS = 1 << 20, 1 << 24
NULL, SHAPE, ALIGN, WORKSPACE, UNSUPPORTED, VALUE = 1, 2, 5, 7, 8, 12


def c_norm(**kw):
    a = dict(ptrs=P, ends=P, dtypes=P, n=3, total=100, sumsq=P, acc=0, ws=WS, wsb=1 << 20)
    a.update(kw)
    return B.load_library().gg_grad_norm(*(a[k] for k in ("ptrs", "ends", "dtypes", "n", "total", "sumsq",
                                                          "acc", "ws", "wsb")), None)


def c_clip(**kw):
    a = dict(ptrs=P, ends=P, dtypes=P, n=3, total=100, sumsq=P, max_norm=1.0, eps=1e-6, norm=P, out=None)
    a.update(kw)
    return B.load_library().gg_grad_clip(*(a[k] for k in ("ptrs", "ends", "dtypes", "n", "total", "sumsq",
                                                          "max_norm", "eps", "norm", "out")), None)


@pytest.mark.parametrize("call", [c_norm, c_clip])
@pytest.mark.parametrize("kw,status", [
    (dict(ptrs=None), NULL), (dict(ends=None), NULL), (dict(dtypes=None), NULL), (dict(sumsq=None), NULL),
    (dict(n=-1), SHAPE), (dict(n=0, total=5), SHAPE), (dict(total=-1), SHAPE),
    (dict(total=(1 << 40) + 1), UNSUPPORTED), (dict(ptrs=P + 4), ALIGN), (dict(sumsq=P + 4), ALIGN),
    (dict(dtypes=P + 2), ALIGN),
])
def test_grads_reject(call, kw, status):
    assert call(**kw) == status
    assert B.gg_last_error() != ""


@pytest.mark.parametrize("call,kw,status", [
    (c_norm, dict(ws=None), NULL), (c_norm, dict(ws=WS + 8), ALIGN), (c_norm, dict(wsb=64), WORKSPACE),
    (c_clip, dict(norm=None), NULL), (c_clip, dict(norm=P + 2), ALIGN), (c_clip, dict(out=P + 4), ALIGN),
    (c_clip, dict(max_norm=-1.0), VALUE), (c_clip, dict(max_norm=float("nan")), VALUE),
    (c_clip, dict(eps=-1.0), VALUE), (c_clip, dict(eps=float("inf")), VALUE),
])
def test_grads_reject_own(call, kw, status):
    assert call(**kw) == status


def test_table_rejects():
    with pytest.raises(B.GGError):
        B.grad_table([torch.zeros(4, dtype=torch.float64)])
    with pytest.raises(B.GGError):
        B.grad_table([torch.zeros(4, 4).t()[:, :2]])
    ptrs, ends, dtypes, total = B.grad_table([torch.zeros(3), torch.zeros(0), torch.zeros(2).half()])
    assert ends.tolist() == [3, 3, 5] and dtypes.tolist() == [2, 2, 1] and total == 5
