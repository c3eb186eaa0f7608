"""gg_mx4_quant and gg_mx4_dequant against plain implementations in 64 bits
(GPU), and their refusals (CPU).  Codes, scales and values are exact: the scale
is a power of two found from the bit pattern, the code's rounding the only one,
and every value but those past a type's largest fits fp32 and bf16."""
import pytest
import torch

from moe_grouped_gemm_offset_amd import binding as B
from tests import mx4_util as mx
from tests.parity_util import say

DTYPES = [torch.bfloat16, torch.float16, torch.float32]
P = 1 << 20


def bits(t):
    return t.view({2: torch.int16, 4: torch.int32}[t.element_size()])


def quant(x, rows=None, width=None, end=None):
    n, w = rows or x.shape[0], width or x.shape[1]
    codes = torch.full((n, w // 2), 0x5A, dtype=torch.uint8, device="cuda")
    scales = torch.full((n, w // 32), 0x5A, dtype=torch.uint8, device="cuda")
    B.gg_mx4_quant(x, codes, scales, end=end)
    return codes, scales


def awkward(dtype, rows, width, seed):
    """Blocks of every kind: ordinary, ties, zeros of both signs, subnormal,
    the largest values, infinities and NaNs."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, width, generator=g) * torch.exp2(torch.randint(-12, 12, (rows, width), generator=g).float())
    x = x.reshape(-1, 32)
    kind = torch.arange(x.shape[0]) % 11
    tie = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])
    pick = tie[torch.randint(0, 8, x.shape, generator=g)] * torch.where(torch.rand(x.shape, generator=g) < 0.5, -1.0, 1.0)
    x = torch.where((kind == 1)[:, None], pick * 2.0 ** -3, x)
    x = torch.where((kind == 2)[:, None], 0.0, x)
    x = torch.where((kind == 3)[:, None], -0.0, x)
    tiny = torch.finfo(dtype).smallest_normal
    x = torch.where((kind == 4)[:, None], torch.randn(x.shape, generator=g) * tiny / 4, x)
    x = torch.where((kind == 5)[:, None], torch.sign(x) * torch.finfo(dtype).max * torch.rand(x.shape, generator=g), x)
    x = torch.where((kind == 6)[:, None], torch.sign(x) * torch.finfo(dtype).max, x)
    x[kind == 7, 5] = float("inf")
    x[kind == 8, 31] = -float("inf")
    x[kind == 9, 0] = float("nan")
    # the border of the scale: the largest at 6 2^e and just above
    x = torch.where((kind == 10)[:, None], x.clamp(-1, 1), x)
    x[kind == 10, 3] = 1.5
    x[(kind == 10).nonzero()[::2], 4] = 1.5 * (1 + 2 * torch.finfo(dtype).eps)
    return x.reshape(rows, width).to(dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("rows,width,pitch", [(1, 32, 32), (3, 64, 64), (7, 96, 101), (1, 8224, 8224), (257, 2080, 2083),
                                              (1500, 32, 33), (33, 32768, 32768), (2, 1 << 20, 1 << 20)])
def test_quant(dtype, rows, width, pitch):
    say("quant", dtype, rows, width, pitch)
    x = awkward(dtype, rows, width, rows + width)
    room = torch.zeros(rows * pitch + 1, dtype=dtype, device="cuda")[1:]     # at element alignment
    dev = room.as_strided((rows, width), (pitch, 1))
    dev.copy_(x)
    codes, scales = quant(dev)
    want_c, want_s = mx.quantise(x)
    assert torch.equal(scales.cpu(), want_s)
    assert torch.equal(codes.cpu(), want_c)


@pytest.mark.gpu
def test_quant_every_bf16():
    """Every finite bf16 as the largest of its block, beside every fraction of it."""
    top = torch.arange(0, 0x7F80, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    x = top[:, None].float() * torch.linspace(-1, 1, 32)[None, :]
    x[:, 7] = top.float()
    x = x.bfloat16()
    codes, scales = quant(x.cuda())
    want_c, want_s = mx.quantise(x)
    assert torch.equal(scales.cpu(), want_s) and torch.equal(codes.cpu(), want_c)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_dequant_every_code(dtype):
    codes = torch.arange(256, dtype=torch.uint8).repeat(256, 1).reshape(256, 256)
    codes = codes.reshape(256 * 16, 16)                      # blocks of 32 values
    scales = torch.arange(256, dtype=torch.uint8).repeat_interleave(16).reshape(-1, 1)
    out = torch.zeros(4096, 35, dtype=dtype, device="cuda")[:, :32]
    B.gg_mx4_dequant(codes.cuda(), scales.cuda(), out)
    want = mx.values(codes, scales).float().to(dtype)
    got = out.cpu()
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan)
    assert torch.equal(bits(got)[~nan], bits(want)[~nan])


@pytest.mark.gpu
@pytest.mark.parametrize("rows,end", [(0, None), (5, 0), (5, -3), (5, 3), (5, 9), (2000, 1025)])
def test_rows_behind_the_end(rows, end):
    g = torch.Generator().manual_seed(3)
    x = torch.randn(rows, 160, generator=g)
    e = None if end is None else torch.tensor([end], dtype=torch.int32, device="cuda")
    codes, scales = quant(x.cuda(), end=e) if rows else quant(x.cuda(), 0, 160)
    n = rows if end is None else max(0, min(rows, end))
    want_c, want_s = mx.quantise(x)
    assert torch.equal(codes.cpu()[:n], want_c[:n]) and torch.equal(scales.cpu()[:n], want_s[:n])
    assert (codes[n:] == 0x5A).all() and (scales[n:] == 0x5A).all()
    out = torch.full((rows, 160), 7.0, device="cuda")
    B.gg_mx4_dequant(codes, scales, out, end=e)
    assert torch.equal(out.cpu()[:n].double(), mx.values(want_c, want_s)[:n]) and (out[n:] == 7.0).all()


@pytest.mark.gpu
def test_typed_tensors_and_unaligned_bytes():
    g = torch.Generator().manual_seed(4)
    x = torch.randn(9, 64, generator=g)
    want_c, want_s = mx.quantise(x)
    c = torch.zeros(9, 32, dtype=torch.uint8, device="cuda")
    s = torch.zeros(9, 2, dtype=torch.uint8, device="cuda")
    B.gg_mx4_quant(x.cuda(), c.view(torch.float4_e2m1fn_x2), s.view(torch.float8_e8m0fnu))
    assert torch.equal(c.cpu(), want_c) and torch.equal(s.cpu(), want_s)
    c1 = torch.zeros(9 * 32 + 3, dtype=torch.uint8, device="cuda")[3:].view(9, 32)
    s1 = torch.zeros(9 * 2 + 1, dtype=torch.uint8, device="cuda")[1:].view(9, 2)
    B.gg_mx4_quant(x.cuda(), c1, s1)
    out = torch.zeros(9, 64, device="cuda")
    B.gg_mx4_dequant(c1, s1, out)
    assert torch.equal(c1.cpu(), want_c) and torch.equal(out.cpu().double(), mx.values(want_c, want_s))


@pytest.mark.gpu
def test_past_4_gib():
    """Rows past 2^32 bytes, and more of them than one pass of the blocks takes."""
    rows, width = (1 << 27) + 3, 32
    x = torch.zeros(rows, width, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator().manual_seed(5)
    tail = torch.randn(1000, width, generator=g).bfloat16()
    x[-1000:] = tail.cuda()
    codes, scales = quant(x)
    want_c, want_s = mx.quantise(tail)
    assert torch.equal(codes[-1000:].cpu(), want_c) and torch.equal(scales[-1000:].cpu(), want_s)
    assert not codes[:-1000].any() and not scales[:-1000].any()
    x.zero_()
    B.gg_mx4_dequant(codes, scales, x)
    assert torch.equal(x[-1000:].cpu().double(), mx.values(want_c, want_s))


# --------------------------------------------------------------------------
# refusals (CPU)
# --------------------------------------------------------------------------

def c_quant(L, **kw):
    a = dict(x=P, dtype=B.GG_BF16, ldx=64, rows=4, width=64, codes=P, scales=P, end=None)
    a.update(kw)
    return L.gg_mx4_quant(a["x"], a["dtype"], a["ldx"], a["rows"], a["width"], a["codes"], a["scales"], a["end"], None)


def c_dequant(L, **kw):
    a = dict(x=P, dtype=B.GG_BF16, ldx=64, rows=4, width=64, codes=P, scales=P, end=None)
    a.update(kw)
    return L.gg_mx4_dequant(a["codes"], a["scales"], a["rows"], a["width"], a["x"], a["dtype"], a["ldx"], a["end"], None)


@pytest.mark.parametrize("call", [c_quant, c_dequant])
@pytest.mark.parametrize("kw,status", [
    (dict(dtype=B.GG_F8E4M3), 3), (dict(dtype=B.GG_MXFP4), 3), (dict(rows=-1), 2), (dict(width=48), 2), (dict(width=0), 2),
    (dict(width=-32), 2), (dict(rows=(1 << 30) + 1), 8), (dict(width=(1 << 20) + 32, ldx=1 << 21), 8), (dict(ldx=63), 4),
    (dict(ldx=1 << 31), 4), (dict(x=None), 1), (dict(codes=None), 1), (dict(scales=None), 1), (dict(x=P + 1), 5),
    (dict(dtype=B.GG_F32, x=P + 2), 5), (dict(end=P + 2), 5)])
def test_refused(call, kw, status):
    assert call(B.load_library(), **kw) == status
    assert B.gg_last_error()


def test_binding_refuses():
    x = torch.zeros(4, 64)
    c, s = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8)
    for bad in [dict(x=x.double()), dict(x=x[0]), dict(x=x.t()), dict(c=c[:, :31]), dict(c=c.int()), dict(s=s[:3]),
                dict(s=s.t().contiguous().t()), dict(end=torch.zeros(2, dtype=torch.int32)), {}]:
        a = dict(x=x, c=c, s=s, end=None)
        a.update(bad)
        for call in (lambda: B.gg_mx4_quant(a["x"], a["c"], a["s"], end=a["end"]),
                     lambda: B.gg_mx4_dequant(a["c"], a["s"], a["x"], end=a["end"])):
            with pytest.raises(B.GGError):
                call()


def test_a_torch_without_the_types():
    """Where torch has no float4_e2m1fn_x2 or float8_e8m0fnu, codes and scales are
    uint8, and every call is there."""
    import os
    import subprocess
    import sys
    code = """
import torch
for name in ("float4_e2m1fn_x2", "float8_e8m0fnu"):
    if hasattr(torch, name):
        delattr(torch, name)
from moe_grouped_gemm_offset_amd import binding as B
assert B._CODES == B._SCALES == (torch.uint8,)
assert all(hasattr(B.load_library(), name) for name in B.EXPORTS)
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
