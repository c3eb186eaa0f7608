"""gg_gemm_mx4 against the product in 64 bits (GPU), and its refusals (CPU).

Most cases are exact: codes are multiples of 1/2 up to 6 and scales 2^-1 .. 2^1,
so a product is a multiple of 2^-4 up to 144, and any partial sum of at most
4096 of them has 20 + 4 = 24 bits: fp32 holds it whatever the order.  With alpha
a power of two and the bias a multiple of 2^-4 below 2^10 times it, the result is
exact too, and only rounded to its type."""
import pytest
import torch

from moe_grouped_gemm_offset_amd import binding as B
from tests import mx4_util as mx
from tests.parity_util import say

DTYPES = [torch.bfloat16, torch.float16, torch.float32]
P = 1 << 20


def case(sizes, K, N, seed=0, tail=0, bias=False, lo=126, hi=128):
    g = torch.Generator().manual_seed(seed)
    L, m = len(sizes), sum(sizes) + tail
    s = dict(K=K, N=N, sizes=sizes, m=m)
    s["a"], s["sfa"] = mx.random_mx4(g, (m, K), lo, hi)
    s["b"], s["sfb"] = mx.random_mx4(g, (L, N, K), lo, hi)
    s["ends"] = torch.tensor(sizes, dtype=torch.int64).cumsum(0).to(torch.int32)
    s["alpha"] = torch.exp2(torch.randint(-2, 3, (L,), generator=g).float())
    s["bias"] = torch.randint(-4000, 4000, (L, N), generator=g).float() / 16 * s["alpha"][:, None] if bias else None
    return s


def want(s, ends=None):
    """(float64 result, float64 sum of magnitudes), 0 behind the last group."""
    d, mag = torch.zeros(s["m"], s["N"], dtype=torch.float64), torch.zeros(s["m"], s["N"], dtype=torch.float64)
    a, at = mx.values(s["a"], s["sfa"]), 0
    for e, end in enumerate((s["ends"] if ends is None else ends).tolist()):
        end = max(at, min(end, s["m"]))
        if end > at:
            b = mx.values(s["b"][e], s["sfb"][e])
            al = 1.0 if s["alpha"] is None else float(s["alpha"][e])
            d[at:end] = al * (a[at:end] @ b.T) + (0 if s["bias"] is None else s["bias"][e].double())
            mag[at:end] = al * (a[at:end].abs() @ b.abs().T) + (0 if s["bias"] is None else s["bias"][e].abs().double())
        at = end
    return d, mag, at


def run(s, dtype=torch.float32, ends=None, ptrs=False, fill=77.0, **kw):
    dev = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in s.items()}
    d = torch.full((s["m"], s["N"]), fill, dtype=dtype, device="cuda")
    kw.setdefault("workspace", torch.full((256,), 255, dtype=torch.uint8, device="cuda"))
    b, sfb = dev["b"], dev["sfb"]
    if ptrs:
        parts = [(x.clone(), y.clone()) for x, y in zip(b, sfb)]
        kw["b_ptrs"] = torch.tensor([x.data_ptr() for x, _ in parts], dtype=torch.int64, device="cuda")
        kw["sfb_ptrs"] = torch.tensor([y.data_ptr() for _, y in parts], dtype=torch.int64, device="cuda")
        b = sfb = None
    ws = B.gg_gemm_mx4(dev["a"], dev["sfa"], b, sfb, dev["ends"] if ends is None else ends.cuda(), d, alpha=dev["alpha"],
                       bias=dev["bias"], **kw)
    err = B.gg_device_error(ws)
    return d.cpu(), err


def check_exact(s, d, dtype, ends=None, fill=77.0):
    w, _, last = want(s, ends)
    assert torch.equal(d[:last].double(), w[:last].float().to(dtype).double())
    assert (d[last:] == fill).all()


# few rows a group (16 or 64 to a tile) and many, K of one stage to several
# groups of scales with an odd number of stages among them, N off the tiles
SHAPES = [([1], 128, 32), ([5], 256, 64), ([0, 3, 0], 384, 96), ([16, 1, 17, 0, 2], 640, 160),
          ([33, 64, 65, 1], 1152, 224), ([0, 0], 128, 64), ([40] * 5, 2176, 320), ([1] * 200, 256, 64),
          ([300], 128, 32), ([257, 0, 255], 256, 288), ([130, 513, 90], 384, 256), ([600], 640, 544),
          ([256, 256], 1024, 512), ([1000, 1, 0, 250], 1920, 288), ([700], 4096, 256)]


@pytest.mark.gpu
@pytest.mark.parametrize("sizes,K,N", SHAPES, ids=lambda v: str(v)[:24].replace(" ", ""))
@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_exact(sizes, K, N, dtype):
    i = SHAPES.index((sizes, K, N))
    say("gemm_mx4", sizes[:6], K, N, dtype)
    s = case(sizes, K, N, seed=i, tail=(0, 3, 40)[i % 3], bias=i % 2 == 0)
    if i % 4 == 3:
        s["alpha"] = None
    if dtype == torch.float16:                               # (within fp16's range)
        s["sfb"] = s["sfb"] - 6
        if s["bias"] is not None:
            s["bias"] = s["bias"] / 64
    d, err = run(s, dtype, ptrs=i % 3 == 1)
    assert err == 0
    check_exact(s, d, dtype)


# tiles of 128 x 128 and of 256 x 256, on ragged groups, K of an odd number of
# stages, of one unit, of several groups of scales; N off the tiles
TILES = [(128, [130, 513, 0, 90] * 3, 384, 1056), (128, [1, 127, 128, 129] * 8, 1152, 544), (128, [700] * 4, 256, 1216),
         (256, [2500, 1000], 128, 4064), (256, [3300, 0], 512, 4096), (256, [1700, 1999], 1920, 3872)]


@pytest.mark.gpu
@pytest.mark.parametrize("tile,sizes,K,N", TILES, ids=lambda v: str(v)[:24].replace(" ", ""))
@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_tiles(tile, sizes, K, N, dtype, monkeypatch, capfd):
    i = TILES.index((tile, sizes, K, N))
    s = case(sizes, K, N, seed=20 + i, tail=(7, 0)[i % 2], bias=i % 2 == 1)
    s["sfb"] = s["sfb"] - 6                                  # (within fp16's range)
    if s["bias"] is not None:
        s["bias"] = s["bias"] / 64
    monkeypatch.setenv("GG_LOG", "1")
    d, err = run(s, dtype, ptrs=i % 3 == 1)
    monkeypatch.setenv("GG_LOG", "0")
    assert err == 0 and f"{tile}x{tile}" in capfd.readouterr().err
    # (fp64 on the device: the products are exact there too)
    a, b = mx.values(s["a"], s["sfa"]).cuda(), [mx.values(x, y).cuda() for x, y in zip(s["b"], s["sfb"])]
    at = 0
    for e, end in enumerate(s["ends"].tolist()):
        w = float(s["alpha"][e]) * (a[at:end] @ b[e].T)
        w += 0 if s["bias"] is None else s["bias"][e].double().cuda()
        assert torch.equal(d[at:end].double(), w.float().to(dtype).double().cpu())
        at = end
    assert (d[at:] == 77.0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("L,rows", [(65, 3), (700, 5), (1024, 1), (130, 100)])
def test_many_groups(L, rows):
    """More groups than lanes, some empty."""
    sizes = [(i * 7 % 5) * rows for i in range(L)]
    s = case(sizes, 128, 32, seed=L, tail=9)
    d, err = run(s)
    assert err == 0
    check_exact(s, d, torch.float32)


@pytest.mark.gpu
@pytest.mark.parametrize("per", [4, 40, 300])
def test_random_scales(per):
    """Scales of any size, fp32: off by at most a rounding of each of K + 2
    additions, (K + 2) 2^-24 of the sum of the magnitudes."""
    K = 1408
    s = case([per, 2 * per, 0, per // 2], K, 288, seed=per, bias=True, lo=97, hi=157)
    d, err = run(s)
    w, mag, last = want(s)
    tol = (K + 2) * 2.0 ** -24 * mag[:last]
    assert err == 0 and ((d[:last].double() - w[:last]).abs() <= tol).all()


@pytest.mark.gpu
@pytest.mark.parametrize("per,K", [(4, 384), (40, 384), (300, 384), (300, 512), (4, 128)])
def test_nan_scales_stay_in_their_rows(per, K):
    """A scale of 255 makes NaN of its row of d (A) or column (B), of nothing
    else; also in the first scale of the row behind an odd number of stages."""
    s = case([per, per], K, 96, seed=1)
    s["sfa"][1::3, 0] = 255
    s["sfa"][2::6, -1] = 255
    s["sfb"][1, 5::8, 0] = 255
    d, _ = run(s)
    w, _, last = want(s)
    assert torch.equal(torch.isnan(d), torch.isnan(w))
    ok = ~torch.isnan(w)
    assert torch.equal(d[ok].double(), w[ok])


@pytest.mark.gpu
@pytest.mark.parametrize("per", [6, 40, 300])
def test_malformed_ends(per):
    """Ends that fall, are negative or lie past m_rows: flagged, groups by the
    running maximum, nothing written outside them."""
    s = case([per, per, per, per], 256, 96, seed=2, tail=5)
    for ends, flag in [([per, per // 2, 2 * per, 3 * per], 1), ([-4, per, per, 2 * per], 1),
                       ([per, 2 * per, 4 * per + 6, 4 * per + 6], 4), ([2 ** 31 - 1, -2 ** 31, 0, 5], 5)]:
        ends = torch.tensor(ends, dtype=torch.int32)
        d, err = run(s, ends=ends)
        assert err == flag
        top = torch.cummax(ends.clamp(0, s["m"]), 0).values
        check_exact(s, d, torch.float32, ends=top)
    d, err = run(s)                                          # the word is cleared
    assert err == 0


@pytest.mark.gpu
@pytest.mark.parametrize("tile,sizes,K,N", [(128, [300, 127, 129], 384, 1568), (128, [300, 127, 129], 512, 1568),
                                            (256, [2500, 1000], 384, 4064), (256, [2500, 1000], 512, 4064)],
                         ids=lambda v: str(v).replace(" ", ""))
def test_nan_and_ends_in_tiles(tile, sizes, K, N, monkeypatch, capfd):
    """NaN scales in the rows and columns next to a tile's edges, in the first
    block of the row behind an odd number of stages, in rows behind the last
    group; then ends that fall and lie past m_rows."""
    s = case(sizes, K, N, seed=3, tail=9)
    edge = torch.tensor([0, 1, 126, 127, 128, 255, 256, 257, s["m"] - 9])
    s["sfa"][edge, 0] = 255
    s["sfa"][4::97, -1] = 255
    s["sfa"][-8:] = 255
    s["sfb"][1, torch.tensor([0, 31, 127, 128, 255, 256, N - 1]), 0] = 255
    s["sfb"][0, 5::61, -1] = 255
    s["alpha"] = None
    a, b = mx.values(s["a"], s["sfa"]).cuda(), [mx.values(x, y).cuda() for x, y in zip(s["b"], s["sfb"])]
    m = s["m"]
    for ends, flag in [(s["ends"].tolist(), 0), ([sizes[0], -5] + sizes[2:], 1), ([sizes[0]] + [m + 1] * (len(sizes) - 1), 4)]:
        monkeypatch.setenv("GG_LOG", "1")
        d, err = run(s, ends=torch.tensor(ends, dtype=torch.int32))
        monkeypatch.setenv("GG_LOG", "0")
        assert f"{tile}x{tile}" in capfd.readouterr().err and err in (flag, flag | 1)
        at = 0
        for e, end in enumerate(ends):
            end = max(at, min(end, m))
            w = (a[at:end] @ b[e].T).cpu()
            assert torch.equal(torch.isnan(d[at:end]), torch.isnan(w))
            ok = ~torch.isnan(w)
            assert torch.equal(d[at:end][ok].double(), w[ok])
            at = end
        assert (d[at:] == 77.0).all()


@pytest.mark.gpu
def test_no_rows():
    s = case([0, 0, 0], 128, 32)
    ws = torch.full((256,), 255, dtype=torch.uint8, device="cuda")
    d, err = run(s, workspace=ws)
    assert err == 0 and d.numel() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [70000, 140])
def test_past_4_gib(rows):
    """d past 2^32 bytes (tiled), weights past them (thin)."""
    if rows == 70000:
        N, L, K = 32768, 1, 128
    else:
        N, L, K = 32768, 68, 4096
    g = torch.Generator().manual_seed(0)
    a, sfa = mx.random_mx4(g, (rows, K))
    b = torch.zeros(L, N, K // 2, dtype=torch.uint8, device="cuda")
    sfb = torch.full((L, N, K // 32), 127, dtype=torch.uint8, device="cuda")
    bc, bs = mx.random_mx4(g, (N, K))
    b[-1], sfb[-1] = bc.cuda(), bs.cuda()
    ends = torch.zeros(L, dtype=torch.int32)
    ends[-1] = rows
    d = torch.zeros(rows, N, dtype=torch.bfloat16, device="cuda")
    B.gg_gemm_mx4(a.cuda(), sfa.cuda(), b, sfb, ends.cuda(), d)
    pick = torch.tensor([0, rows // 2, rows - 2, rows - 1])
    w = mx.values(a[pick], sfa[pick]) @ mx.values(bc, bs).T
    assert torch.equal(d[pick.cuda()].cpu().double(), w.float().bfloat16().double())


# --------------------------------------------------------------------------
# refusals (CPU)
# --------------------------------------------------------------------------

def c_gemm(**kw):
    a = dict(a=P, sfa=P, m=64, k=256, b=P, sfb=P, bp=None, sp=None, n=64, off=P, L=2, alpha=None, bias=None, d=P,
             dt=B.GG_BF16, flags=0, ws=P, nb=256)
    a.update(kw)
    return B.load_library().gg_gemm_mx4(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(dt=B.GG_F8E4M3), 3), (dict(L=0), 2), (dict(L=1025), 2), (dict(m=-1), 2), (dict(m=1 << 31), 2), (dict(k=64), 2),
    (dict(k=192), 2), (dict(n=48), 2), (dict(n=0), 2), (dict(k=(1 << 21) + 128), 8), (dict(n=(1 << 21) + 32), 8),
    (dict(bp=P, sp=P), 6), (dict(b=None, sfb=None), 6), (dict(sfb=None), 1), (dict(b=None, sfb=None, bp=P), 1),
    (dict(off=None), 1), (dict(a=None), 1), (dict(sfa=None), 1), (dict(d=None), 1), (dict(a=P + 8), 5), (dict(b=P + 8), 5),
    (dict(d=P + 8), 5), (dict(sfa=P + 2), 5), (dict(sfb=P + 1), 5), (dict(off=P + 2), 5), (dict(alpha=P + 2), 5),
    (dict(bias=P + 1), 5), (dict(b=None, sfb=None, bp=P + 4, sp=P), 5), (dict(flags=4), 6), (dict(ws=None), 1),
    (dict(ws=P + 128), 5), (dict(nb=255), 7), (dict(m=(1 << 31) - 1, n=1 << 21), 8)])
def test_refused(kw, status):
    assert c_gemm(**kw) == status
    assert B.gg_last_error()


def test_binding_refuses():
    u8 = dict(dtype=torch.uint8)
    good = dict(a=torch.zeros(4, 64, **u8), sfa=torch.zeros(4, 4, **u8), b=torch.zeros(2, 32, 64, **u8),
                sfb=torch.zeros(2, 32, 4, **u8), offsets=torch.zeros(2, dtype=torch.int32), d=torch.zeros(4, 32))
    for bad in [dict(a=good["a"].float()), dict(sfa=good["sfa"][:3]), dict(b=good["b"][:1]), dict(b=good["b"][0]),
                dict(sfb=good["sfb"].transpose(1, 2)), dict(offsets=good["offsets"].long()),
                dict(offsets=good["offsets"][None]), dict(d=torch.zeros(4, 40)[:, :32]), dict(d=torch.zeros(3, 32)),
                dict(alpha=torch.ones(3)), dict(bias=torch.zeros(2, 31)), dict(b_ptrs=torch.zeros(2)), {}]:
        a = dict(good)
        a.update(bad)
        with pytest.raises(B.GGError):
            B.gg_gemm_mx4(**a)


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [1 << 30, (1 << 31) - 1])
def test_rows_by_the_billion(rows):
    """More tiles of 128 x 128 than a launch holds: the larger ones take the call,
    up to the most rows that there can be (132 and 264 GiB of operands)."""
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 133 * rows + (6 << 30):
        pytest.skip("not enough free memory on this device")
    K, N = 128, 32
    g = torch.Generator().manual_seed(0)
    pick = torch.tensor([0, 1, 255, 256, rows // 2, rows // 2 + 1, rows - 257, rows - 256, rows - 255, rows - 2, rows - 1])
    codes, scales = mx.random_mx4(g, (len(pick), K))
    b, sfb = mx.random_mx4(g, (1, N, K))
    a = torch.zeros(rows, K // 2, dtype=torch.uint8, device="cuda")
    sfa = torch.full((rows, K // 32), 127, dtype=torch.uint8, device="cuda")
    a[pick.cuda()], sfa[pick.cuda()] = codes.cuda(), scales.cuda()
    d = torch.full((rows, N), 7.0, dtype=torch.bfloat16, device="cuda")
    ends = torch.tensor([rows], dtype=torch.int32, device="cuda")
    ws = B.gg_gemm_mx4(a, sfa, b.cuda(), sfb.cuda(), ends, d)
    assert B.gg_device_error(ws) == 0
    w = mx.values(codes, scales) @ mx.values(b[0], sfb[0]).T
    assert torch.equal(d[pick.cuda()].cpu().double(), w.float().bfloat16().double())
    for at in range(2, rows, 1 << 24):                       # rows of zeros between the picked ones
        if not bool((pick >= at).logical_and(pick < at + 64).any()):
            assert not d[at:at + 64].any()


# --------------------------------------------------------------------------
# long reduction axes: scale buffers that are used again
# --------------------------------------------------------------------------

def logged(s, tile, capfd, monkeypatch, *args, **kw):
    """run(), whose report names the tile."""
    capfd.readouterr()
    monkeypatch.setenv("GG_LOG", "1")
    out = run(s, *args, **kw)
    monkeypatch.setenv("GG_LOG", "0")
    err = capfd.readouterr().err
    assert f"tile {tile}," in err and ("thin_kernel" in err) == tile.endswith("x32"), err
    return out


# The tiles' scales come in groups of 1024 values, in two buffers in turn, the thin
# kernel's 4096 values at a time for each of four waves.  Odd numbers of stages of 128
# among them, parts of a tile.
LONG = [("256x256", [2500, 1000], 4096, 4064), ("256x256", [2500, 1000], 3968, 4064),
        ("256x256", [1700, 1999], 2176, 4064), ("256x256", [1700, 1999], 8320, 3872),
        ("128x128", [700] * 4, 4096, 1216), ("128x128", [700] * 4, 3968, 1216),
        ("128x128", [130, 513, 0, 90] * 3, 2176, 1056), ("32x32", [16], 20480, 64), ("16x32", [5, 0, 30], 20608, 96),
        ("32x32", [40, 9], 20608, 96), ("32x32", [100], 16896, 160)]


@pytest.mark.gpu
@pytest.mark.parametrize("tile,sizes,K,N", LONG, ids=lambda v: str(v)[:24].replace(" ", ""))
@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_long_reductions(tile, sizes, K, N, dtype, monkeypatch, capfd):
    """Exact: products are multiples of 2^-4, and their magnitudes (with the bias,
    all before alpha) add up to less than 2^20, which is checked."""
    i = LONG.index((tile, sizes, K, N))
    say("gemm_mx4 long", tile, sizes[:4], K, N, dtype)
    s = case(sizes, K, N, seed=40 + i, tail=(0, 7)[i % 2], bias=i % 2 == 0)
    a = mx.values(s["a"], s["sfa"]).cuda()
    b = [mx.values(x, y).cuda() for x, y in zip(s["b"], s["sfb"])]
    down = 1.0
    if dtype == torch.float16:                               # (within fp16's range)
        down = 2.0 ** -8
        s["sfb"] = s["sfb"] - 8
        if s["bias"] is not None:
            s["bias"] = s["bias"] * down
    d, err = logged(s, tile, capfd, monkeypatch, dtype, ptrs=i % 3 == 1)
    assert err == 0
    at = 0
    for e, end in enumerate(s["ends"].tolist()):
        al, bias = float(s["alpha"][e]) * down, 0.0
        if s["bias"] is not None:
            bias = s["bias"][e].double().cuda() / al
        w = a[at:end] @ b[e].T + bias
        if end > at:
            mag = a[at:end].abs() @ b[e].abs().T + (bias.abs() if s["bias"] is not None else 0)
            assert float(mag.max()) < 2.0 ** 20
        assert torch.equal(d[at:end].double(), (al * w).float().to(dtype).double().cpu())
        at = end
    assert (d[at:] == 77.0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("tile,sizes,N", [("128x128", [300, 127, 129], 1568), ("256x256", [2500, 1000], 4064),
                                          ("16x32", [3, 0, 20], 96), ("32x32", [40, 9, 30], 96)],
                         ids=lambda v: str(v).replace(" ", ""))
def test_flags_of_the_ends_alone(tile, sizes, N, monkeypatch, capfd):
    """The error word of each tile's kernel has the flag of what is wrong, no other."""
    s = case(sizes, 384, N, seed=4, tail=9)
    m, last = s["m"], sum(sizes)
    for ends, flag in [(s["ends"].tolist(), 0), ([sizes[0], sizes[0] - 1] + [last] * (len(sizes) - 2), 1),
                       ([-1] + [last] * (len(sizes) - 1), 1), ([sizes[0]] + [m + 1] * (len(sizes) - 1), 4),
                       ([m + 1, -5] + [m] * (len(sizes) - 2), 5), ([0] * len(sizes), 0), ([m] * len(sizes), 0)]:
        _, err = logged(s, tile, capfd, monkeypatch, ends=torch.tensor(ends, dtype=torch.int32))
        assert err == flag, (ends, err)


@pytest.mark.gpu
def test_thin_past_4_gib(monkeypatch, capfd):
    """The thin kernel on weights past 2^32 bytes, their scales past 2^28.  Exact:
    products are multiples of 2^-6, their magnitudes add up to less than 2^18."""
    K, N, L, rows = (1 << 18) + (1 << 13), 32, 1024, 5
    g = torch.Generator().manual_seed(0)
    a, sfa = mx.random_mx4(g, (rows, K), 125, 126)
    bc, bs = mx.random_mx4(g, (N, K), 125, 126)
    b = torch.zeros(L, N, K // 2, dtype=torch.uint8, device="cuda")
    sfb = torch.full((L, N, K // 32), 127, dtype=torch.uint8, device="cuda")
    b[-1], sfb[-1] = bc.cuda(), bs.cuda()
    ends = torch.zeros(L, dtype=torch.int32)
    ends[-1] = rows
    s = dict(m=rows, N=N, ends=ends, a=a, sfa=sfa, b=b, sfb=sfb, alpha=None, bias=None)
    d, err = logged(s, "16x32", capfd, monkeypatch)
    w, x = mx.values(a, sfa), mx.values(bc, bs)
    assert err == 0 and b.numel() > 2 ** 32 and float((w.abs() @ x.abs().T).max()) < 2.0 ** 18
    assert torch.equal(d.double(), w @ x.T)
