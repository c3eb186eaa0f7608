"""gg_plan, gg_permute, gg_combine and gg_combine_bwd against plain
implementations (GPU), and their refusals (CPU).

Tolerances, from the arithmetic: rows and copies are exact.  A combined value
is a sum of k products in fp32, each fma of relative error u = 2^-24: off by
at most k u sum_j |w y|, then rounded once to its type (half an ulp of the
value: 2^-8 bf16, 2^-11 fp16, plus half of fp16's smallest subnormal, 2^-25).
A row gradient is one fp32 product, rounded once.  A weight gradient sums
`width` products over 256 threads: off by at most (width / 256 + 16) u
sum |d y|; a thread's own run is width / 256 long, and vectors add up to 8.
"""
import itertools

import pytest
import torch

from moe_grouped_gemm_offset_amd import binding as B
from tests.parity_util import say

U = 2.0 ** -24
HALF_ULP = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
FLOOR = {torch.float32: 0.0, torch.bfloat16: 0.0, torch.float16: 2.0 ** -25}


def ref_plan(ids, E, granule, m_rows):
    """(counts, ends, row_of, flags) by plain loops."""
    T, k = ids.shape
    flags = 0
    kept = [[] for _ in range(E)]
    for t in range(T):
        seen = set()
        for j in range(k):
            e = int(ids[t, j])
            if e == -1:
                continue
            if e < 0 or e >= E or e in seen:
                flags |= B.GG_DEVERR_IDS
                continue
            seen.add(e)
            kept[e].append((t, j))
    limit = m_rows // granule * granule
    row_of = torch.full((T, k), -1, dtype=torch.int32)
    counts, ends, at = [], [], 0
    for e in range(E):
        begin = min(at, limit)
        at += -(-len(kept[e]) // granule) * granule
        end = min(at, limit)
        n = min(len(kept[e]), end - begin)
        if n < len(kept[e]):
            flags |= B.GG_DEVERR_LAST
        for r, (t, j) in enumerate(kept[e][:n]):
            row_of[t, j] = begin + r
        counts.append(n)
        ends.append(end)
    return torch.tensor(counts, dtype=torch.int32), torch.tensor(ends, dtype=torch.int32), row_of, flags


def make_ids(T, k, E, seed, empty=0.1, skew=0.0):
    g = torch.Generator().manual_seed(seed)
    like = -skew * torch.arange(1, E + 1).float().log()
    noise = -(-torch.rand(T, E, generator=g).clamp_min(1e-7).log()).log()
    ids = (like + noise).argsort(1, descending=True)[:, :k].to(torch.int32)
    ids[torch.rand(T, k, generator=g) < empty] = -1
    ids[torch.rand(T, generator=g) < empty / 2] = -1
    return ids


def run_plan(ids, E, granule, m_rows, prob=None):
    T, k = ids.shape
    dev = torch.device("cuda")
    o = dict(counts=torch.full((E,), -7, dtype=torch.int32, device=dev),
             ends=torch.full((E,), -7, dtype=torch.int32, device=dev),
             row_of=torch.full((T, k), -7, dtype=torch.int32, device=dev),
             prob_rows=None if prob is None else torch.full((m_rows,), float("nan"), device=dev))
    ws = B.gg_plan(ids.cuda(), o["counts"], o["ends"], o["row_of"], m_rows, granule=granule,
                   prob=None if prob is None else prob.cuda(), prob_rows=o["prob_rows"])
    o["flags"] = B.gg_device_error(ws)
    return o


def check_plan(ids, E, granule, m_rows=None):
    T, k = ids.shape
    if m_rows is None:
        m_rows = B.gg_plan_max_rows(T, k, E, granule)
    prob = torch.rand(T, k, generator=torch.Generator().manual_seed(T)) + 0.5
    counts, ends, row_of, flags = ref_plan(ids, E, granule, m_rows)
    o = run_plan(ids, E, granule, m_rows, prob)
    assert torch.equal(o["counts"].cpu(), counts)
    assert torch.equal(o["ends"].cpu(), ends)
    assert torch.equal(o["row_of"].cpu(), row_of)
    assert o["flags"] == flags
    end = int(ends[-1])
    assert end <= m_rows
    rows = torch.zeros(end)
    rows[row_of[row_of >= 0].long()] = prob[row_of >= 0]
    got = o["prob_rows"].cpu()
    assert torch.equal(got[:end], rows)
    assert bool(torch.isnan(got[end:]).all()), "rows past the groups were written"


@pytest.mark.gpu
@pytest.mark.parametrize("T,k,E,granule", [
    (0, 2, 4, 256), (1, 1, 1, 1), (1, 8, 64, 256), (7, 8, 64, 8), (255, 3, 5, 256), (256, 2, 16, 16),
    (257, 4, 61, 256), (512, 2, 1024, 1), (513, 2, 1024, 2), (777, 32, 40, 256), (3000, 6, 128, 64),
    (1500, 1, 2, 256)])
def test_plan(T, k, E, granule):
    say("plan", T, k, E, granule)
    check_plan(make_ids(T, k, E, T + E, skew=0.8), E, granule)


@pytest.mark.gpu
def test_plan_many_chunks():
    """More tokens than 256 blocks of one chunk: several chunks to a block."""
    say("plan chunks")
    T, E = 256 * 256 + 700, 9
    ids = make_ids(T, 2, E, 5)
    m = B.gg_plan_max_rows(T, 2, E, 256)
    o = run_plan(ids, E, 256, m)
    # rows by a stable sort of the choices by expert
    flat = ids.flatten()
    counts = torch.bincount(flat[flat >= 0], minlength=E)
    padded = (counts + 255) // 256 * 256
    begin = torch.cat([torch.zeros(1, dtype=torch.int64), padded.cumsum(0)[:-1]])
    order = torch.where(flat >= 0, flat, torch.full_like(flat, E)).argsort(stable=True)
    order = order[: int(counts.sum())]
    rank = torch.arange(order.numel()) - (counts.cumsum(0) - counts)[flat[order].long()]
    want = torch.full_like(flat, -1)
    want[order] = (begin[flat[order].long()] + rank).to(torch.int32)
    assert torch.equal(o["row_of"].cpu().flatten(), want)
    assert torch.equal(o["counts"].cpu().long(), counts) and o["flags"] == 0


@pytest.mark.gpu
@pytest.mark.parametrize("T", [6, 900])
def test_plan_bad_ids(T):
    """Ids outside the experts and repeated ones have no row and are flagged;
    nothing else moves."""
    say("plan bad ids", T)
    ids = make_ids(T, 4, 12, 3, empty=0.0)
    ids[1, 2] = 12
    ids[2, 0] = -5
    ids[3, 3] = ids[3, 1]
    ids[T - 1] = 7
    ids[4, 1] = 2147483647
    check_plan(ids, 12, 256)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [40, 1200])
@pytest.mark.parametrize("m", [0, 100, 256, 600, 1024])
def test_plan_too_few_rows(T, m):
    """Groups are cut off at m_rows; what is left is consistent."""
    say("plan cut", T, m)
    check_plan(make_ids(T, 3, 6, 11), 6, 256, m_rows=m)
    check_plan(make_ids(T, 3, 6, 11), 6, 8, m_rows=m)


def max_rows(T, k, E, g):
    return B.gg_plan_max_rows(T, k, E, g)


def test_plan_max_rows():
    """The bound holds every way to deal n choices to E experts."""
    assert max_rows(0, 4, 8, 256) == 0
    assert max_rows(1, 1, 8, 256) == 256
    assert max_rows(1, 8, 64, 256) == 8 * 256
    assert max_rows(1000, 2, 4, 1) == 2000
    for n, E, g in itertools.product(range(9), range(1, 4), (1, 2, 4)):
        cuts = [c for c in itertools.product(range(n + 1), repeat=E) if sum(c) == n]
        worst = max(sum(-(-c // g) * g for c in cut) for cut in cuts)
        assert worst <= max_rows(n, 1, E, g) < worst + g * E + 1
    assert max_rows(-1, 1, 1, 1) == 0 and max_rows(1, 33, 64, 1) == 0


def rows_case(T, k, E, H, dtype, granule, seed, spare=3):
    ids = make_ids(T, k, E, seed)
    m = B.gg_plan_max_rows(T, k, E, granule) + spare
    counts, ends, row_of, _ = ref_plan(ids, E, granule, m)
    g = torch.Generator().manual_seed(seed)
    return counts, ends, row_of, m, g


CASES = [(1, 1, 1, 1, 256), (1, 2, 4, 7, 1), (5, 3, 8, 64, 8), (9, 8, 16, 1000, 256), (130, 2, 5, 2047, 16),
         (33, 4, 9, 4096, 256), (3, 32, 40, 7168, 1), (300, 2, 3, 129, 256), (0, 2, 4, 64, 256)]
FLOATS = [torch.bfloat16, torch.float16, torch.float32]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", FLOATS + [torch.float8_e4m3fn, torch.uint8])
def test_permute(dtype):
    for i, (T, k, E, H, granule) in enumerate(CASES):
        say("permute", T, k, E, H, granule, dtype)
        counts, ends, row_of, m, g = rows_case(T, k, E, H, dtype, granule, 20 + i)
        x = torch.randn(T, H + 5, generator=g)
        x[torch.rand(x.shape, generator=g) < 0.02] = float("nan")
        x = (x * 20).nan_to_num(nan=3.0).to(torch.uint8) if dtype == torch.uint8 else x.to(dtype)
        size = x.element_size()
        as_int = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[size]
        x = x[:, 2:2 + H] if i % 2 else x[:, :H].contiguous()
        out = torch.full((m, H), 7.0, device="cuda").to(dtype)
        before = out.clone().view(as_int)
        B.gg_permute(x.cuda() if x.is_contiguous() else torch.empty_strided(
            x.shape, x.stride(), dtype=dtype, device="cuda").copy_(x), row_of.cuda(), counts.cuda(),
            ends.cuda(), out)
        torch.cuda.synchronize()
        want = before.cpu()
        want[: int(ends[-1])] = 0
        t = torch.arange(T)[:, None].expand(T, k)
        ok = row_of >= 0
        want[row_of[ok].long()] = x.contiguous().view(as_int)[t[ok]]
        assert torch.equal(out.view(as_int).cpu(), want)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("weighted", [False, True])
def test_combine(dtype, weighted):
    for i, (T, k, E, H, granule) in enumerate(CASES):
        say("combine", T, k, E, H, granule, dtype, weighted)
        counts, ends, row_of, m, g = rows_case(T, k, E, H, dtype, granule, 60 + i)
        y = torch.randn(m, H, generator=g).to(dtype)
        w = torch.randn(T, k, generator=g) if weighted else None
        wide = torch.full((T, H + 5), 9.0, dtype=dtype, device="cuda")
        out = wide[:, 3:3 + H]
        B.gg_combine(y.cuda(), row_of.cuda(), out, weights=None if w is None else w.cuda())
        torch.cuda.synchronize()
        yy = torch.where((row_of >= 0)[:, :, None], y.double()[row_of.clamp_min(0).long()],
                         torch.zeros(1, dtype=torch.float64))
        ww = torch.ones(T, k, dtype=torch.float64) if w is None else w.double()
        terms = yy * ww[:, :, None]
        want = terms.sum(1)
        tol = (k + 1) * U * terms.abs().sum(1) + HALF_ULP[dtype] * (1 + 2 ** -7) * want.abs() + FLOOR[dtype]
        assert bool(((out.cpu().double() - want).abs() <= tol).all())
        rest = torch.cat([wide[:, :3], wide[:, 3 + H:]], 1)
        assert bool((rest == 9.0).all()), "columns outside the output were written"


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32, torch.uint8])
def test_widths_around_a_vector(dtype):
    """Widths just below and past whole 16-byte vectors, waves and blocks, at
    odd starts: permute writes its rows and nothing else, and combine of one
    choice without weights is a copy back, bit for bit."""
    n = 16 // torch.empty(0, dtype=dtype).element_size()
    for H in (1, n - 1, n, n + 1, 2 * n - 1, 2 * n + 1, 64 * n - 1, 64 * n + 1, 256 * n + 1, 513 * n - 1):
        say("widths", H, dtype)
        T, E = 37, 5
        counts, ends, row_of, m, g = rows_case(T, 1, E, H, dtype, 8, H)
        x = torch.randint(1, 100, (T, H + 3), generator=g).to(dtype)[:, 1:1 + H]
        out = torch.full((m + 1, H), 7, dtype=dtype, device="cuda")
        wide = torch.empty(T, H + 3, dtype=dtype, device="cuda")
        wide[:, 1:1 + H] = x.cuda()
        B.gg_permute(wide[:, 1:1 + H], row_of.cuda(), counts.cuda(), ends.cuda(), out[:m])
        torch.cuda.synchronize()
        want = torch.full((m + 1, H), 7, dtype=dtype)
        want[: int(ends[-1])] = 0
        ok = row_of[:, 0] >= 0
        want[row_of[ok, 0].long()] = x[ok]
        assert torch.equal(out.cpu(), want)
        if dtype == torch.uint8:
            continue
        back = torch.full((T, H + 3), 9, dtype=dtype, device="cuda")
        B.gg_combine(out[:m], row_of.cuda(), back[:, 1:1 + H])
        torch.cuda.synchronize()
        want = torch.full((T, H + 3), 9, dtype=dtype)
        want[:, 1:1 + H] = torch.where(ok[:, None], x, torch.zeros_like(x))
        assert torch.equal(back.cpu(), want)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", FLOATS)
def test_combine_bwd(dtype):
    for i, (T, k, E, H, granule) in enumerate(CASES):
        say("combine_bwd", T, k, E, H, granule, dtype)
        counts, ends, row_of, m, g = rows_case(T, k, E, H, dtype, granule, 90 + i)
        y = torch.randn(m, H, generator=g).to(dtype)
        wide = torch.randn(T, H + 4, generator=g).to(dtype)
        d = wide[:, 1:1 + H]
        w = torch.randn(T, k, generator=g)
        dy = torch.full((m, H), 7.0, dtype=dtype, device="cuda")
        dw = torch.full((T, k), float("nan"), device="cuda")
        B.gg_combine_bwd(wide.cuda()[:, 1:1 + H], y.cuda(), row_of.cuda(), w.cuda(), counts.cuda(),
                         ends.cuda(), dy, dw)
        torch.cuda.synchronize()
        want = torch.full((m, H), 7.0, dtype=torch.float64)
        want[: int(ends[-1])] = 0
        t = torch.arange(T)[:, None].expand(T, k)
        ok = row_of >= 0
        want[row_of[ok].long()] = w[ok].double()[:, None] * d.double()[t[ok]]
        tol = (HALF_ULP[dtype] * (1 + 2 ** -7) + U) * want.abs() + FLOOR[dtype]
        assert bool(((dy.cpu().double() - want).abs() <= tol).all())
        yy = torch.where(ok[:, :, None], y.double()[row_of.clamp_min(0).long()],
                         torch.zeros(1, dtype=torch.float64))
        terms = yy * d.double()[:, None, :]
        tol = (H / 256 + 32) * U * terms.abs().sum(2)
        assert bool(((dw.cpu().double() - terms.sum(2)).abs() <= tol).all())


@pytest.mark.gpu
def test_combine_bwd_differences():
    """Gradients against differences of the 64-bit sum, which is linear in y
    and in w: exact but for the outputs' own rounding."""
    T, k, E, H = 3, 2, 4, 24
    counts, ends, row_of, m, g = rows_case(T, k, E, H, torch.float32, 8, 7)
    y, w, d = torch.randn(m, H, generator=g), torch.randn(T, k, generator=g), torch.randn(T, H, generator=g)
    dy = torch.zeros(m, H, device="cuda")
    dw = torch.zeros(T, k, device="cuda")
    B.gg_combine_bwd(d.cuda(), y.cuda(), row_of.cuda(), w.cuda(), counts.cuda(), ends.cuda(), dy, dw)
    torch.cuda.synchronize()

    def loss(y, w):
        yy = torch.where((row_of >= 0)[:, :, None], y[row_of.clamp_min(0).long()], torch.zeros(1).double())
        return float(((yy * w[:, :, None]).sum(1) * d.double()).sum())

    y, w = y.double(), w.double()
    for r in range(0, int(ends[-1]), 3):
        for c in (0, 7, 23):
            z = y.clone()
            z[r, c] += 1.0
            assert abs(loss(z, w) - loss(y, w) - float(dy[r, c])) <= 1e-5
    for t in range(T):
        for j in range(k):
            z = w.clone()
            z[t, j] += 1.0
            assert abs(loss(y, z) - loss(y, w) - float(dw[t, j])) <= 1e-4


@pytest.mark.gpu
def test_rows_out_of_range_are_left_out():
    """A row_of outside the rows (here: of a larger plan) reads and writes
    nothing."""
    T, k, H, m = 6, 2, 96, 16
    row_of = torch.arange(T * k, dtype=torch.int32).reshape(T, k)
    row_of[2, 1], row_of[3, 0], row_of[4, 1] = m, 1 << 30, -3
    counts = torch.tensor([m], dtype=torch.int32)
    ends = torch.tensor([1 << 20], dtype=torch.int32)      # past the rows as well
    ok = (row_of >= 0) & (row_of < m)
    x = torch.randn(T, H)
    out = torch.zeros(m, H, device="cuda")
    B.gg_permute(x.cuda(), row_of.cuda(), counts.cuda(), ends.cuda(), out)
    back = torch.zeros(T, H, device="cuda")
    B.gg_combine(out, row_of.cuda(), back)
    torch.cuda.synchronize()
    assert torch.equal(back.cpu(), x * ok.sum(1, keepdim=True))


@pytest.mark.gpu
def test_combine_is_the_gradient_of_permute():
    T, k, E, H = 40, 3, 6, 200
    counts, ends, row_of, m, g = rows_case(T, k, E, H, torch.float32, 16, 31)
    x, dr = torch.randn(T, H, generator=g), torch.randn(m, H, generator=g)
    rows = torch.zeros(m, H, device="cuda")
    B.gg_permute(x.cuda(), row_of.cuda(), counts.cuda(), ends.cuda(), rows)
    dx = torch.zeros(T, H, device="cuda")
    B.gg_combine(dr.cuda(), row_of.cuda(), dx)
    torch.cuda.synchronize()
    a = float((rows.cpu().double() * dr.double()).sum())
    b = float((x.double() * dx.cpu().double()).sum())
    size = float((x.abs().double().sum())) * 10
    assert abs(a - b) <= 4 * k * U * size


# --------------------------------------------------------------------------
# rows that pass the cache by: more than 256 MB of expert rows
# --------------------------------------------------------------------------

def big_case(T, k, E, H, dtype, seed):
    """(row_of, counts, ends, x, weights, rows in use) on the GPU, groups padded
    to 16; some choices without a row."""
    counts, ends, row_of, m, _ = rows_case(T, k, E, H, dtype, 16, seed)
    size = torch.empty(0, dtype=dtype).element_size()
    assert T * k * H * size > 256 << 20
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randint(-99, 100, (T, H), generator=g, device="cuda", dtype=torch.int32)
    x = (x.abs() if dtype == torch.uint8 else x.float() / 64).to(dtype)
    w = torch.randn(T, k, generator=g, device="cuda")
    return row_of.cuda(), counts.cuda(), ends.cuda(), x, w, m


BIG = [(9001, 4, 8191, torch.uint8), (9001, 4, 4096, torch.bfloat16), (5003, 7, 4097, torch.float16),
       (17_003, 2, 2050, torch.float32)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,k,H,dtype", BIG)
def test_permute_past_the_cache(T, k, H, dtype):
    say("permute past the cache", T, k, H, dtype)
    row_of, counts, ends, x, _, m = big_case(T, k, 12, H, dtype, T)
    out = torch.full((m, H), 7, dtype=dtype, device="cuda")
    B.gg_permute(x, row_of, counts, ends, out)
    torch.cuda.synchronize()
    want = torch.full((m, H), 7, dtype=dtype, device="cuda")
    want[: int(ends[-1])] = 0
    ok = row_of >= 0
    t = torch.arange(T, device="cuda")[:, None].expand(T, k)
    want[row_of[ok].long()] = x[t[ok]]
    assert torch.equal(out, want)


@pytest.mark.gpu
@pytest.mark.parametrize("T,k,H,dtype", BIG[1:])
def test_combine_past_the_cache(T, k, H, dtype):
    say("combine past the cache", T, k, H, dtype)
    row_of, counts, ends, x, w, m = big_case(T, k, 12, H, dtype, T)
    y = torch.randn(m, H, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(dtype)
    out = torch.full((T, H), 9.0, dtype=dtype, device="cuda")
    B.gg_combine(y, row_of, out, weights=w)
    torch.cuda.synchronize()
    want = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    size = torch.zeros_like(want)
    for j in range(k):
        term = torch.where(row_of[:, j:j + 1] >= 0, y[row_of[:, j].clamp_min(0).long()].double() *
                           w[:, j:j + 1].double(), 0.0)
        want += term
        size += term.abs()
    tol = (k + 1) * U * size + HALF_ULP[dtype] * (1 + 2 ** -7) * want.abs() + FLOOR[dtype]
    assert bool(((out.double() - want).abs() <= tol).all())


@pytest.mark.gpu
@pytest.mark.parametrize("T,k,H,dtype", BIG[1:])
def test_combine_bwd_past_the_cache(T, k, H, dtype):
    say("combine_bwd past the cache", T, k, H, dtype)
    row_of, counts, ends, d, w, m = big_case(T, k, 12, H, dtype, T)
    y = torch.randn(m, H, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda").to(dtype)
    dy = torch.full((m, H), 7.0, dtype=dtype, device="cuda")
    dw = torch.full((T, k), float("nan"), device="cuda")
    B.gg_combine_bwd(d, y, row_of, w, counts, ends, dy, dw)
    torch.cuda.synchronize()
    end = int(ends[-1])
    assert bool((dy[end:] == 7.0).all())
    padding = torch.ones(end, dtype=torch.bool, device="cuda")
    padding[row_of[row_of >= 0].long()] = False
    assert bool((dy[:end][padding] == 0).all())
    for j in range(k):
        ok = row_of[:, j] >= 0
        r = row_of[ok, j].long()
        want = w[ok, j:j + 1].double() * d[ok].double()
        tol = (HALF_ULP[dtype] * (1 + 2 ** -7) + U) * want.abs() + FLOOR[dtype]
        assert bool(((dy[r].double() - want).abs() <= tol).all())
        terms = y[r].double() * d[ok].double()
        tol = (H / 256 + 32) * U * terms.abs().sum(1)
        assert bool(((dw[ok, j].double() - terms.sum(1)).abs() <= tol).all())
        assert bool((dw[~ok, j] == 0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("k", [1, 2, 3, 5, 6, 7, 9, 17])
def test_combine_bwd_every_count_of_choices(k):
    """Choices that fill a block's rows in flight in part, or in several turns."""
    T, E, H = 50, 40, 515
    say("combine_bwd choices", k)
    counts, ends, row_of, m, g = rows_case(T, k, E, H, torch.float32, 8, k)
    y, d, w = torch.randn(m, H, generator=g), torch.randn(T, H, generator=g), torch.randn(T, k, generator=g)
    y[0] = float("nan")                                # not to be taken by a choice without a row
    nan = row_of == 0
    dy, dw = torch.full((m, H), 7.0, device="cuda"), torch.full((T, k), float("nan"), device="cuda")
    B.gg_combine_bwd(d.cuda(), y.cuda(), row_of.cuda(), w.cuda(), counts.cuda(), ends.cuda(), dy, dw)
    torch.cuda.synchronize()
    ok = row_of >= 0
    yy = torch.where(ok[:, :, None], y.double()[row_of.clamp_min(0).long()], torch.zeros(1).double())
    terms = yy * d.double()[:, None, :]
    near = (dw.cpu().double() - terms.sum(2)).abs() <= (H / 256 + 32) * U * terms.abs().sum(2)
    assert bool(near[~nan].all()) and bool(torch.isnan(dw.cpu()[nan]).all()) and int(nan.sum()) == 1
    want = torch.full((m, H), 7.0, dtype=torch.float64)
    want[: int(ends[-1])] = 0
    t = torch.arange(T)[:, None].expand(T, k)
    want[row_of[ok].long()] = w[ok].double()[:, None] * d.double()[t[ok]]
    assert bool(((dy.cpu().double() - want).abs() <= U * want.abs()).all())


# --------------------------------------------------------------------------
# refusals, on the host (no GPU)
# --------------------------------------------------------------------------

P, WS = 1 << 20, 1 << 24
NULL, SHAPE, DTYPE, LAYOUT, ALIGN, MODE, WORKSPACE, UNSUPPORTED = 1, 2, 3, 4, 5, 6, 7, 8


def c_plan(**kw):
    a = dict(ids=P, T=16, k=4, E=64, g=256, m=4096, prob=P, counts=P, ends=P, row_of=P, rows=P, ws=WS,
             wsb=1 << 20)
    a.update(kw)
    return B.load_library().gg_plan(*(a[n] for n in ("ids", "T", "k", "E", "g", "m", "prob", "counts",
                                                     "ends", "row_of", "rows", "ws", "wsb")), None)


@pytest.mark.parametrize("kw,status", [
    (dict(ids=None), NULL), (dict(counts=None), NULL), (dict(ends=None), NULL), (dict(row_of=None), NULL),
    (dict(ws=None), NULL), (dict(rows=None), MODE), (dict(prob=None), MODE), (dict(E=0), SHAPE),
    (dict(E=1025), SHAPE), (dict(k=0), SHAPE), (dict(k=33), UNSUPPORTED), (dict(T=-1), SHAPE),
    (dict(T=1 << 24), UNSUPPORTED), (dict(g=0), SHAPE), (dict(g=3), SHAPE), (dict(g=512), SHAPE),
    (dict(m=-1), SHAPE), (dict(m=1 << 31), SHAPE), (dict(row_of=P + 2), ALIGN), (dict(ws=WS + 4), ALIGN),
    (dict(wsb=8), WORKSPACE),
])
def test_plan_rejects(kw, status):
    assert c_plan(**kw) == status
    assert B.gg_last_error() != ""


def test_plan_max_rows_out_of_range():
    """0 for a granule that gg_plan refuses."""
    for g in (0, 3, 6, 100, 255, 257, 512):
        assert c_plan(g=g) == SHAPE
        assert max_rows(10, 2, 4, g) == 0


def c_permute(**kw):
    a = dict(x=P, dt=0, ld=64, T=16, H=64, row_of=P, k=4, counts=P, ends=P, E=8, m=512, out=P)
    a.update(kw)
    return B.load_library().gg_permute(*(a[n] for n in ("x", "dt", "ld", "T", "H", "row_of", "k", "counts",
                                                        "ends", "E", "m", "out")), None)


def c_combine(**kw):
    a = dict(y=P, dt=0, m=512, H=64, row_of=P, T=16, k=4, w=None, out=P, ld=64)
    a.update(kw)
    return B.load_library().gg_combine(*(a[n] for n in ("y", "dt", "m", "H", "row_of", "T", "k", "w", "out",
                                                        "ld")), None)


def c_combine_bwd(**kw):
    a = dict(d=P, dt=0, ld=64, T=16, H=64, y=P, m=512, w=P, row_of=P, k=4, counts=P, ends=P, E=8, dy=P, dw=P)
    a.update(kw)
    return B.load_library().gg_combine_bwd(*(a[n] for n in ("d", "dt", "ld", "T", "H", "y", "m", "w",
                                                            "row_of", "k", "counts", "ends", "E", "dy",
                                                            "dw")), None)


@pytest.mark.parametrize("call", [c_permute, c_combine, c_combine_bwd])
@pytest.mark.parametrize("kw,status", [
    (dict(row_of=None), NULL), (dict(dt=7), DTYPE), (dict(H=0), SHAPE), (dict(H=(1 << 20) + 1), UNSUPPORTED),
    (dict(ld=63), LAYOUT), (dict(T=-1), SHAPE), (dict(k=0), SHAPE), (dict(k=40), UNSUPPORTED),
    (dict(m=-1), SHAPE), (dict(m=1 << 31), SHAPE), (dict(row_of=P + 1), ALIGN),
])
def test_rows_reject(call, kw, status):
    assert call(**kw) == status


@pytest.mark.parametrize("call,kw,status", [
    (c_permute, dict(x=None), NULL), (c_permute, dict(out=None), NULL), (c_permute, dict(counts=None), NULL),
    (c_permute, dict(ends=None), NULL), (c_permute, dict(x=P + 1), ALIGN), (c_permute, dict(E=0), SHAPE),
    (c_combine, dict(y=None), NULL), (c_combine, dict(out=None), NULL), (c_combine, dict(dt=3), DTYPE),
    (c_combine, dict(w=P + 2), ALIGN), (c_combine_bwd, dict(w=None), NULL), (c_combine_bwd, dict(dw=None), NULL),
    (c_combine_bwd, dict(dy=None), NULL), (c_combine_bwd, dict(d=None), NULL), (c_combine_bwd, dict(dt=4), DTYPE),
    (c_combine_bwd, dict(dy=P + 1), ALIGN), (c_combine_bwd, dict(E=2000), SHAPE),
])
def test_rows_reject_own(call, kw, status):
    assert call(**kw) == status


def test_binding_rejects():
    i32 = torch.int32
    x, row_of = torch.zeros(4, 8), torch.zeros(4, 2, dtype=i32)
    c, e = torch.zeros(3, dtype=i32), torch.zeros(3, dtype=i32)
    ws = torch.zeros(1 << 16, dtype=torch.uint8)
    for call in (lambda: B.gg_permute(x, row_of, c, e, torch.zeros(16, 9)),
                 lambda: B.gg_permute(x, row_of, c, e, torch.zeros(16, 8).half()),
                 lambda: B.gg_permute(x, row_of.long(), c, e, torch.zeros(16, 8)),
                 lambda: B.gg_permute(x.t(), row_of[:2], c, e, torch.zeros(16, 4)),
                 lambda: B.gg_permute(x.expand(4, 8)[:1].expand(4, 8), row_of, c, e, torch.zeros(16, 8)),
                 lambda: B.gg_combine(torch.zeros(16, 8), row_of, x.half()),
                 lambda: B.gg_combine(torch.zeros(16, 8), row_of, x, weights=torch.zeros(4, 3)),
                 lambda: B.gg_combine(torch.zeros(16, 16)[:, ::2], row_of, x),
                 lambda: B.gg_combine_bwd(x, torch.zeros(16, 8), row_of, torch.zeros(4, 2), c, e,
                                          torch.zeros(15, 8), torch.zeros(4, 2)),
                 lambda: B.gg_plan(row_of, c, e[:2], row_of, 16, workspace=ws),
                 lambda: B.gg_plan(row_of, c, e, row_of, 16, prob=torch.zeros(4, 2),
                                   prob_rows=torch.zeros(15), workspace=ws)):
        with pytest.raises(B.GGError):
            call()


def test_binding_rejects_another_device(monkeypatch):
    """The library launches on the current device; a call whose arguments are
    on another one is refused before anything is launched there."""
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    with pytest.raises(B.GGError) as e:
        B._raw_stream(None, 1)
    assert e.value.status == 9
    assert B._raw_stream(1234, 0) == 1234


def host_calls(dev="cpu", ws="cpu"):
    """Every call around the GEMMs with well-formed arguments on a device."""
    f, i32, u8 = torch.zeros, torch.int32, torch.uint8
    kw = dict(device=dev)
    x, x_rows = f(4, 8, **kw), f(16, 8, **kw)
    ids, p = f(4, 2, dtype=i32, **kw), f(4, 2, **kw)
    c, one, fone = f(3, dtype=i32, **kw), f(1, dtype=i32, **kw), f(1, **kw)
    logits, d = f(4, 3, **kw), f(4, 3, **kw)
    tab = f(2, dtype=torch.int64, **kw), f(2, dtype=torch.int64, **kw), f(2, dtype=i32, **kw), 0
    s = f(1, dtype=torch.float64, **kw)
    w = None if ws is None else f(1 << 16, dtype=u8, device=ws)
    return dict(
        route=lambda: B.gg_route(logits, ids, p, c, one, fone, workspace=w),
        route_bwd=lambda: B.gg_route_bwd(logits, ids, c, one, p, d),
        plan=lambda: B.gg_plan(ids, c, c.clone(), ids.clone(), 16, workspace=w),
        permute=lambda: B.gg_permute(x, ids, c, c, x_rows),
        combine=lambda: B.gg_combine(x_rows, ids, x),
        combine_bwd=lambda: B.gg_combine_bwd(x, x_rows, ids, p, c, c, x_rows.clone(), p.clone()),
        grad_norm=lambda: B.gg_grad_norm(*tab, s, workspace=w),
        grad_clip=lambda: B.gg_grad_clip(*tab, s, 1.0, f(2, **kw)))


@pytest.mark.parametrize("ws", ["cpu", None])
@pytest.mark.parametrize("call", list(host_calls()))
def test_binding_rejects_host_tensors(call, ws):
    """Kernels cannot read them: refused by the binding, with or without a GPU."""
    with pytest.raises(B.GGError) as e:
        host_calls(ws=ws)[call]()
    assert e.value.status == 9


@pytest.mark.gpu
@pytest.mark.parametrize("call", ["route", "plan", "grad_norm"])
def test_binding_rejects_a_host_workspace(call):
    with pytest.raises(B.GGError) as e:
        host_calls(dev="cuda", ws="cpu")[call]()
    assert e.value.status == 9


def test_binding_rejects_scalars():
    z = torch.zeros((), dtype=torch.int32)
    x, ids, p, c = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2), torch.zeros(8).int()
    for call in (lambda: B.gg_route(x, z, p, c, c[:1]), lambda: B.gg_route_bwd(x, z, c, c[:1], p, x),
                 lambda: B.gg_plan(z, c, c, ids, 16), lambda: B.gg_permute(x, z, c, c, x),
                 lambda: B.gg_permute(x, ids, c, c, z.float()), lambda: B.gg_permute(z.float(), ids, c, c, x),
                 lambda: B.gg_combine(z.float(), ids, x), lambda: B.gg_combine(x, z, x),
                 lambda: B.gg_combine_bwd(x, x, z, p, c, c, x, p), lambda: B.gg_grad_norm(z, z, z, 0, z)):
        with pytest.raises(B.GGError) as e:
            call()
        assert e.value.status == 2
