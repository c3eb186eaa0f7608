"""MXFP4 in 64 bits on the CPU, for the tests of the 4-bit calls."""
import torch

LEVELS = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def quantise(x):
    """(codes, scales) of a CPU tensor (rows, width): every code by comparing
    the distances to all eight levels, ties to the even one."""
    rows, width = x.shape
    v = x.double().reshape(rows, width // 32, 32)
    odd = ~torch.isfinite(v).all(2, keepdim=True)
    v = torch.where(odd, torch.zeros_like(v), v)
    top = v.abs().amax(2, keepdim=True)
    m, ex = torch.frexp(top)                       # m in [1/2, 1)
    e = torch.where(top > 0, torch.where(m <= 0.75, ex - 3, ex - 2), -127).clamp_min(-127)
    r = v.abs() * torch.exp2(-e.double())
    code = torch.zeros_like(r, dtype=torch.int64)
    for i in range(1, 8):
        lower, mid = LEVELS[i - 1], (LEVELS[i - 1] + LEVELS[i]) / 2
        code = torch.where((r > mid) | ((r == mid) & (i % 2 == 0)), i, code)
        assert bool((lower <= mid))
    code = code + 8 * (torch.signbit(v) & ~odd)
    pair = code.reshape(rows, width // 2, 2)
    scales = torch.where(odd, 255, e + 127).reshape(rows, width // 32)
    return (pair[..., 0] + 16 * pair[..., 1]).to(torch.uint8), scales.to(torch.uint8)


def values(codes, scales):
    """The float64 values of CPU codes (..., width / 2) and scales."""
    c = torch.stack([codes & 15, codes >> 4], dim=-1).long()
    v = LEVELS[c & 7] * torch.where(c >= 8, -1.0, 1.0).double()
    v = v.reshape(*scales.shape, 32)
    s = torch.where(scales == 255, float("nan"), torch.exp2(scales.double() - 127))
    return (v * s[..., None]).reshape(*codes.shape[:-1], 2 * codes.shape[-1])


def random_mx4(g, shape, lo=126, hi=128):
    """Random codes (..., width / 2) and scales of 2^(lo - 127) .. 2^(hi - 127)."""
    *head, width = shape
    codes = torch.randint(0, 256, (*head, width // 2), generator=g, dtype=torch.uint8)
    scales = torch.randint(lo, hi + 1, (*head, width // 32), generator=g, dtype=torch.uint8)
    return codes, scales
