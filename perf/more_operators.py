"""What the operators of 4-bit experts are measured on: quantisation, the gated
activation, the grouped product, and a whole layer for a few tokens.

`run` computes each operator either in elementary torch operations (`own`
False) or with the package's entry points (`own` True); both take what
`prepare` holds.  `exact` gives the same outputs from the definitions in 64
bits.

MXFP4 is blocks of 32 values along a row: a 4-bit code each (E2M1: 0, 0.5, 1,
1.5, 2, 3, 4, 6 and their negatives; two to a byte, the first in the low half)
and one E8M0 scale 2^(s - 127) a block.

  quant   x (rows, width) -> codes and scales, with 2^e the smallest power of
          two for which max|x| of the block is at most 6 * 2^e, x / 2^e
          rounded to the nearest code, ties to the even one; and back to the
          values the codes stand for, in x's type
  glu     c (rows, 2n), 32-wide blocks of inputs and gates in turn, to the
          gated activation (rows, n), times a factor per row
  gemm    the rows of expert g times its weights, both MXFP4:
          d[m] = alpha_g a[m] b_g^T + bias_g; rows behind the last group stay
  few     a layer for a few tokens: y[t] = sum_j prob[t, j] (w2_e act(w1_e
          x[t] + bias1_e) + bias2_e), e = ids[t, j] (-1: none), weights in
          bf16 or MXFP4

Sizes are those of the library's workloads: 64 experts of 4096 x 2048, 32 of
4096 x 1536, 16 of 7168 x 2048, 8 of 2048 x 1024, 65536 rows.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
# the constants of the clamped GeGLU and of SiTU-GLU
ALPHA, CLAMP, OFFSET = 1.702, 7.0, 1.0
BETA1, BETA2 = 4.0, 25.0


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def listed():
    return [
        # the activations of a few decoded tokens: two calls' latency
        dict(name="quant_few", op="quant", rows=5, width=4096, pitch=0, dtype="bf16"),
        # the dispatched rows of a training batch
        dict(name="quant_rows", op="quant", rows=65536, width=4096, pitch=0, dtype="bf16"),
        # fp32 rows out of a wider tensor, an odd number of blocks
        dict(name="quant_odd", op="quant", rows=4097, width=2080, pitch=2083, dtype="f32"),
        # a micro-batch's rows through the clamped GeGLU
        dict(name="glu_small", op="glu", rows=515, n=1536, act="geglu", dtype="f16", out="f16", prob=True),
        # the rows of the 64-expert layer
        dict(name="glu_rows", op="glu", rows=65536, n=2048, act="swiglu", dtype="bf16", out="bf16",
             prob=True),
        # a batch of 512 decoded tokens' choices: eight rows an expert
        dict(name="gemm_decode", op="gemm", L=64, K=4096, N=4096, rows=512, skew=0.3, tail=0,
             out="bf16", bias=False),
        # a short prefill over few experts, groups of any size, K and N off the tiles
        dict(name="gemm_odd", op="gemm", L=8, K=1920, N=2080, rows=5003, skew=0.8, tail=37, out="f32",
             bias=True),
        # the first product of the 64-expert layer, Zipf-skewed over the experts
        dict(name="gemm_batch", op="gemm", L=64, K=4096, N=4096, rows=65536, skew=1.2, tail=512,
             out="bf16", bias=False),
        # one decoded token over 64 experts, 4-bit weights
        dict(name="few_one", op="few", T=1, E=64, k=8, H=4096, I=2048, weights="mx4", act="swiglu",
             out="bf16", bias=False, masked=0.0),
        # a small layer, three tokens, bf16 weights: latency
        dict(name="few_small", op="few", T=3, E=8, k=2, H=2048, I=1024, weights="bf16", act="geglu",
             out="bf16", bias=True, masked=0.0),
        # a padded batch of 24 over 32 experts
        dict(name="few_padded", op="few", T=24, E=32, k=4, H=4096, I=1536, weights="mx4", act="geglu",
             out="f32", bias=True, masked=0.2),
        # the largest batch: every one of 64 experts is read, bf16 weights
        dict(name="few_batch", op="few", T=64, E=64, k=8, H=4096, I=2048, weights="bf16", act="swiglu",
             out="bf16", bias=False, masked=0.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quant", "glu", "gemm", "gemm", "few", "few"])
    if op == "quant":
        width = 32 * _log_int(rng, 1, 256)
        dtype = rng.choice(["bf16", "f16", "f32"])
        rows = _log_int(rng, 1, min(65536, (1 << 29) // (width * BYTES[dtype])))
        return dict(op=op, rows=rows, width=width, dtype=dtype,
                    pitch=rng.choice([0, 0, width + rng.randint(1, 64)]))
    if op == "glu":
        n = 32 * _log_int(rng, 4, 224)
        dtype = rng.choice(["bf16", "f16", "f32"])
        rows = _log_int(rng, 1, min(65536, (1 << 28) // (n * BYTES[dtype])))
        return dict(op=op, rows=rows, n=n, act=rng.choice(["swiglu", "geglu", "situ"]), dtype=dtype,
                    out=rng.choice(["bf16", "f16", "f32"]), prob=rng.random() < 0.7)
    if op == "gemm":
        K, N = 128 * _log_int(rng, 2, 56), 32 * _log_int(rng, 8, 224)
        return dict(op=op, L=rng.choice([1, 8, 16, 32, 60, 64]), K=K, N=N,
                    rows=_log_int(rng, 1, min(65536, (1 << 40) // (K * N))),
                    skew=rng.choice([0.0, 0.6, 1.2]), tail=rng.choice([0, 0, 37, 256]),
                    out=rng.choice(["bf16", "f16", "f32"]), bias=rng.random() < 0.5)
    E = rng.choice([8, 16, 32, 60, 64, 128])
    H, I = 32 * _log_int(rng, 16, 224), 32 * _log_int(rng, 8, 100)
    I = min(I, (64 * 4096 * 2048 // (E * H)) // 32 * 32)
    return dict(op=op, T=_log_int(rng, 1, 64), E=E, k=rng.randint(1, 8), H=H, I=max(32, I),
                weights=rng.choice(["bf16", "mx4", "mx4"]), act=rng.choice(["swiglu", "geglu", "situ"]),
                out=rng.choice(["bf16", "f16", "f32"]), bias=rng.random() < 0.5,
                masked=rng.choice([0.0, 0.0, 0.2]))


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _sizes(case, seed):
    """Rows of every group: in proportion to Zipf weights in a shuffled order,
    as whole numbers that add up."""
    L, rows = case["L"], case["rows"]
    g = torch.Generator().manual_seed(seed)
    p = torch.arange(1, L + 1, dtype=torch.float64) ** -case["skew"]
    p = p[torch.randperm(L, generator=g)]
    p = p * (0.7 + 0.6 * torch.rand(L, generator=g, dtype=torch.float64))
    ends = (p.cumsum(0) / p.sum() * rows).round().long().tolist()
    ends[-1] = rows
    return [b - a for a, b in zip([0] + ends, ends)]


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    op, s = case["op"], dict(case)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    def activations(rows, width):
        # some channels are larger than others, as in a trained network
        return normal(rows, width) * (0.7 * normal(width)).exp()

    if op == "quant":
        rows, width = case["rows"], case["width"]
        room = torch.zeros(rows, max(width, case["pitch"]), dtype=DTYPES[case["dtype"]], device=dev)
        s["x"] = room[:, :width]
        for a in range(0, rows, 8192):
            s["x"][a:a + 8192] = activations(min(8192, rows - a), width)
        s["codes"] = torch.zeros(rows, width // 2, dtype=torch.uint8, device=dev)
        s["scales"] = torch.zeros(rows, width // 32, dtype=torch.uint8, device=dev)
        s["values"] = torch.zeros(rows, width, dtype=DTYPES[case["dtype"]], device=dev)
        return s
    if op == "glu":
        rows, n = case["rows"], case["n"]
        s["c"] = torch.zeros(rows, 2 * n, dtype=DTYPES[case["dtype"]], device=dev)
        for a in range(0, rows, 8192):
            s["c"][a:a + 8192] = 2.0 * normal(min(8192, rows - a), 2 * n)
        s["prob_rows"] = torch.rand(rows, generator=g, device=dev) if case["prob"] else None
        s["y"] = torch.zeros(rows, n, dtype=DTYPES[case["out"]], device=dev)
        return s
    if op == "gemm":
        L, K, N, rows = case["L"], case["K"], case["N"], case["rows"]
        s["sizes"] = _sizes(case, seed)
        s["offsets"] = torch.tensor(s["sizes"], dtype=torch.int64).cumsum(0).to(torch.int32).to(dev)
        m = rows + case["tail"]
        s["a"] = torch.zeros(m, K // 2, dtype=torch.uint8, device=dev)
        s["sfa"] = torch.zeros(m, K // 32, dtype=torch.uint8, device=dev)
        for i in range(0, m, 8192):
            s["a"][i:i + 8192], s["sfa"][i:i + 8192] = _quantise(activations(min(8192, m - i), K))
        s["b"] = torch.zeros(L, N, K // 2, dtype=torch.uint8, device=dev)
        s["sfb"] = torch.zeros(L, N, K // 32, dtype=torch.uint8, device=dev)
        for e in range(L):
            s["b"][e], s["sfb"][e] = _quantise(normal(N, K) * K ** -0.5)
        s["alpha"] = 0.5 + torch.rand(L, generator=g, device=dev)
        s["bias_t"] = 0.1 * normal(L, N) if case["bias"] else None
        s["d"] = torch.zeros(m, N, dtype=DTYPES[case["out"]], device=dev)
        s["workspace"] = torch.zeros(4096, dtype=torch.uint8, device=dev)
        return s

    T, E, H, I = case["T"], case["E"], case["H"], case["I"]
    k = s["k"] = min(case["k"], E)
    s["x"] = normal(T, H).bfloat16()
    ids = torch.rand(T, E, generator=g, device=dev).topk(k, dim=1).indices.to(torch.int32)
    # a padded batch: some tokens are none, and some choices were dropped
    none = torch.rand(T, 1, generator=g, device=dev) < case["masked"]
    drop = torch.rand(T, k, generator=g, device=dev) < case["masked"] / 4
    s["ids"] = torch.where(none | drop, torch.full_like(ids, -1), ids)
    s["prob"] = torch.softmax(normal(T, k), dim=1)
    if case["weights"] == "bf16":
        s["w1"] = torch.zeros(E, 2 * I, H, dtype=torch.bfloat16, device=dev)
        s["w2"] = torch.zeros(E, H, I, dtype=torch.bfloat16, device=dev)
        s["sf1"] = s["sf2"] = None
        for e in range(E):
            s["w1"][e], s["w2"][e] = normal(2 * I, H) * H ** -0.5, normal(H, I) * I ** -0.5
    else:
        s["w1"] = torch.zeros(E, 2 * I, H // 2, dtype=torch.uint8, device=dev)
        s["sf1"] = torch.zeros(E, 2 * I, H // 32, dtype=torch.uint8, device=dev)
        s["w2"] = torch.zeros(E, H, I // 2, dtype=torch.uint8, device=dev)
        s["sf2"] = torch.zeros(E, H, I // 32, dtype=torch.uint8, device=dev)
        for e in range(E):
            s["w1"][e], s["sf1"][e] = _quantise(normal(2 * I, H) * H ** -0.5)
            s["w2"][e], s["sf2"][e] = _quantise(normal(H, I) * I ** -0.5)
    s["bias1"] = 0.1 * normal(E, 2 * I) if case["bias"] else None
    s["bias2"] = 0.1 * normal(E, H) if case["bias"] else None
    s["y"] = torch.zeros(T, H, dtype=DTYPES[case["out"]], device=dev)
    s["workspace"] = torch.zeros(1 << 24, dtype=torch.uint8, device=dev)
    return s


# --------------------------------------------------------------------------
# the plain forms
# --------------------------------------------------------------------------

_LEVELS = {}


def _levels(device):
    """The values of the 16 codes."""
    if device not in _LEVELS:
        half = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
        _LEVELS[device] = torch.tensor(half + [-v for v in half], device=device)
    return _LEVELS[device]


def _quantise(x):
    """(codes, scales) of rows whose width is a multiple of 32."""
    rows, width = x.shape
    v = x.float().reshape(rows, width // 32, 32)
    top = v.abs().amax(2, keepdim=True)
    m, ex = torch.frexp(top)                       # top = m 2^ex, 6 = 0.75 * 2^3
    e = torch.where(m <= 0.75, ex - 3, ex - 2).clamp(-127, 127)
    e = torch.where(top > 0, e, torch.full_like(e, -127))
    a = torch.ldexp(v.abs(), -e)
    # the grid's step is 0.5 up to 2, 1 up to 4, 2 up to 6
    index = torch.where(a < 2, (2 * a).round(), torch.where(a < 4, a.round() + 2, (a / 2).round() + 4))
    index = (index.clamp_max(7) + 8 * torch.signbit(v)).to(torch.uint8).reshape(rows, width // 2, 2)
    return index[:, :, 0] | index[:, :, 1] << 4, (e + 127).to(torch.uint8).reshape(rows, width // 32)


def _dequantise(codes, scales):
    """The fp32 values that codes and scales stand for."""
    pair = torch.stack([codes & 15, codes >> 4], dim=-1)
    v = _levels(codes.device)[pair.int()].reshape(*scales.shape, 32)
    v = torch.ldexp(v, scales.int().unsqueeze(-1) - 127)
    return v.reshape(*codes.shape[:-1], 2 * codes.shape[-1])


def _sigmoid(x):
    return 1 / (1 + (-x).exp())


def _activate(c, act):
    """(rows, 2n) in 32-wide blocks, input then gate, to (rows, n)."""
    pair = c.float().reshape(c.shape[0], -1, 2, 32)
    u, g = pair[:, :, 0], pair[:, :, 1]
    if act == "swiglu":
        y = g * _sigmoid(g) * u
    elif act == "geglu":
        g, u = g.clamp_max(CLAMP), u.clamp(-CLAMP, CLAMP)
        y = g * _sigmoid(ALPHA * g) * (u + OFFSET)
    else:
        y = BETA1 * (g / BETA1).tanh() * _sigmoid(g) * BETA2 * (u / BETA2).tanh()
    return y.reshape(c.shape[0], -1)


def _quant(s):
    codes, scales = _quantise(s["x"])
    return _dequantise(codes, scales).to(s["x"].dtype)


def _glu(s):
    y = _activate(s["c"], s["act"])
    if s["prob_rows"] is not None:
        y = y * s["prob_rows"][:, None]
    return y.to(s["y"].dtype)


def _gemm(s):
    at = 0
    for e, n in enumerate(s["sizes"]):
        if n:
            a = _dequantise(s["a"][at:at + n], s["sfa"][at:at + n])
            b = _dequantise(s["b"][e], s["sfb"][e])
            d = (a @ b.t()) * s["alpha"][e]
            s["d"][at:at + n] = d if s["bias_t"] is None else d + s["bias_t"][e]
        at += n
    return s["d"]


def _weights(s, name, scales, e):
    w = s[name].index_select(0, e)[0]
    return w.float() if s[scales] is None else _dequantise(w, s[scales].index_select(0, e)[0])


def _few(s):
    T, k, E, ids = s["T"], s["k"], s["E"], s["ids"].long()
    x, y = s["x"].float(), torch.zeros(T, s["H"], device=s["x"].device)
    prob = torch.where(ids >= 0, s["prob"], torch.zeros_like(s["prob"]))
    if T * k < E:                                  # choice by choice
        turns = [(t, t + 1, ids[t, j:j + 1].clamp_min(0), prob[t, j].reshape(1))
                 for t in range(T) for j in range(k)]
    else:                                          # every expert on all tokens
        every = torch.arange(E, device=ids.device)
        turns = [(0, T, every[e:e + 1], (prob * (ids == e)).sum(1)) for e in range(E)]
    for a, b, e, w in turns:
        c = x[a:b] @ _weights(s, "w1", "sf1", e).t()
        if s["bias1"] is not None:
            c = c + s["bias1"][e]
        v = _activate(c, s["act"]) @ _weights(s, "w2", "sf2", e).t()
        if s["bias2"] is not None:
            v = v + s["bias2"][e]
        y[a:b] += w[:, None] * v
    return y.to(s["y"].dtype)


PLAIN = {"quant": _quant, "glu": _glu, "gemm": _gemm, "few": _few}


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def run(s):
    if not own:
        return PLAIN[s["op"]](s)
    from moe_grouped_gemm_offset_amd import binding as b
    op = s["op"]
    if op == "quant":
        b.gg_mx4_quant(s["x"], s["codes"], s["scales"])
        b.gg_mx4_dequant(s["codes"], s["scales"], s["values"])
        return s["values"]
    if op == "gemm":
        b.gg_gemm_mx4(s["a"], s["sfa"], s["b"], s["sfb"], s["offsets"], s["d"], alpha=s["alpha"],
                      bias=s["bias_t"], workspace=s["workspace"])
        return s["d"]
    act = {"swiglu": b.GG_DSWIGLU, "geglu": b.GG_DGEGLU, "situ": b.GG_DSITUGLU}[s["act"]]
    if op == "glu":
        b.gg_glu(s["c"], s["y"], prob=s["prob_rows"], act=act)
    else:
        b.gg_moe_few(s["x"], s["ids"], s["prob"], s["w1"], s["w2"], s["y"], sf1=s["sf1"], sf2=s["sf2"],
                     bias1=s["bias1"], bias2=s["bias2"], act=act, workspace=s["workspace"])
    return s["y"]


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "quant":
        n, b = case["rows"] * case["width"], BYTES[case["dtype"]]
        return dict(bytes=2 * n * b + n // 2 + n // 32, flops=4 * n)
    if op == "glu":
        n = case["rows"] * case["n"]
        return dict(bytes=n * (2 * BYTES[case["dtype"]] + BYTES[case["out"]]) + 4 * case["rows"],
                    flops=8 * n)
    if op == "gemm":
        L, K, N, rows = (case[x] for x in ("L", "K", "N", "rows"))
        # the weights of the groups that have rows, each counted as one that may
        used = min(L, rows)
        return dict(bytes=(rows + used * N) * (K // 2 + K // 32) + rows * N * BYTES[case["out"]],
                    flops=2 * rows * N * K)
    T, E, H, I = (case[x] for x in ("T", "E", "H", "I"))
    k = min(case["k"], E)
    # experts that T random choices of k reach, on average
    used = E * (1 - (1 - k / E) ** (T * (1 - case["masked"])))
    each = 3 * H * I * (2.0 if case["weights"] == "bf16" else 0.5 + 1 / 32)
    return dict(bytes=int(used * each) + T * H * (2 + BYTES[case["out"]]) + 8 * T * k,
                flops=6 * T * k * H * I)


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------

def _decode(codes, scales):
    """E2M1 by its fields: exponent 0 is m / 2, else (1 + m / 2) 2^(exponent - 1)."""
    out = torch.empty(*codes.shape, 2, dtype=torch.float64, device=codes.device)
    for i, nib in enumerate((codes & 15, codes >> 4)):
        m, ex = (nib & 1).double(), (nib >> 1 & 3).double()
        mag = torch.where(ex == 0, m / 2, (1 + m / 2) * torch.exp2(ex - 1))
        out[..., i] = torch.where(nib >= 8, -mag, mag)
    out = out.reshape(*scales.shape, 32) * torch.exp2(scales.double() - 127).unsqueeze(-1)
    return out.reshape(*codes.shape[:-1], 2 * codes.shape[-1])


def _gated(c, act):
    c = c.reshape(c.shape[0], -1, 64)
    u, g = c[..., :32], c[..., 32:]
    if act == "swiglu":
        y = torch.nn.functional.silu(g) * u
    elif act == "geglu":
        gc = torch.minimum(g, torch.full_like(g, CLAMP))
        y = torch.sigmoid(ALPHA * gc) * gc * (u.clamp(min=-CLAMP, max=CLAMP) + OFFSET)
    else:
        y = (BETA1 * torch.tanh(g / BETA1) * torch.sigmoid(g)) * (BETA2 * torch.tanh(u / BETA2))
    return y.reshape(c.shape[0], -1)


def exact(case, seed):
    op, s = case["op"], prepare(case, seed)
    f = torch.float64
    if op == "quant":
        out = torch.empty(case["rows"], case["width"], dtype=f, device="cuda")
        # a magnitude lies between two levels: the nearer, of two as near the even one
        level = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=f, device="cuda")
        middle = (level[1:] + level[:-1]) / 2
        for a in range(0, case["rows"], 8192):
            v = s["x"][a:a + 8192].to(f)
            v = v.reshape(v.shape[0], -1, 32)
            top = v.abs().amax(2, keepdim=True)
            e = torch.floor(torch.log2(top.clamp_min(1e-30))) - 3
            for _ in range(2):                     # up until 6 * 2^e reaches top
                e = torch.where(6 * torch.exp2(e) < top, e + 1, e)
            unit = torch.exp2(e)
            r = (v.abs() / unit).contiguous()
            up, down = torch.bucketize(r, middle, right=True), torch.bucketize(r, middle)
            code = torch.where(up % 2 == 0, up, down)
            q = torch.where(top > 0, level[code] * unit, torch.zeros_like(r))
            out[a:a + 8192] = torch.copysign(q, v).reshape(v.shape[0], -1)
        return out
    if op == "glu":
        out = torch.empty(case["rows"], case["n"], dtype=f, device="cuda")
        for a in range(0, case["rows"], 8192):
            out[a:a + 8192] = _gated(s["c"][a:a + 8192].to(f), case["act"])
        return out if s["prob_rows"] is None else out * s["prob_rows"].to(f)[:, None]
    if op == "gemm":
        d, begin = torch.zeros(s["d"].shape, dtype=f, device="cuda"), 0
        for e, end in enumerate(s["offsets"].tolist()):
            if end > begin:
                rows = slice(begin, end)
                d[rows] = s["alpha"][e].to(f) * torch.mm(
                    _decode(s["a"][rows], s["sfa"][rows]), _decode(s["b"][e], s["sfb"][e]).T)
                if case["bias"]:
                    d[rows] += s["bias_t"][e].to(f)
            begin = end
        return d
    y = torch.zeros(case["T"], case["H"], dtype=f, device="cuda")
    for e in sorted(set(s["ids"].flatten().tolist()) - {-1}):
        t, j = (s["ids"] == e).nonzero(as_tuple=True)
        w1, w2 = ((s[n][e].to(f) if s[q] is None else _decode(s[n][e], s[q][e]))
                  for n, q in (("w1", "sf1"), ("w2", "sf2")))
        c = torch.mm(s["x"][t].to(f), w1.T)
        if case["bias"]:
            c += s["bias1"][e].to(f)
        v = torch.mm(_gated(c, case["act"]), w2.T)
        if case["bias"]:
            v += s["bias2"][e].to(f)
        y.index_add_(0, t, v * s["prob"][t, j].to(f)[:, None])
    return y
