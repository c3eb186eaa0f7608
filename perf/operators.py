"""What the routing, dispatch and gradient-clipping operators are measured on.

`run` computes each operator either in elementary torch operations (`own`
False) or with the package's entry points (`own` True); both take what
`prepare` holds.  `exact` gives the same outputs from the definitions in 64
bits.

The operators, for T tokens, E experts and k choices a token:

  route        logits (T, E) -> the k largest of logit + bias per token
               (`ids`, -1 where fewer than k are above -inf), their weights
               (softmax or sigmoid, divided by their sum if `normalize`,
               times `scale`), tokens per expert, routed tokens N and the
               balance loss E sum_e (counts_e / (k N)) (sum_t p_te / N)
  route_bwd    the gradient of the logits, from the gradient of the weights
               (given by row of the dispatched layout) and of the loss
  dispatch     ids -> group ends in multiples of `granule`, the row of every
               (token, choice) in the expert-sorted layout, and the tokens
               copied there, zeros in the padding
  combine      out[t] = sum_j w[t, j] y[row(t, j)]
  combine_bwd  dy[row(t, j)] = w[t, j] dout[t], dw[t, j] = <dout[t], y[row]>
  clip         the 2-norm over many tensors, each scaled by
               min(1, max_norm / (norm + 1e-6))

Token counts and widths are those of the library's workloads: 65536 rows of
64 experts at hidden 4096 are 8192 tokens with 8 choices each, 65536 rows of
16 experts at 7168 are 32768 tokens with 2.
"""
import math

import torch

own = False

INF = float("inf")
EPS = 1e-6          # added to the norm in the clip factor
TINY = 1e-20        # added to sums of sigmoids
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def listed():
    return [
        # routing a few tokens of a decode step: launch latency
        dict(name="route_few", op="route", T=5, E=256, k=8, dtype="bf16", score="sigmoid",
             normalize=True, bias=True, masked=0.0),
        # a training batch over many experts, some tokens padding (every logit masked)
        dict(name="route_batch", op="route", T=65536, E=256, k=8, dtype="bf16", score="sigmoid",
             normalize=True, bias=True, masked=0.02),
        # 64 experts, fp32 logits, plain softmax weights
        dict(name="route_bwd_odd", op="route_bwd", T=8191, E=61, k=6, dtype="f32", score="softmax",
             normalize=False, bias=False, masked=0.02),
        # the gradient of the large batch
        dict(name="route_bwd_batch", op="route_bwd", T=65536, E=256, k=8, dtype="bf16",
             score="softmax", normalize=True, bias=True, masked=0.02),
        # a handful of tokens in a compact layout
        dict(name="dispatch_few", op="dispatch", T=7, E=64, k=8, H=4096, dtype="bf16", granule=8,
             skew=0.0),
        # the 64-expert workload's rows, Zipf-skewed over the experts
        dict(name="dispatch_batch", op="dispatch", T=8192, E=64, k=8, H=4096, dtype="bf16",
             granule=256, skew=1.2),
        # odd width, no weights: the gradient of a dispatch
        dict(name="combine_odd", op="combine", T=1001, E=8, k=3, H=2047, dtype="f32", granule=256,
             skew=0.0, weights=False),
        # the 64-expert workload's rows, weighted
        dict(name="combine_batch", op="combine", T=8192, E=64, k=8, H=4096, dtype="bf16",
             granule=256, skew=1.2, weights=True),
        # a small fp16 micro-batch
        dict(name="combine_bwd_small", op="combine_bwd", T=515, E=32, k=4, H=4096, dtype="f16",
             granule=256, skew=0.0, weights=True),
        # 16 experts, two choices, the widest rows
        dict(name="combine_bwd_wide", op="combine_bwd", T=32768, E=16, k=2, H=7168, dtype="bf16",
             granule=256, skew=0.0, weights=True),
        # the many small tensors beside the experts: norms, biases, routers, mixed types
        dict(name="clip_small", op="clip", shape="mixed", n=96, size=20000, dtype="mixed",
             max_norm=1.0),
        # the 64 experts' weight gradients, (4096, 2048) each
        dict(name="clip_experts", op="clip", shape="even", n=64, size=4096 * 2048, dtype="bf16",
             max_norm=1.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route_bwd", "dispatch", "combine", "combine_bwd", "clip"])
    if op in ("route", "route_bwd"):
        E = rng.choice([8, 16, 32, 61, 64, 96, 128, 160, 200, 256])
        return dict(op=op, T=_log_int(rng, 1, 65536), E=E, k=rng.randint(1, min(E, 10)),
                    dtype=rng.choice(["bf16", "f16", "f32"]),
                    score=rng.choice(["softmax", "sigmoid"]), normalize=rng.random() < 0.5,
                    bias=rng.random() < 0.5, masked=rng.choice([0.0, 0.02, 0.2]))
    if op == "clip":
        n = _log_int(rng, 1, 300)
        return dict(op=op, shape=rng.choice(["even", "mixed"]), n=n,
                    size=_log_int(rng, 16, min(1 << 22, (1 << 28) // n)),
                    dtype=rng.choice(["bf16", "f16", "f32", "mixed"]),
                    max_norm=rng.choice([0.5, 1.0, 1e6]))
    E = rng.choice([8, 16, 32, 60, 64, 128])
    k = rng.randint(1, 8)
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    H = rng.choice([2048, 2880, 4096, 5000, 7168, rng.randint(64, 7168)])
    T = _log_int(rng, 1, max(2, 230_000_000 // (k * H)))
    return dict(op=op, T=T, E=E, k=k, H=H, dtype=dtype, granule=rng.choice([1, 8, 256, 256]),
                skew=rng.choice([0.0, 0.6, 1.2]), **({} if op == "dispatch" else
                dict(weights=op == "combine_bwd" or rng.random() < 0.6)))


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _rows_bound(T, E, k, granule):
    """Rows that hold T k choices over E groups, whatever the choices are."""
    n = T * k
    return (n + (granule - 1) * min(E, n)) // granule * granule


def _clip_sizes(case):
    """Element counts of the tensors: all alike, or from nothing to four
    times the mean, odd ones among them."""
    if case["shape"] == "even":
        return [case["size"]] * case["n"]
    return [case["size"] * (i * 37 % 101) // 25 + i % 3 for i in range(case["n"])]


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    op, s = case["op"], dict(case)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    if op == "clip":
        sizes = _clip_sizes(case)
        kinds = [case["dtype"] if case["dtype"] != "mixed" else ("bf16", "f32", "f16")[i % 3]
                 for i in range(case["n"])]
        # gradients of the magnitude that makes the norm a few times max_norm = 1
        std = 3.0 / math.sqrt(max(1, sum(sizes)))
        s["grads"] = [(normal(n) * std).to(DTYPES[d]) for n, d in zip(sizes, kinds)]
        # the clipped values go end to end into one flat buffer of each type
        flat, s["out"], at = {}, [], {}
        for d in sorted(set(kinds)):
            flat[d] = torch.zeros(sum(n for n, e in zip(sizes, kinds) if e == d), dtype=DTYPES[d], device=dev)
        for n, d in zip(sizes, kinds):
            s["out"].append(flat[d][at.get(d, 0):at.get(d, 0) + n])
            at[d] = at.get(d, 0) + n
        s["flat"] = list(flat.values())
        code = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
        s["ptrs"] = torch.tensor([t.data_ptr() for t in s["grads"]], dtype=torch.int64, device=dev)
        s["out_ptrs"] = torch.tensor([t.data_ptr() for t in s["out"]], dtype=torch.int64, device=dev)
        s["ends"] = torch.tensor(sizes, dtype=torch.int64).cumsum(0).to(dev)
        s["dtypes"] = torch.tensor([code[t.dtype] for t in s["grads"]], dtype=torch.int32, device=dev)
        s["total"] = sum(sizes)
        s["sumsq"] = torch.zeros(1, dtype=torch.float64, device=dev)
        s["norm"] = torch.zeros(2, dtype=torch.float32, device=dev)
        s["workspace"] = torch.zeros(1 << 16, dtype=torch.uint8, device=dev)
        return s

    T, E, k = case["T"], case["E"], case["k"]
    if op in ("route", "route_bwd"):
        # some experts are liked more than others
        logits = 1.5 * normal(T, E) + 0.5 * normal(1, E)
        drop = torch.rand(T, generator=g, device=dev) < case["masked"]
        few = torch.rand(T, E, generator=g, device=dev) < case["masked"]
        logits = torch.where(drop[:, None] | few, torch.full_like(logits, -INF), logits)
        s["logits"] = logits.to(DTYPES[case["dtype"]])
        s["bias_t"] = 0.2 * normal(E) if case["bias"] else None
        s["scale"] = 2.5 if case["score"] == "sigmoid" else 1.0
        s["workspace"] = torch.zeros(1 << 24, dtype=torch.uint8, device=dev)
        if op == "route":
            s["ids"] = torch.zeros(T, k, dtype=torch.int32, device=dev)
            s["prob"] = torch.zeros(T, k, device=dev)
            s["counts"] = torch.zeros(E, dtype=torch.int32, device=dev)
            s["routed"] = torch.zeros(1, dtype=torch.int32, device=dev)
            s["balance"] = torch.zeros(1, device=dev)
            return s
        s["ids"], _, s["counts"], s["routed"], _ = _route(s)
        s["rows"] = _rows_bound(T, E, k, 256)
        s["row_of"] = _plan(s["ids"], E, 256)[2]
        s["dprob_rows"] = normal(s["rows"]) / max(1, T)
        s["dbalance"] = torch.full((1,), 0.01, device=dev)
        s["dlogits"] = torch.zeros_like(s["logits"])
        return s

    H, dt = case["H"], DTYPES[case["dtype"]]
    like = -case["skew"] * torch.arange(1, E + 1, device=dev, dtype=torch.float32).log()
    like = like[torch.randperm(E, generator=g, device=dev)]
    noise = -(-torch.rand(T, E, generator=g, device=dev).clamp_min(1e-7).log()).log()
    k = min(k, E)
    s["ids"] = (like + noise).topk(k, dim=1).indices.to(torch.int32)
    s["rows"] = _rows_bound(T, E, k, case["granule"])
    w = torch.softmax(normal(T, k), dim=1)
    if op == "dispatch":
        s["prob"] = w
        s["x"] = normal(T, H).to(dt)
        s["counts"] = torch.zeros(E, dtype=torch.int32, device=dev)
        s["ends"] = torch.zeros(E, dtype=torch.int32, device=dev)
        s["row_of"] = torch.zeros(T, k, dtype=torch.int32, device=dev)
        s["prob_rows"] = torch.zeros(s["rows"], device=dev)
        s["x_rows"] = torch.zeros(s["rows"], H, dtype=dt, device=dev)
        s["workspace"] = torch.zeros(1 << 24, dtype=torch.uint8, device=dev)
        return s
    s["counts"], s["ends"], s["row_of"] = _plan(s["ids"], E, case["granule"])
    s["w"] = w if case["weights"] else None
    s["y_rows"] = torch.zeros(s["rows"], H, dtype=dt, device=dev)
    s["y_rows"][s["row_of"].flatten().long()] = normal(T * k, H).to(dt)
    if op == "combine":
        s["out"] = torch.zeros(T, H, dtype=dt, device=dev)
        return s
    s["dout"] = normal(T, H).to(dt)
    s["dy_rows"] = torch.zeros(s["rows"], H, dtype=dt, device=dev)
    s["dw"] = torch.zeros(T, k, device=dev)
    return s


# --------------------------------------------------------------------------
# the plain forms
# --------------------------------------------------------------------------

def _scores(s):
    """fp32 logits, the scores (softmax or sigmoid) and the probabilities of
    the balance loss (the scores over their sum), 0 in rows without a finite
    logit."""
    x = s["logits"].float()
    if s["score"] == "softmax":
        top = x.max(1, keepdim=True).values
        e = (x - torch.where(top > -INF, top, torch.zeros_like(top))).exp()
        p = e / e.sum(1, keepdim=True).clamp_min(TINY)
        return x, p, p
    sig = 1 / (1 + (-x).exp())
    return x, sig, sig / (sig.sum(1, keepdim=True) + TINY)


def _weights(s, x, score, ids):
    """(T, k) weights before `scale` of the chosen experts."""
    safe, there = ids.clamp_min(0).long(), ids >= 0
    if s["score"] == "softmax" and s["normalize"]:
        v = torch.where(there, x.gather(1, safe), torch.full_like(x[:, :1], -INF))
        top = v.max(1, keepdim=True).values
        e = (v - torch.where(top > -INF, top, torch.zeros_like(top))).exp()
        return e / e.sum(1, keepdim=True).clamp_min(TINY)
    w = torch.where(there, score.gather(1, safe), torch.zeros_like(x[:, :1]))
    return w / (w.sum(1, keepdim=True) + TINY) if s["normalize"] else w


def _route(s):
    T, E, k = s["T"], s["E"], s["k"]
    x, score, p = _scores(s)
    key = x if s["bias_t"] is None else x + s["bias_t"]
    order = key.sort(dim=1, descending=True, stable=True)
    there = order.values[:, :k] > -INF
    ids = torch.where(there, order.indices[:, :k], -torch.ones_like(order.indices[:, :k]))
    prob = s["scale"] * _weights(s, x, score, ids)
    counts = torch.zeros(E + 1, dtype=torch.int64, device=x.device)
    counts.scatter_add_(0, torch.where(there, ids, torch.full_like(ids, E)).flatten(),
                        torch.ones_like(ids).flatten())
    counts = counts[:E]
    routed = (ids[:, 0] >= 0).sum()
    n = routed.clamp_min(1).float()
    balance = E * ((counts.float() / (k * n)) * (p.sum(0) / n)).sum()
    return (ids.to(torch.int32), prob, counts.to(torch.int32), routed.to(torch.int32).reshape(1),
            balance.reshape(1))


def _route_bwd(s):
    E, k, ids = s["E"], s["k"], s["ids"]
    x, score, p = _scores(s)
    there, safe = ids >= 0, ids.clamp_min(0).long()
    row = s["row_of"]
    g = torch.where(there & (row >= 0), s["dprob_rows"][row.clamp_min(0).long()],
                    torch.zeros_like(s["dprob_rows"][:1])) * s["scale"]
    n = s["routed"].clamp_min(1).float()
    c = s["dbalance"] * E * (s["counts"].float() / (k * n)) / n
    soft = s["score"] == "softmax"
    pull = c - (p * c).sum(1, keepdim=True)
    if s["normalize"]:
        q = _weights(s, x, score, ids)
        pick = g - (q * g).sum(1, keepdim=True)
    if soft:
        dx = p * pull
        if s["normalize"]:
            dx = dx.scatter_add(1, safe, torch.where(there, q * pick, torch.zeros_like(q)))
        else:
            at = torch.zeros_like(x).scatter_add(1, safe, torch.where(there, g, torch.zeros_like(g)))
            dx = dx + p * (at - (p * at).sum(1, keepdim=True))
    else:
        ds = pull / (score.sum(1, keepdim=True) + TINY)
        if s["normalize"]:
            chosen = torch.where(there, score.gather(1, safe), torch.zeros_like(g))
            g = pick / (chosen.sum(1, keepdim=True) + TINY)
        ds = ds.scatter_add(1, safe, torch.where(there, g, torch.zeros_like(g)))
        dx = ds * score * (1 - score)
    dx = torch.where(there[:, :1], dx, torch.zeros_like(dx))
    return dx.to(s["logits"].dtype)


def _plan(ids, E, granule):
    """Tokens per expert, ends of the padded groups and the row of every
    (token, choice): within a group the tokens keep their order."""
    T, k = ids.shape
    lanes = torch.arange(E, device=ids.device, dtype=torch.int32)
    chosen = torch.zeros(T, E + 1, dtype=torch.int32, device=ids.device)
    chosen.scatter_(1, torch.where(ids >= 0, ids, torch.full_like(ids, E)).long(), 1)
    before = chosen.cumsum(0, dtype=torch.int32)
    counts = before[-1, :E]
    ends = ((counts + granule - 1) // granule * granule).cumsum(0, dtype=torch.int32)
    begins = torch.where(lanes > 0, ends.roll(1), torch.zeros_like(ends))
    safe = ids.clamp_min(0).long()
    rows = begins[safe] + before.gather(1, safe) - 1
    return counts, ends, torch.where(ids >= 0, rows, -torch.ones_like(rows)).to(torch.int32)


def _dispatch(s):
    counts, ends, row_of = _plan(s["ids"], s["E"], s["granule"])
    at = row_of.flatten().long()
    prob_rows = torch.zeros_like(s["prob_rows"])
    prob_rows[at] = s["prob"].flatten()
    x_rows = torch.zeros_like(s["x_rows"])
    x_rows[at] = s["x"].repeat_interleave(row_of.shape[1], dim=0)
    return counts, ends, row_of, prob_rows, x_rows


def _combine(s):
    y = s["y_rows"][s["row_of"].long()].float()
    if s["w"] is not None:
        y = y * s["w"][:, :, None]
    return y.sum(1).to(s["out"].dtype)


def _combine_bwd(s):
    at = s["row_of"].long()
    d = s["dout"].float()[:, None, :]
    dw = (s["y_rows"][at].float() * d).sum(2)
    dy = torch.zeros_like(s["dy_rows"])
    dy[at] = (s["w"][:, :, None] * d).to(dy.dtype)
    return dy, dw


def _clip(s):
    sums = torch.stack([t.float().square().sum() for t in s["grads"]])
    norm = sums.sum().sqrt()
    factor = (s["max_norm"] / (norm + EPS)).clamp_max(1.0)
    [o.copy_(t.float() * factor) for o, t in zip(s["out"], s["grads"])]
    return s["flat"] + [torch.stack([norm, factor])]


PLAIN = {"route": _route, "route_bwd": _route_bwd, "dispatch": _dispatch, "combine": _combine,
         "combine_bwd": _combine_bwd, "clip": _clip}


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def run(s):
    if not own:
        return PLAIN[s["op"]](s)
    from moe_grouped_gemm_offset_amd import binding as b
    op = s["op"]
    if op in ("route", "route_bwd"):
        kind = dict(score=b.GG_SOFTMAX if s["score"] == "softmax" else b.GG_SIGMOID,
                    scale=s["scale"], flags=b.GG_FLAG_NORMALIZE if s["normalize"] else 0)
        if op == "route":
            b.gg_route(s["logits"], s["ids"], s["prob"], s["counts"], s["routed"], s["balance"],
                       bias=s["bias_t"], workspace=s["workspace"], **kind)
            return s["ids"], s["prob"], s["counts"], s["routed"], s["balance"]
        b.gg_route_bwd(s["logits"], s["ids"], s["counts"], s["routed"], s["dprob_rows"],
                       s["dlogits"], row_of=s["row_of"], dbalance=s["dbalance"], **kind)
        return s["dlogits"]
    if op == "dispatch":
        b.gg_plan(s["ids"], s["counts"], s["ends"], s["row_of"], s["rows"], granule=s["granule"],
                  prob=s["prob"], prob_rows=s["prob_rows"], workspace=s["workspace"])
        b.gg_permute(s["x"], s["row_of"], s["counts"], s["ends"], s["x_rows"])
        return s["counts"], s["ends"], s["row_of"], s["prob_rows"], s["x_rows"]
    if op == "combine":
        b.gg_combine(s["y_rows"], s["row_of"], s["out"], weights=s["w"])
        return s["out"]
    if op == "combine_bwd":
        b.gg_combine_bwd(s["dout"], s["y_rows"], s["row_of"], s["w"], s["counts"], s["ends"],
                         s["dy_rows"], s["dw"])
        return s["dy_rows"], s["dw"]
    b.gg_grad_norm(s["ptrs"], s["ends"], s["dtypes"], s["total"], s["sumsq"],
                   workspace=s["workspace"])
    b.gg_grad_clip(s["ptrs"], s["ends"], s["dtypes"], s["total"], s["sumsq"], s["max_norm"],
                   s["norm"], eps=EPS, out_ptrs=s["out_ptrs"])
    return s["flat"] + [s["norm"]]


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "clip":
        sizes = _clip_sizes(case)
        each = [BYTES[case["dtype"] if case["dtype"] != "mixed" else ("bf16", "f32", "f16")[i % 3]]
                for i in range(case["n"])]
        moved = sum(n * b for n, b in zip(sizes, each))
        # read once for the norm and the scaled values, written once
        return dict(bytes=2 * moved, flops=3 * sum(sizes))
    T, E = case["T"], case["E"]
    k, b = min(case["k"], E), BYTES[case["dtype"]]
    if op == "route":
        return dict(bytes=T * E * b + 8 * T * k + 8 * E, flops=T * E * (6 + k))
    if op == "route_bwd":
        return dict(bytes=2 * T * E * b + 12 * T * k + 4 * E, flops=T * E * 12)
    H, n = case["H"], T * k
    if op == "dispatch":
        return dict(bytes=(T + n) * H * b + 16 * n, flops=n)
    if op == "combine":
        return dict(bytes=(T + n) * H * b + 8 * n, flops=2 * n * H)
    return dict(bytes=(T + 2 * n) * H * b + 12 * n, flops=3 * n * H)


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------

def exact(case, seed):
    op = case["op"]
    if op == "dispatch":
        return None                  # copies and whole numbers
    s = prepare(case, seed)
    f = torch.float64
    if op == "clip":
        total = torch.zeros((), dtype=f, device="cuda")
        for t in s["grads"]:
            total = total + torch.dot(t.to(f), t.to(f))
        norm = total ** 0.5
        factor = torch.minimum(torch.ones_like(norm), s["max_norm"] / (norm + EPS))
        flat = [torch.cat([t.to(f) * factor for t in s["grads"] if t.dtype == o.dtype])
                for o in s["flat"]]
        return flat + [torch.cat([norm[None], factor[None]])]
    if op == "combine":
        T, k = s["row_of"].shape
        total = torch.zeros(T, s["H"], dtype=f, device="cuda")
        for j in range(k):
            part = s["y_rows"][s["row_of"][:, j].long()].to(f)
            total += part if s["w"] is None else part * s["w"][:, j:j + 1].to(f)
        return total
    if op == "combine_bwd":
        T, k = s["row_of"].shape
        dy = torch.zeros(s["rows"], s["H"], dtype=f, device="cuda")
        dw = torch.zeros(T, k, dtype=f, device="cuda")
        d = s["dout"].to(f)
        for j in range(k):
            r = s["row_of"][:, j].long()
            dy[r] = d * s["w"][:, j:j + 1].to(f)
            dw[:, j] = torch.linalg.vecdot(s["y_rows"][r].to(f), d)
        return dy, dw

    T, E, k = s["T"], s["E"], s["k"]
    x = s["logits"].to(f)
    live = x > -INF
    some = live.any(1)
    if s["score"] == "softmax":
        z = torch.nan_to_num(torch.logsumexp(x, 1), neginf=0.0)
        a = p = torch.exp(x - z[:, None])
    else:
        a = torch.sigmoid(x)
        p = a / (a.sum(1)[:, None] + TINY)
    if op == "route":
        # the choice goes by the sum rounded to 32 bits; ties to the lower index
        key = (s["logits"].float() + s["bias_t"] if case["bias"] else s["logits"].float()).to(f)
        left = key.clone()
        ids = torch.full((T, k), -1, dtype=torch.int64, device="cuda")
        at = torch.arange(E, device="cuda").expand(T, E)
        for j in range(k):
            best = left.amax(1, keepdim=True)
            first = torch.where(left == best, at, E).amin(1)
            got = best[:, 0] > -INF
            ids[:, j] = torch.where(got, first, -1)
            left.scatter_(1, first[:, None], -INF)
    else:
        ids = s["ids"].long()
    on = torch.zeros(T, E, dtype=f, device="cuda")
    for j in range(k):
        on.scatter_add_(1, ids[:, j:j + 1].clamp_min(0), (ids[:, j:j + 1] >= 0).to(f))
    if s["normalize"]:
        if s["score"] == "softmax":
            zc = torch.nan_to_num(torch.logsumexp(torch.where(on > 0, x, -INF), 1), neginf=0.0)
            w = torch.where(on > 0, torch.exp(x - zc[:, None]), 0.0)
        else:
            w = on * a / ((on * a).sum(1)[:, None] + TINY)
    else:
        w = on * a
    n_e, n = on.sum(0), some.sum().clamp_min(1).to(f)
    if op == "route":
        prob = torch.where(ids >= 0, s["scale"] * w.gather(1, ids.clamp_min(0)), 0.0)
        loss = E / (k * n * n) * torch.dot(n_e, p.sum(0))
        return ids.to(torch.int32), prob, n_e.to(torch.int32), some.sum().to(torch.int32)[None], loss[None]

    # by the chain rule, for the whole row at once: gw the gradient of the
    # weights, gp that of the balance probabilities
    gw = torch.zeros(T, E, dtype=f, device="cuda")
    for j in range(k):
        r = s["row_of"][:, j].long()
        ok = (ids[:, j] >= 0) & (r >= 0)
        val = torch.where(ok, s["scale"] * s["dprob_rows"].to(f)[r.clamp_min(0)], 0.0)
        gw.scatter_add_(1, ids[:, j:j + 1].clamp_min(0), val[:, None])
    gp = (s["dbalance"].to(f) * E / (k * n * n) * n_e).expand(T, E)
    if s["score"] == "softmax":
        dx = p * gp - p * (p * gp).sum(1)[:, None]
        dx = dx + w * gw - (w if s["normalize"] else a) * (w * gw).sum(1)[:, None]
    else:
        da = (gp - (p * gp).sum(1)[:, None]) / (a.sum(1)[:, None] + TINY)
        if s["normalize"]:
            da = da + on * (gw - (w * gw).sum(1)[:, None]) / ((on * a).sum(1)[:, None] + TINY)
        else:
            da = da + gw
        dx = da * a * (1 - a)
    return torch.where(some[:, None], dx, 0.0)
