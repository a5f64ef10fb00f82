"""Cases of the vocabulary-side operators: token scoring with its gradient, the 4-bit head, the embedding with its
gradient.

``run`` computes each operator in its plain form (elementary torch operations in 32 bits, rounded once), or, with
``own`` set, through the library's entry points. ``exact`` gives the same outputs in 64 bits.
"""
import math

import torch

own = False

IGNORE = -100   # a row (or token) that is not scored and gets no gradient

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "bf16": 2}

# no case is larger than the largest listed ones
MOST_LOGITS = 2048 * 151936
MOST_WEIGHTS = 4096 * 151936
MOST_PRODUCTS = 24 * 2560 * 151936


def listed():
    return [
        # one decode step of four requests under a grammar: half of the vocabulary masked, rows padded to an odd stride
        dict(name="score step", kind="score", B=4, V=32000, pad=7, dtype="f32", n_alt=5, masked=True, ignored=0,
             temps=True),
        # a full serving batch that returns the 20 most probable alternatives per token
        dict(name="score batch", kind="score", B=256, V=151936, pad=0, dtype="bf16", n_alt=20, masked=False, ignored=0,
             temps=True),
        # a training micro-batch: log-probability and entropy of every target, a quarter of the rows are prompt
        dict(name="score train", kind="score", B=2048, V=151936, pad=0, dtype="bf16", n_alt=0, masked=False,
             ignored=512, temps=False),
        # gradient of a short masked answer, rows of an odd length
        dict(name="score grad odd", kind="score_grad", B=33, V=100003, pad=0, dtype="f32", masked=True, ignored=3,
             temps=True),
        # gradient of the training micro-batch
        dict(name="score grad train", kind="score_grad", B=2048, V=151936, pad=0, dtype="bf16", masked=False,
             ignored=512, temps=False),
        # single-token decode of a small model
        dict(name="head one small", kind="head", M=1, V=32000, D=2048, group=64, zeros=False, scales="bf16",
             dtype="bf16", out="f32"),
        # single-token decode of a large model
        dict(name="head one large", kind="head", M=1, V=151936, D=4096, group=128, zeros=False, scales="bf16",
             dtype="bf16", out="bf16"),
        # a batch of 24 sequences (an odd number of column tiles), small groups with zero points
        dict(name="head batch", kind="head", M=24, V=151936, D=2560, group=32, zeros=True, scales="bf16",
             dtype="bf16", out="f32"),
        # the drawn tokens of one decode step become the next step's inputs
        dict(name="embed step", kind="embed", N=4, V=32000, D=2048, dtype="bf16", out="bf16"),
        # the tokens of several packed prompts
        dict(name="embed prompt", kind="embed", N=16384, V=151936, D=4096, dtype="bf16", out="bf16"),
        # a short sequence added to the tied head's gradient, an odd number of tokens, rows of an odd length
        dict(name="embed grad odd", kind="embed_grad", N=509, V=32000, D=1001, dtype="f32", out="f32",
             accumulate=True, ignored=5),
        # the gradient of a training micro-batch, written whole
        dict(name="embed grad train", kind="embed_grad", N=16384, V=151936, D=4096, dtype="bf16", out="bf16",
             accumulate=False, ignored=0),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _plain_size(n):
    return n + 1 if n == 3072 else n


def draw(rng):
    kind = rng.choice(["score", "score", "score_grad", "head", "head", "embed", "embed_grad"])
    V = _plain_size(_log_uniform(rng, 1000, 262144))
    if kind in ("score", "score_grad"):
        dtype = rng.choice(["f32", "bf16"])
        B = _plain_size(_log_uniform(rng, 1, max(1, min(4096, MOST_LOGITS * 2 // (V * BYTES[dtype])))))
        c = dict(kind=kind, B=B, V=V, pad=rng.choice([0, 0, 1, 8, 13]), dtype=dtype, masked=rng.random() < 0.4,
                 ignored=rng.choice([0, 0, B // 4]), temps=rng.random() < 0.5)
        if kind == "score":
            c["n_alt"] = rng.choice([0, 1, 5, 20, 64])
        return c
    if kind == "head":
        group = rng.choice([32, 64, 128])
        D = group * _log_uniform(rng, max(1, 256 // group), 8192 // group)
        D = D + group if D == 3072 else D
        V = min(V, MOST_WEIGHTS // D)
        M = min(_log_uniform(rng, 1, 64), max(1, MOST_PRODUCTS // (V * D)))
        return dict(kind=kind, M=M, V=_plain_size(V), D=D, group=group, zeros=rng.random() < 0.5,
                    scales=rng.choice(["bf16", "bf16", "f32"]), dtype=rng.choice(["bf16", "bf16", "f32"]),
                    out=rng.choice(["f32", "bf16"]))
    D = _plain_size(_log_uniform(rng, 64, 8192))
    V = _plain_size(min(V, MOST_WEIGHTS // D))
    N = _plain_size(_log_uniform(rng, 1, max(1, min(65536, 16384 * 4096 // D))))
    c = dict(kind=kind, N=N, V=V, D=D, dtype=rng.choice(["f32", "bf16"]), out=rng.choice(["f32", "bf16"]))
    if V * D * BYTES[c["out"]] > MOST_WEIGHTS * 2 or N * D * BYTES[c["dtype"]] > 16384 * 4096 * 2:
        c["out"] = c["dtype"] = "bf16"
    if kind == "embed_grad":
        c["accumulate"] = rng.random() < 0.5
        c["ignored"] = rng.choice([0, N // 5])
        if c["accumulate"]:
            c["out"] = "f32"
            c["V"] = _plain_size(min(V, MOST_WEIGHTS // (2 * D)))
    return c


def _tokens(n, V, gen, dev):
    """Token ids with the frequencies of text: rank r about in proportion to 1 / r, ids scattered over the table."""
    u = torch.rand(n, generator=gen, device=dev, dtype=torch.float64)
    r = torch.exp(u * math.log(V)).long().clamp_(1, V) - 1
    return ((r * 7919 + 13) % V).to(torch.int32)


def _ignore(token, count, gen, dev):
    if count:
        token[torch.randperm(token.numel(), generator=gen, device=dev)[:count]] = IGNORE
    return token


def _score_inputs(case, gen, dev):
    B, V, ld = case["B"], case["V"], case["V"] + case["pad"]
    x = torch.randn((B, ld), generator=gen, device=dev).mul_(2.5)
    rows = torch.arange(B, device=dev)
    token = torch.randint(0, V, (B,), generator=gen, device=dev)
    # most given tokens are likely ones: raised by up to 16
    x[rows, token] += torch.rand(B, generator=gen, device=dev) * 16
    if case["masked"]:
        # a grammar allows half of the tokens, the given one among them
        hide = torch.rand((1, ld), generator=gen, device=dev) < 0.5
        keep = x[rows, token].clone()
        x.masked_fill_(hide, -math.inf)
        x[rows, token] = keep
    s = {"logits": x.to(DTYPES[case["dtype"]])[:, :V], "token": _ignore(token.to(torch.int32), case["ignored"], gen, dev)}
    s["temperature"] = torch.rand(B, generator=gen, device=dev) + 0.5 if case["temps"] else None
    return s


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    kind = case["kind"]
    s = {"case": dict(case)}
    if kind in ("score", "score_grad"):
        s.update(_score_inputs(case, gen, dev))
        B, V = case["B"], case["V"]
        if kind == "score":
            n = case["n_alt"]
            s["out"] = {"logprob": torch.empty(B, device=dev), "entropy": torch.empty(B, device=dev),
                        "rank": torch.empty(B, dtype=torch.int32, device=dev),
                        "row_max": torch.empty(B, device=dev), "row_logsum": torch.empty(B, device=dev)}
            if n:
                s["out"]["alt_idx"] = torch.empty((B, n), dtype=torch.int32, device=dev)
                s["out"]["alt_lp"] = torch.empty((B, n), device=dev)
            s["row_status"] = torch.empty(B, dtype=torch.int32, device=dev)
        else:
            # what the forward pass kept, and the gradients that the loss gives
            m, logsum, entropy = _row_stats(s["logits"], s["temperature"], torch.float64)
            s["row_max"], s["row_logsum"], s["entropy"] = m.float(), logsum.float(), entropy.float()
            s["dlogprob"] = -torch.rand(B, generator=gen, device=dev) / B
            s["dentropy"] = -0.01 * torch.rand(B, generator=gen, device=dev) / B
            s["out"] = torch.empty((B, V), dtype=DTYPES[case["dtype"]], device=dev)
            s["row_status"] = torch.empty(B, dtype=torch.int32, device=dev)
    elif kind == "head":
        M, V, D, G = case["M"], case["V"], case["D"], case["group"]
        q = torch.randn((V, D), generator=gen, device=dev).mul_(2.6).add_(8).round_().clamp_(0, 15).to(torch.uint8)
        s["codes"] = q[:, 0::2] | (q[:, 1::2] << 4)
        s["scales"] = (torch.rand((V, D // G), generator=gen, device=dev) * 0.02 + 0.002).to(DTYPES[case["scales"]])
        s["zeros"] = None
        if case["zeros"]:
            s["zeros"] = torch.randint(4, 12, (V, D // G), generator=gen, device=dev).to(torch.uint8)
        s["hidden"] = torch.randn((M, D), generator=gen, device=dev).to(DTYPES[case["dtype"]])
        s["out"] = torch.empty((M, V), dtype=DTYPES[case["out"]], device=dev)
        if own:
            # a server lays its weights out once, when it loads them
            import top_sampling_gb300 as ts
            s["head"] = ts.vsamp_head_pack(s["codes"], s["scales"], zeros=s["zeros"], group=G)
    else:
        N, V, D = case["N"], case["V"], case["D"]
        s["token"] = _ignore(_tokens(N, V, gen, dev), case.get("ignored", 0), gen, dev)
        s["scale"] = math.sqrt(D)
        if kind == "embed":
            s["table"] = torch.randn((V, D), generator=gen, device=dev).mul_(0.02).to(DTYPES[case["dtype"]])
            s["out"] = torch.empty((N, D), dtype=DTYPES[case["out"]], device=dev)
            s["row_status"] = torch.empty(N, dtype=torch.int32, device=dev)
        else:
            s["dout"] = torch.randn((N, D), generator=gen, device=dev).to(DTYPES[case["dtype"]])
            if case["accumulate"]:
                s["out"] = torch.randn((V, D), generator=gen, device=dev).to(DTYPES[case["out"]])
            else:
                s["out"] = torch.empty((V, D), dtype=DTYPES[case["out"]], device=dev)
    return s


def _scaled(logits, temperature, kind):
    x = logits.to(kind)
    m = x.amax(dim=1)
    sc = x - m[:, None]
    if temperature is not None:
        sc = sc / temperature.to(kind)[:, None]
    return x, m, sc


def _row_stats(logits, temperature, kind):
    _, m, sc = _scaled(logits, temperature, kind)
    e = torch.exp(sc)
    total = e.sum(dim=1)
    logsum = torch.log(total)
    first = torch.where(e > 0, e * sc, torch.zeros((), dtype=kind, device=e.device)).sum(dim=1)
    return m, logsum, logsum - first / total


def _order_key(x):
    """Whole numbers in the order of the fp32 values, -0 equal to +0."""
    b = (x + 0.0).view(torch.int32).long()
    return torch.where(b < 0, -(b & 0x7FFFFFFF), b)


def _run_score(s):
    case, token = s["case"], s["token"].long()
    x, m, sc = _scaled(s["logits"], s["temperature"], torch.float32)
    B, V = x.shape
    ignored = token == IGNORE
    t = torch.where(ignored, 0, token)
    e = torch.exp(sc)
    total = e.sum(dim=1)
    logsum = torch.log(total)
    first = torch.where(e > 0, e * sc, 0.0).sum(dim=1)
    lp = (sc.gather(1, t[:, None])[:, 0] - logsum).clamp(max=0)
    xt = x.gather(1, t[:, None])
    at = torch.arange(V, device=x.device)[None, :]
    rank = ((x > xt) | ((x == xt) & (at < t[:, None]))).sum(dim=1)
    zero = torch.zeros_like(m)
    out = {"logprob": torch.where(ignored, zero, lp), "entropy": torch.where(ignored, zero, logsum - first / total),
           "rank": torch.where(ignored, -1, rank).int(), "row_max": torch.where(ignored, zero, m),
           "row_logsum": torch.where(ignored, zero, logsum)}
    n = case["n_alt"]
    if n:
        key = _order_key(x) * (1 << 32) + ((1 << 32) - 1 - at)
        best = torch.topk(key, n, dim=1, sorted=True)[1]
        got = (x.gather(1, best) > -math.inf) & ~ignored[:, None]
        alt = (sc.gather(1, best) - logsum[:, None]).clamp(max=0)
        out["alt_idx"] = torch.where(got, best, -1).int()
        out["alt_lp"] = torch.where(got, alt, math.nan)
    return out


def _run_score_grad(s):
    token = s["token"].long()
    x = s["logits"].float()
    B, V = x.shape
    ignored = token == IGNORE
    t = torch.where(ignored, 0, token)
    inv = 1.0 / s["temperature"][:, None] if s["temperature"] is not None else torch.ones((B, 1), device=x.device)
    lp = (x - s["row_max"][:, None]) * inv - s["row_logsum"][:, None]
    p = torch.exp(lp)
    g, h = s["dlogprob"][:, None], s["dentropy"][:, None]
    d = torch.where(p > 0, -p * (g + h * (lp + s["entropy"][:, None])), 0.0)
    d.scatter_add_(1, t[:, None], g)
    d = torch.where(ignored[:, None], 0.0, d * inv)
    return d.to(s["logits"].dtype)


def _weights(s, kind):
    case = s["case"]
    V, D, G = case["V"], case["D"], case["group"]
    q = torch.stack([s["codes"] & 15, s["codes"] >> 4], dim=2).view(V, D // G, G).to(kind)
    z = s["zeros"].to(kind)[:, :, None] if s["zeros"] is not None else 8.0
    return ((q - z) * s["scales"].to(kind)[:, :, None]).view(V, D)


def run(state):
    s = state
    kind = s["case"]["kind"]
    if own:
        import top_sampling_gb300 as ts
        if kind == "score":
            ts.vsamp_score_tokens(s["logits"], s["token"], temperature=s["temperature"], n_alt=s["case"]["n_alt"],
                                  row_status=s["row_status"], **s["out"])
        elif kind == "score_grad":
            ts.vsamp_score_tokens_backward(s["logits"], s["token"], s["dlogprob"], s["row_max"], s["row_logsum"],
                                           entropy=s["entropy"], dentropy=s["dentropy"],
                                           temperature=s["temperature"], dlogits=s["out"], row_status=s["row_status"])
        elif kind == "head":
            ts.vsamp_head_logits(s["hidden"], s["head"], out=s["out"])
        elif kind == "embed":
            ts.vsamp_embed(s["token"], s["table"], scale=s["scale"], out=s["out"], row_status=s["row_status"])
        else:
            ts.vsamp_embed_backward(s["token"], s["dout"], s["case"]["V"], scale=s["scale"], dtable=s["out"],
                                    accumulate=s["case"]["accumulate"])
        return s["out"]
    if kind == "score":
        return _run_score(s)
    if kind == "score_grad":
        return _run_score_grad(s)
    if kind == "head":
        return torch.matmul(s["hidden"].float(), _weights(s, torch.float32).t()).to(s["out"].dtype)
    ignored = s["token"] == IGNORE
    t = torch.where(ignored, 0, s["token"]).long()
    if kind == "embed":
        rows = s["table"][t].float() * s["scale"]
        return torch.where(ignored[:, None], 0.0, rows).to(s["out"].dtype)
    rows = torch.where(ignored[:, None], 0.0, s["dout"].float() * s["scale"])
    total = torch.zeros(s["out"].shape, device=rows.device).index_add_(0, t, rows)
    if s["case"]["accumulate"]:
        total += s["out"].float()
    return s["out"].copy_(total)


def _distinct(case):
    """Expected number of different tokens among the case's."""
    n, V = case["N"] - case.get("ignored", 0), case["V"]
    r = torch.arange(1, V + 1, dtype=torch.float64)
    p = torch.log((r + 1) / r)
    p = p / p.sum()
    return float((1 - torch.exp(n * torch.log1p(-p.clamp(max=1 - 1e-12)))).sum())


def work(case):
    kind = case["kind"]
    if kind in ("score", "score_grad"):
        B, V, es = case["B"], case["V"], BYTES[case["dtype"]]
        rows = B - case["ignored"]
        per_row = 4 + (4 if case["temps"] else 0)
        if kind == "score":
            # per element: shift, scale, exponential, two sums, maximum, comparison
            return {"bytes": rows * V * es + B * (per_row + 5 * 4 + case["n_alt"] * 8), "flops": 7 * rows * V}
        # per element: shift and scale, exponential, three products and sums
        return {"bytes": rows * V * es + B * V * es + B * (per_row + 5 * 4), "flops": 7 * rows * V}
    if kind == "head":
        M, V, D, G = case["M"], case["V"], case["D"], case["group"]
        weights = V * D // 2 + V * (D // G) * (BYTES[case["scales"]] + (1 if case["zeros"] else 0))
        return {"bytes": weights + M * D * BYTES[case["dtype"]] + M * V * BYTES[case["out"]], "flops": 2 * M * V * D}
    N, V, D, es, eo = case["N"], case["V"], case["D"], BYTES[case["dtype"]], BYTES[case["out"]]
    if kind == "embed":
        return {"bytes": 4 * N + int(_distinct(case)) * D * es + N * D * eo, "flops": N * D}
    rows = N - case["ignored"]
    out = 2 * int(_distinct(case)) * D * eo if case["accumulate"] else V * D * eo
    return {"bytes": 4 * N + rows * D * es + out, "flops": 2 * rows * D}


def _exact_score(s):
    case = s["case"]
    x = s["logits"].double()
    B, V = x.shape
    T = s["temperature"].double()[:, None] if s["temperature"] is not None else 1.0
    z = x / T
    skip = s["token"] == IGNORE
    lse = torch.logsumexp(z, dim=1)
    lps = z - lse[:, None]
    top = x.max(dim=1).values
    h = -torch.nan_to_num(torch.exp(lps) * lps, nan=0.0).sum(dim=1)
    t = s["token"].long().masked_fill(skip, 0)
    out = {"logprob": lps[torch.arange(B, device=x.device), t].masked_fill(skip, 0.0), "entropy": h.masked_fill(skip, 0.0),
           "rank": None, "row_max": top.masked_fill(skip, 0.0),
           "row_logsum": (lse - z.max(dim=1).values).masked_fill(skip, 0.0)}
    if case["n_alt"]:
        v, i = torch.sort(x, dim=1, descending=True, stable=True)
        i, v = i[:, : case["n_alt"]], v[:, : case["n_alt"]]
        out["alt_idx"] = None
        alt = lps.gather(1, i)
        out["alt_lp"] = alt.masked_fill(torch.isinf(v) | skip[:, None], math.nan)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "score":
        return _exact_score(s)
    if kind == "score_grad":
        # the softmax's own Jacobian: d lp_t / dz = e_t - p and d H / dz_v = -p_v (log p_v + H), z = x / T
        T = s["temperature"].double()[:, None] if s["temperature"] is not None else 1.0
        lps = torch.log_softmax(s["logits"].double() / T, dim=1)
        p = torch.exp(lps)
        plogp = torch.nan_to_num(p * lps, nan=0.0)
        ent = -plogp.sum(dim=1, keepdim=True)
        d = -s["dentropy"].double()[:, None] * (plogp + p * ent) - s["dlogprob"].double()[:, None] * p
        skip = s["token"] == IGNORE
        t = s["token"].long().masked_fill(skip, 0)
        d[torch.arange(case["B"], device=d.device), t] += s["dlogprob"].double()
        return (d / T).masked_fill(skip[:, None], 0.0)
    if kind == "head":
        V, D, G = case["V"], case["D"], case["group"]
        x = s["hidden"].double()
        total = torch.zeros((case["M"], V), dtype=torch.float64, device=x.device)
        for g in range(D // G):
            b = s["codes"][:, g * G // 2:(g + 1) * G // 2]
            z = 8.0 if s["zeros"] is None else s["zeros"][:, g:g + 1].double()
            dot = x[:, g * G:(g + 1) * G:2] @ ((b % 16).double() - z).t() + \
                x[:, g * G + 1:(g + 1) * G:2] @ ((b // 16).double() - z).t()
            total += dot * s["scales"][:, g].double()[None, :]
        return total
    skip = s["token"] == IGNORE
    if kind == "embed":
        t = s["token"].long().masked_fill(skip, 0)
        return (torch.index_select(s["table"], 0, t).double() * s["scale"]).masked_fill(skip[:, None], 0.0)
    # sums of equal tokens as differences of a running sum over the sorted tokens
    keep = torch.nonzero(~skip)[:, 0]
    tok, order = torch.sort(s["token"][keep].long(), stable=True)
    run_sum = torch.cumsum(s["dout"][keep[order]].double() * s["scale"], dim=0)
    values, counts = torch.unique_consecutive(tok, return_counts=True)
    ends = run_sum[torch.cumsum(counts, dim=0) - 1]
    sums = ends.clone()
    sums[1:] -= ends[:-1]
    total = s["out"].double() if case["accumulate"] else torch.zeros(s["out"].shape, dtype=torch.float64,
                                                                     device=sums.device)
    total[values] += sums
    return total
