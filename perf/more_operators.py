"""Cases of the 8-bit blocks and of the optimiser: quantisation into e4m3 blocks of 128, the product of two such matrices,
the AdamW step over many tensors.

``run`` computes each operator in its plain form (elementary torch operations in 32 bits, rounded once), or, with ``own``
set, through the library's entry points. ``exact`` gives the same outputs in 64 bits.
"""
import math
import random

import torch

own = False

BLOCK = 128             # elements of a block along the inner dimension
TOP = 448.0             # the largest e4m3 value
LEAST = 2.0 ** -126     # the smallest scale
F8 = torch.float8_e4m3fn

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "bf16": 2}

# no case is larger than the largest listed ones
MOST_PRODUCTS = 2048 * 151936 * 4096
MOST_OPERAND = 4096 * 151936
MOST_OUT = 2048 * 151936
MOST_QUANT = 2048 * 151936
MOST_PARAMS = 2048 * 151936

LR, BETA1, BETA2, EPS, DECAY = 1e-5, 0.9, 0.999, 1e-8, 0.05


def listed():
    return [
        # the hidden states of one decode step of 16 requests, before an 8-bit head
        dict(name="quantise step", kind="quant", R=16, C=2048, dtype="bf16", tile=False, plain=True, turned=False, pad=0),
        # a short sequence's hidden states in both directions, odd sizes, rows at an odd stride
        dict(name="quantise odd", kind="quant", R=509, C=1001, dtype="f32", tile=False, plain=True, turned=True, pad=3),
        # the gradient of a training micro-batch's logits: rows for the hidden states' gradient, columns for the weights'
        dict(name="quantise train", kind="quant", R=2048, C=151936, dtype="bf16", tile=False, plain=True, turned=True,
             pad=0),
        # a head's weights after an optimiser step, for the logits and for the hidden states' gradient
        dict(name="quantise weights", kind="quant", R=32000, C=2048, dtype="f32", tile=True, plain=True, turned=True,
             pad=0),
        # logits of one decode step of a small model
        dict(name="product step", kind="product", M=4, N=32000, K=2048, tile=True, out="f32", add=False),
        # logits of a full serving batch of a large model
        dict(name="product batch", kind="product", M=64, N=151936, K=4096, tile=True, out="bf16", add=False),
        # logits of a training micro-batch, or of the prompts whose tokens are scored
        dict(name="product train", kind="product", M=2048, N=151936, K=4096, tile=True, out="bf16", add=False),
        # gradient of that micro-batch's hidden states: the vocabulary is summed over
        dict(name="product hidden grad", kind="product", M=2048, N=4096, K=151936, tile=True, out="f32", add=False),
        # gradient of a head's weights added to a tied table's: both operands with a scale per row, odd sizes
        dict(name="product weight grad", kind="product", M=32003, N=2050, K=1501, tile=False, out="f32", add=True),
        # all matrices and norms of a small model, packed one behind the other: many short tensors at any alignment
        dict(name="adamw many", kind="adamw", tensors=150, largest=100000, packed=True, param="f32", grad="f32", bits=32,
             master=False, step=3),
        # a table in bf16 with fp32 masters, beside the other matrices of its model
        dict(name="adamw masters", kind="adamw", tensors=3, largest=32000 * 2048, packed=False, param="bf16", grad="bf16",
             bits=32, master=True, step=1000),
        # a large tied table with 8-bit states
        dict(name="adamw table", kind="adamw", tensors=1, largest=2048 * 151936, packed=False, param="f32", grad="bf16",
             bits=8, master=False, step=200),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["quant", "product", "product", "product", "adamw", "adamw"])
    if kind == "quant":
        C = _log_uniform(rng, 64, 151936)
        R = _log_uniform(rng, 1, max(1, min(32768, MOST_QUANT // C)))
        plain, turned = rng.choice([(True, False), (True, True), (True, True), (False, True)])
        return dict(kind=kind, R=R, C=C, dtype=rng.choice(["f32", "bf16"]) if R * C <= MOST_QUANT // 2 else "bf16",
                    tile=rng.random() < 0.4, plain=plain, turned=turned, pad=rng.choice([0, 0, 1, 8, 13]))
    if kind == "product":
        K = _log_uniform(rng, 128, 151936)
        N = _log_uniform(rng, 64, min(151936, MOST_OPERAND // K))
        M = _log_uniform(rng, 1, max(1, min(16384, MOST_PRODUCTS // (N * K), MOST_OPERAND // K, MOST_OUT // N)))
        tile = rng.random() < 0.6
        add = not tile and rng.random() < 0.7
        return dict(kind=kind, M=M, N=N, K=K, tile=tile, out="f32" if add else rng.choice(["f32", "bf16"]), add=add)
    tensors = _log_uniform(rng, 1, 300)
    param = rng.choice(["f32", "f32", "bf16"])
    return dict(kind=kind, tensors=tensors, largest=_log_uniform(rng, 1000, MOST_PARAMS // (3 * tensors)),
                packed=rng.random() < 0.5, param=param, grad=rng.choice(["f32", "bf16"]), bits=rng.choice([32, 8]),
                master=param == "bf16" and rng.random() < 0.5, step=_log_uniform(rng, 1, 100000))


def _blocks(n):
    return -(-n // BLOCK)


def _up(n, m):
    return -(-n // m) * m


def _sizes(case):
    """Numbers of elements of the case's tensors: the largest one, others down to a norm's, and where each begins."""
    rng = random.Random(case["tensors"] * 1000003 + case["largest"])
    sizes = [case["largest"]]
    sizes += [_log_uniform(rng, 64, max(64, case["largest"])) for _ in range(case["tensors"] - 1)]
    at, begins = 0, []
    for n in sizes:
        begins.append(at)
        at += n if case["packed"] else _up(n, 1024)
    return sizes, begins, at


def _scale_plane(rows, cols, tile, dev):
    """Where the scales of a matrix's blocks go: [row blocks, column blocks] of 128 x 128 blocks, else [column blocks,
    rows], rows of whole 16 bytes."""
    if tile:
        return torch.empty((_blocks(rows), _blocks(cols)), device=dev)
    return torch.empty((_blocks(cols), _up(rows, 4)), device=dev)[:, :rows]


def _code_plane(rows, cols, dev):
    return torch.empty((rows, _up(cols, 16)), dtype=F8, device=dev)[:, :cols]


def _operand(rows, cols, tile, gen, dev):
    """Codes and scales as a quantisation leaves them: every block reaches 448, scales of several magnitudes."""
    codes = torch.empty((rows, _up(cols, 16)), dtype=F8, device=dev)
    part = max(1, (1 << 28) // codes.shape[1])
    for r in range(0, rows, part):
        x = torch.randn((min(part, rows - r), codes.shape[1]), generator=gen, device=dev).mul_(120).clamp_(-TOP, TOP)
        codes[r:r + part] = x.to(F8)
    scales = _scale_plane(rows, cols, tile, dev)
    scales.copy_(torch.exp2(torch.rand(scales.shape, generator=gen, device=dev) * 4 - 14))
    return codes[:, :cols], scales


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    s = {"case": dict(case)}
    kind = case["kind"]
    if kind == "quant":
        R, C = case["R"], case["C"]
        x = torch.randn((R, C + case["pad"]), generator=gen, device=dev)
        # channels and rows of other magnitudes, as hidden states and gradients have them
        x.mul_(torch.exp2(torch.randn((1, C + case["pad"]), generator=gen, device=dev)))
        x.mul_(torch.exp2(torch.randn((R, 1), generator=gen, device=dev) * 2 - 6))
        s["x"] = x.to(DTYPES[case["dtype"]])[:, :C]
        if case["plain"]:
            s["codes"], s["scales"] = _code_plane(R, C, dev), _scale_plane(R, C, case["tile"], dev)
        if case["turned"]:
            s["codes_t"], s["scales_t"] = _code_plane(C, R, dev), _scale_plane(C, R, case["tile"], dev)
        if own:
            import top_sampling_gb300 as ts
            if case["plain"]:
                s["to"] = ts.BlockTensor(s["codes"], s["scales"], tile=case["tile"])
            if case["turned"]:
                s["to_t"] = ts.BlockTensor(s["codes_t"], s["scales_t"], tile=case["tile"])
    elif kind == "product":
        M, N, K = case["M"], case["N"], case["K"]
        s["a"], s["sa"] = _operand(M, K, False, gen, dev)
        s["b"], s["sb"] = _operand(N, K, case["tile"], gen, dev)
        s["out"] = torch.empty((M, N), dtype=DTYPES[case["out"]], device=dev)
        if case["add"]:
            s["out"].normal_(generator=gen)
        if own:
            import top_sampling_gb300 as ts
            s["A"], s["B"] = ts.BlockTensor(s["a"], s["sa"]), ts.BlockTensor(s["b"], s["sb"], tile=case["tile"])
    else:
        sizes, begins, total = _sizes(case)
        size = torch.exp2(torch.randn(total, generator=gen, device=dev) * 1.5 - 10)   # an element's usual gradient
        value = torch.randn(total, generator=gen, device=dev).mul_(0.05)
        grad = torch.randn(total, generator=gen, device=dev).mul_(size)
        first = torch.randn(total, generator=gen, device=dev).mul_(size).mul_(0.25)
        root = torch.rand(total, generator=gen, device=dev).add_(0.5).mul_(size)
        del size
        parts = [slice(b, b + n) for b, n in zip(begins, sizes)]
        s["param"] = value.to(DTYPES[case["param"]])
        s["grad"] = grad.to(DTYPES[case["grad"]])
        if case["master"]:
            s["master"] = value
        s["grad_scale"] = torch.full((1,), 0.75, device=dev)
        if case["bits"] == 32:
            s["m"], s["v"] = first, root.square_()
        else:
            # a tensor's blocks begin at its first element; the codes and scales of all tensors lie in one buffer each
            s["m"], s["v"] = (torch.zeros(total, dtype=F8, device=dev) for _ in range(2))
            at = [0]
            for n in sizes:
                at.append(at[-1] + _blocks(n))
            s["m_scale"], s["v_scale"] = (torch.zeros(at[-1], device=dev) for _ in range(2))
            s["blocks"] = [slice(at[i], at[i + 1]) for i in range(len(sizes))]
            for p, b in zip(parts, s["blocks"]):
                for x, codes, scales in ((first, s["m"], s["m_scale"]), (root, s["v"], s["v_scale"])):
                    y, sc = _to_blocks(x[p])
                    codes[p] = y.clamp(-TOP, TOP).to(F8).reshape(-1)[:x[p].numel()]
                    scales[b] = sc
        s["parts"], s["grads"] = parts, [s["grad"][p] for p in parts]
        if own:
            # an optimiser's object: the tensors that it updates, checked once
            import top_sampling_gb300 as ts
            more = {}
            if case["bits"] == 8:
                more = dict(m_scale=[s["m_scale"][b] for b in s["blocks"]], v_scale=[s["v_scale"][b] for b in s["blocks"]])
            s["state"] = ts.vsamp_adamw_state([s["param"][p] for p in parts], bits=case["bits"],
                                              masters=[s["master"][p] for p in parts] if case["master"] else None,
                                              m=[s["m"][p] for p in parts], v=[s["v"][p] for p in parts], **more)
    return s


def _whole_blocks(x, rows):
    """x [R, C] with zeros up to whole blocks, as [row blocks, rows, column blocks, 128]."""
    R, C = x.shape
    x = torch.nn.functional.pad(x, (0, _up(C, BLOCK) - C, 0, _up(R, rows) - R))
    return x.view(x.shape[0] // rows, rows, x.shape[1] // BLOCK, BLOCK)


def _scale_of(amax):
    return torch.where(torch.isfinite(amax), (amax / TOP).clamp(min=LEAST), math.nan)


def _to_blocks(x):
    """Values of a vector in units of their block's scale [blocks, 128], and the scales."""
    n = x.numel()
    x = torch.nn.functional.pad(x, (0, _up(n, BLOCK) - n)).view(-1, BLOCK)
    scale = _scale_of(x.abs().amax(dim=1))
    return x * (1 / scale)[:, None], scale


def _quantise(x, tile):
    R, C = x.shape
    rows = BLOCK if tile else 1
    x = _whole_blocks(x.float(), rows)
    scale = _scale_of(x.abs().amax(dim=(1, 3)))
    y = (x * (1 / scale)[:, None, :, None]).nan_to_num(nan=0.0).clamp(-TOP, TOP).to(F8)
    return y.view(x.shape[0] * rows, -1)[:R, :C], scale if tile else scale.t()


def _dequantise(codes, scales, tile, kind):
    R, C = codes.shape
    x = codes.to(kind)
    s = scales.to(kind)
    s = s.repeat_interleave(BLOCK, 0)[:R] if tile else s.t()
    return x * s.repeat_interleave(BLOCK, 1)[:, :C]


def _philox(i, high, step, tensor, seed):
    """The four words of Philox4x32-10 at the counters (i, high, step, tensor), in 64-bit whole numbers."""
    low = 0xFFFFFFFF
    c0, c1, c2, c3 = i & low, torch.full_like(i, high), torch.full_like(i, step & low), torch.full_like(i, tensor)
    k0, k1 = seed & low, seed >> 32
    for _ in range(10):
        p0, p1 = _wide(c0, 0xD2511F53), _wide(c2, 0xCD9E8D57)
        c0, c1, c2, c3 = p1[0] ^ c1 ^ k0, p1[1], p0[0] ^ c3 ^ k1, p0[1]
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    return c0, c1, c2, c3


def _wide(c, by):
    """High and low words of a 32 x 32 bit product."""
    low = c * (by & 0xFFFF)
    high = c * (by >> 16) + (low >> 16)
    return high >> 16, ((high & 0xFFFF) << 16) | (low & 0xFFFF)


def _random_words(n, high, step, tensor, seed, dev):
    words = _philox(torch.arange(_up(n, 4) // 4, device=dev), high, step, tensor, seed)
    return torch.stack(words, dim=1).view(-1)[:n]


def _round_up_or_down(y, h):
    """e4m3 values next to y at random: y is rounded up with the probability of its place between them."""
    size = y.abs()
    e = (torch.frexp(size)[1] - 1).clamp(min=-6)
    step = torch.exp2((e - 3).to(y.dtype))
    q = torch.floor(size / step + (h.to(y.dtype) + 0.5) * 2.0 ** -16) * step
    return torch.copysign(q.clamp(max=TOP), y)


def _adamw_one(s, k):
    case, p = s["case"], s["parts"][k]
    step, n = case["step"], p.stop - p.start
    value = (s["master"] if case["master"] else s["param"])[p].float()
    g = s["grads"][k].float() * s["grad_scale"]
    b = s["blocks"][k] if case["bits"] == 8 else None
    if b is None:
        m, v = s["m"][p], s["v"][p]
    else:
        m = s["m"][p].float() * s["m_scale"][b].repeat_interleave(BLOCK)[:n]
        v = (s["v"][p].float() * s["v_scale"][b].repeat_interleave(BLOCK)[:n]).square()
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * g * g
    size = torch.sqrt(v)
    change = m / (1 - BETA1 ** step) / (size / math.sqrt(1 - BETA2 ** step) + EPS)
    value = value * (1 - LR * DECAY) - LR * change
    if case["master"]:
        s["master"][p] = value
    if case["param"] == "bf16" and not case["master"]:
        # stochastic: 16 random bits below the kept ones
        h = _random_words(n, 1 << 31, step, k, 0, value.device).to(torch.int32) & 0xFFFF
        value = ((value.view(torch.int32) + h) & -65536).view(torch.float32)
    s["param"][p] = value.to(s["param"].dtype)
    if b is None:
        s["m"][p], s["v"][p] = m, v
        return
    w = _random_words(n, 0, step, k, 0, m.device)
    for x, codes, scales, h in ((m, s["m"], s["m_scale"], w >> 16), (size, s["v"], s["v_scale"], w & 0xFFFF)):
        y, scales[b] = _to_blocks(x)
        y = _round_up_or_down(y.view(-1)[:n], h)
        if x is size:
            y = torch.where(x > 0, y.clamp(min=2.0 ** -9), y)
        codes[p] = y.to(F8)


def _adamw_out(s):
    return {k: s[k] for k in ("param", "master", "m", "v", "m_scale", "v_scale") if k in s}


def run(state):
    s = state
    case = s["case"]
    kind = case["kind"]
    if own:
        import top_sampling_gb300 as ts
        if kind == "quant":
            ts.vsamp_block_quantize(s["x"], tile=case["tile"], plain=case["plain"], transposed=case["turned"],
                                    out=s.get("to"), out_t=s.get("to_t"))
            return {k: s[k] for k in ("codes", "scales", "codes_t", "scales_t") if k in s}
        if kind == "product":
            return ts.vsamp_block_matmul(s["A"], s["B"], out=s["out"], accumulate=case["add"])
        ts.vsamp_adamw(s["state"], s["grads"], lr=LR, step=case["step"], beta1=BETA1, beta2=BETA2,
                       eps=EPS, weight_decay=DECAY, grad_scale=s["grad_scale"])
        return _adamw_out(s)
    if kind == "quant":
        out = {}
        if case["plain"]:
            out["codes"], out["scales"] = _quantise(s["x"], case["tile"])
        if case["turned"]:
            out["codes_t"], out["scales_t"] = _quantise(s["x"].t(), case["tile"])
        return out
    if kind == "product":
        a = _dequantise(s["a"], s["sa"], False, torch.float32)
        b = _dequantise(s["b"], s["sb"], case["tile"], torch.float32)
        y = torch.matmul(a, b.t())
        return s["out"].copy_(y + s["out"] if case["add"] else y)
    [_adamw_one(s, k) for k in range(len(s["parts"]))]
    return _adamw_out(s)


def work(case):
    kind = case["kind"]
    if kind == "quant":
        R, C = case["R"], case["C"]
        ways = case["plain"] + case["turned"]
        if case["tile"]:
            scales = 4 * ways * _blocks(R) * _blocks(C)
        else:
            scales = 4 * (case["plain"] * R * _blocks(C) + case["turned"] * C * _blocks(R))
        # per element: the largest magnitude, and per direction a product and a conversion
        return {"bytes": R * C * (BYTES[case["dtype"]] + ways) + scales, "flops": R * C * (1 + 2 * ways)}
    if kind == "product":
        M, N, K = case["M"], case["N"], case["K"]
        scales = 4 * _blocks(K) * (M + (_blocks(N) if case["tile"] else N))
        out = M * N * BYTES[case["out"]] * (2 if case["add"] else 1)
        return {"bytes": (M + N) * K + scales + out, "flops": 2 * M * N * K}
    n = sum(_sizes(case)[0])
    state = 8 if case["bits"] == 32 else 2 + 8 / BLOCK
    each = 2 * state + BYTES[case["grad"]]
    each += 8 + 2 if case["master"] else 2 * BYTES[case["param"]]
    return {"bytes": int(n * each) + 4, "flops": 16 * n}


# ---- 64 bits, apart from the above ------------------------------------------------------------------------------------


def _exact_codes(x, tile):
    """Codes and scales of a matrix in 64 bits, row block by row block."""
    R, C = x.shape
    high = BLOCK if tile else max(1, min(R, (1 << 25) // max(C, 1)))
    codes = torch.empty((R, C), dtype=F8, device=x.device)
    scales = torch.empty((_blocks(R), _blocks(C)) if tile else (_blocks(C), R), dtype=torch.float64, device=x.device)
    for r in range(0, R, high):
        part = x[r:r + high].double()
        size = torch.zeros((part.shape[0], _blocks(C) * BLOCK), dtype=torch.float64, device=x.device)
        size[:, :C] = part.abs()
        top = size.view(part.shape[0], -1, BLOCK).max(dim=2).values / TOP
        if tile:
            top = top.max(dim=0, keepdim=True).values
            scales[r // BLOCK] = top[0]
        else:
            scales[:, r:r + high] = top.t()
        unit = torch.where(top > 0, top, 1.0).expand(part.shape[0], -1).repeat_interleave(BLOCK, 1)[:, :C]
        codes[r:r + high] = (part / unit).to(F8)
    return codes, scales


def _exact_product(s):
    case = s["case"]
    M, N, K, tile = case["M"], case["N"], case["K"], case["tile"]
    total = s["out"].double() if case["add"] else torch.zeros((M, N), dtype=torch.float64, device=s["a"].device)
    span = BLOCK * max(1, min(_blocks(K), (1 << 27) // (max(M, N) * BLOCK)))   # columns per product
    for k in range(0, K, span):
        at = torch.arange(k, min(K, k + span), device=total.device) // BLOCK
        a = s["a"][:, k:k + span].double() * s["sa"].double()[at].t()
        if tile:
            b = s["b"][:, k:k + span].double() * s["sb"].double()[torch.arange(N, device=at.device) // BLOCK][:, at]
        else:
            b = s["b"][:, k:k + span].double() * s["sb"].double()[at].t()
        total += a @ b.t()
    return total


def _exact_words(n, high, step, tensor, dev):
    """Philox4x32-10 with the key 0, products in binary64 halves."""
    i = torch.arange(-(-n // 4), device=dev)
    c = [i, torch.full_like(i, high), torch.full_like(i, step), torch.full_like(i, tensor)]
    key = [0, 0]

    def product(by, x):
        top, rest = x >> 16, x & 0xFFFF
        mid = by * top                                  # below 2^48
        whole = (mid & 0xFFFFFFFFFF) * 65536 + by * rest   # bits up to 2^57
        carry = (mid >> 40) << 56
        return (whole + carry) >> 32, (whole + carry) & 0xFFFFFFFF

    for r in range(10):
        h0, l0 = product(0xD2511F53, c[0])
        h1, l1 = product(0xCD9E8D57, c[2])
        # 2^63 and more wraps to a negative number: its high word is taken modulo 2^32
        h0, h1 = h0 & 0xFFFFFFFF, h1 & 0xFFFFFFFF
        c = [h1 ^ c[1] ^ key[0], l1, h0 ^ c[3] ^ key[1], l0]
        key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
    return torch.cat([w[:, None] for w in c], dim=1).reshape(-1)[:n]


def _exact_adamw(s):
    case = s["case"]
    out = {k: v.clone() if v.dtype in (F8, torch.bfloat16) else v.double() for k, v in _adamw_out(s).items()}
    t = case["step"]
    for k, p in enumerate(s["parts"]):
        n = p.stop - p.start
        g = s["grad"][p].double() * s["grad_scale"].double()
        theta = s["master" if case["master"] else "param"][p].double()
        m, v = s["m"][p].double(), s["v"][p].double()
        if case["bits"] == 8:
            block = torch.arange(n, device=g.device) // BLOCK
            at = s["blocks"][k]
            m *= s["m_scale"][at].double()[block]
            v = (v * s["v_scale"][at].double()[block]) ** 2
        m = m + (1 - BETA1) * (g - m)
        v = v + (1 - BETA2) * (g ** 2 - v)
        root = v ** 0.5
        theta = theta - LR * DECAY * theta - LR * (m / -math.expm1(t * math.log(BETA1))) / (
            root / (-math.expm1(t * math.log(BETA2))) ** 0.5 + EPS)
        if case["master"]:
            out["master"][p] = theta
        if case["param"] == "f32":
            out["param"][p] = theta
        elif case["master"]:
            out["param"][p] = theta.to(torch.bfloat16)
        else:
            # up with the probability that 16 random bits and the bits below the kept ones carry
            h = (_exact_words(n, 1 << 31, t, k, g.device) & 0xFFFF).double()
            e = torch.exp2((torch.frexp(theta)[1] - 8).double())
            out["param"][p] = (torch.trunc(theta.abs() / e + h / 65536) * e * torch.sign(theta)).to(torch.bfloat16)
        if case["bits"] == 32:
            out["m"][p], out["v"][p] = m, v
            continue
        w = _exact_words(n, 0, t, k, g.device)
        for x, name, h in ((m, "m", w // 65536), (root, "v", w % 65536)):
            size = torch.zeros(_blocks(n) * BLOCK, dtype=torch.float64, device=g.device)
            size[:n] = x.abs()
            unit = size.view(-1, BLOCK).max(dim=1).values / TOP
            out[name + "_scale"][at] = unit
            y = size[:n] / torch.where(unit > 0, unit, 1.0)[block]
            e = torch.exp2((torch.frexp(y)[1].clamp(min=-5) - 4).double())
            y = (torch.floor(y / e + (h.double() + 0.5) / 65536) * e).clamp(max=TOP)
            if name == "v":
                y = torch.where(x > 0, y.clamp(min=2.0 ** -9), y)
            out[name][p] = (y * torch.sign(x)).to(F8)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "quant":
        out = {}
        if case["plain"]:
            out["codes"], out["scales"] = _exact_codes(s["x"], case["tile"])
        if case["turned"]:
            out["codes_t"], out["scales_t"] = _exact_codes(s["x"].t(), case["tile"])
        return out
    if case["kind"] == "product":
        return _exact_product(s)
    return _exact_adamw(s)
