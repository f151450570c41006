"""What a decoding step does around a quantised head, as cases to measure: the
residual's addition with the RMS norm in front of the head, microscaled (MX)
quantisation, the product of microscaled operands, and sampling of the next
token from the logits.

Each case names its operator in ``op``.  ``run`` computes it in plain torch
operations in 32 bits, or, where ``own`` is set, through the framework.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EMAX = {"fp4": 2, "fp8": 8}     # exponent of the largest element of a microscaled format
FP4_VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
LOG2E = 1.4426950408889634
EPS = 1e-6


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    head = {"n": 151936, "k": 1024}      # the head whose figures this repository quotes
    large = {"n": 248320, "k": 5120}     # the largest head it is configured for
    return [
        # one sequence's hidden state before the head: the smallest call, latency alone
        {"name": "norm 1x1024 bf16", "op": "norm", "m": 1, "k": 1024, "dtype": "bf16",
         "out": "same"},
        # a ragged batch and a width that no vector divides
        {"name": "norm 333x4099 f16", "op": "norm", "m": 333, "k": 4099, "dtype": "f16",
         "out": "same"},
        # a prompt's hidden states, 8 bits with a scale per row
        {"name": "norm 4096x5120 e4m3", "op": "norm", "m": 4096, "k": 5120, "dtype": "bf16",
         "out": "e4m3"},
        # a step's activations for an 8-bit x 4-bit product
        {"name": "quantize 61x5120 fp8", "op": "quantize", "m": 61, "k": 5120, "dtype": "bf16",
         "fmt": "fp8"},
        # a whole head at load time
        {"name": "quantize 151936x1024 fp4", "op": "quantize", "m": head["n"], "k": head["k"],
         "dtype": "f16", "fmt": "fp4"},
        # one sequence decoding
        {"name": "logits 1 151936x1024 fp8", "op": "logits", "m": 1, "dtype": "f16", "fmt": "fp8",
         **head},
        # a batch of sequences decoding on the largest head
        {"name": "logits 32 248320x5120 fp8", "op": "logits", "m": 32, "dtype": "bf16",
         "fmt": "fp8", **large},
        # a large batch, or a prompt's scores, both operands in 4 bits
        {"name": "logits 256 151936x1024 fp4", "op": "logits", "m": 256, "dtype": "f16",
         "fmt": "fp4", **head},
        # one sequence, the usual sampling settings
        {"name": "sample 1x151936 top-k", "op": "sample", "m": 1, "n": 151936, "dtype": "bf16",
         "mode": "top_k"},
        # a batch with other settings in each row, and an odd vocabulary
        {"name": "sample 33x50303 mixed", "op": "sample", "m": 33, "n": 50303, "dtype": "f16",
         "mode": "mixed"},
        # 32-bit logits, temperature alone: the draw runs over the whole vocabulary
        {"name": "sample 64x248320 plain", "op": "sample", "m": 64, "n": 248320, "dtype": "f32",
         "mode": "plain"},
        # a large batch with a nucleus
        {"name": "sample 256x151936 top-p", "op": "sample", "m": 256, "n": 151936,
         "dtype": "bf16", "mode": "top_p"},
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["norm", "quantize", "logits", "logits", "sample", "sample"])
    half = rng.choice(["f16", "bf16"])
    if op == "norm":
        out = rng.choice(["same", "e4m3", "e4m3"])
        return {"op": op, "m": log_int(1, 4096), "k": log_int(64, 5120), "dtype": half,
                "out": out}
    if op == "quantize":
        k = 32 * log_int(2, 160)
        return {"op": op, "m": min(log_int(1, 151936), 150_000_000 // k), "k": k,
                "dtype": rng.choice(["f16", "bf16", "f32"]), "fmt": rng.choice(["fp4", "fp8"])}
    if op == "logits":
        k = 32 * log_int(4, 160)
        n = min(log_int(1000, 248320), 400_000_000 // k)
        return {"op": op, "m": log_int(1, 256), "dtype": half, "fmt": rng.choice(["fp4", "fp8"]),
                "n": n, "k": k}
    n = log_int(1000, 248320)
    return {"op": op, "m": min(log_int(1, 256), 32_000_000 // n), "n": n,
            "dtype": rng.choice(["f16", "bf16", "f32"]),
            "mode": rng.choice(["top_k", "top_p", "mixed", "plain"])}


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op, m = case["op"], case["m"]
    dt = DTYPES[case["dtype"]]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    def rand(*shape):
        return torch.rand(*shape, generator=g, device=DEV)

    st = {"case": case}
    if op == "norm":
        k = case["k"]
        # a residual stream grows over the layers and has a few large channels
        loud = 1.0 + 15.0 * (rand(k) < 0.004)
        st["x"] = randn(m, k).to(dt)
        st["residual"] = (4.0 * randn(m, k) * loud).to(dt)
        st["gamma"] = (1.0 + 0.2 * randn(k)).to(dt)
    elif op == "quantize":
        k = case["k"]
        # activations have large channels, rows of a weight differ in size
        st["x"] = torch.empty(m, k, dtype=dt, device=DEV)
        loud = 1.0 + 15.0 * (rand(k) < 0.004)
        for i in range(0, m, 16384):
            r = min(16384, m - i)
            st["x"][i:i + r] = (randn(r, k) * loud * (0.5 + rand(r, 1))).to(dt)
    elif op == "logits":
        n, k = case["n"], case["k"]
        loud = 1.0 + 7.0 * (rand(k) < 0.004)
        st["x"] = (randn(m, k) * loud).to(dt)
        st["w_codes"] = torch.empty(n, k // 2, dtype=torch.uint8, device=DEV)
        exps = torch.empty(n, k // 32, dtype=torch.uint8, device=DEV)
        for i in range(0, n, 32768):
            r = min(32768, n - i)
            st["w_codes"][i:i + r], exps[i:i + r] = plain_mx(0.02 * randn(r, k), "fp4")
        st["w_scales"] = tile_scales(exps)
    else:
        n = case["n"]
        # next-token logits fall off with the rank, by a power that differs from
        # row to row: 1.4 is a hesitant model (some 600 tokens make up 0.9 of the
        # mass), 2.5 a sure one
        power = 1.4 + 1.1 * rand(m, 1)
        rank = 2.0 + n * rand(m, n)
        st["logits"] = (12.0 - power * rank.log() + 0.2 * randn(m, n)).to(dt)
        mode = case["mode"]
        t = 0.6 + 0.4 * rand(m)
        top_k = torch.full((m,), 50, dtype=torch.int32, device=DEV)
        top_p = 0.8 + 0.18 * rand(m)
        min_p = 0.02 + 0.1 * rand(m)
        if mode == "mixed":              # by row: greedy, top-k, top-p, min-p, all of them, none
            kind = torch.arange(m, device=DEV) % 6
            t = torch.where(kind == 0, 0.0, t)
            top_k = torch.where((kind == 1) | (kind == 4), top_k, 0).to(torch.int32)
            top_p = torch.where((kind == 2) | (kind == 4), top_p, 1.0)
            min_p = torch.where((kind == 3) | (kind == 4), min_p, 0.0)
        st["temperature"] = t
        st["top_k"] = top_k if mode in ("top_k", "mixed") else None
        st["top_p"] = top_p if mode in ("top_k", "top_p", "mixed") else None
        st["min_p"] = min_p if mode == "mixed" else None
        st["u"] = rand(m)
    return st


def work(case):
    op, m = case["op"], case["m"]
    size = 4 if case["dtype"] == "f32" else 2
    if op == "norm":
        k = case["k"]
        out = size * m * k if case["out"] == "same" else m * k + 4 * m
        return {"bytes": 3 * size * m * k + size * k + out, "flops": 6 * m * k}
    if op == "quantize":
        # in, and the values that come back
        k = case["k"]
        return {"bytes": m * k * (size + (4 if case["dtype"] == "f32" else 2)),
                "flops": 4 * m * k}
    if op == "logits":
        n, k = case["n"], case["k"]
        return {"bytes": n * k // 2 + n * k // 32 + 2 * m * k + 2 * m * n, "flops": 2 * m * n * k}
    return {"bytes": size * m * case["n"] + 8 * m, "flops": 4 * m * case["n"]}


def run(state):
    return OWN[state["case"]["op"]](state) if own else PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# The framework's calls
# ---------------------------------------------------------------------------
def own_norm(st):
    import weight_only_quantized_wql_gb300 as wql
    case = st["case"]
    fmt = wql.NORM_SAME if case["out"] == "same" else wql.NORM_E4M3
    y, residual, scales = wql.wql_add_rmsnorm(st["x"], st["gamma"], st["residual"], eps=EPS,
                                              fmt=fmt)
    if case["out"] == "same":
        return {"y": y, "residual": residual}
    return {"y": y, "residual": residual, "scales": scales}


def own_quantize(st):
    import weight_only_quantized_wql_gb300 as wql
    fmt = wql.MX_FP4 if st["case"]["fmt"] == "fp4" else wql.MX_FP8
    return wql.wql_mx_dequantize(wql.wql_mx_quantize(st["x"], fmt), st["x"].dtype)


def own_logits(st):
    import weight_only_quantized_wql_gb300 as wql
    case = st["case"]
    w = wql.MXMatrix(st["w_codes"], st["w_scales"], wql.MX_FP4, case["n"], case["k"])
    x = wql.wql_mx_quantize(st["x"], wql.MX_FP4 if case["fmt"] == "fp4" else wql.MX_FP8)
    return wql.wql_mx_logits(x, w, st["x"].dtype)


def own_sample(st):
    import weight_only_quantized_wql_gb300 as wql
    ids, logp = wql.wql_sample(st["logits"], st["u"], temperature=st["temperature"],
                               top_k=st["top_k"], top_p=st["top_p"], min_p=st["min_p"])
    return {"ids": ids, "logp": logp}


OWN = {"norm": own_norm, "quantize": own_quantize, "logits": own_logits, "sample": own_sample}


# ---------------------------------------------------------------------------
# The plain forms, 32 bits, elementary operations
# ---------------------------------------------------------------------------
def plain_norm(st):
    x = st["x"]
    h = x.float() + st["residual"].float()
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * st["gamma"].float()
    if st["case"]["out"] == "same":
        return {"y": y.to(x.dtype), "residual": h.to(x.dtype)}
    s = (y.abs().amax(-1) * (1.0 / 448.0)).clamp(min=1e-8)
    q = (y / s[:, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return {"y": q, "residual": h.to(x.dtype), "scales": s}


def power_of_two(biased):
    """2^(biased - 127) for whole numbers 0..254, exactly (exp2 need not be)."""
    b = biased.to(torch.int32)
    return torch.where(b > 0, b << 23, 1 << 22).to(torch.int32).view(torch.float32)


def plain_mx(x, fmt):
    """Codes and scale exponents (biased by 127) of 32-bit rows."""
    rows, k = x.shape
    b = x.reshape(rows, k // 32, 32)
    top = (b.abs().amax(-1).view(torch.int32) >> 23) & 255     # floor(log2) + 127
    e = (top - EMAX[fmt]).clamp(min=0)
    v = b * power_of_two(254 - e)[..., None]
    if fmt == "fp8":
        q = v.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8).reshape(rows, k)
        return q, e.to(torch.uint8)
    a = v.abs()
    q = sum((a > t if up else a >= t).to(torch.uint8) for t, up in
            ((0.25, 1), (0.75, 0), (1.25, 1), (1.75, 0), (2.5, 1), (3.5, 0), (5.0, 1)))
    q = (q | (torch.signbit(v).to(torch.uint8) << 3)).reshape(rows, k)
    return q[:, 0::2] | (q[:, 1::2] << 4), e.to(torch.uint8)


def plain_values(codes, exps, fmt):
    """The 32-bit values that codes and scale exponents stand for."""
    if fmt == "fp8":
        q = codes.view(torch.float8_e4m3fn).float()
    else:
        lut = torch.tensor(FP4_VALUES + tuple(-v for v in FP4_VALUES), device=codes.device)
        q = lut[torch.stack((codes & 15, codes >> 4), -1).int()].reshape(codes.shape[0], -1)
    rows, k = q.shape
    s = power_of_two(exps)
    return (q.reshape(rows, k // 32, 32) * s[..., None]).reshape(rows, k)


def tile_scales(exps):
    """[rows, k/32] -> tiles of 128 rows x 4 blocks, 512 bytes each: byte
    16 * (row % 32) + 4 * (row / 32 % 4) + block % 4; the rest is zero."""
    rows, nb = exps.shape
    rt, kt = -(-rows // 128), -(-nb // 4)
    p = torch.zeros(rt * 128, kt * 4, dtype=torch.uint8, device=exps.device)
    p[:rows, :nb] = exps
    return p.reshape(rt, 4, 32, kt, 4).permute(0, 3, 2, 1, 4).reshape(rt, kt, 512).contiguous()


def untile_scales(tiles, rows, nb):
    rt, kt = tiles.shape[:2]
    p = tiles.reshape(rt, kt, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rt * 128, kt * 4)
    return p[:rows, :nb]


def plain_quantize(st):
    x, fmt = st["x"], st["case"]["fmt"]
    codes, exps = plain_mx(x.float(), fmt)
    return plain_values(codes, exps, fmt).to(x.dtype)


def plain_logits(st):
    case = st["case"]
    n, k, fmt = case["n"], case["k"], case["fmt"]
    codes, exps = plain_mx(st["x"].float(), fmt)
    x = plain_values(codes, exps, fmt)
    w = plain_values(st["w_codes"], untile_scales(st["w_scales"], n, k // 32), "fp4")
    return (x @ w.t()).to(st["x"].dtype)


def plain_sample(st):
    """Weights are integers (2^31 for the likeliest token), so that their sums
    are the same in every order; order: logit descending, index ascending."""
    lf = st["logits"].float()
    n = lf.shape[1]
    top, best = lf.max(-1, keepdim=True)
    best = (lf == top).int().argmax(-1)
    t = st["temperature"]
    c = torch.full_like(t, LOG2E) / t.clamp(min=1e-30)
    e = torch.exp2((lf - top) * c[:, None])
    w = (e * 2147483648.0).to(torch.int64)
    order = lf.sort(dim=-1, descending=True, stable=True).indices
    ws = w.gather(1, order)
    keep = torch.ones_like(ws, dtype=torch.bool)
    if st["top_k"] is not None:
        k = torch.where(st["top_k"] > 0, st["top_k"].long(), n)
        keep = torch.arange(n, device=lf.device)[None] < k[:, None]
    ws = ws * keep
    if st["top_p"] is not None:
        before = ws.cumsum(-1) - ws
        target = ws.sum(-1).double() * st["top_p"].double()
        inside = (before.double() < target[:, None]) | (st["top_p"] >= 1.0)[:, None]
        inside[:, 0] = True
        keep = keep & inside
    if st["min_p"] is not None:
        keep = keep & (e.gather(1, order) >= st["min_p"].clamp(max=1.0)[:, None])
    w = w * torch.zeros_like(keep).scatter(1, order, keep)
    total = w.sum(-1)
    r = (st["u"].double() * total.double()).to(torch.int64).clamp(min=0)
    r = torch.minimum(r, total - 1)
    ids = (w.cumsum(-1) > r[:, None]).int().argmax(-1)
    ids = torch.where(t > 0, ids, best)
    p = w.gather(1, ids[:, None])[:, 0].float() / total.float()
    return {"ids": ids.to(torch.int32), "logp": torch.where(t > 0, p.log(), torch.zeros_like(p))}


PLAIN = {"norm": plain_norm, "quantize": plain_quantize, "logits": plain_logits,
         "sample": plain_sample}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    st = prepare(case, seed)
    return EXACT[case["op"]](case, st)


def exact_norm(case, st):
    h = st["x"].double() + st["residual"].double()
    y = h / (h.pow(2).sum(-1, keepdim=True) / case["k"] + EPS).sqrt() * st["gamma"].double()
    if case["out"] == "same":
        return {"y": y, "residual": h}
    s = (y.abs().max(-1).values / 448.0).clamp(min=1e-8)
    return {"y": y / s[:, None], "residual": h, "scales": s}


def two_to(e):
    """2^e in 64 bits for whole numbers e, from the bits of the exponent."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def nearest(v, fmt):
    """Nearest element of the format, ties to the even code, saturated; 64 bits."""
    bits, low, most = (1, 0, 6.0) if fmt == "fp4" else (3, -6, 448.0)
    e = torch.frexp(v)[1].clamp(min=low + 1) - 1        # v in [2^e, 2^(e+1)), or subnormal
    step = two_to(e - bits)
    return (torch.round(v / step) * step).clamp(-most, most)


def exact_mx(x, fmt):
    rows, k = x.shape
    out = torch.empty(rows, k, dtype=torch.float64, device=x.device)
    for i in range(0, rows, 16384):
        b = x[i:i + 16384].double().reshape(-1, k // 32, 32)
        top = b.abs().max(-1, keepdim=True).values
        e = torch.where(top > 0, torch.frexp(top)[1] - 1 - EMAX[fmt], -127).clamp(min=-127)
        s = two_to(e)
        out[i:i + 16384] = (nearest(b / s, fmt) * s).reshape(-1, k)
    return out


def exact_quantize(case, st):
    return exact_mx(st["x"], case["fmt"])


def exact_logits(case, st):
    n, k = case["n"], case["k"]
    x = exact_mx(st["x"], case["fmt"])
    tiles = st["w_scales"].reshape(-1, -(-k // 128), 32, 4, 4)
    out = torch.empty(case["m"], n, dtype=torch.float64, device=x.device)
    for i in range(0, n, 32768):
        codes = st["w_codes"][i:i + 32768].long()
        r = codes.shape[0]
        row = torch.arange(i, i + r, device=x.device)[:, None]
        blk = torch.arange(k // 32, device=x.device)[None]
        s = tiles[row // 128, blk // 4, row % 32, row // 32 % 4, blk % 4].long() - 127
        q = torch.stack((codes % 16, codes // 16), -1).reshape(r, k)
        mag = q % 8
        man, ex = (mag % 2).double(), mag // 2
        v = torch.where(ex > 0, (2.0 + man) * two_to(ex - 2), man / 2.0)
        v = torch.where(q >= 8, -v, v).reshape(r, k // 32, 32) * two_to(s)[..., None]
        out[:, i:i + r] = x @ v.reshape(r, k).t()
    return out


def exact_sample(case, st):
    z = st["logits"].double()
    n = case["n"]
    t = st["temperature"].double()
    greedy = t <= 0
    p = torch.softmax(z / torch.where(greedy, torch.ones_like(t), t)[:, None], -1)
    order = torch.argsort(z, dim=-1, descending=True, stable=True)
    ps = p.gather(1, order)
    rank = torch.arange(n, device=z.device)[None]
    if st["top_k"] is not None:
        k = st["top_k"].long()[:, None]
        ps = torch.where((rank < k) | (k <= 0), ps, 0.0)
    first = ps[:, :1].clone()
    if st["top_p"] is not None:
        share = (ps / ps.sum(-1, keepdim=True)).cumsum(-1)
        share = torch.cat((torch.zeros_like(first), share[:, :-1]), -1)
        tp = st["top_p"].double()[:, None]
        ps = torch.where((share < tp) | (tp >= 1) | (rank == 0), ps, 0.0)
    if st["min_p"] is not None:
        ps = torch.where(ps >= st["min_p"].double().clamp(max=1.0)[:, None] * first, ps, 0.0)
    p = torch.zeros_like(p).scatter(1, order, ps)
    cum = p.cumsum(-1)
    ids = (cum > (st["u"].double() * cum[:, -1])[:, None]).int().argmax(-1)
    logp = (p.gather(1, ids[:, None])[:, 0] / cum[:, -1]).log()
    ids = torch.where(greedy, order[:, 0], ids)
    return {"ids": ids, "logp": torch.where(greedy, torch.zeros_like(logp), logp)}


EXACT = {"norm": exact_norm, "quantize": exact_quantize, "logits": exact_logits,
         "sample": exact_sample}
