"""What a decoding step needs around the head when requests bring adapters of
their own or are decoded by beam search, as cases to measure: the low-rank
adapters of many requests added to a shared projection's result, the selection
of beams over beams and vocabulary, and the reordering of the beams' states.

Each case names its operator in ``op``.  ``run`` computes it in plain torch
operations, or, where ``own`` is set, through the framework.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one request's token on a head with its own adapter: the smallest call, latency alone
        {"name": "lora 1 151936x1024 r16", "op": "lora", "m": 1, "n": 151936, "k": 1024, "r": 16,
         "adapters": 4, "ids": "mixed", "dtype": "bf16"},
        # a ragged batch on an odd vocabulary
        {"name": "lora 33 50303x512 r8", "op": "lora", "m": 33, "n": 50303, "k": 512, "r": 8,
         "adapters": 5, "ids": "mixed", "dtype": "f16"},
        # a batch in which every request has its own adapter, on the largest head
        {"name": "lora 64 248320x5120 r16", "op": "lora", "m": 64, "n": 248320, "k": 5120, "r": 16,
         "adapters": 64, "ids": "mixed", "dtype": "bf16"},
        # a large batch over a few adapters of a high rank
        {"name": "lora 256 151936x1024 r64", "op": "lora", "m": 256, "n": 151936, "k": 1024,
         "r": 64, "adapters": 8, "ids": "mixed", "dtype": "bf16"},
        # the prompts of a few requests beside a projection inside the model
        {"name": "lora 4096 5120x5120 r32", "op": "lora", "m": 4096, "n": 5120, "k": 5120, "r": 32,
         "adapters": 4, "ids": "runs", "dtype": "f16"},
        # one request, four beams: the smallest selection
        {"name": "select 1x4x151936 bf16", "op": "select", "batch": 1, "beams": 4, "n": 151936,
         "dtype": "bf16", "order": "ranked", "eos": True},
        # an odd number of beams on an odd vocabulary
        {"name": "select 7x5x50303 f16", "op": "select", "batch": 7, "beams": 5, "n": 50303,
         "dtype": "f16", "order": "anchored", "eos": True},
        # the batch whose logits the head's benchmark computes at its widest
        {"name": "select 64x4x151936 bf16", "op": "select", "batch": 64, "beams": 4, "n": 151936,
         "dtype": "bf16", "order": "anchored", "eos": True},
        # wide beams, 32-bit logits, no end token
        {"name": "select 16x16x248320 f32", "op": "select", "batch": 16, "beams": 16, "n": 248320,
         "dtype": "f32", "order": "ranked", "eos": False},
        # one request's caches after a step: 24 layers, keys and values
        {"name": "reorder 1x4, 48 states", "op": "reorder", "batch": 1, "beams": 4, "states": 48,
         "heads": 2, "positions": 300, "dim": 64, "order": "ranked", "lengths": False,
         "dtype": "bf16"},
        # a batch of ragged sequences in caches with room behind them
        {"name": "reorder 16x4, 32 states", "op": "reorder", "batch": 16, "beams": 4, "states": 32,
         "heads": 4, "positions": 1024, "dim": 64, "order": "ranked", "lengths": True,
         "dtype": "bf16"},
        # the same kind where the selection left survivors in place; odd sizes
        {"name": "reorder 9x8, 12 states", "op": "reorder", "batch": 9, "beams": 8, "states": 12,
         "heads": 3, "positions": 777, "dim": 80, "order": "anchored", "lengths": True,
         "dtype": "f32"},
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["lora", "lora", "select", "select", "reorder"])
    half = rng.choice(["f16", "bf16"])
    if op == "lora":
        m, r, k = log_int(1, 4096), 8 * rng.randint(1, 8), 8 * log_int(8, 640)
        adapters = min(m, log_int(1, 64))
        n = log_int(1000, 248320)
        n = max(64, min(n, 400_000_000 // (4 * m + 2 * adapters * r),
                        80_000_000_000 // (2 * m * r)))
        return {"op": op, "m": m, "n": n, "k": k, "r": r, "adapters": adapters,
                "ids": rng.choice(["mixed", "runs"]), "dtype": half}
    if op == "select":
        n, beams = log_int(1000, 248320), log_int(1, 16)
        batch = max(1, min(log_int(1, 64), 60_000_000 // (n * beams)))
        return {"op": op, "batch": batch, "beams": beams, "n": n,
                "dtype": rng.choice(["f16", "bf16", "f32"]),
                "order": rng.choice(["ranked", "anchored"]), "eos": rng.random() < 0.75}
    beams, states = rng.randint(2, 16), log_int(1, 48)
    heads, dim, positions = rng.randint(1, 8), 8 * rng.randint(2, 16), log_int(8, 1024)
    per_row = 2 * states * heads * dim * positions
    return {"op": op, "batch": max(1, min(log_int(1, 32), 400_000_000 // (per_row * beams))),
            "beams": beams, "states": states, "heads": heads, "positions": positions, "dim": dim,
            "order": rng.choice(["ranked", "anchored"]), "lengths": rng.random() < 0.7,
            "dtype": half}


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    def rand(*shape):
        return torch.rand(*shape, generator=g, device=DEV)

    st = {"case": case}
    if case["op"] == "lora":
        m, n, k, r, count = (case[v] for v in ("m", "n", "k", "r", "adapters"))
        loud = 1.0 + 7.0 * (rand(k) < 0.004)        # activations have large channels
        st["x"] = (randn(m, k) * loud).to(dt)
        st["y"] = torch.empty(m, n, dtype=dt, device=DEV)       # what the projection gave
        for i in range(0, m, 64):
            st["y"][i:i + 64] = (2.0 * randn(min(64, m - i), n)).to(dt)
        st["a"] = (randn(count, r, k) / k ** 0.5).to(dt)
        st["b"] = torch.empty(count, n, r, dtype=dt, device=DEV)
        for i in range(count):
            st["b"][i] = (0.1 * randn(n, r)).to(dt)
        st["scale"] = 0.5 + 1.5 * rand(count)
        if case["ids"] == "runs":                   # prompts, token after token
            st["ids"] = (torch.arange(m, device=DEV) * count // m).to(torch.int32)
        else:                                       # a batch; some requests have no adapter
            at = torch.arange(m, device=DEV)
            none = at % 16 == 7
            ids = torch.where(none, -1, ((~none).cumsum(0) - 1) % count)
            st["ids"] = ids[torch.randperm(m, generator=g, device=DEV)].to(torch.int32)
    elif case["op"] == "select":
        batch, beams, n = case["batch"], case["beams"], case["n"]
        rows = batch * beams
        st["logits"] = torch.empty(batch, beams, n, dtype=dt, device=DEV)
        flat = st["logits"].view(rows, n)
        for i in range(0, rows, 32):
            # next-token logits fall off with the rank, by a power that differs
            # from row to row
            c = min(32, rows - i)
            power = 1.4 + 1.1 * rand(c, 1)
            rank = 2.0 + n * rand(c, n)
            flat[i:i + c] = (12.0 - power * rank.log() + 0.2 * randn(c, n)).to(dt)
        # log-probabilities of the beams so far, best first, near one another
        st["scores"] = (-8.0 - 2.0 * rand(batch, beams).cumsum(-1)).float()
        st["eos"] = None
        if case["eos"]:
            st["eos"] = n // 2
            # the end is likely in some rows
            flat[:, n // 2] = torch.where(rand(rows) < 0.3, 11.0 - rand(rows),
                                          flat[:, n // 2].float()).to(dt)
    else:
        batch, beams = case["batch"], case["beams"]
        rows, h, p, d = batch * beams, case["heads"], case["positions"], case["dim"]
        st["states"] = [randn(rows, h, p, d).to(dt) for _ in range(case["states"])]
        st["lengths"] = None
        if case["lengths"]:
            st["lengths"] = (p // 4 + (p - p // 4 + 1) * rand(batch)).to(torch.int32).clamp(max=p)
        # the first half of the beams lives on, twice each: what a selection gives
        # when the better beams push out the others
        parents = torch.arange(beams, device=DEV).div(2, rounding_mode="floor")
        if case["order"] == "anchored":             # survivors stay, their doubles fill the rest
            keep = (beams + 1) // 2
            at = torch.arange(beams, device=DEV)
            parents = torch.where(at < keep, at, at - keep)
        st["parents"] = parents.to(torch.int32).expand(batch, beams).contiguous()
    return st


def used_adapters(case):
    m = case["m"]
    return min(case["adapters"], m if case["ids"] == "runs" else m - (m + 8) // 16)


def moved_beams(case):
    """(read, written) beams of a sequence: those whose parent is another beam,
    and those parents."""
    beams = case["beams"]
    if case["order"] == "anchored":
        doubles = beams - (beams + 1) // 2
        return doubles, doubles
    return (beams + 1) // 2, beams - 1              # beam 0 keeps itself


def work(case):
    if case["op"] == "lora":
        m, n, k, r = (case[v] for v in ("m", "n", "k", "r"))
        rows = m if case["ids"] == "runs" else m - (m + 8) // 16
        return {"bytes": 2 * (2 * m * n + m * k + used_adapters(case) * r * (n + k)) + 4 * m,
                "flops": 2 * rows * r * (n + k)}
    if case["op"] == "select":
        rows, size = case["batch"] * case["beams"], 4 if case["dtype"] == "f32" else 2
        return {"bytes": rows * (size * case["n"] + 20), "flops": 4 * rows * case["n"]}
    size = 4 if case["dtype"] == "f32" else 2
    # lengths are spread evenly from a quarter to the whole
    share = 0.625 if case["lengths"] else 1.0
    row = size * case["states"] * case["heads"] * case["dim"] * case["positions"] * share
    return {"bytes": int(case["batch"] * sum(moved_beams(case)) * row), "flops": 0}


def run(state):
    return OWN[state["case"]["op"]](state) if own else PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# The framework's calls
# ---------------------------------------------------------------------------
def own_lora(st):
    import weight_only_quantized_wql_gb300 as wql
    adapters = wql.LoraAdapters(st["a"], st["b"], st["scale"])
    return wql.wql_lora_add(st["y"], st["x"], adapters, st["ids"])


def own_select(st):
    import weight_only_quantized_wql_gb300 as wql
    order = wql.BEAM_RANKED if st["case"]["order"] == "ranked" else wql.BEAM_ANCHORED
    tokens, parents, scores, ended = wql.wql_beam_select(st["logits"], st["scores"],
                                                         eos=st["eos"], order=order)
    out = {"tokens": tokens, "parents": parents, "scores": scores}
    return out if ended is None else {**out, "ended": ended}


def own_reorder(st):
    import weight_only_quantized_wql_gb300 as wql
    return wql.wql_beam_reorder(st["states"], st["parents"], lengths=st["lengths"],
                                position_dim=2)


OWN = {"lora": own_lora, "select": own_select, "reorder": own_reorder}


# ---------------------------------------------------------------------------
# The plain forms: 32 bits, elementary operations; the scores, whose order
# decides, in 64
# ---------------------------------------------------------------------------
def plain_lora(st):
    case = st["case"]
    m, n, k, r, count = (case[v] for v in ("m", "n", "k", "r", "adapters"))
    # every adapter's projection of every token, those of other adapters set to zero
    u = (st["x"].float() @ st["a"].float().view(count * r, k).t()).view(m, count, r)
    mine = st["ids"][:, None] == torch.arange(count, device=DEV)
    u = (u * torch.where(mine, st["scale"], 0.0)[..., None]).view(m, count * r)
    b = st["b"].float().transpose(1, 2).reshape(count * r, n)
    return (st["y"].float() + u @ b).to(st["y"].dtype)


def plain_select(st):
    case = st["case"]
    batch, beams, n = case["batch"], case["beams"], case["n"]
    l = st["logits"].double()
    top = l.amax(-1, keepdim=True)
    lse = (l - top).exp().sum(-1, keepdim=True).log() + top
    s = st["scores"].double()[..., None] + (l - lse)
    del l
    out = {}
    if st["eos"] is not None:
        end = s[..., st["eos"]].clone()
        s[..., st["eos"]] = -math.inf
    # stable: ties go to the lower beam, then the lower token
    best, at = (v[:, :beams] for v in s.view(batch, beams * n).sort(
        dim=-1, descending=True, stable=True))
    tokens, parents = at % n, at.div(n, rounding_mode="floor")
    if st["eos"] is not None:
        # the end of a beam counts where fewer than `beams` continuations of any
        # kind have a larger score
        better = (best[:, None, :] > end[..., None]).sum(-1)
        better = better + (end[:, None, :] > end[..., None]).sum(-1)
        out["ended"] = torch.where(better < beams, end, -math.inf).float()
    if case["order"] == "anchored":
        slot = torch.arange(beams, device=DEV)
        first = ~((parents[:, :, None] == parents[:, None, :]) & (slot[None] < slot[:, None])).any(-1)
        taken = ((parents[:, :, None] == slot) & first[..., None]).any(1)
        free = taken.int().sort(dim=-1, stable=True).indices
        place = torch.where(first, parents, free.gather(1, ((~first).cumsum(-1) - 1).clamp(min=0)))
        tokens, parents, best = (torch.empty_like(v).scatter(1, place, v)
                                 for v in (tokens, parents, best))
    return {"tokens": tokens.to(torch.int32), "parents": parents.to(torch.int32),
            "scores": best.float(), **out}


def plain_reorder(st):
    case = st["case"]
    beams, parents = case["beams"], st["parents"].long()
    source = (torch.arange(case["batch"], device=DEV)[:, None] * beams + parents).view(-1)
    if st["lengths"] is None:
        return [s.copy_(s[source]) for s in st["states"]]
    at = torch.arange(case["positions"], device=DEV)
    inside = (at < st["lengths"].repeat_interleave(beams)[:, None])[:, None, :, None]
    return [s.copy_(torch.where(inside, s[source], s)) for s in st["states"]]


PLAIN = {"lora": plain_lora, "select": plain_select, "reorder": plain_reorder}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    return EXACT[case["op"]](case, prepare(case, seed))


def exact_lora(case, st):
    out = st["y"].double()
    ids = st["ids"].tolist()
    for i in sorted(set(ids)):
        if i < 0:
            continue
        rows = torch.tensor([j for j, v in enumerate(ids) if v == i], device=DEV)
        u = torch.einsum("mk,rk->mr", st["x"][rows].double(), st["a"][i].double())
        for c in range(0, case["n"], 65536):
            part = torch.einsum("mr,nr->mn", u, st["b"][i, c:c + 65536].double())
            out[rows, c:c + 65536] += float(st["scale"][i]) * part
    return out


def exact_select(case, st):
    batch, beams, n, eos = case["batch"], case["beams"], case["n"], st["eos"]
    out = {v: [] for v in ("tokens", "parents", "scores", "ended")}
    for i in range(batch):
        s = st["scores"][i].double()[:, None] + torch.log_softmax(st["logits"][i].double(), -1)
        s = s.view(-1).clone()
        kept, ended, seen = [], [-math.inf] * beams, []
        while True:                                 # the best one left, until enough go on
            top = s.max()
            if len(kept) >= beams and top < kept[beams - 1][0]:
                break
            at = int((s == top).nonzero()[0])
            beam, token = divmod(at, n)
            s[at] = -math.inf
            if token != eos:
                kept.append((float(top), beam, token))
            elif sum(v > top for v in seen) < beams:
                ended[beam] = float(top)
            seen.append(float(top))
        kept = kept[:beams]
        if case["order"] == "anchored":
            slots = [None] * beams
            rest = []
            for c in kept:
                if slots[c[1]] is None:
                    slots[c[1]] = c
                else:
                    rest.append(c)
            for j in range(beams):
                if slots[j] is None:
                    slots[j] = rest.pop(0)
            kept = slots
        for j, v in enumerate(("scores", "parents", "tokens")):
            out[v].append([c[j] for c in kept])
        out["ended"].append(ended)
    if eos is None:
        del out["ended"]
    return {v: torch.tensor(w, dtype=torch.float64 if v in ("scores", "ended") else torch.int64)
            for v, w in out.items()}


def exact_reorder(case, st):
    beams = case["beams"]
    parents = st["parents"].tolist()
    lengths = [case["positions"]] * case["batch"] if st["lengths"] is None else st["lengths"].tolist()
    out = []
    for s in st["states"]:
        new = s.double()
        for i, (chosen, length) in enumerate(zip(parents, lengths)):
            for j, parent in enumerate(chosen):
                new[i * beams + j, :, :length] = s[i * beams + parent, :, :length].double()
        out.append(new)
    return out


EXACT = {"lora": exact_lora, "select": exact_select, "reorder": exact_reorder}
