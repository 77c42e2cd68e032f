"""The experts' feed-forward block and per-request adapters: cases, inputs and
plain forms for measurement.

Four operations around the 1x128 quantizer (E4M3 codes, one power-of-two scale
per 128 columns) and weights that carry one such scale per 128x128 block:

  route    the k experts of every token, their weights, and the slots of all
           (token, expert) pairs in the experts' order
  expert   one product of the experts: the rows of a list are quantised and
           each expert's are multiplied with its own weights; gated: the weights
           hold gate rows and then up rows, and silu(gate) * up comes out
  combine  each token's weighted sum of its slots, on top of another row
  adapt    low-rank adapters of many requests beside a shared projection: every
           request's rows get scale * B (A x) of its own adapter added

Each has a plain form in elementary float32 tensor operations (`own` false) and
the library's kernels (`own` true).
"""

import math

import torch

own = False

FLOOR = 1e-4      # smallest block magnitude the scale rule looks at


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one decoded token chooses its experts: nothing but latency
        dict(name="route_1", op="route", tokens=1, experts=64, k=8, score="sigmoid", normalize=True, dtype="bfloat16"),
        # a prompt's tokens over many experts
        dict(name="route_4632", op="route", tokens=4632, experts=256, k=8, score="softmax", normalize=False,
             dtype="float32"),
        # the experts' outputs of a decode batch, summed per token
        dict(name="combine_64", op="combine", tokens=64, k=8, cols=7168, add=False),
        # the same for a prompt, on top of a shared expert's output
        dict(name="combine_4632", op="combine", tokens=4632, k=8, cols=7168, add=True),
        # one token through the first product of its eight experts: reading the weights
        dict(name="expert_up_1", op="expert", tokens=1, experts=64, k=8, skew=0.0, in_dim=7168, out_dim=4096, gated=True),
        # a decode batch: every expert has a few rows
        dict(name="expert_up_64", op="expert", tokens=64, experts=64, k=8, skew=0.5, in_dim=7168, out_dim=4096,
             gated=True),
        # a prompt, first product: 37056 rows, experts of all sizes
        dict(name="expert_up_4632", op="expert", tokens=4632, experts=64, k=8, skew=0.7, in_dim=7168, out_dim=4096,
             gated=True),
        # a prompt, second product
        dict(name="expert_down_4632", op="expert", tokens=4632, experts=64, k=8, skew=0.7, in_dim=2048, out_dim=7168,
             gated=False),
        # few experts, odd sizes: an output width that fills no tile
        dict(name="expert_odd_333", op="expert", tokens=333, experts=5, k=2, skew=1.0, in_dim=1536, out_dim=1544,
             gated=False),
        # one user's decode step with an adapter
        dict(name="adapt_1", op="adapt", requests=1, len_lo=1, len_hi=1, adapters=4, rank=16, in_dim=1536, out_dim=8192),
        # a decode batch of 64 requests over 48 adapters
        dict(name="adapt_64", op="adapt", requests=64, len_lo=1, len_hi=1, adapters=48, rank=64, in_dim=7168,
             out_dim=8192),
        # prompts of several requests at once, ragged
        dict(name="adapt_prompts_5", op="adapt", requests=5, len_lo=1, len_hi=1852, adapters=3, rank=32, in_dim=7168,
             out_dim=1536),
    ]


def draw(rng):
    def size(lo, hi):                     # log-uniform, odd
        return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi)))) | 1)

    op = rng.choice(["route", "combine", "expert", "expert", "expert", "adapt", "adapt"])
    if op == "route":
        E = size(2, 512)
        return dict(op=op, tokens=size(1, 16384), experts=E, k=rng.randint(1, min(E, 16)),
                    score=rng.choice(["softmax", "sigmoid"]), normalize=rng.random() < 0.5,
                    dtype=rng.choice(["float32", "bfloat16"]))
    if op == "combine":
        c = dict(op=op, tokens=size(1, 8192), k=rng.randint(1, 16), cols=8 * size(16, 1024), add=rng.random() < 0.5)
    elif op == "expert":
        E = rng.choice([1, 2, size(3, 128)])
        c = dict(op=op, tokens=size(1, 4632), experts=E, k=rng.randint(1, min(E, 8)), skew=rng.choice([0.0, 0.5, 1.0]),
                 in_dim=128 * size(2, 56), gated=rng.random() < 0.5)
        c["out_dim"] = 256 * size(1, 32) if c["gated"] else 8 * size(16, 1024)
    else:
        c = dict(op=op, requests=size(1, 64), len_lo=1, adapters=size(1, 64), rank=8 * rng.randint(1, 16),
                 in_dim=8 * size(32, 896), out_dim=8 * size(16, 1024))
        c["len_hi"] = 1 if rng.random() < 0.5 else size(1, 8192 // c["requests"])
    while work(c)["bytes"] > 2e9 or work(c)["flops"] > 2e12:     # no dearer than the largest listed ones
        c["tokens"] = max(1, c["tokens"] // 2)
        if "experts" in c:
            c["experts"] = max(c["k"], c["experts"] // 2)
    return c


def _counts(case):
    """Rows of each expert, in a mixed order: experts' shares fall as a power
    of their rank, no expert gets more rows than there are tokens."""
    T, E, S = case["tokens"], case["experts"], case["tokens"] * case["k"]
    share = [(i + 1.0) ** -case["skew"] for i in range(E)]
    left, n = S, [0] * E
    for i in range(E):
        n[i] = min(T, left, int(round(left * share[i] / sum(share[i:]))))
        left -= n[i]
    for i in range(E):                    # what rounding and the limit left over
        more = min(T - n[i], left)
        n[i] += more
        left -= more
    step = next(s for s in (37, 41, 43, 47, 53) if math.gcd(s, E) == 1)
    return [n[i * step % E] for i in range(E)]


def _lengths(case):
    """Rows of each request: both ends of the range among them, in a mixed order."""
    lo, hi, n = case["len_lo"], case["len_hi"], case["requests"]
    if n == 1:
        return [hi]
    step = next(s for s in (37, 41, 43, 47, 53) if math.gcd(s, n) == 1)
    return [lo + (hi - lo) * ((i * step) % n) // (n - 1) for i in range(n)]


def _used(case):
    """Adapter of each request; the last request of several has none."""
    n = case["requests"]
    return [-1 if n > 1 and i == n - 1 else i * 7 % case["adapters"] for i in range(n)]


def work(case):
    if case["op"] == "route":
        T, E, k = case["tokens"], case["experts"], case["k"]
        return {"bytes": T * E * (4 if case["dtype"] == "float32" else 2) + 16 * T * k + 4 * (E + 1), "flops": 0}
    if case["op"] == "combine":
        T, k, N = case["tokens"], case["k"], case["cols"]
        return {"bytes": 2 * T * N * (k + 1 + case["add"]) + 8 * T * k, "flops": 2 * T * k * N}
    if case["op"] == "expert":
        n = _counts(case)
        S, K, N, hit = sum(n), case["in_dim"], case["out_dim"], sum(1 for m in n if m)
        blocks = -(-N // 128) * (K // 128)
        out = N // 2 if case["gated"] else N
        return {"bytes": 2 * min(S, case["tokens"]) * K + hit * (N * K + blocks) + 2 * S * out + 4 * (S + len(n) + 1),
                "flops": 2 * S * N * K}
    T, K, N, r = sum(_lengths(case)), case["in_dim"], case["out_dim"], case["rank"]
    rows = sum(m for m, a in zip(_lengths(case), _used(case)) if a >= 0)
    hit = len({a for a in _used(case) if a >= 0})
    return {"bytes": 2 * rows * K + 4 * T * N + 2 * hit * r * (K + N) + 4 * hit + 4 * (2 * case["requests"] + 1),
            "flops": 2 * rows * r * (K + N)}


# ------------------------------------------------------------------ inputs

def _randn(shape, gen, dev):
    return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32)


def _ceil_exponent(amax):
    """Smallest e with 448 * 2^e >= max(amax, 1e-4)."""
    m, x = torch.frexp(amax.clamp_min(FLOOR))
    return x - 9 + (m > 0.875).to(x.dtype)


def _weights(E, N, K, gen, dev):
    """E4M3 codes [E, N, K] of normal weights whose 128x128 blocks differ in
    magnitude, and the blocks' scale bytes [E, ceil(N / 128), K / 128]."""
    Nb, Kb = -(-N // 128), K // 128
    codes = torch.empty((E, N, K), dtype=torch.uint8, device=dev)
    sf = torch.empty((E, Nb, Kb), dtype=torch.uint8, device=dev)
    for e in range(E):
        w = _randn((Nb, 128, Kb, 128), gen, dev) * K ** -0.5
        w *= torch.exp2(torch.rand((Nb, 1, Kb, 1), generator=gen, device=dev) * 2 - 1)
        x = _ceil_exponent(w.abs().amax(dim=(1, 3), keepdim=True))
        q = (w * torch.exp2(-x.float())).to(torch.float8_e4m3fn).view(torch.uint8)
        codes[e] = q.view(Nb * 128, K)[:N]
        sf[e] = (x + 127).view(Nb, Kb).to(torch.uint8)
    return codes, sf


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    op = case["op"]
    if op == "route":
        T, E = case["tokens"], case["experts"]
        x = 2 * _randn((T, E), gen, dev) + _randn((1, E), gen, dev)      # some experts are preferred
        return {"op": op, "logits": x.to(getattr(torch, case["dtype"])), "k": case["k"], "score": case["score"],
                "normalize": case["normalize"], "scale": 2.5}
    if op == "combine":
        T, k, N = case["tokens"], case["k"], case["cols"]
        w = torch.rand((T, k), generator=gen, device=dev) + 0.05
        return {"op": op, "y": _randn((T * k, N), gen, dev).to(torch.bfloat16),
                "slots": torch.randperm(T * k, generator=gen, device=dev).to(torch.int32).view(T, k),
                "weights": w / w.sum(dim=1, keepdim=True),
                "add": _randn((T, N), gen, dev).to(torch.bfloat16) if case["add"] else None}
    if op == "expert":
        T, n = case["tokens"], _counts(case)
        x = _randn((T, case["in_dim"]), gen, dev)
        x *= torch.exp2(torch.rand((T, 1), generator=gen, device=dev) * 4 - 2)
        start = [sum(n[:e]) for e in range(len(n) + 1)]
        rows = torch.argsort(torch.rand((len(n), T), generator=gen, device=dev), dim=1)
        rows = torch.cat([rows[e, :m].sort().values for e, m in enumerate(n)])
        w, w_sf = _weights(case["experts"], case["out_dim"], case["in_dim"], gen, dev)
        return {"op": op, "x": x.to(torch.bfloat16), "rows": rows.to(torch.int32), "w": w, "w_sf": w_sf, "counts": n,
                "row_start": torch.tensor(start, dtype=torch.int32, device=dev), "gated": case["gated"]}
    n, used = _lengths(case), _used(case)
    T, K, N, r, A = sum(n), case["in_dim"], case["out_dim"], case["rank"], case["adapters"]
    return {"op": op, "lengths": n, "used": used, "x": _randn((T, K), gen, dev).to(torch.bfloat16),
            "base": _randn((T, N), gen, dev).to(torch.bfloat16),
            "a": (_randn((A, r, K), gen, dev) * K ** -0.5).to(torch.bfloat16),
            "b": (_randn((A, N, r), gen, dev) * r ** -0.5).to(torch.bfloat16),
            "scale": torch.rand((A,), generator=gen, device=dev) + 0.5,
            "row_start": torch.tensor([sum(n[:i]) for i in range(len(n) + 1)], dtype=torch.int32, device=dev),
            "adapter": torch.tensor(used, dtype=torch.int32, device=dev)}


# ------------------------------------------------------------- plain forms

def _route(s):
    l = s["logits"].float()
    T, E = l.shape
    k = s["k"]
    top, experts = torch.sort(l, dim=1, descending=True, stable=True)
    top, experts = top[:, :k], experts[:, :k]
    if s["score"] == "softmax":
        p = torch.exp(top - top[:, :1])
        total = p if s["normalize"] else torch.exp(l - top[:, :1])
        weights = p / total.sum(dim=1, keepdim=True)
    else:
        weights = 1 / (1 + torch.exp(-top))
        if s["normalize"]:
            weights = weights / weights.sum(dim=1, keepdim=True)
    flat = experts.reshape(-1)
    order = torch.argsort(flat * T + torch.arange(T, device=l.device).repeat_interleave(k))
    slots = torch.empty_like(order)
    slots[order] = torch.arange(T * k, device=l.device)
    start = (flat[None, :] < torch.arange(E + 1, device=l.device)[:, None]).sum(dim=1)
    return {"weights": weights * s["scale"], "experts": experts.to(torch.int32), "slots": slots.view(T, k).to(torch.int32),
            "rows": (order // k).to(torch.int32), "row_start": start.to(torch.int32)}


def _expert(s):
    x = s["x"][s["rows"].long()].float()
    S, K = x.shape
    x = x.view(S, K // 128, 128)
    e = _ceil_exponent(x.abs().amax(dim=2, keepdim=True)).float()
    x = ((x * torch.exp2(-e)).to(torch.float8_e4m3fn).float() * torch.exp2(e)).view(S, K)
    N = s["w"].shape[1]
    out = torch.empty((S, N // 2 if s["gated"] else N), dtype=torch.bfloat16, device=x.device)
    at = 0
    for i, n in enumerate(s["counts"]):
        if n == 0:
            continue
        f = torch.exp2(s["w_sf"][i].float() - 127).repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)
        y = torch.matmul(x[at:at + n], (s["w"][i].view(torch.float8_e4m3fn).float() * f).t())
        if s["gated"]:
            g, u = y[:, :N // 2], y[:, N // 2:]
            y = g * u / (1 + torch.exp(-g))
        out[at:at + n] = y
        at += n
    return out


def _combine(s):
    y = s["y"][s["slots"].long()].float()
    o = (y * s["weights"][:, :, None]).sum(dim=1)
    return (o if s["add"] is None else o + s["add"].float()).to(torch.bfloat16)


def _adapt(s):
    out = s["base"].clone()
    at = 0
    for n, a in zip(s["lengths"], s["used"]):
        if a >= 0 and n > 0:
            v = torch.matmul(s["x"][at:at + n].float(), s["a"][a].float().t())
            out[at:at + n] = s["base"][at:at + n].float() + s["scale"][a] * torch.matmul(v, s["b"][a].float().t())
        at += n
    return out


# --------------------------------------------------------------------- run

def run(s):
    op = s["op"]
    if not own:
        return {"route": _route, "expert": _expert, "combine": _combine, "adapt": _adapt}[op](s)
    from fp4_fp8_quant_gb300 import iq
    if op == "route":
        return iq.moe_route(s["logits"], s["k"], score=s["score"], normalize=s["normalize"], scale=s["scale"])._asdict()
    if op == "expert":
        xq, x_sf = iq.fp8_quant_1x128_ue8m0(s["x"], rows=s["rows"])
        return iq.grouped_gemm(xq, x_sf, s["w"], s["w_sf"], s["row_start"], gated=s["gated"])
    if op == "combine":
        return iq.moe_combine(s["y"], s["slots"], s["weights"], add=s["add"])
    return iq.adapters(s["x"], s["base"], s["a"], s["b"], s["scale"], s["row_start"], s["adapter"])


# ------------------------------------------------- the definition in 64 bits

def _e4m3_table(dev):
    """The 256 E4M3 values from the format's definition (no infinities; 0x7F is NaN)."""
    t = []
    for c in range(256):
        sign, e, m = (-1.0 if c & 128 else 1.0), (c >> 3) & 15, c & 7
        mag = math.nan if (c & 127) == 127 else (m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
        t.append(sign * mag)
    return torch.tensor(t, dtype=torch.float64, device=dev)


def _round_e4m3(y):
    """float64 to the nearest E4M3 value, ties to even, |y| <= 448."""
    _, x = torch.frexp(y)
    step = torch.exp2((x - 4).clamp_min(-9).double())
    return (y / step).round() * step      # torch.round takes ties to even


def _exact_route(s):
    l = s["logits"].double()
    T, E = l.shape
    k = s["k"]
    if s["score"] == "softmax":
        p = torch.softmax(l, dim=1)
    else:
        p = torch.sigmoid(l)
    left, ids = l.clone(), []
    low = torch.full((), -math.inf, dtype=torch.float64, device=l.device)
    e = torch.arange(E, device=l.device)[None, :]
    for _ in range(k):                    # the largest that is left, the lowest index of equal ones
        best = torch.where(left == left.amax(dim=1, keepdim=True), e, E).amin(dim=1, keepdim=True)
        ids.append(best)
        left = torch.where(e == best, low, left)
    ids = torch.cat(ids, dim=1)
    w = p.gather(1, ids)
    if s["normalize"]:
        w = w / w.sum(dim=1, keepdim=True)
    chosen = torch.zeros((E, T), dtype=torch.long, device=l.device)
    chosen[ids.t(), torch.arange(T, device=l.device)[None, :]] = 1
    place = (chosen.view(-1).cumsum(0) - 1).view(E, T)
    slots = place.t().gather(1, ids)
    start = torch.cat([torch.zeros(1, dtype=torch.long, device=l.device), chosen.sum(dim=1).cumsum(0)])
    return {"weights": w * s["scale"], "experts": ids.to(torch.int32), "slots": slots.to(torch.int32),
            "rows": chosen.nonzero()[:, 1].to(torch.int32), "row_start": start.to(torch.int32)}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        return _exact_route(s)
    if case["op"] == "combine":
        T, k = s["slots"].shape
        o = torch.zeros((T, s["y"].shape[1]), dtype=torch.float64, device=s["y"].device)
        for j in range(k):
            o += s["y"].index_select(0, s["slots"][:, j].long()).double() * s["weights"][:, j:j + 1].double()
        return o if s["add"] is None else o.add_(s["add"].double())
    if case["op"] == "adapt":
        o = s["base"].double()
        seq = torch.repeat_interleave(torch.arange(len(s["used"]), device=o.device), torch.diff(s["row_start"]).long())
        which = s["adapter"].long()[seq]
        for a in sorted({a for a in s["used"] if a >= 0}):
            t = (which == a).nonzero()[:, 0]
            v = torch.einsum("tk,rk->tr", s["x"][t].double(), s["a"][a].double())
            o[t] += s["scale"][a].double() * torch.einsum("tr,nr->tn", v, s["b"][a].double())
        return o
    tab = _e4m3_table(s["x"].device)
    S, K, N = sum(s["counts"]), case["in_dim"], case["out_dim"]
    out = torch.empty((S, N // 2 if case["gated"] else N), dtype=torch.float64, device=s["x"].device)
    for i, n in enumerate(s["counts"]):
        at = sum(s["counts"][:i])
        x = s["x"][s["rows"][at:at + n].long()].double().view(n, K // 128, 128)
        a = x.abs().amax(dim=2, keepdim=True).clamp_min(FLOOR)
        e = torch.ceil(torch.log2(a / 448.0))
        e = torch.where(448.0 * torch.exp2(e - 1) >= a, e - 1, e)                # log2's own rounding
        e = torch.where(448.0 * torch.exp2(e) < a, e + 1, e)
        x = _round_e4m3(x * torch.exp2(-e)) * torch.exp2(e)
        y = torch.zeros((n, N), dtype=torch.float64, device=x.device)
        for j in range(K // 128):
            w = tab[s["w"][i, :, 128 * j:128 * j + 128].int()]
            f = torch.exp2(s["w_sf"][i, :, j].double() - 127).repeat_interleave(128)[:N]
            y += torch.matmul(x[:, j], (w * f[:, None]).t())
        out[at:at + n] = y[:, :N // 2] * torch.sigmoid(y[:, :N // 2]) * y[:, N // 2:] if case["gated"] else y
    return out
