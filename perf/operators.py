"""The token-selected operators beside the low-bit projection, as cases.

Three operators whose weights a token selects:

  moe       a mixture-of-experts layer on packed low-bit experts for a few
            tokens (`ttq.moe_lowbit`)
  route     the router that picks a token's experts (`ttq.moe_route`)
  adapters  low-rank adapters of many requests added to one shared
            projection's output (`ttq.adapters_add`)

`own` false runs each in elementary torch operations, `own` true through the
package's calls. A case is a plain dict; `listed()` has the fixed ones and
`draw(rng)` makes more of the same ranges.
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token of an interactive request, many small experts
        dict(name="moe-t1", op="moe", T=1, E=64, top_k=6, K=2048, I=1408,
             bits=4, group=128, dtype="bf16", act="silu", pad=0),
        # a handful of requests, many small experts, fine groups
        dict(name="moe-t5", op="moe", T=5, E=128, top_k=8, K=2048, I=768,
             bits=4, group=32, dtype="bf16", act="silu", pad=0),
        # a decode batch with two padded rows, three-bit codes
        dict(name="moe-t16", op="moe", T=16, E=32, top_k=4, K=2560, I=1728,
             bits=3, group=64, dtype="f16", act="gelu", pad=2),
        # the MLP size of a 7B model as each of few large experts
        dict(name="moe-t33", op="moe", T=33, E=8, top_k=2, K=4096, I=11008,
             bits=4, group=128, dtype="bf16", act="silu", pad=0),
        # a large decode batch over many experts
        dict(name="moe-t64", op="moe", T=64, E=64, top_k=8, K=4096, I=1408,
             bits=5, group=128, dtype="bf16", act="silu", pad=0),
        # the router of one token, and of a prompt chunk
        dict(name="route-t1", op="route", T=1, E=64, top_k=6, K=2048,
             dtype="bf16", wtype="bf16", score="softmax", bias=False,
             renormalize=False),
        dict(name="route-t1000", op="route", T=1000, E=128, top_k=8, K=4096,
             dtype="bf16", wtype="f32", score="sigmoid", bias=True,
             renormalize=True),
        # one token of one request with an adapter
        dict(name="adapters-t1", op="adapters", T=1, L=8, r=16, K=4096,
             N=4096, dtype="bf16", mix="each", none=0.0),
        # a decode batch, every request with an adapter of its own
        dict(name="adapters-t32", op="adapters", T=32, L=32, r=16, K=4096,
             N=11008, dtype="bf16", mix="each", none=0.0),
        # a large decode batch over two dozen adapters, some rows without
        dict(name="adapters-t301", op="adapters", T=301, L=24, r=64, K=4096,
             N=4096, dtype="f16", mix="random", none=0.1),
        # single precision, ragged sizes
        dict(name="adapters-t77-f32", op="adapters", T=77, L=5, r=8, K=1152,
             N=6912, dtype="f32", mix="runs", none=0.2),
        # several prompts in one chunk
        dict(name="adapters-t4096", op="adapters", T=4096, L=16, r=32,
             K=4096, N=11008, dtype="bf16", mix="runs", none=0.0),
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return min(hi, max(lo, int(round(v / step)) * step))


def _draw_moe(rng):
    group = rng.choice([16, 32, 64, 128])
    step = max(32, group)
    E = rng.choice([8, 16, 24, 32, 60, 64, 96, 128])
    c = dict(op="moe", T=_log_int(rng, 1, 64), E=E,
             top_k=rng.randint(1, min(8, E // 2)),
             K=_log_int(rng, 512, 4096, step), I=_log_int(rng, 256, 11008,
                                                          step),
             bits=rng.randint(2, 8), group=group,
             dtype=rng.choice(["bf16", "bf16", "f16", "f32"]),
             act=rng.choice(["silu", "silu", "gelu"]), pad=0)
    if c["T"] > 2 and rng.random() < 0.3:
        c["pad"] = rng.randint(1, c["T"] // 2)
    return c


def _draw_route(rng):
    return dict(op="route", T=_log_int(rng, 1, 1000),
                E=rng.choice([8, 16, 60, 64, 96, 128, 160, 256]),
                top_k=rng.randint(1, 8), K=_log_int(rng, 512, 4096, 8),
                dtype=rng.choice(["bf16", "f16", "f32"]),
                wtype=rng.choice(["bf16", "f16", "f32"]),
                score=rng.choice(["softmax", "sigmoid"]),
                bias=rng.random() < 0.5, renormalize=rng.random() < 0.5)


def _draw_adapters(rng):
    T = _log_int(rng, 1, 4096)
    return dict(op="adapters", T=T, L=rng.randint(1, 64),
                r=rng.choice([4, 8, 16, 24, 32, 48, 64]),
                K=_log_int(rng, 768, 11008, 8),
                N=_log_int(rng, 768, 11008, rng.choice([1, 8, 64])),
                dtype=rng.choice(["bf16", "bf16", "f16", "f32"]),
                mix=rng.choice(["each", "random", "runs"]),
                none=rng.choice([0.0, 0.0, 0.2]))


def draw(rng):
    make = rng.choice([_draw_moe, _draw_moe, _draw_route, _draw_adapters,
                       _draw_adapters])
    while True:
        c = make(rng)
        if c["op"] == "moe":
            # at most the weights and the products of the largest listed case
            if c["E"] * 3 * c["K"] * c["I"] > 1_082_130_432 or \
                    _moe_work(c)["bytes"] > 600_000_000 or \
                    _moe_work(c)["flops"] > 17_000_000_000:
                continue
        if c["op"] == "adapters" and \
                _adapters_work(c)["bytes"] > 215_000_000:
            continue
        return c


# ------------------------------------------------------------------ work

def _size(dtype):
    return 4 if dtype == "f32" else 2


def _moe_work(c):
    live = c["T"] - c["pad"]
    hit = c["E"] * (1 - (1 - c["top_k"] / c["E"]) ** live)
    w = 3 * c["K"] * c["I"]
    b = hit * w * (c["bits"] / 8 + 5 / c["group"]) + hit * c["I"] * 4
    b += c["T"] * (2 * c["K"] * _size(c["dtype"]) + 8 * c["top_k"])
    return {"bytes": int(b + 4 * c["K"]),
            "flops": int(2 * w * live * c["top_k"])}


def _route_work(c):
    b = c["T"] * c["K"] * _size(c["dtype"]) + \
        c["E"] * c["K"] * _size(c["wtype"]) + c["T"] * c["top_k"] * 8
    return {"bytes": b, "flops": 2 * c["T"] * c["E"] * c["K"]}


def _adapters_work(c):
    live = c["T"] * (1 - c["none"])
    hit = min(c["L"], max(1, round(live)))
    if c["mix"] == "random":
        hit = c["L"] * (1 - (1 - 1 / c["L"]) ** live)
    e = _size(c["dtype"])
    b = live * c["K"] * e + 2 * c["T"] * c["N"] * e + \
        hit * c["r"] * (c["K"] + c["N"]) * e
    return {"bytes": int(b),
            "flops": int(2 * live * c["r"] * (c["K"] + c["N"]))}


def work(case):
    return {"moe": _moe_work, "route": _route_work,
            "adapters": _adapters_work}[case["op"]](case)


# ------------------------------------------------------------------ inputs

def _outliers(n, g, frac, factor):
    """Per-channel sizes: a few channels far larger than the rest, as the
    inputs of a language model's projections have them."""
    f = torch.ones(n, device="cuda")
    k = max(1, int(n * frac))
    f[torch.randperm(n, generator=g, device="cuda")[:k]] = factor
    return f


def _scales(sizes):
    """s = c^(1/4) of the shrunk second moment c (alpha 0.5, p 2)."""
    m = sizes * sizes
    return (0.9 * m + 0.1 * m.mean(-1, keepdim=True)) ** 0.25


def _pitch(n, to):
    return (n + to - 1) // to * to


def _quantize(W, bits, group):
    """Group-wise round-to-nearest of W [N, K] into the packed layout: codes
    int32 [N, pitch], delta fp32 and zero uint8 [N, group pitch]."""
    N, K = W.shape
    top = 2 ** bits - 1
    w = W.view(N, K // group, group)
    lo = w.amin(-1).clamp(max=0)
    hi = w.amax(-1).clamp(min=0)
    d = (hi - lo) / top
    d = torch.where(d == 0, torch.ones_like(d), d)
    z = torch.round(-lo / d).clamp(0, top)
    q = (torch.round(w / d[..., None]) + z[..., None]).clamp(0, top)
    q = q.to(torch.int32).view(N, K // 32, 32, 1)
    bit = torch.arange(bits, device=W.device, dtype=torch.int32)
    at = torch.arange(32, device=W.device, dtype=torch.int32)
    stream = ((q >> bit) & 1).view(N, K // 32, bits, 32)
    words = (stream << at).sum(-1, dtype=torch.int32).view(N, -1)
    codes = torch.zeros(N, _pitch(K * bits // 32, 4), dtype=torch.int32,
                        device=W.device)
    codes[:, :words.shape[1]] = words
    delta = torch.zeros(N, _pitch(K // group, 16), device=W.device)
    zero = torch.zeros(N, delta.shape[1], dtype=torch.uint8, device=W.device)
    delta[:, :K // group] = d
    zero[:, :K // group] = z.to(torch.uint8)
    return codes, delta, zero


def _experts(E, N, K, s, bits, group, g):
    """E quantized [N, K] weights stacked by rows; s [E or 1, K]."""
    parts = []
    for e in range(E):
        W = torch.randn(N, K, generator=g, device="cuda") / math.sqrt(K)
        parts.append(_quantize(W * s[e % s.shape[0]], bits, group))
    return tuple(torch.cat(p) for p in zip(*parts))


def _prepare_moe(c, g):
    T, E, k, K, I = c["T"], c["E"], c["top_k"], c["K"], c["I"]
    sizes = _outliers(K, g, 0.005, 20.0)
    X = torch.randn(T, K, generator=g, device="cuda") * sizes
    # experts are not equally popular
    popular = 0.7 * torch.randn(E, generator=g, device="cuda")
    logits = torch.randn(T, E, generator=g, device="cuda") + popular
    vals, ids = torch.topk(logits, k, dim=-1)
    weights = torch.softmax(vals, -1)
    ids = ids.to(torch.int32)
    if c["pad"]:
        ids[T - c["pad"]:] = -1
    s_in = _scales(sizes)[None]
    mid = torch.exp(0.7 * torch.randn(E, I, generator=g, device="cuda"))
    s_mid = _scales(mid)
    up = _experts(E, 2 * I, K, s_in, c["bits"], c["group"], g)
    down = _experts(E, K, I, s_mid, c["bits"], c["group"], g)
    return dict(c=c, X=X.to(DT[c["dtype"]]), ids=ids.contiguous(),
                weights=weights.contiguous(), inv_s=1 / s_in[0], up=up,
                inv_s_mid=(1 / s_mid).contiguous(), down=down)


def _prepare_route(c, g):
    X = torch.randn(c["T"], c["K"], generator=g, device="cuda")
    W = torch.randn(c["E"], c["K"], generator=g, device="cuda")
    W = W * 1.5 / math.sqrt(c["K"])
    bias = 0.1 * torch.randn(c["E"], generator=g, device="cuda") \
        if c["bias"] else None
    return dict(c=c, X=X.to(DT[c["dtype"]]), W=W.to(DT[c["wtype"]]),
                bias=bias)


def _prepare_adapters(c, g):
    T, L, r, K, N, dt = c["T"], c["L"], c["r"], c["K"], c["N"], DT[c["dtype"]]
    X = torch.randn(T, K, generator=g, device="cuda")
    X = X * _outliers(K, g, 0.005, 20.0)
    A = torch.randn(L, r, K, generator=g, device="cuda") / math.sqrt(K)
    B = torch.randn(L, N, r, generator=g, device="cuda") / math.sqrt(r)
    Y = torch.randn(T, N, generator=g, device="cuda")
    scale = 0.25 + torch.rand(L, generator=g, device="cuda")
    if c["mix"] == "each":        # token t has adapter t, wrapped
        index = torch.randperm(T, generator=g, device="cuda") % L
    elif c["mix"] == "random":
        index = torch.randint(0, L, (T,), generator=g, device="cuda")
    else:                         # one request's tokens stand together
        index = torch.randint(0, L, (T,), generator=g, device="cuda")
        index = torch.sort(index).values.roll(T // 3)
    drop = torch.rand(T, generator=g, device="cuda") < c["none"]
    index = torch.where(drop, torch.full_like(index, -1), index)
    st = dict(c=c, X=X.to(dt), A=A.to(dt), B=B.to(dt), Y=Y.to(dt),
              scale=scale, index=index.to(torch.int32), plan=None)
    if own:  # a batch's plan serves every projection of every layer
        from test_weight_quantization_b200 import ttq
        st["plan"] = ttq.adapters_plan(st["index"], L)
    return st


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return {"moe": _prepare_moe, "route": _prepare_route,
            "adapters": _prepare_adapters}[case["op"]](case, g)


# ------------------------------------------------------------------ plain

def _dequantize(packed, K, bits, group):
    """(q - z) * delta of the packed layout, fp32 [N, K]."""
    codes, delta, zero = packed
    N, dev = codes.shape[0], codes.device
    words = codes[:, :K * bits // 32].reshape(N, K // 32, bits)
    bit = torch.arange(32, device=dev) * bits
    wd, sh = bit // 32, (bit % 32).to(torch.int32)
    low = torch.clamp(32 - sh, max=bits)            # bits in the first word
    q = (words[..., wd] >> sh) & ((1 << low) - 1)
    high = words[..., torch.clamp(wd + 1, max=bits - 1)]
    q = q | ((high & ((1 << (bits - low)) - 1)) << low)
    q = q.view(N, K // group, group).to(torch.float32)
    G = K // group
    w = (q - zero[:, :G, None].to(torch.float32)) * delta[:, :G, None]
    return w.view(N, K)


def _plain_moe(st):
    c = st["c"]
    T, E, K, I = c["T"], c["E"], c["K"], c["I"]
    x = st["X"].float() * st["inv_s"]
    w1 = _dequantize(st["up"], K, c["bits"], c["group"])
    gu = (x @ w1.t()).view(T, E, 2 * I)
    del w1
    gate, up = gu[..., :I], gu[..., I:]
    if c["act"] == "silu":
        gate = gate / (1 + torch.exp(-gate))
    else:
        inner = math.sqrt(2 / math.pi) * (gate + 0.044715 * gate ** 3)
        gate = 0.5 * gate * (1 + torch.tanh(inner))
    h = gate * up * st["inv_s_mid"]                              # [T, E, I]
    w2 = _dequantize(st["down"], I, c["bits"], c["group"]).view(E, K, I)
    y = torch.bmm(h.transpose(0, 1), w2.transpose(1, 2))         # [E, T, K]
    ids = st["ids"].long()
    live = ids >= 0
    share = torch.zeros(T, E, device=x.device)
    share.scatter_add_(1, ids.clamp(min=0),
                       torch.where(live, st["weights"], 0.0))
    return (share.t()[:, :, None] * y).sum(0).to(st["X"].dtype)


def _plain_route(st):
    c = st["c"]
    # scores next to one another decide which expert is picked: 64 bits
    logits = st["X"].double() @ st["W"].double().t()
    if c["score"] == "softmax":
        score = torch.softmax(logits, -1)
        rank = logits
    else:
        score = torch.sigmoid(logits)
        rank = score
    if st["bias"] is not None:
        rank = score + st["bias"].double()
    ids = torch.sort(rank, dim=-1, descending=True, stable=True).indices
    ids = ids[:, :c["top_k"]]
    w = torch.gather(score, 1, ids)
    if c["renormalize"]:
        w = w / w.sum(-1, keepdim=True)
    return ids.to(torch.int32), w.to(torch.float32)


def _plain_adapters(st):
    index = st["index"].long()
    live = index >= 0
    L, r, K = st["A"].shape
    # every adapter's U, then each token's own: no adapter is gathered whole
    U = (st["X"].float() @ st["A"].float().view(L * r, K).t())
    pick = torch.arange(L, device=index.device) == index[:, None]
    U = U.view(-1, L, r) * (pick * st["scale"])[:, :, None]
    B = st["B"].float().transpose(0, 1).reshape(-1, L * r)
    y = st["Y"].float()
    y = y + torch.where(live[:, None], U.view(-1, L * r) @ B.t(), 0.0)
    return y.to(st["Y"].dtype)


# ------------------------------------------------------------------ run

def _own_moe(st):
    from test_weight_quantization_b200 import ttq
    c = st["c"]
    return ttq.moe_lowbit(st["X"], st["ids"], st["weights"], st["inv_s"],
                          st["up"], st["inv_s_mid"], st["down"], c["bits"],
                          c["group"], act=c["act"])


def _own_route(st):
    from test_weight_quantization_b200 import ttq
    c = st["c"]
    return ttq.moe_route(st["X"], st["W"], c["top_k"], bias=st["bias"],
                         score=c["score"], renormalize=c["renormalize"])


def _own_adapters(st):
    from test_weight_quantization_b200 import ttq
    return ttq.adapters_add(st["X"], st["A"], st["B"], st["plan"], st["Y"],
                            scale=st["scale"], out=torch.empty_like(st["Y"]))


def run(state):
    op = state["c"]["op"]
    if own:
        return {"moe": _own_moe, "route": _own_route,
                "adapters": _own_adapters}[op](state)
    return {"moe": _plain_moe, "route": _plain_route,
            "adapters": _plain_adapters}[op](state)


# ------------------------------------------------------------------ exact

def _expert_rows(packed, e, rows, K, bits, group):
    """Expert e's weight in 64 bits, read code by code from its bit stream."""
    codes, delta, zero = (p[e * rows:(e + 1) * rows] for p in packed)
    words = codes.long() & 0xFFFFFFFF
    W = torch.empty(rows, K, dtype=torch.float64, device=codes.device)
    for j in range(32):  # code j of every 32-code block
        first, sh = divmod(j * bits, 32)
        cols = torch.arange(K // 32, device=codes.device) * bits + first
        v = words[:, cols] >> sh
        if sh + bits > 32:
            v = v | (words[:, cols + 1] << (32 - sh))
        G = (torch.arange(K // 32, device=codes.device) * 32 + j) // group
        W[:, j::32] = ((v & (2 ** bits - 1)).double() -
                       zero[:, G].double()) * delta[:, G].double()
    return W


def _exact_moe(st):
    c = st["c"]
    K, I = c["K"], c["I"]
    x = st["X"].double() * st["inv_s"].double()
    y = torch.zeros(c["T"], K, dtype=torch.float64, device=x.device)
    for e in torch.unique(st["ids"]).tolist():
        if e < 0:
            continue
        t, slot = torch.nonzero(st["ids"] == e, as_tuple=True)
        W1 = _expert_rows(st["up"], e, 2 * I, K, c["bits"], c["group"])
        a = torch.einsum("nk,tk->tn", W1[:I], x[t])
        b = torch.einsum("nk,tk->tn", W1[I:], x[t])
        if c["act"] == "silu":
            a = a * torch.sigmoid(a)
        else:
            a = torch.nn.functional.gelu(a, approximate="tanh")
        h = a * b * st["inv_s_mid"][e].double()
        W2 = _expert_rows(st["down"], e, K, I, c["bits"], c["group"])
        y.index_add_(0, t, torch.einsum("ni,ti->tn", W2, h) *
                     st["weights"][t, slot].double()[:, None])
    return y


def _exact_route(st):
    c = st["c"]
    z = torch.einsum("tk,ek->te", st["X"].double(), st["W"].double())
    p = torch.exp(z - z.amax(1, keepdim=True)) if c["score"] == "softmax" \
        else 1 / (1 + torch.exp(-z))
    if c["score"] == "softmax":
        p = p / p.sum(1, keepdim=True)
    left = (z if c["score"] == "softmax" and st["bias"] is None else p).clone()
    if st["bias"] is not None:
        left = left + st["bias"].double()
    ids, w = [], []
    rows = torch.arange(c["T"], device=z.device)
    for _ in range(c["top_k"]):
        best = left.amax(1, keepdim=True)
        e = (left == best).to(torch.int8).argmax(1)  # the lowest index
        ids.append(e)
        w.append(p[rows, e])
        left[rows, e] = -math.inf
    w = torch.stack(w, 1)
    if c["renormalize"]:
        w = w / w.sum(1, keepdim=True)
    return torch.stack(ids, 1).to(torch.int32), w


def _exact_adapters(st):
    y = st["Y"].double()
    for a in torch.unique(st["index"]).tolist():
        if a < 0:
            continue
        t = torch.nonzero(st["index"] == a)[:, 0]
        u = st["X"][t].double() @ st["A"][a].double().t()
        y[t] += st["scale"][a].double() * (u @ st["B"][a].double().t())
    return y


def exact(case, seed):
    st = prepare(case, seed)
    return {"moe": _exact_moe, "route": _exact_route,
            "adapters": _exact_adapters}[case["op"]](st)
