"""The calls on weights a token selects (router, low-bit experts, request
adapters) against plain implementations in 64 bits.

Tolerances are bounds, not fits. Notation: a value rounded to a type t is off
by at most eps(t)/2 relative. The kernels keep
  - the activations x and h of the experts in one fp16 term for a bf16 output
    (2^-11) and in two for fp16 and fp32 outputs (the second term rounds a
    residual of at most 2^-11: 2^-22), scaled by a power of two so that the
    row's largest value is near fp16's top: what falls below fp16's normal
    range is off by at most 2^-24 of a unit at a largest value of 2^13, 2^-37
    of that value in the first term;
  - the adapters' U = X A^T in two 16-bit terms (bf16: 2^-16, fp16: 2^-22) or
    three bf16 terms (2^-24);
  - every sum in fp32: n additions are off by at most n 2^-23 of the sum of
    the terms' sizes (2^-23 and not 2^-24: a tensor-core addition may
    truncate).
Each bound is carried through the formulas with absolute values, element by
element."""
import math
import zlib

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11,
        torch.float32: 2.0 ** -24}
TERMS = {torch.bfloat16: 2.0 ** -11, torch.float16: 2.0 ** -21,
         torch.float32: 2.0 ** -21}
UTERM = {torch.bfloat16: 2.0 ** -16, torch.float16: 2.0 ** -21,
         torch.float32: 2.0 ** -23}


@pytest.fixture(scope="module")
def ttq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from test_weight_quantization_b200 import ttq as mod
    mod.device_error(clear=True)
    return mod


def gen(*key):
    return torch.Generator().manual_seed(zlib.crc32(repr(key).encode()))


def dense(packed, N, K, bits, group):
    """(q - z) * delta in 64 bits, [N, K]."""
    c, d, z = (p.cpu().numpy() for p in packed)
    c = c.view(np.uint32)[:, :K * bits // 32]  # without the pitch's padding
    q = oracle.unpack_codes(c, K, bits).astype(np.float64)
    G = K // group
    w = (q.reshape(N, G, group) - z[:, :G, None]) * \
        d[:, :G, None].astype(np.float64)
    return torch.from_numpy(w.reshape(N, K))


# ------------------------------------------------------------------- experts

def silu(v):
    return v * torch.sigmoid(v)


def gelu(v):
    return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) *
                                     (v + 0.044715 * v ** 3)))


def make_moe(ttq, T, E, k, K, I, bits, group, dt, seed=0, size=1.0,
             ids=None):
    g = gen("moe", T, E, k, K, I, bits, group, seed)
    X = (torch.randn(T, K, generator=g) * size).to(dt).cuda()
    W1 = (torch.randn(E * 2 * I, K, generator=g) / math.sqrt(K)).cuda()
    W2 = (torch.randn(E * K, I, generator=g) / math.sqrt(I)).cuda()
    s = torch.exp(0.5 * torch.randn(K, generator=g)).cuda()
    s_mid = torch.exp(0.5 * torch.randn(E, I, generator=g))
    up = ttq.quantize_rtn_grouped(W1, s, bits, group)
    parts = [ttq.quantize_rtn_grouped(W2[e * K:(e + 1) * K],
                                      s_mid[e].cuda(), bits, group)
             for e in range(E)]
    down = tuple(torch.cat(p).contiguous() for p in zip(*parts))
    if ids is None:
        ids = torch.stack([torch.randperm(E, generator=g)[:k]
                           for _ in range(T)])
    w = torch.rand(T, k, generator=g)
    return dict(X=X, ids=ids.to(torch.int32).cuda(), weights=w.cuda(),
                inv_s=1 / s, up=up, inv_s_mid=(1 / s_mid).contiguous().cuda(),
                down=down, bits=bits, group=group)


def moe_reference(m, act, out_dt):
    """(Y, bound) in 64 bits on the host."""
    X, ids, w = m["X"].double().cpu(), m["ids"].cpu(), m["weights"].double()
    w = w.cpu()
    bits, group = m["bits"], m["group"]
    E, I = m["inv_s_mid"].shape
    T, K = X.shape
    W1 = dense(m["up"], E * 2 * I, K, bits, group).view(E, 2 * I, K)
    W2 = dense(m["down"], E * K, I, bits, group).view(E, K, I)
    mid = m["inv_s_mid"].double().cpu()
    x = X * m["inv_s"].double().cpu()
    term = TERMS[out_dt]
    Y, err = torch.zeros(T, K, dtype=torch.float64), \
        torch.zeros(T, K, dtype=torch.float64)
    f = silu if act == "silu" else gelu
    n1, n2 = (K / 8 + 64) * 2.0 ** -23, (I / 8 + 64) * 2.0 ** -23
    for t in range(T):
        top = x[t].abs().max()
        ex = x[t].abs() * term + top * 2.0 ** -36
        for j in range(ids.shape[1]):
            e = int(ids[t, j])
            if e < 0 or e >= E:
                continue
            gu, size = W1[e] @ x[t], W1[e].abs() @ x[t].abs()
            egu = W1[e].abs() @ ex + n1 * size
            g, u, eg, eu = gu[:I], gu[I:], egu[:I], egu[I:]
            # |act'| <= 1.13 for both; the function itself in fp32
            a = f(g)
            ea = 1.13 * eg + 2.0 ** -20 * (a.abs() + g.abs() * 2.0 ** -4)
            h = a * u * mid[e]
            eh = (ea * (u.abs() + eu) + a.abs() * eu) * mid[e] + \
                h.abs() * 2.0 ** -22
            eh = eh + h.abs() * term + h.abs().max() * 2.0 ** -36
            y = W2[e] @ h
            ey = W2[e].abs() @ eh + n2 * (W2[e].abs() @ h.abs())
            Y[t] += w[t, j] * y
            err[t] += w[t, j].abs() * (ey + ids.shape[1] * 2.0 ** -22 *
                                       y.abs())
    return Y, err + HALF[out_dt] * (Y.abs() + err) + 1e-30


def check_moe(ttq, m, act="silu", out_dt=None, **kw):
    out_dt = out_dt or m["X"].dtype
    got = ttq.moe_lowbit(m["X"], m["ids"], m["weights"], m["inv_s"], m["up"],
                         m["inv_s_mid"], m["down"], m["bits"], m["group"],
                         act=act, out_dtype=out_dt, **kw)
    ref, bound = moe_reference(m, act, out_dt)
    err = (got.double().cpu() - ref).abs()
    assert torch.isfinite(got).all()
    worst = (err / bound).max().item()
    assert worst <= 1, f"error {worst:.3g} of its bound"
    # the same in the 2-norm, where roundings do not add up: three rounded
    # operands (x into both factors, h) and the output's rounding
    fro = (err.norm() / max(ref.norm().item(), 1e-300)).item()
    assert fro <= HALF[out_dt] + 4 * TERMS[out_dt], f"{fro:.3g}"
    return got


@pytest.mark.parametrize("bits", [2, 3, 4, 5, 6, 7, 8])
@pytest.mark.parametrize("group", [16, 32, 64, 128])
def test_moe_every_width_and_group(ttq, bits, group):
    m = make_moe(ttq, 3, 4, 2, 256, 384, bits, group, torch.bfloat16)
    check_moe(ttq, m)
    check_moe(ttq, m, out_dt=torch.float32)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("out_dt", [torch.float32, torch.bfloat16,
                                    torch.float16])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_moe_types(ttq, dt, out_dt, act):
    check_moe(ttq, make_moe(ttq, 5, 3, 2, 160, 96, 4, 32, dt), act, out_dt)


@pytest.mark.parametrize("T,E,k,K,I,bits,group", [
    (1, 1, 1, 32, 32, 4, 32),        # the smallest
    (1, 8, 8, 96, 32, 3, 16),        # every expert, one token
    (2, 512, 3, 32, 32, 2, 16),      # the most experts
    (7, 5, 4, 2080, 160, 4, 32),     # K past the 128-channel chunks
    (9, 2, 1, 288, 1056, 5, 32),     # nine tokens: one past a column tile
    (17, 2, 2, 160, 224, 4, 32),     # all tokens on both experts
    (33, 1, 1, 128, 128, 8, 128),    # one past the widest column tile
    (64, 3, 3, 128, 256, 4, 128),    # the most tokens, two column tiles
    (64, 40, 32, 64, 64, 6, 64),     # the most choices
    (16, 16, 2, 4096, 64, 4, 64),    # wide in, narrow middle
    (16, 16, 2, 64, 4096, 4, 64),    # narrow out, wide middle
    (16, 64, 8, 64, 1024, 4, 32),    # whole rounds of tiles per CTA
    (12, 64, 8, 160, 1024, 3, 16),   # and a rest, chunks that end early
])
def test_moe_sizes(ttq, T, E, k, K, I, bits, group):
    check_moe(ttq, make_moe(ttq, T, E, k, K, I, bits, group, torch.bfloat16))


def test_moe_padding_repeats_and_empty_rows(ttq):
    ids = torch.tensor([[2, 2, -1], [-1, -1, -1], [0, 1, 0], [3, -1, 3],
                        [-5, 1, 1]])
    m = make_moe(ttq, 5, 4, 3, 128, 96, 4, 32, torch.bfloat16, ids=ids)
    Y = check_moe(ttq, m)
    assert (Y[1] == 0).all()
    # nobody has an expert
    m["ids"].fill_(-1)
    Y = ttq.moe_lowbit(m["X"], m["ids"], m["weights"], m["inv_s"], m["up"],
                       m["inv_s_mid"], m["down"], 4, 32)
    assert (Y == 0).all()
    assert ttq.device_error() == 0


def test_moe_expert_out_of_range_adds_nothing_and_is_flagged(ttq):
    m = make_moe(ttq, 3, 4, 2, 128, 96, 4, 32, torch.bfloat16)
    m["ids"][0, 1] = 4
    m["ids"][2, 0] = 2 ** 31 - 1
    check_moe(ttq, m)
    assert ttq.device_error() == ttq.DEVERR_INDEX


@pytest.mark.parametrize("size", [1e-4, 3e3])
@pytest.mark.parametrize("out_dt", [torch.bfloat16, torch.float32])
def test_moe_small_and_large_activations(ttq, size, out_dt):
    m = make_moe(ttq, 3, 4, 2, 128, 96, 4, 32, torch.float32, size=size)
    check_moe(ttq, m, out_dt=out_dt)


def test_moe_pitched_rows_workspace_and_untouched_memory(ttq):
    m = make_moe(ttq, 6, 4, 2, 128, 96, 3, 32, torch.bfloat16)
    wide = torch.full((6, 200), 7.0, dtype=torch.bfloat16, device="cuda")
    wide[:, :128] = m["X"]
    plain = check_moe(ttq, m)
    m["X"] = wide[:, :128]
    need = ttq.moe_lowbit_workspace_size(6, 128, 96, 2)
    ws = torch.full((need + 64,), 171, dtype=torch.uint8, device="cuda")
    out = torch.full((7, 131), 5.0, dtype=torch.bfloat16, device="cuda")
    ttq.moe_lowbit(m["X"], m["ids"], m["weights"], m["inv_s"], m["up"],
                   m["inv_s_mid"], m["down"], 3, 32, out=out[:6, :128],
                   workspace=ws[:need])
    torch.cuda.synchronize()
    assert torch.equal(out[:6, :128], plain)
    assert (out[:6, 128:] == 5).all() and (out[6] == 5).all()
    assert (ws[need:] == 171).all()
    assert (wide[:, 128:] == 7).all()


def test_moe_a_bad_token_stays_alone(ttq):
    """NaN and infinity in one token leave the other rows' bits alone, also
    where they share an expert."""
    m = make_moe(ttq, 10, 2, 2, 128, 96, 4, 32, torch.bfloat16)
    good = check_moe(ttq, m)
    for bad in (float("nan"), float("inf")):
        X = m["X"].clone()
        X[4, 17] = bad
        got = ttq.moe_lowbit(X, m["ids"], m["weights"], m["inv_s"], m["up"],
                             m["inv_s_mid"], m["down"], 4, 32)
        keep = torch.arange(10) != 4
        assert torch.equal(got[keep], good[keep])
        assert not torch.isfinite(got[4]).any()


def test_moe_repeats_bit_for_bit_and_is_captured(ttq):
    m = make_moe(ttq, 16, 8, 4, 512, 256, 4, 64, torch.float16)
    ws = torch.empty(ttq.moe_lowbit_workspace_size(16, 512, 256, 4),
                     dtype=torch.uint8, device="cuda")
    out = torch.empty(16, 512, dtype=torch.float16, device="cuda")

    def call(o):
        return ttq.moe_lowbit(m["X"], m["ids"], m["weights"], m["inv_s"],
                              m["up"], m["inv_s_mid"], m["down"], 4, 64,
                              out=o, workspace=ws)
    first = call(out).clone()
    for _ in range(5):
        assert torch.equal(call(out), first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call(out)
    # replayed on other inputs: nothing of the capture's inputs is kept
    m2 = make_moe(ttq, 16, 8, 4, 512, 256, 4, 64, torch.float16, seed=1)
    second = ttq.moe_lowbit(m2["X"], m2["ids"], m2["weights"], m2["inv_s"],
                            m["up"], m["inv_s_mid"], m["down"], 4, 64)
    m["X"].copy_(m2["X"])
    m["ids"].copy_(m2["ids"])
    m["weights"].copy_(m2["weights"])
    m["inv_s"].copy_(m2["inv_s"])
    for _ in range(3):
        out.fill_(0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, second)


def test_moe_on_two_streams_at_once(ttq):
    ms = [make_moe(ttq, 8, 8, 4, 512, 512, 4, 64, torch.bfloat16, seed=i)
          for i in range(2)]

    def call(m):
        return ttq.moe_lowbit(m["X"], m["ids"], m["weights"], m["inv_s"],
                              m["up"], m["inv_s_mid"], m["down"], 4, 64)
    want = [call(m) for m in ms]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ms]
    got = [[], []]
    for _ in range(10):
        for i, m in enumerate(ms):
            with torch.cuda.stream(streams[i]):
                got[i].append(call(m))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in got[i])


# -------------------------------------------------------------------- router

def route_reference(X, W, bias, score):
    """(scores, ranking values, error of the logits [T, 1]) in 64 bits."""
    x, w = X.double().cpu(), W.double().cpu()
    z = x @ w.t()
    # at most K/32 + 48 fp32 additions in one partial sum
    ez = ((x.abs() @ w.abs().t()) * (X.shape[1] / 32 + 48) *
          2.0 ** -23).amax(1, keepdim=True)
    p = torch.softmax(z, -1) if score == "softmax" else torch.sigmoid(z)
    rank = z if score == "softmax" and bias is None else p
    if bias is not None:
        rank = rank + bias.double().cpu()
    return p, rank, ez


@pytest.mark.parametrize("T,E,k,K,dt,wt,score,bias,renorm", [
    (1, 1, 1, 8, torch.bfloat16, torch.bfloat16, "softmax", False, True),
    (1, 64, 6, 2048, torch.bfloat16, torch.bfloat16, "softmax", False, False),
    (3, 60, 4, 1000, torch.float16, torch.float16, "softmax", True, True),
    (17, 128, 8, 712, torch.bfloat16, torch.float32, "sigmoid", True, True),
    (33, 512, 32, 264, torch.float32, torch.float32, "sigmoid", False, False),
    (130, 33, 5, 520, torch.float16, torch.float32, "softmax", False, True),
    (65, 100, 7, 1032, torch.float32, torch.bfloat16, "softmax", True, False),
    (300, 256, 8, 128, torch.bfloat16, torch.float16, "sigmoid", False, True),
    (16, 16, 16, 40, torch.float16, torch.bfloat16, "softmax", False, True),
    (700, 64, 4, 1536, torch.bfloat16, torch.float32, "softmax", False, True),
    (601, 512, 3, 136, torch.float16, torch.float16, "sigmoid", True, True),
])
def test_route(ttq, T, E, k, K, dt, wt, score, bias, renorm):
    g = gen("route", T, E, k, K, score)
    X = torch.randn(T, K, generator=g).to(dt).cuda()
    W = (torch.randn(E, K, generator=g) * 1.5 / math.sqrt(K)).to(wt).cuda()
    b = (0.1 * torch.randn(E, generator=g)).cuda() if bias else None
    ids, w = ttq.moe_route(X, W, k, bias=b, score=score, renormalize=renorm,
                           scaling=2.5)
    p, rank, ez = route_reference(X, W, b, score)
    best = torch.sort(rank, dim=-1, descending=True, stable=True)
    got = ids.cpu().long()
    # every row: the i-th choice ranks within the logits' error of the i-th
    # best (|d softmax|, |d sigmoid| <= |d logit|), none is taken twice
    off = (torch.gather(rank, 1, got) - best.values[:, :k]).abs()
    assert (off <= 2 * ez).all(), (off / ez).max()
    assert all(len(set(r)) == k for r in got.tolist())
    # where the neighbours are further apart than that, the very expert
    gaps = torch.full((T, E + 1), math.inf, dtype=torch.float64)
    gaps[:, 1:E] = best.values[:, :-1] - best.values[:, 1:]
    apart = torch.minimum(gaps[:, :k], gaps[:, 1:k + 1]) > 2 * ez
    assert torch.equal(got[apart], best.indices[:, :k][apart])
    # and nearly everywhere, since real errors are far below the bound
    assert (got == best.indices[:, :k]).double().mean() > 0.999
    rw = torch.gather(p, 1, got)
    if renorm:
        rw = rw / rw.sum(1, keepdim=True)
    rw = rw * 2.5
    err = (w.double().cpu() - rw).abs()
    # d log softmax and d log sigmoid are at most 2 d logit; twice that
    # for the renormalised quotient
    assert (err <= rw * (4 * ez + 2.0 ** -23) + 1e-40).all()


def test_route_ties_go_to_the_lowest_expert(ttq):
    W = torch.randn(1, 64, generator=gen(1)).repeat(40, 1).cuda()
    W[7] *= 2
    W[31] = W[7]
    X = W[:1].clone()
    for score in ("softmax", "sigmoid"):
        ids, w = ttq.moe_route(X, W * 0.05, 6, score=score)
        assert ids[0].tolist() == [7, 31, 0, 1, 2, 3]
        assert torch.allclose(w.sum(), torch.ones((), device="cuda"))
    # bias decides alone where the scores are equal
    bias = torch.zeros(40, device="cuda")
    bias[22], bias[5] = 3.0, 2.0
    ids, _ = ttq.moe_route(X, W * 0.05, 2, bias=bias, score="sigmoid")
    assert ids[0].tolist() == [22, 5]


def test_route_nan_ranks_last_and_ids_stay_valid(ttq):
    X = torch.randn(5, 64, generator=gen(2)).cuda()
    W = torch.randn(12, 64, generator=gen(3)).cuda() * 0.1
    good, _ = ttq.moe_route(X, W, 4)
    X2 = X.clone()
    X2[2, 5] = float("nan")
    X2[3, 5] = float("inf")
    ids, w = ttq.moe_route(X2, W, 4)
    assert torch.equal(ids[[0, 1, 4]], good[[0, 1, 4]])
    assert ids[2].tolist() == [0, 1, 2, 3] and torch.isnan(w[2]).all()
    for row in ids.tolist():
        assert len(set(row)) == 4 and all(0 <= e < 12 for e in row)
    # one expert with a NaN row never displaces a number under sigmoid
    W[4, 0] = float("nan")
    ids, _ = ttq.moe_route(X, W, 11, score="sigmoid")
    assert (ids != 4).all()
    ids, _ = ttq.moe_route(X, W, 12, score="sigmoid")
    assert (ids[:, 11] == 4).all()


def test_route_pitched_rows_and_all_zero_scores(ttq):
    X = torch.randn(9, 96, generator=gen(4)).cuda()
    W = torch.randn(24, 136, generator=gen(5)).cuda()
    wide = torch.full((9, 128), 9.0, device="cuda")
    wide[:, :96] = X
    a = ttq.moe_route(X, W[:, :96].contiguous(), 3)
    b = ttq.moe_route(wide[:, :96], W[:, :96], 3)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    # sigmoids that underflow to nothing: weights of 0, not NaN
    X1 = torch.full((1, 8), 1e4, device="cuda")
    ids, w = ttq.moe_route(X1, torch.full((4, 8), -1.0, device="cuda"), 2,
                           score="sigmoid")
    assert ids[0].tolist() == [0, 1] and (w == 0).all()


# ------------------------------------------------------------------ adapters

def make_adapters(T, L, r, K, N, dt, ydt=None, seed=0):
    g = gen("ad", T, L, r, K, N, seed)
    return dict(X=torch.randn(T, K, generator=g).to(dt).cuda(),
                A=(torch.randn(L, r, K, generator=g) /
                   math.sqrt(K)).to(dt).cuda(),
                B=torch.randn(L, N, r, generator=g).to(dt).cuda(),
                Y=torch.randn(T, N, generator=g).to(ydt or dt).cuda(),
                scale=(torch.rand(L, generator=g) * 2 - 0.5).cuda(),
                index=torch.randint(-1, L, (T,), generator=g,
                                    dtype=torch.int32).cuda())


def adapters_reference(a, scale):
    X, A, B, Y = (a[n].double().cpu() for n in "XABY")
    K, r = A.shape[2], A.shape[1]
    dt = a["X"].dtype
    out, err = Y.clone(), torch.zeros_like(Y)
    live = torch.zeros(Y.shape[0], dtype=torch.bool)
    for t, i in enumerate(a["index"].cpu().tolist()):
        if i < 0 or i >= A.shape[0]:
            continue
        live[t] = True
        s = 1.0 if scale is None else float(scale[i].double())
        U, size = A[i] @ X[t], A[i].abs() @ X[t].abs()
        eU = size * (K / 8 + 64) * 2.0 ** -23 + U.abs() * UTERM[dt] + \
            U.abs().max() * 2.0 ** -30
        out[t] += s * (B[i] @ U)
        err[t] = abs(s) * (B[i].abs() @ (eU + U.abs() * (r + 8) * 2.0 ** -23))
    h = HALF[a["Y"].dtype]
    return out, err + h * (out.abs() + err) + 2.0 ** -22 * Y.abs(), live


def check_adapters(ttq, a, scale="given", in_place=False):
    scale = a["scale"] if scale == "given" else None
    plan = ttq.adapters_plan(a["index"], a["A"].shape[0])
    ref, bound, live = adapters_reference(a, scale)
    Y = a["Y"].clone()
    out = None if in_place else torch.full_like(Y, float("nan"))
    got = ttq.adapters_add(a["X"], a["A"], a["B"], plan, Y, scale=scale,
                           out=out)
    if not in_place:
        assert torch.equal(Y, a["Y"])
    assert torch.equal(got.cpu()[~live], a["Y"].cpu()[~live])
    err = (got.double().cpu() - ref).abs()
    worst = (err / bound)[live].max().item() if live.any() else 0.0
    assert worst <= 1, f"error {worst:.3g} of its bound"
    return got


@pytest.mark.parametrize("T,L,r,K,N", [
    (1, 1, 4, 8, 1),            # the smallest
    (1, 8, 16, 256, 320),
    (5, 3, 8, 72, 33),          # N odd: rows that start off 16 bytes
    (8, 8, 12, 1000, 100),
    (9, 2, 16, 264, 136),       # nine tokens on few adapters
    (33, 1, 64, 512, 512),      # one past a tile
    (100, 40, 20, 136, 257),
    (257, 5, 32, 640, 384),
    (64, 3, 48, 2056, 1544),
    (700, 1000, 24, 128, 64),   # more adapters than tokens
])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16, torch.float16])
def test_adapters_sizes(ttq, T, L, r, K, N, dt):
    a = make_adapters(T, L, r, K, N, dt)
    out = check_adapters(ttq, a)
    assert torch.equal(check_adapters(ttq, a, in_place=True), out)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("ydt", [torch.float32, torch.bfloat16,
                                 torch.float16])
def test_adapters_types(ttq, dt, ydt):
    a = make_adapters(40, 4, 16, 256, 272, dt, ydt)
    check_adapters(ttq, a)
    check_adapters(ttq, a, scale=None, in_place=True)


def test_adapters_nobody_everybody_and_out_of_range(ttq):
    a = make_adapters(50, 6, 16, 128, 96, torch.bfloat16)
    a["index"].fill_(-1)
    check_adapters(ttq, a)
    a["index"].fill_(5)
    check_adapters(ttq, a)
    assert ttq.device_error() == 0
    a["index"][3] = 6
    a["index"][9] = 2 ** 31 - 1
    a["index"][11] = -2 ** 31
    check_adapters(ttq, a)
    assert ttq.device_error() == ttq.DEVERR_INDEX


def test_adapters_plan_covers_every_token_once(ttq):
    for T, L in ((1, 1), (31, 3), (32, 1), (1025, 70), (5000, 8192)):
        index = torch.randint(-1, L, (T,), generator=gen(T),
                              dtype=torch.int32).cuda()
        plan = ttq.adapters_plan(index, L).cpu()
        n, tile = int(plan[0]), int(plan[1])
        most = min(T, (T + tile - 1) // tile + L + 1)
        assert n <= most
        tiles = plan[4:4 + 4 * n].view(n, 4).tolist()
        order = plan[4 + 4 * most:4 + 4 * most + T]
        assert torch.equal(order.sort().values, torch.arange(T).int())
        at = 0
        for ad, start, count, _ in tiles:
            assert start == at and 1 <= count <= tile
            at += count
            assert (index.cpu()[order[start:start + count].long()] ==
                    ad).all()
        assert at == T


def test_adapters_a_plan_of_another_batch_is_flagged(ttq):
    a = make_adapters(20, 4, 16, 128, 96, torch.bfloat16)
    big = ttq.adapters_plan(torch.zeros(40, dtype=torch.int32,
                                        device="cuda"), 4)
    out = torch.full_like(a["Y"], 3.0)
    ttq.adapters_add(a["X"], a["A"], a["B"], big, a["Y"], out=out)
    torch.cuda.synchronize()
    assert ttq.device_error() == ttq.DEVERR_INDEX
    assert (out == 3).all()


def test_adapters_pitched_rows_and_untouched_memory(ttq):
    a = make_adapters(21, 4, 8, 128, 96, torch.float16)
    want = check_adapters(ttq, a)
    plan = ttq.adapters_plan(a["index"], 4)
    X = torch.full((21, 136), 7.0, dtype=torch.float16, device="cuda")
    X[:, :128] = a["X"]
    Y = torch.full((21, 101), 4.0, dtype=torch.float16, device="cuda")
    Y[:, 2:98] = a["Y"]
    out = torch.full((22, 104), 5.0, dtype=torch.float16, device="cuda")
    ttq.adapters_add(X[:, :128], a["A"], a["B"], plan, Y[:, 2:98],
                     scale=a["scale"], out=out[:21, 8:])
    assert torch.equal(out[:21, 8:], want)
    assert (out[:21, :8] == 5).all() and (out[21] == 5).all()
    ttq.adapters_add(X[:, :128], a["A"], a["B"], plan, Y[:, 2:98],
                     scale=a["scale"])
    assert torch.equal(Y[:, 2:98], want)
    assert (Y[:, :2] == 4).all() and (Y[:, 98:] == 4).all()


def test_adapters_a_bad_token_stays_alone(ttq):
    a = make_adapters(40, 2, 16, 128, 96, torch.bfloat16)
    a["index"].fill_(1)
    plan = ttq.adapters_plan(a["index"], 2)

    def call(X):
        return ttq.adapters_add(X, a["A"], a["B"], plan, a["Y"],
                                out=torch.empty_like(a["Y"]))
    good = call(a["X"])
    X = a["X"].clone()
    X[7, 3] = float("nan")
    got = call(X)
    keep = torch.arange(40) != 7
    assert torch.equal(got[keep], good[keep])
    assert torch.isnan(got[7]).all()


def test_adapters_results_do_not_depend_on_the_batch(ttq):
    """A token's result is the same bits in a batch of another order and
    size (where as many CTAs share a tile)."""
    a = make_adapters(90, 3, 16, 256, 192, torch.bfloat16)
    all_out = check_adapters(ttq, a)
    pick = torch.tensor([0, 17, 44, 89])
    b = {n: (v[pick].contiguous() if n in ("X", "Y", "index") else v)
         for n, v in a.items()}
    assert torch.equal(check_adapters(ttq, b), all_out[pick])


def test_adapters_captured_and_replayed(ttq):
    a = make_adapters(48, 6, 16, 256, 320, torch.bfloat16)
    n = int(ttq.adapters_plan(a["index"], 6).numel())
    plan = torch.empty(n, dtype=torch.int32, device="cuda")
    out = torch.empty_like(a["Y"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        ttq.adapters_plan(a["index"], 6, plan=plan)
        ttq.adapters_add(a["X"], a["A"], a["B"], plan, a["Y"],
                         scale=a["scale"], out=out)
    for seed in range(3):
        b = make_adapters(48, 6, 16, 256, 320, torch.bfloat16, seed=seed)
        for n in ("X", "A", "B", "Y", "scale", "index"):
            a[n].copy_(b[n])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, check_adapters(ttq, b))


# ------------------------------------------------------------------ together

def make_layer(ttq, E, k, K, I, act="silu", dt=torch.bfloat16, score="softmax"):
    g = gen("layer", E, K, I)
    router = (torch.randn(E, K, generator=g) / math.sqrt(K)).to(dt).cuda()
    W1 = (torch.randn(E, 2 * I, K, generator=g) / math.sqrt(K)).to(dt).cuda()
    W2 = (torch.randn(E, K, I, generator=g) / math.sqrt(I)).to(dt).cuda()
    return ttq.TTQMoE(router, W1, W2, ttq.TTQParams(4, 32), k, act=act,
                      score=score)


@pytest.mark.parametrize("act,score", [("silu", "softmax"),
                                       ("gelu", "sigmoid")])
def test_moe_layer_prompt_then_decode(ttq, act, score):
    layer = make_layer(ttq, 6, 2, 256, 128, act, torch.float32, score)
    X = torch.randn(40, 256, generator=gen("px")).cuda()
    Y = layer.prompt(X)
    # the same tokens by the decode form, against its own bound
    ids, w = layer.route(X)
    m = dict(X=X, ids=ids, weights=w, inv_s=layer.inv_s, up=layer.up,
             inv_s_mid=layer.inv_s_mid, down=layer.down, bits=4, group=32)
    D = check_moe(ttq, m, act)
    assert torch.equal(layer.decode(X), D)
    # and the prompt's pass within the projection's tolerance (2e-3 each),
    # twice through h (both factors), once through the down projection
    fro = ((Y - D).norm() / D.norm()).item()
    assert fro <= 3 * 2e-3, fro
    # the scales are the framework's own statistics of this prompt
    s, inv = ttq.awq_scales(ttq.act_stats(X), 40)
    assert torch.allclose(layer.inv_s, inv, rtol=1e-5)
    # an expert that no token picked keeps scales of 1
    one = make_layer(ttq, 6, 1, 256, 128)
    one.prompt(X[:1].bfloat16())
    hit = int(one.route(X[:1].bfloat16())[0][0, 0])
    rest = [e for e in range(6) if e != hit]
    assert (one.inv_s_mid[rest] == 1).all()
    assert not (one.inv_s_mid[hit] == 1).all()


def test_linear_with_adapters(ttq):
    T, K, N, L = 37, 256, 320, 5
    g = gen("lin")
    W = (torch.randn(N, K, generator=g) / math.sqrt(K)).bfloat16().cuda()
    a = make_adapters(T, L, 16, K, N, torch.bfloat16)
    lin = ttq.TTQLinear(W, ttq.TTQParams(4, 32))
    bank = ttq.AdapterBank(a["A"], a["B"], a["scale"])
    plan = bank.plan(a["index"])
    base = lin(a["X"])
    got = lin.project(a["X"], adapters=(bank, plan))
    a["Y"] = base
    ref, bound, live = adapters_reference(a, a["scale"])
    assert ((got.double().cpu() - ref).abs() <= bound)[live].all()
    assert torch.equal(got[~live.cuda()], base[~live.cuda()])
    assert torch.equal(lin(a["X"], adapters=(bank, plan)), got)


def test_a_decode_step_of_all_of_them_captured(ttq):
    """A projection with its requests' adapters, then the expert layer, as one
    graph: replayed on new tokens and adapters it gives the eager bits."""
    T, K, L = 12, 256, 7
    layer = make_layer(ttq, 8, 2, K, 128)
    layer.prompt(torch.randn(90, K, generator=gen("p")).bfloat16().cuda())
    W = (torch.randn(K, K, generator=gen("w")) / 16).bfloat16().cuda()
    lin = ttq.TTQLinear(W, ttq.TTQParams(4, 32))
    lin.calibrate(torch.randn(90, K, generator=gen("q")).bfloat16().cuda())
    a = make_adapters(T, L, 8, K, K, torch.bfloat16)
    bank = ttq.AdapterBank(a["A"], a["B"], a["scale"])

    def step(X, index):
        Y = lin.project(X, adapters=(bank, bank.plan(index)))
        return layer.decode(Y)
    X, index = a["X"].clone(), a["index"].clone()
    step(X, index)  # workspaces exist before the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(X, index)
    for seed in range(3):
        b = make_adapters(T, L, 8, K, K, torch.bfloat16, seed=seed)
        want = step(b["X"], b["index"])
        X.copy_(b["X"])
        index.copy_(b["index"])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert ttq.device_error() == 0


def test_calls_on_a_side_stream_follow_its_work(ttq):
    """Inputs written on the same side stream just before the calls."""
    m = make_moe(ttq, 1, 8, 4, 512, 256, 4, 64, torch.bfloat16)
    want = check_moe(ttq, m)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(20):
            up = tuple(torch.zeros_like(p) for p in m["up"])
            X, ids = torch.zeros_like(m["X"]), torch.zeros_like(m["ids"])
            w = torch.zeros_like(m["weights"])
            for d, s in zip(up + (X, ids, w),
                            m["up"] + (m["X"], m["ids"], m["weights"])):
                d.copy_(s)
            got = ttq.moe_lowbit(X, ids, w, m["inv_s"], up, m["inv_s_mid"],
                                 m["down"], 4, 64)
            assert torch.equal(got, want)


def test_one_token_right_behind_its_router_and_quantizer(ttq):
    """The layer's first kernel may start while the kernel before it still
    runs: it must not read that kernel's ids or codes early."""
    g = gen("behind")
    E, K, I, k = 256, 512, 128, 4
    layer = make_layer(ttq, E, k, K, I)
    layer.prompt(torch.randn(300, K, generator=g).bfloat16().cuda())
    xs = [torch.randn(1, K, generator=g).bfloat16().cuda() for _ in range(40)]
    want = []
    for x in xs:
        ids, w = layer.route(x)
        torch.cuda.synchronize()
        want.append(ttq.moe_lowbit(x, ids, w, layer.inv_s, layer.up,
                                   layer.inv_s_mid, layer.down, 4, 32))
        torch.cuda.synchronize()
    got = [layer.decode(x) for x in xs]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # the up weights quantized anew just before the call
    W = layer.W_up.view(E * 2 * I, K)
    ids, w = layer.route(xs[0])
    for _ in range(20):
        for b in layer.up:
            b.zero_()
        ttq.quantize_rtn_grouped(W, layer.s, 4, 32, *layer.up)
        out = ttq.moe_lowbit(xs[0], ids, w, layer.inv_s, layer.up,
                             layer.inv_s_mid, layer.down, 4, 32)
        assert torch.equal(out, want[0])


@pytest.mark.parametrize("K,T", [(10000, 40), (11008, 8)])
def test_adapters_fp32_over_a_long_input(ttq, K, T):
    """fp32 stays fp32 over a long K: the error's 2-norm within 1e-6 of the
    result's. Rounded additions of n random terms are off by about sqrt(n)
    2^-24 of a term's size, 2^-24 of the sum's; sums that the tensor core cuts
    are off by up to n / 16 times 2^-24 of it."""
    a = make_adapters(T, 2, 16, K, 256, torch.float32)
    a["Y"].zero_()
    a["index"].fill_(1)
    out = check_adapters(ttq, a)
    ref = adapters_reference(a, a["scale"])[0]
    err = ((out.double().cpu() - ref).norm() / ref.norm()).item()
    assert err < 1e-6, err
