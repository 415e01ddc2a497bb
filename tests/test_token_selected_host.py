"""Refusals of the calls on weights a token selects, on the host: the C ABI
returns an error before any launch, and the Python binding refuses wrong
buffers before the library is called."""
import pytest
import torch

from test_weight_quantization_b200 import ttq


def far(i):
    """Fake pointers, 1 TiB apart; never dereferenced: checks fail first."""
    return (i + 1) << 40


def route_args(**kw):
    a = dict(X=far(0), xt=1, T=4, K=64, ldx=64, W=far(1), wt=1, E=16, ldw=64,
             bias=None, top_k=2, score=0, renormalize=1, scaling=1.0,
             ids=far(2), weights=far(3), stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("bad", [
    dict(X=None), dict(W=None), dict(ids=None), dict(weights=None),
    dict(T=0), dict(T=1 << 31), dict(K=0), dict(K=60), dict(K=1 << 21),
    dict(E=0), dict(E=513), dict(top_k=0), dict(top_k=17),
    dict(top_k=33, E=64), dict(xt=3), dict(wt=-1), dict(ldx=56),
    dict(ldw=56), dict(ldx=68), dict(ldw=65), dict(X=far(0) + 8),
    dict(W=far(1) + 2), dict(score=2), dict(renormalize=2),
    dict(scaling=float("nan")), dict(scaling=float("inf")),
    dict(ids=far(2) + 2), dict(bias=far(4) + 1), dict(weights=far(2) + 16),
    dict(ids=far(0) + 64), dict(weights=far(1) + 64),
])
def test_route_refuses(bad):
    assert ttq._lib.ttq_moe_route(*route_args(**bad)) == 1


def moe_args(**kw):
    a = dict(X=far(0), xt=1, T=4, K=128, ldx=128, ids=far(1),
             weights=far(2), top_k=2, E=8, inv_s=far(3), uc=far(4),
             ud=far(5), uz=far(6), I=64, mid=far(7), dc=far(8), dd=far(9),
             dz=far(10), bits=4, group=32, act=0, Y=far(11), yt=1, ldy=128,
             ws=far(12), wsb=1 << 30, stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("bad", [
    *[{n: None} for n in ("X", "ids", "weights", "inv_s", "uc", "ud", "uz",
                          "mid", "dc", "dd", "dz", "Y", "ws")],
    dict(T=0), dict(K=0), dict(K=120), dict(I=0), dict(I=48), dict(E=0),
    dict(E=513), dict(top_k=0), dict(top_k=33), dict(bits=1), dict(bits=9),
    dict(group=24), dict(group=128, I=64), dict(group=128, K=192, ldx=192),
    dict(act=2), dict(xt=3), dict(yt=5), dict(ldx=120), dict(ldx=132),
    dict(ldy=127), dict(X=far(0) + 8), dict(Y=far(11) + 1),
    dict(inv_s=far(3) + 4), dict(uc=far(4) + 4), dict(ud=far(5) + 4),
    dict(uz=far(6) + 1), dict(dc=far(8) + 8), dict(dd=far(9) + 8),
    dict(dz=far(10) + 2), dict(ws=far(12) + 8), dict(wsb=16),
    dict(ws=far(0) - 256), dict(ws=far(11)), dict(ws=far(1) - 64),
    dict(Y=far(1) - 16),
])
def test_moe_refuses(bad):
    assert ttq._lib.ttq_moe_lowbit(*moe_args(**bad)) == 1


def test_moe_is_for_a_few_tokens():
    assert ttq._lib.ttq_moe_lowbit(*moe_args(T=65)) == 2
    size = ttq.moe_lowbit_workspace_size
    assert size(64, 128, 64, 2) > size(1, 128, 64, 2) > 0
    for a in ((0, 128, 64, 2), (65, 128, 64, 2), (4, 100, 64, 2),
              (4, 128, 63, 2), (4, 128, 64, 0), (4, 128, 64, 33)):
        assert size(*a) == 0


def plan_args(**kw):
    a = dict(index=far(0), T=40, L=4, plan=far(1), n=1 << 20, stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("bad", [
    dict(index=None), dict(plan=None), dict(T=0), dict(T=(1 << 20) + 1),
    dict(L=0), dict(L=8193), dict(index=far(0) + 2), dict(plan=far(1) + 4),
    dict(n=59), dict(plan=far(0) + 16),
])
def test_plan_refuses(bad):
    assert ttq._lib.ttq_adapters_plan(*plan_args(**bad)) == 1


def add_args(**kw):
    a = dict(X=far(0), xt=1, T=40, K=64, ldx=64, A=far(1), B=far(2),
             scale=None, L=4, r=16, N=32, plan=far(3), n=1 << 20, Y=far(4),
             yt=1, ldy=32, out=far(5), ldo=32, stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("bad", [
    *[{n: None} for n in ("X", "A", "B", "plan", "Y", "out")],
    dict(T=0), dict(K=0), dict(K=60), dict(N=0), dict(r=0), dict(r=6),
    dict(r=68), dict(L=0), dict(xt=4), dict(yt=-1), dict(ldx=63),
    dict(ldx=68), dict(ldy=31), dict(ldo=31), dict(X=far(0) + 4),
    dict(A=far(1) + 8), dict(B=far(2) + 8), dict(plan=far(3) + 4),
    dict(n=59), dict(Y=far(4) + 1), dict(out=far(5) + 1),
    dict(scale=far(6) + 2),
    dict(out=far(4) + 64),           # overlaps Y without being Y
    dict(out=far(4), ldo=40),        # Y itself, but with another pitch
    dict(out=far(0)), dict(out=far(1)), dict(out=far(2)), dict(out=far(3)),
    dict(out=far(6), scale=far(6) + 4),
])
def test_adapters_add_refuses(bad):
    assert ttq._lib.ttq_adapters_add(*add_args(**bad)) == 1


# --------------------------------------------------------------- the binding

class Recorder:
    def __init__(self, real):
        self.real, self.calls = real, []

    def __getattr__(self, name):
        if name.endswith(("_ld", "_size", "status_string")):
            return getattr(self.real, name)

        def call(*args):
            self.calls.append((name, args))
            return ttq.TTQ_OK
        return call


@pytest.fixture
def rec(monkeypatch):
    r = Recorder(ttq._lib)
    monkeypatch.setattr(ttq, "_lib", r)
    monkeypatch.setattr(ttq, "_stream", lambda: 0)

    def host_dev(t, name):
        if not isinstance(t, torch.Tensor):
            raise ttq.TTQError(f"{name} must be a tensor")
    monkeypatch.setattr(ttq, "_dev", host_dev)
    return r


def moe_buffers(T=3, E=4, k=2, K=128, I=64, b=4, g=32):
    def packed(rows, cols):
        return (torch.zeros(rows, ttq.codes_ld(cols, b), dtype=torch.int32),
                torch.zeros(rows, ttq.groups_ld(cols, g)),
                torch.zeros(rows, ttq.groups_ld(cols, g), dtype=torch.uint8))
    return dict(X=torch.zeros(T, K, dtype=torch.bfloat16),
                ids=torch.zeros(T, k, dtype=torch.int32),
                weights=torch.zeros(T, k), inv_s=torch.zeros(K),
                up=packed(E * 2 * I, K), inv_s_mid=torch.zeros(E, I),
                down=packed(E * K, I), bits=b, group=g)


def test_binding_passes_documented_calls(rec):
    m = moe_buffers()
    Y = ttq.moe_lowbit(**m)
    assert Y.shape == (3, 128) and Y.dtype == torch.bfloat16
    name, a = rec.calls[-1]
    assert name == "ttq_moe_lowbit" and a[2:5] == (3, 128, 128)
    assert a[7:9] == (2, 4) and a[13] == 64 and a[18:21] == (4, 32, 0)
    ttq.moe_lowbit(**m, act="gelu", out=torch.zeros(3, 130)[:, :128])
    assert rec.calls[-1][1][20] == 1 and rec.calls[-1][1][22:24] == (0, 130)
    X = m["X"]
    W = torch.zeros(16, 128, dtype=torch.float32)
    ids, w = ttq.moe_route(X, W, 4, bias=torch.zeros(16), score="sigmoid",
                           renormalize=False, scaling=2.0)
    assert ids.shape == w.shape == (3, 4) and ids.dtype == torch.int32
    a = rec.calls[-1][1]
    assert a[6] == 0 and a[10:14] == (4, 1, 0, 2.0)
    plan = ttq.adapters_plan(torch.zeros(3, dtype=torch.int32), 2)
    A, B = torch.zeros(2, 8, 128, dtype=torch.bfloat16), \
        torch.zeros(2, 40, 8, dtype=torch.bfloat16)
    Y = torch.zeros(3, 40, dtype=torch.bfloat16)
    assert ttq.adapters_add(X, A, B, plan, Y) is Y
    out = torch.zeros(3, 44, dtype=torch.bfloat16)[:, :40]
    assert ttq.adapters_add(X, A, B, plan, Y, torch.ones(2), out) is out
    a = rec.calls[-1][1]
    assert a[8:11] == (2, 8, 40) and a[15] == 40 and a[17] == 44


def test_binding_refuses_bad_buffers(rec):
    m = moe_buffers()
    X = m["X"]
    plan = ttq.adapters_plan(torch.zeros(3, dtype=torch.int32), 2)
    A, B = torch.zeros(2, 8, 128, dtype=torch.bfloat16), \
        torch.zeros(2, 40, 8, dtype=torch.bfloat16)
    Y = torch.zeros(3, 40, dtype=torch.bfloat16)
    W = torch.zeros(16, 128, dtype=torch.bfloat16)
    before = len(rec.calls)

    def moe(**kw):
        return lambda: ttq.moe_lowbit(**{**m, **kw})
    bad = [
        moe(ids=m["ids"].long()), moe(ids=m["ids"][0]),
        moe(ids=m["ids"][:2]), moe(weights=m["weights"].half()),
        moe(weights=torch.zeros(3, 3)), moe(inv_s=torch.zeros(96)),
        moe(inv_s_mid=torch.zeros(64)), moe(inv_s_mid=torch.zeros(5, 64)),
        moe(up=m["down"]), moe(down=m["up"]), moe(bits=5), moe(group=24),
        moe(act="relu"), moe(out=torch.zeros(3, 64)),
        moe(out=torch.zeros(3, 128, dtype=torch.float64)),
        moe(workspace=torch.zeros(16, dtype=torch.uint8)),
        moe(X=X.t()),
        lambda: ttq.moe_route(X, W[:, :64], 2),
        lambda: ttq.moe_route(X, W, 2, score="top"),
        lambda: ttq.moe_route(X, W, 2, bias=torch.zeros(15)),
        lambda: ttq.moe_route(X, W, 2, ids=torch.zeros(3, 2)),
        lambda: ttq.moe_route(X, W, 2, weights=torch.zeros(3, 3)),
        lambda: ttq.moe_route(X, W.double(), 2),
        lambda: ttq.adapters_plan(torch.zeros(3), 2),
        lambda: ttq.adapters_plan(torch.zeros(3, dtype=torch.int32), 0),
        lambda: ttq.adapters_plan(torch.zeros(3, dtype=torch.int32), 2,
                                  torch.zeros(5, dtype=torch.int32)),
        lambda: ttq.adapters_add(X, A[0], B, plan, Y),
        lambda: ttq.adapters_add(X, A.float(), B, plan, Y),
        lambda: ttq.adapters_add(X, A, B[:1], plan, Y),
        lambda: ttq.adapters_add(X, A[:, :4], B, plan, Y),
        lambda: ttq.adapters_add(X, A, B, plan[:8], Y),
        lambda: ttq.adapters_add(X, A, B, plan, Y[:, :32]),
        lambda: ttq.adapters_add(X, A, B, plan, Y, torch.ones(1)),
        lambda: ttq.adapters_add(X, A, B, plan, Y, out=Y.float()),
    ]
    for i, fn in enumerate(bad):
        with pytest.raises(ttq.TTQError):
            fn()
        assert len(rec.calls) == before, f"case {i} reached the library"


def test_index_error_bit_matches_the_header():
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = open(os.path.join(root, "include", "ttq.h")).read()
    bit = re.search(r"#define TTQ_DEVERR_INDEX (0x[0-9a-f]+)u", src).group(1)
    assert int(bit, 16) == ttq.DEVERR_INDEX
