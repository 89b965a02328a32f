"""Host side of the input layer's C ABI (include/onetrans_input.h), without a
GPU: exports, workspace sizes, and argument errors found before any launch.
Device pointers are fake aligned addresses; nothing here reaches a kernel."""
import ctypes
import os
import re

import pytest
import torch

import unified_transformer_recommender_b200 as ot
from test_host_abi import FAKE, FakeModel

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "onetrans_input.h")
BIG = 1 << 40


def size_of(fm, op, n, L):
    out = ot.SZ(0)
    return ot.lib.onetrans_input_workspace_size(fm.h, op, n, L, ctypes.byref(out)), out.value


def test_exports():
    names = set(re.findall(r"ONETRANS_API\s+[\w\s\*]+?\b(onetrans_\w+)\s*\(", open(HEADER).read()))
    assert names == set(ot.INPUT_SYMBOLS)
    for n in names:
        assert hasattr(ot.lib, n), n


def test_embedding_workspace():
    fm = FakeModel()
    st, a = size_of(fm, ot.OP_EMBEDDING_BACKWARD, 1000, 64)
    st2, b = size_of(fm, ot.OP_EMBEDDING_BACKWARD, 100_000, 64)
    assert st == st2 == ot.OK and 16 * 1000 <= a < b and b >= 16 * 100_000
    assert size_of(fm, ot.OP_EMBEDDING_BACKWARD, -1, 64)[0] == ot.ERR_SHAPE
    assert size_of(fm, ot.OP_EMBEDDING_BACKWARD, 2 ** 26 + 1, 64)[0] == ot.ERR_SHAPE
    assert size_of(fm, ot.OP_EMBEDDING_BACKWARD, 10, 0)[0] == ot.ERR_SHAPE
    assert size_of(fm, 99, 10, 1)[0] == ot.ERR_INVALID_ARG
    assert ot.lib.onetrans_input_workspace_size(None, 0, 1, 1, ctypes.byref(ot.SZ(0))) == ot.ERR_INVALID_ARG


def test_a_workspace_serves_every_smaller_call():
    """Sizes never fall as ids, events, width or choices grow: the sizes on both sides of every rule that picks larger
    tiles or chunks, and of the numbers between, each against the largest before it."""
    fm = FakeModel(n_beh=3, event_dim=64)
    ends = [37_888, 81_920, 327_680, (1 << 20) - 1] + [i << 20 for i in range(1, 65)]
    ns = sorted({n for e in ends for n in (e - 1, e, e + 1, e + 3000) if n <= 1 << 26} | {1, 31, 4096, 4097, 40_000, 400_000})
    for w in (1, 8, 64, 256, 5000):
        most = 0
        for n in ns:
            st, b = size_of(fm, ot.OP_EMBEDDING_BACKWARD, n, w)
            assert st == ot.OK and b >= most, (n, w, b, most)
            most = b
    for n in ns:
        sizes = [size_of(fm, ot.OP_EMBEDDING_BACKWARD, n, w)[1] for w in (1, 8, 64, 256, 5000)]
        assert sizes == sorted(sizes)
    for op in (ot.OP_ROUTE, ot.OP_ROUTED, ot.OP_ROUTED_BACKWARD):
        for k in (1, 2, 8):
            sizes = [size_of(fm, op, n, k)[1] for n in ns if n * k <= 1 << 26]
            assert sizes == sorted(sizes), (op, k)
        for n in (1, 1000, 40_000):
            sizes = [size_of(fm, op, n, k)[1] for k in range(1, 9)]
            assert sizes == sorted(sizes), (op, n)


def test_lookup_argument_errors():
    fm = FakeModel()
    base = dict(m=fm.h, table=FAKE, tm=ot.BF16, V=100, w=64, ids=FAKE, bits=32, R=8, out=FAKE, ld=64)

    def call(**kw):
        a = dict(base, **kw)
        return ot.lib.onetrans_embedding_lookup(a["m"], a["table"], a["tm"], a["V"], a["w"], a["ids"], a["bits"], a["R"],
                                                1.0, a["out"], a["ld"], None)

    assert call(R=0, table=None, ids=None, out=None) == ot.OK
    for kw in (dict(m=None), dict(tm=2), dict(bits=16), dict(table=None), dict(ids=None), dict(out=None),
               dict(table=FAKE + 8), dict(ids=FAKE + 4), dict(out=FAKE + 2)):
        assert call(**kw) == ot.ERR_INVALID_ARG, kw
    for kw in (dict(V=0), dict(V=2 ** 31), dict(w=0), dict(w=65537, ld=70000), dict(R=-1), dict(R=2 ** 31), dict(ld=63)):
        assert call(**kw) == ot.ERR_SHAPE, kw


def test_gradient_argument_errors():
    fm = FakeModel()
    base = dict(m=fm.h, dout=FAKE, dm=ot.BF16, ld=64, ids=FAKE, bits=32, R=8, V=100, w=64, out=FAKE, uniq=FAKE, n=FAKE,
                ws=FAKE, nb=BIG)

    def dense(**kw):
        a = dict(base, **kw)
        return ot.lib.onetrans_embedding_backward(a["m"], a["dout"], a["dm"], a["ld"], a["ids"], a["bits"], a["R"],
                                                  a["V"], a["w"], 1.0, a["out"], a["ws"], a["nb"], None)

    def sparse(**kw):
        a = dict(base, **kw)
        return ot.lib.onetrans_embedding_backward_sparse(a["m"], a["dout"], a["dm"], a["ld"], a["ids"], a["bits"], a["R"],
                                                         a["V"], a["w"], 1.0, a["uniq"], a["out"], a["n"], a["ws"],
                                                         a["nb"], None)

    for f in (dense, sparse):
        for kw in (dict(m=None), dict(dm=3), dict(bits=8), dict(dout=None), dict(ids=None), dict(ws=None), dict(out=None),
                   dict(dout=FAKE + 2), dict(ids=FAKE + 4), dict(out=FAKE + 4), dict(ws=FAKE + 16)):
            assert f(**kw) == ot.ERR_INVALID_ARG, kw
        for kw in (dict(V=0), dict(V=2 ** 31), dict(w=0), dict(R=-1), dict(R=2 ** 26 + 1), dict(ld=63)):
            assert f(**kw) == ot.ERR_SHAPE, kw
        need = size_of(fm, ot.OP_EMBEDDING_BACKWARD, 8, 64)[1]
        assert f(nb=need - 1) == ot.ERR_CAPACITY
    for kw in (dict(uniq=None), dict(uniq=FAKE + 8), dict(n=None), dict(n=FAKE + 4)):
        assert sparse(**kw) == ot.ERR_INVALID_ARG, kw
    assert dense(R=0, out=None) == ot.ERR_INVALID_ARG      # the zeros still have to go somewhere


def event_grads(n, addr=FAKE):
    g = ot.EventGrads()
    keep = []
    for f in ot._BEH_FIELDS:
        arr = (ot.P * n)(*[addr + 256 * i for i in range(n)])
        keep.append(arr)
        setattr(g, f, ctypes.cast(arr, ot.PP))
    g.type_emb = addr
    return g, keep


def test_routed_workspaces():
    fm = FakeModel(n_beh=3, event_dim=64)
    for op in (ot.OP_ROUTE, ot.OP_ROUTED, ot.OP_ROUTED_BACKWARD):
        st, a = size_of(fm, op, 1000, 1)
        st2, b = size_of(fm, op, 10_000, 1)
        st3, c = size_of(fm, op, 10_000, 3)
        assert st == st2 == st3 == ot.OK and 0 < a < b < c
        assert size_of(fm, op, 10, 0)[0] == ot.ERR_SHAPE
        assert size_of(fm, op, 10, 9)[0] == ot.ERR_SHAPE
        assert size_of(fm, op, -1, 1)[0] == ot.ERR_SHAPE
        assert size_of(fm, op, 2 ** 26, 2)[0] == ot.ERR_SHAPE
        assert size_of(fm, op, 0, 1)[0] == ot.OK
        assert size_of(FakeModel(), op, 10, 1)[0] == ot.ERR_UNSUPPORTED      # no behavior MLPs


def test_routed_argument_errors():
    fm = FakeModel(n_beh=3, event_dim=64)
    d = fm.cfg.d_model
    g, keep = event_grads(3)
    base = dict(m=fm.h, types=FAKE, ev=FAKE, wt=None, R=8, k=2, plan=FAKE, pb=BIG, tok=FAKE, per=8, ld=8 * d, ws=FAKE, nb=BIG,
                dm=ot.BF16, de=FAKE, dw=FAKE, g=ctypes.byref(g))

    def route(**kw):
        a = dict(base, **kw)
        return ot.lib.onetrans_route_events(a["m"], a["types"], a["R"], a["k"], a["plan"], a["pb"], None)

    def tokens(**kw):
        a = dict(base, **kw)
        return ot.lib.onetrans_tokenize_routed(a["m"], a["ev"], a["wt"], a["R"], a["k"], a["plan"], a["pb"], a["tok"],
                                               a["per"], a["ld"], a["ws"], a["nb"], None)

    def grad(**kw):
        a = dict(base, **kw)
        return ot.lib.onetrans_tokenize_routed_backward(a["m"], a["ev"], a["wt"], a["R"], a["k"], a["plan"], a["pb"],
                                                        a["tok"], a["dm"], a["per"], a["ld"], a["de"], a["dw"], a["g"],
                                                        a["ws"], a["nb"], None)

    none = FakeModel()
    for f in (route, tokens, grad):
        assert f(m=None) == ot.ERR_INVALID_ARG
        assert f(m=none.h) == ot.ERR_UNSUPPORTED
        for kw in (dict(R=-1), dict(k=0), dict(k=9), dict(R=2 ** 26)):
            assert f(**kw) == ot.ERR_SHAPE, kw
        for kw in (dict(plan=None), dict(plan=FAKE + 16)):
            assert f(**kw) == ot.ERR_INVALID_ARG, kw
        assert f(pb=size_of(fm, ot.OP_ROUTE, 8, 2)[1] - 1) == ot.ERR_CAPACITY
    assert route(R=0, types=None, plan=None) == ot.OK
    assert route(types=None) == route(types=FAKE + 4) == ot.ERR_INVALID_ARG
    assert tokens(R=0, ev=None, plan=None, tok=None, ws=None) == ot.OK
    for f in (tokens, grad):
        for kw in (dict(ev=None), dict(ev=FAKE + 2), dict(tok=None), dict(tok=FAKE + 8), dict(ws=None), dict(ws=FAKE + 16), dict(wt=FAKE + 4)):
            assert f(**kw) == ot.ERR_INVALID_ARG, kw
        for kw in (dict(per=0), dict(per=4, ld=4 * d - 1)):
            assert f(**kw) == ot.ERR_SHAPE, kw
    assert tokens(nb=size_of(fm, ot.OP_ROUTED, 8, 2)[1] - 1) == ot.ERR_CAPACITY
    assert grad(nb=size_of(fm, ot.OP_ROUTED_BACKWARD, 8, 2)[1] - 1) == ot.ERR_CAPACITY
    for kw in (dict(dm=2), dict(de=FAKE + 8), dict(dw=FAKE + 4), dict(g=None)):
        assert grad(**kw) == ot.ERR_INVALID_ARG, kw
    keep[2][1] = FAKE + 4
    assert grad() == ot.ERR_INVALID_ARG
    keep[2][1] = None
    assert grad() == ot.ERR_INVALID_ARG
    fp = FakeModel(n_beh=3, event_dim=64, mode=ot.FP32)
    keep[2][1] = FAKE
    assert grad(m=fp.h, dm=ot.BF16) == ot.ERR_UNSUPPORTED


def test_rows_per_sample_past_the_events_is_one_sample():
    """Any rows_per_sample of at least R means rows one after another, also one past 32 bits: such a call gets past the
    checks of the token rows, here to the one of the workspace."""
    fm = FakeModel(n_beh=3, event_dim=64)
    d = fm.cfg.d_model
    g, keep = event_grads(3)
    plan = size_of(fm, ot.OP_ROUTE, 8, 2)[1]
    for per in (8, 9, 2 ** 31 - 1, 2 ** 31, 2 ** 40, 2 ** 63 - 1):
        assert ot.lib.onetrans_tokenize_routed(fm.h, FAKE, None, 8, 2, FAKE, plan, FAKE, per, 0, FAKE, 0, None) == ot.ERR_CAPACITY
        assert ot.lib.onetrans_tokenize_routed_backward(fm.h, FAKE, None, 8, 2, FAKE, plan, FAKE, ot.FP32, per, 0, None, None,
                                                        ctypes.byref(g), FAKE, 0, None) == ot.ERR_CAPACITY
    for per in (0, -1, -2 ** 63):
        assert ot.lib.onetrans_tokenize_routed(fm.h, FAKE, None, 8, 2, FAKE, plan, FAKE, per, 8 * d, FAKE, 0, None) == ot.ERR_SHAPE


def test_a_model_on_another_device_is_refused(monkeypatch):
    """The kernels of a routed call run on the current device and read the model's weights there.  Without a second
    device here, the current one is said to be the one the arguments are on, and the weights' another."""
    from onetrans_synth import ModelShape, make_weights
    sh = ModelShape(n_layers=1, d=64, n_heads=1, d_ff=64, L_NS=2, ns_feat=16, ns_hidden=64, behavior_dims=(64, 64))
    m = ot.model_from_arrays(sh, make_weights(sh, 1, "bf16"), device="cpu", event_dim=64)
    ev, tok = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(4, 64, dtype=torch.bfloat16)
    types, ws = torch.zeros(4, dtype=torch.int32), torch.zeros(256, dtype=torch.uint8)
    dev = ev.get_device()
    assert m.device_index == dev
    monkeypatch.setattr(torch.cuda, "current_device", lambda: dev)
    m.device_index = dev + 2
    for call in (lambda: ot.onetrans_tokenize_routed(m, ev, types, None, ws, tok, ws),
                 lambda: ot.onetrans_tokenize_routed_backward(m, ev, types, None, ws, tok, None, None, {"type_emb": tok}, ws)):
        with pytest.raises(ValueError, match="the model's weights must be on the current CUDA device"):
            call()
