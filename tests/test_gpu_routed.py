"""Routed event tokenizer (events sorted by behaviour, each through its
behaviour's MLP, weighted and put back) and its gradient, through the C ABI
against plain float64 implementations.

Tolerances, per element, with S = the sum of the absolute values of the terms
of that element's sum (every operand replaced by its absolute value):
  float32 arithmetic: a sum of n terms is off by at most n * 2^-24 * S; a
    tensor-core sum may truncate instead of rounding, 2^-23; GELU and its
    slope by at most 2^-20 * (1 + |u|) in the accurate form.
  bf16 forward: z rounded to bf16 (2^-8 |z|), with a tanh good to 2^-10.9
    (2^-11.9 |u| of z), and the token rounded once (2^-8 of it).
  bf16 backward: z and du as two bf16 terms (2^-16 of them) for the weight
    gradients, du as one (2^-8) for the event gradient.  float32 dtokens are
    rounded to bf16 on entry: the reference takes the rounded values,
    except in dw's <dtoken, b2 + emb> (2^-8 of those terms)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import unified_transformer_recommender_b200 as ot  # noqa: E402

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
C, A = (2.0 / np.pi) ** 0.5, 0.044715


def make(mode, T, e, d, seed, std=1.0, scale2=1.0):
    """A model with T behaviours and its MLP weights (float64 copies of the rounded values)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DT[mode]

    def n(*s, std=1.0):
        return (torch.randn(*s, device="cuda", generator=g) * std).to(dt)

    H = next(h for h in (1, 2, 3, 4, 5, 6, 8) if d % h == 0 and d // h in (16, 32, 64, 96, 128))
    W = {"Wb1": [n(d, e, std=std * e ** -0.5) for _ in range(T)], "bb1": [n(d, std=0.1) for _ in range(T)],
         "Wb2": [n(d, d, std=scale2 * d ** -0.5) for _ in range(T)], "bb2": [n(d, std=0.1) for _ in range(T)],
         "type_emb": n(T, d, std=0.1)}
    z = {f: [torch.zeros(s, device="cuda", dtype=dt)] for f, s in (
        ("g_attn", (d,)), ("g_ffn", (d,)), ("Wqkv_S", (3 * d, d)), ("Wqkv_NS", (1, 3 * d, d)), ("Wo", (d, d)),
        ("W1_S", (d, d)), ("b1_S", (d,)), ("W2_S", (d, d)), ("b2_S", (d,)), ("W1_NS", (1, d, d)), ("b1_NS", (1, d)),
        ("W2_NS", (1, d, d)), ("b2_NS", (1, d)))}
    m = ot.Model(n_layers=1, d_model=d, n_heads=H, d_ff=d, L_NS=1, weights={**z, **W},
                 mode=ot.BF16 if mode == "bf16" else ot.FP32, n_behaviors=T, event_dim=e)
    return m, W


def make_types(kind, R, k, T, seed):
    g = np.random.default_rng(seed)
    if kind == "none":
        t = np.full((R, k), -1)
    elif kind == "last":
        t = np.full((R, k), T - 1)
    else:
        t = g.integers(0, T, (R, k)) if kind == "uniform" else (T * g.random((R, k)) ** 3).astype(int)
        if kind != "uniform" or k > 1:
            t[g.random((R, k)) < 0.2] = -1
    return torch.from_numpy(t.astype(np.int32)).cuda()


def parts(W, t, x):
    """float64 u, z, slope of behaviour t for events x, and the gelu error scale 1 + |u|."""
    u = x @ W["Wb1"][t].double().t() + W["bb1"][t].double()
    th = torch.tanh(C * (u + A * u ** 3))
    return u, 0.5 * u * (1 + th), 0.5 * (1 + th) + 0.5 * u * (1 - th * th) * C * (1 + 3 * A * u * u)


def forward_ref(W, ev, types, wt, mode):
    """Tokens in float64 and the bound on each element's error."""
    R, k = types.shape
    T, d, e = len(W["Wb1"]), W["Wb1"][0].shape[0], ev.shape[1]
    out = torch.zeros(R, d, device="cuda", dtype=torch.float64)
    tol = torch.zeros_like(out)
    for t in range(T):
        W1, W2 = W["Wb1"][t].double(), W["Wb2"][t].double()
        s = W["bb2"][t].double() + W["type_emb"][t].double()
        sa = W["bb2"][t].double().abs() + W["type_emb"][t].double().abs()
        for j in range(k):
            r = torch.nonzero(types[:, j] == t)[:, 0]
            x, w = ev[r].double(), wt[r, j].double()[:, None]
            u, z, slope = parts(W, t, x)
            out.index_add_(0, r, w * (z @ W2.t() + s))
            ua = x.abs() @ W1.t().abs() + W["bb1"][t].double().abs()
            dz = ua * ((e + 2) * 2.0 ** -23) * 1.13 + (1 + u.abs()) * 2.0 ** -20     # |gelu'| <= 1.13
            if mode == "bf16":
                dz = dz + z.abs() * 2.0 ** -8 * 1.01 + u.abs() * 2.0 ** -11.8
            tol.index_add_(0, r, w.abs() * (dz @ W2.t().abs() + (d + 4) * 2.0 ** -23 * (z.abs() @ W2.t().abs() + sa)))
    half = 2.0 ** -8 if mode == "bf16" else 2.0 ** -24
    return out, tol + (out.abs() + tol) * half + k * 2.0 ** -24 * out.abs()


def backward_ref(W, ev, types, wt, dy, dy_in, mode):
    """float64 gradients and the bounds; dy: the operand values, dy_in: the caller's."""
    R, k = types.shape
    T, d, e = len(W["Wb1"]), W["Wb1"][0].shape[0], ev.shape[1]
    z8 = dict(device="cuda", dtype=torch.float64)
    de, dw = torch.zeros(R, e, **z8), torch.zeros(R, k, **z8)
    tde, tdw = torch.zeros(R, e, **z8), torch.zeros(R, k, **z8)
    g = {"Wb1": torch.zeros(T, d, e, **z8), "bb1": torch.zeros(T, d, **z8), "Wb2": torch.zeros(T, d, d, **z8), "bb2": torch.zeros(T, d, **z8)}
    tg = {f: torch.zeros_like(v) for f, v in g.items()}
    split = 2.0 ** -16 if mode == "bf16" else 0.0
    u23 = 2.0 ** -23
    for t in range(T):
        W1, W2 = W["Wb1"][t].double(), W["Wb2"][t].double()
        s = W["bb2"][t].double() + W["type_emb"][t].double()
        for j in range(k):
            r = torch.nonzero(types[:, j] == t)[:, 0]
            n = r.numel() * k + 16
            x, w, y = ev[r].double(), wt[r, j].double()[:, None], dy[r].double()
            u, z, slope = parts(W, t, x)
            ua = x.abs() @ W1.t().abs() + W["bb1"][t].double().abs()
            eu = ua * (e + 2) * u23 + (1 + u.abs()) * 2.0 ** -20      # of u, z, slope (slopes' own slope <= 1.2)
            dz = y @ W2
            edz = (y.abs() @ W2.abs()) * (d + 2) * u23
            du = w * dz * slope
            edu = w.abs() * (edz * 1.2 + dz.abs() * eu * 1.3) + du.abs() * (split + 4 * u23)
            ez = eu * 1.3 + z.abs() * (split + 4 * u23)
            de.index_add_(0, r, du @ W1)
            one = 2.0 ** -8 * 1.01 if mode == "bf16" else 0.0
            tde.index_add_(0, r, (edu + du.abs() * one) @ W1.abs() + (du.abs() @ W1.abs()) * (2 * d + 2) * u23)
            dw[r, j] = (dz * z).sum(1) + (dy_in[r].double() * s).sum(1)
            tdw[r, j] = ((edz * z.abs() + dz.abs() * ez).sum(1) + (dz * z).abs().sum(1) * (d + 8) * u23
                         + (dy_in[r].double().abs() * (s.abs() + 0.4)).sum(1) * (d + 8) * u23)
            if mode == "bf16":
                tdw[r, j] += ((dy_in[r].double() - y).abs() * s.abs()).sum(1)
            wa, ya, xa = w.abs(), y.abs(), x.abs()
            g["Wb2"][t] += (w * y).t() @ z
            tg["Wb2"][t] += (wa * ya).t() @ (ez + z.abs() * (2 * n * u23))
            g["bb2"][t] += (w * y).sum(0)
            tg["bb2"][t] += (wa * ya).sum(0) * (n * u23 + split)
            g["Wb1"][t] += du.t() @ x
            tg["Wb1"][t] += (edu + du.abs() * (2 * n * u23)).t() @ xa
            g["bb1"][t] += du.sum(0)
            tg["bb1"][t] += (edu + du.abs() * (2 * n * u23)).sum(0)
    tde = tde + (de.abs() + tde) * (2.0 ** -8 if mode == "bf16" else 2.0 ** -24) + k * 2.0 ** -24 * de.abs()
    g["type_emb"], tg["type_emb"] = g["bb2"], tg["bb2"]
    return {"devents": de, "dweights": dw, **g}, {"devents": tde, "dweights": tdw, **tg}


def close(got, ref, tol, what):
    got = got.double()
    assert torch.isfinite(got).all(), what
    over = (got - ref).abs() - tol
    assert (over <= 1e-30).all(), (what, float(over.max()), float((got - ref).abs().max()))


CASES = [
    # mode, R, T, k, e, d, weighted, types
    ("fp32", 1, 1, 1, 1, 16, False, "uniform"),
    ("fp32", 300, 3, 1, 64, 256, True, "uniform"),
    ("fp32", 129, 8, 3, 10, 48, True, "skewed"),
    ("fp32", 200, 2, 2, 24, 64, False, "none"),
    ("bf16", 1, 3, 1, 64, 256, False, "uniform"),
    ("bf16", 2, 2, 1, 16, 64, True, "last"),
    ("bf16", 127, 3, 1, 64, 256, True, "uniform"),
    ("bf16", 1025, 3, 1, 64, 256, False, "skewed"),
    ("bf16", 1024, 5, 2, 32, 128, True, "skewed"),
    ("bf16", 3001, 8, 3, 96, 384, True, "skewed"),
    ("bf16", 700, 4, 1, 128, 256, False, "last"),
    ("bf16", 300, 4, 2, 128, 384, True, "none"),
    ("fp32", 10_007, 4, 2, 40, 80, True, "skewed"),    # many slot tiles on CUDA cores
    ("bf16", 12_001, 3, 1, 20, 96, True, "uniform"),
    ("bf16", 513, 2, 1, 20, 96, True, "skewed"),       # widths the tensor-core kernels do not take
    ("bf16", 777, 3, 8, 48, 320, True, "skewed"),
    ("bf16", 260, 2, 1, 64, 512, False, "skewed"),
    ("bf16", 700, 3, 2, 128, 384, True, "skewed"),     # the smallest rings
    ("bf16", 900, 2, 1, 96, 320, True, "uniform"),
    ("bf16", 1500, 3, 1, 64, 192, False, "skewed"),
    ("bf16", 640, 2, 2, 128, 64, True, "skewed"),
    ("bf16", 30_000, 3, 1, 64, 256, True, "skewed"),
    ("bf16", 20_011, 8, 2, 64, 384, True, "skewed"),
]


def inputs(mode, R, T, k, e, d, weighted, kind):
    m, W = make(mode, T, e, d, R + e)
    g = torch.Generator(device="cuda").manual_seed(R + 7)
    ev = torch.randn(R, e, device="cuda", generator=g).to(DT[mode])
    types = make_types(kind, R, k, T, R + 1)
    wt = torch.randn(R, k, device="cuda", generator=g) if weighted else None
    plan = m.input_workspace(ot.OP_ROUTE, R, k)
    plan.fill_(0x5a)
    return m, W, ev, types, wt, plan, g


@pytest.mark.parametrize("mode,R,T,k,e,d,weighted,kind", CASES)
def test_tokens(mode, R, T, k, e, d, weighted, kind):
    m, W, ev, types, wt, plan, _ = inputs(mode, R, T, k, e, d, weighted, kind)
    ot.onetrans_route_events(m, types, plan)
    tok = torch.full((R, d), float("nan"), device="cuda", dtype=DT[mode])
    ws = m.input_workspace(ot.OP_ROUTED, R, k)
    ws.fill_(0xff)                                       # NaN everywhere: nothing of it may be taken for a value
    ot.onetrans_tokenize_routed(m, ev, types, wt, plan, tok, ws)
    torch.cuda.synchronize()
    assert ot.onetrans_device_status() == 0
    w = wt if weighted else torch.ones(R, k, device="cuda")
    ref, tol = forward_ref(W, ev, types, w, mode)
    close(tok, ref, tol, "tokens")
    assert (tok[(types < 0).all(1)] == 0).all()


@pytest.mark.parametrize("mode,R,T,k,e,d,weighted,kind", CASES)
def test_gradients(mode, R, T, k, e, d, weighted, kind):
    m, W, ev, types, wt, plan, g = inputs(mode, R, T, k, e, d, weighted, kind)
    ot.onetrans_route_events(m, types, plan)
    for dy_t in ({torch.float32, DT[mode]}):
        dy_in = torch.randn(R, d, device="cuda", generator=g).to(dy_t)
        dy = dy_in.to(DT[mode])
        de = torch.full((R, e), float("nan"), device="cuda", dtype=DT[mode])
        dw = torch.full((R, k), float("nan"), device="cuda")
        grads = {f: [torch.full(tuple(x.shape), float("nan"), device="cuda") for x in W[f]] for f in ("Wb1", "bb1", "Wb2", "bb2")}
        grads["type_emb"] = torch.full((T, d), float("nan"), device="cuda")
        ws = m.input_workspace(ot.OP_ROUTED_BACKWARD, R, k)
        ws.fill_(0xff)
        ot.onetrans_tokenize_routed_backward(m, ev, types, wt, plan, dy_in, de, dw, grads, ws)
        torch.cuda.synchronize()
        assert ot.onetrans_device_status() == 0
        w = wt if weighted else torch.ones(R, k, device="cuda")
        ref, tol = backward_ref(W, ev, types, w, dy, dy_in, mode)
        close(de, ref["devents"], tol["devents"], "devents")
        close(dw, ref["dweights"], tol["dweights"], "dweights")
        for f in ("Wb1", "bb1", "Wb2", "bb2"):
            close(torch.stack(grads[f]), ref[f], tol[f], f)
        close(grads["type_emb"], ref["type_emb"], tol["type_emb"], "type_emb")
        again = {f: [torch.empty_like(x) for x in grads[f]] for f in ("Wb1", "bb1", "Wb2", "bb2")}
        again["type_emb"] = torch.empty_like(grads["type_emb"])
        ot.onetrans_tokenize_routed_backward(m, ev, types, wt, plan, dy_in, None, None, again, ws)
        for f in ("Wb1", "bb1", "Wb2", "bb2"):               # a fixed order of additions, outputs left out
            for a, b in zip(again[f], grads[f]):
                assert torch.equal(a, b), f


def test_plan_is_a_stable_sort():
    m, _ = make("fp32", 5, 8, 16, 3)
    for R, k in ((1, 1), (127, 3), (1024, 1), (1025, 1), (20_000, 2), (700_001, 2), (1_400_001, 2)):   # the last with scanned counts
        types = make_types("skewed", R, k, 5, R)
        plan = m.input_workspace(ot.OP_ROUTE, R, k)
        ot.onetrans_route_events(m, types, plan)
        p = plan.view(torch.int32).cpu().numpy()
        n, t = R * k, types.cpu().numpy().reshape(-1)
        cap = -(-n // 128) * 128 + 128 * 5
        order, pos = p[64:64 + cap], p[64 + -(-cap // 64) * 64:][:n]
        at = 0
        for b in range(5):
            mine = np.nonzero(t == b)[0]
            assert p[8 + b] == len(mine) and p[16 + b] == at
            assert (order[at:at + len(mine)] == mine).all()
            assert (pos[mine] == at + np.arange(len(mine))).all()
            end = at + -(-len(mine) // 128) * 128
            assert (order[at + len(mine):end] == -1).all()
            at = end
        assert p[16 + 5] == at and (pos[t < 0] == -1).all()
    assert ot.onetrans_device_status() == 0


@pytest.mark.parametrize("d,e,k", [(256, 64, 1), (384, 32, 3)])
def test_both_kernel_sets(d, e, k):
    """The same call on tensor cores and (kernel policy 1) on CUDA cores, each within the bounds."""
    m, W, ev, types, wt, plan, g = inputs("bf16", 1300, 4, k, e, d, True, "skewed")
    dy = torch.randn(1300, d, device="cuda", generator=g).bfloat16()
    ot.onetrans_route_events(m, types, plan)
    ws, wsb = m.input_workspace(ot.OP_ROUTED, 1300, k), m.input_workspace(ot.OP_ROUTED_BACKWARD, 1300, k)
    ftok, ttok = forward_ref(W, ev, types, wt, "bf16")
    ref, tol = backward_ref(W, ev, types, wt, dy, dy, "bf16")
    try:
        for policy in (0, 1):
            ot.onetrans_set_kernel_policy(policy)
            tok = torch.empty(1300, d, device="cuda", dtype=torch.bfloat16)
            ot.onetrans_tokenize_routed(m, ev, types, wt, plan, tok, ws)
            close(tok, ftok, ttok, "tokens")
            grads = {f: [torch.empty(tuple(x.shape), device="cuda") for x in W[f]] for f in ("Wb1", "bb1", "Wb2", "bb2")}
            grads["type_emb"] = torch.empty(4, d, device="cuda")
            de, dw = torch.empty_like(ev), torch.empty(1300, k, device="cuda")
            ot.onetrans_tokenize_routed_backward(m, ev, types, wt, plan, dy, de, dw, grads, wsb)
            close(de, ref["devents"], tol["devents"], "devents")
            close(dw, ref["dweights"], tol["dweights"], "dweights")
            for f in ("Wb1", "bb1", "Wb2", "bb2"):
                close(torch.stack(grads[f]), ref[f], tol[f], f)
            assert ot.onetrans_device_status() == 0
    finally:
        ot.onetrans_set_kernel_policy(0)


def test_types_out_of_range_are_flagged_and_take_no_part():
    m, W = make("bf16", 2, 16, 64, 5)
    ev = torch.randn(4, 16, device="cuda").bfloat16()
    types = torch.tensor([0, 2, -5, 1], device="cuda", dtype=torch.int32)
    plan = m.input_workspace(ot.OP_ROUTE, 4, 1)
    ot.onetrans_route_events(m, types, plan)
    assert ot.onetrans_device_status() == 3
    tok = torch.full((4, 64), 9.0, device="cuda", dtype=torch.bfloat16)
    ot.onetrans_tokenize_routed(m, ev, types, None, plan, tok, m.input_workspace(ot.OP_ROUTED, 4, 1))
    assert ot.onetrans_device_status() == 0
    assert (tok[1:3] == 0).all() and (tok[0] != 0).any() and (tok[3] != 0).any()


@pytest.mark.parametrize("mode", ["bf16", "fp32"])
def test_a_plan_of_other_sizes_is_refused_on_the_device(mode):
    m, W = make(mode, 2, 16, 64, 5)
    R = 200
    ev = torch.randn(R, 16, device="cuda").to(DT[mode])
    types = torch.zeros(R, device="cuda", dtype=torch.int32)
    plan = m.input_workspace(ot.OP_ROUTE, R, 1)
    tok = torch.full((R, 64), 9.0, device="cuda", dtype=DT[mode])
    ws = m.input_workspace(ot.OP_ROUTED, R, 1)
    plan.zero_()                                         # never made
    ot.onetrans_tokenize_routed(m, ev, types, None, plan, tok, ws)
    assert ot.onetrans_device_status() == 3
    ot.onetrans_route_events(m, types[:100].contiguous(), plan)   # made for fewer events
    ot.onetrans_tokenize_routed(m, ev, types, None, plan, tok, ws)
    assert ot.onetrans_device_status() == 3
    assert (tok == 9.0).all()
    grads = {f: [torch.full(tuple(x.shape), 9.0, device="cuda") for x in W[f]] for f in ("Wb1", "bb1", "Wb2", "bb2")}
    grads["type_emb"] = torch.full((2, 64), 9.0, device="cuda")
    de, dw = torch.full_like(ev, 9.0), torch.full((R, 1), 9.0, device="cuda")
    ot.onetrans_tokenize_routed_backward(m, ev, types, None, plan, tok, de, dw, grads, m.input_workspace(ot.OP_ROUTED_BACKWARD, R, 1))
    assert ot.onetrans_device_status() == 3
    assert all((x == 9.0).all() for f in ("Wb1", "bb1", "Wb2", "bb2") for x in grads[f])
    assert (de == 9.0).all() and (dw == 9.0).all() and (grads["type_emb"] == 9.0).all()


@pytest.mark.parametrize("mode,d,k", [("bf16", 256, 1), ("bf16", 128, 2), ("fp32", 48, 1)])
def test_rows_inside_a_stack_input(mode, d, k):
    """Tokens written into x0's S rows, their gradient read from a float32 dx0, in place."""
    B, L, L_NS, e, T = 3, 117, 5, 32, 3
    m, W = make(mode, T, e, d, 11)
    R = B * L
    ev = torch.randn(R, e, device="cuda").to(DT[mode])
    types = make_types("skewed", R, k, T, 12)
    plan = m.input_workspace(ot.OP_ROUTE, R, k)
    ot.onetrans_route_events(m, types, plan)
    flat = torch.empty(R, d, device="cuda", dtype=DT[mode])
    ws = m.input_workspace(ot.OP_ROUTED, R, k)
    ot.onetrans_tokenize_routed(m, ev, types, None, plan, flat, ws)
    x0 = torch.full((B, L + L_NS, d), 5.0, device="cuda", dtype=DT[mode])
    ot.onetrans_tokenize_routed(m, ev, types, None, plan, x0[:, :L], ws)
    assert torch.equal(x0[:, :L].reshape(R, d), flat)
    assert (x0[:, L:] == 5.0).all()
    dx0 = torch.randn(B, L + L_NS, d, device="cuda")
    out = []
    for dy in (dx0[:, :L], dx0[:, :L].reshape(R, d)):
        grads = {f: [torch.empty(tuple(x.shape), device="cuda") for x in W[f]] for f in ("Wb1", "bb1", "Wb2", "bb2")}
        grads["type_emb"] = torch.empty(T, d, device="cuda")
        de, dw = torch.empty_like(ev), torch.empty(R, k, device="cuda")
        ot.onetrans_tokenize_routed_backward(m, ev, types, None, plan, dy, de, dw, grads,
                                             m.input_workspace(ot.OP_ROUTED_BACKWARD, R, k))
        out.append([de, dw, grads["type_emb"]] + [x for f in ("Wb1", "bb1", "Wb2", "bb2") for x in grads[f]])
    for a, b in zip(*out):
        assert torch.equal(a, b)
    assert ot.onetrans_device_status() == 0


def test_equals_the_event_tokenizer():
    """One unweighted choice per event is onetrans_tokenize_events' function."""
    m, W = make("fp32", 3, 64, 256, 17)
    R = 400
    ev = torch.randn(R, 64, device="cuda")
    types = torch.randint(0, 3, (R,), device="cuda", dtype=torch.int32)
    a, b = torch.empty(R, 256, device="cuda"), torch.empty(R, 256, device="cuda")
    ot.onetrans_tokenize_events(m, ev, types, a)
    plan = m.input_workspace(ot.OP_ROUTE, R, 1)
    ot.onetrans_route_events(m, types, plan)
    ot.onetrans_tokenize_routed(m, ev, types, None, plan, b, m.input_workspace(ot.OP_ROUTED, R, 1))
    ref, tol = forward_ref(W, ev, types[:, None], torch.ones(R, 1, device="cuda"), "fp32")
    close(a, ref, tol, "onetrans_tokenize_events")
    close(b, ref, tol, "onetrans_tokenize_routed")


def test_nan_stays_with_its_events():
    """Events, weights and gradients of choices that are none never reach a sum; a NaN event reaches its own token,
    its behaviour's weight gradients and no other behaviour's."""
    for mode in ("bf16", "fp32"):
        T, k, e, d, R = 3, 2, 64, 256, 500
        m, W = make(mode, T, e, d, 23)
        types = make_types("skewed", R, k, T, 24)
        types[7] = torch.tensor([2, -1])
        types[9] = -1
        ev = torch.randn(R, e, device="cuda").to(DT[mode])
        wt = torch.randn(R, k, device="cuda")
        dy = torch.randn(R, d, device="cuda").to(DT[mode])
        ev[7, 3], ev[9, 4], dy[9, 1], wt[types < 0] = float("nan"), float("nan"), float("nan"), float("nan")
        plan = m.input_workspace(ot.OP_ROUTE, R, k)
        ot.onetrans_route_events(m, types, plan)
        tok = torch.empty(R, d, device="cuda", dtype=DT[mode])
        ot.onetrans_tokenize_routed(m, ev, types, wt, plan, tok, m.input_workspace(ot.OP_ROUTED, R, k))
        bad = ~torch.isfinite(tok).all(1)
        assert bad[7] and int(bad.sum()) == 1 and (tok[9] == 0).all()
        grads = {f: [torch.empty(tuple(x.shape), device="cuda") for x in W[f]] for f in ("Wb1", "bb1", "Wb2", "bb2")}
        grads["type_emb"] = torch.empty(T, d, device="cuda")
        de, dw = torch.empty_like(ev), torch.empty(R, k, device="cuda")
        ot.onetrans_tokenize_routed_backward(m, ev, types, wt, plan, dy, de, dw, grads,
                                             m.input_workspace(ot.OP_ROUTED_BACKWARD, R, k))
        bad = ~torch.isfinite(de).all(1)
        assert bad[7] and int(bad.sum()) == 1 and (de[9] == 0).all()
        assert torch.isfinite(dw).sum() == R * k - 1 and (dw[types < 0] == 0).all()
        for t in range(2):
            assert all(torch.isfinite(grads[f][t]).all() for f in ("Wb1", "bb1", "Wb2", "bb2"))
        assert torch.isfinite(grads["type_emb"]).all() and not torch.isfinite(grads["Wb1"][2]).all()


def test_finite_differences():
    """d sum(c * tokens) along random directions of the events, the weights and every MLP weight, float32 mode,
    against central differences of the tokenizer."""
    T, k, e, d, R = 3, 2, 24, 64, 150
    m, W = make("fp32", T, e, d, 31)
    g = torch.Generator(device="cuda").manual_seed(32)
    types = make_types("skewed", R, k, T, 33)
    ev, wt = torch.randn(R, e, device="cuda", generator=g), torch.randn(R, k, device="cuda", generator=g)
    c = torch.randn(R, d, device="cuda", generator=g)
    plan = m.input_workspace(ot.OP_ROUTE, R, k)
    ws = m.input_workspace(ot.OP_ROUTED, R, k)
    ot.onetrans_route_events(m, types, plan)
    grads = {f: [torch.empty(tuple(x.shape), device="cuda") for x in W[f]] for f in ("Wb1", "bb1", "Wb2", "bb2")}
    grads["type_emb"] = torch.empty(T, d, device="cuda")
    de, dw = torch.empty_like(ev), torch.empty(R, k, device="cuda")
    ot.onetrans_tokenize_routed_backward(m, ev, types, wt, plan, c, de, dw, grads, m.input_workspace(ot.OP_ROUTED_BACKWARD, R, k))

    def f():
        tok = torch.empty(R, d, device="cuda")
        ot.onetrans_tokenize_routed(m, ev, types, wt, plan, tok, ws)
        return float((tok.double() * c.double()).sum()), float((tok.double() * c.double()).abs().sum())

    pairs = [([ev], [de]), ([wt], [dw]), ([W["type_emb"]], [grads["type_emb"]])] + [(W[n], grads[n]) for n in ("Wb1", "bb1", "Wb2", "bb2")]
    h = 2.0 ** -7
    for xs, gs in pairs:
        vs = [torch.randn(tuple(x.shape), device="cuda", generator=g) for x in xs]
        ref = sum(float((a.double() * v.double()).sum()) for a, v in zip(gs, vs))
        keep = [x.clone() for x in xs]
        val = []
        for s in (h, -h, 2 * h, -2 * h):
            for x, x0, v in zip(xs, keep, vs):
                x.copy_(x0 + s * v)
            val.append(f())
        for x, x0 in zip(xs, keep):
            x.copy_(x0)
        # two central differences extrapolated: error of order h^4, plus the tokens' float32 roundings
        # (about d sums of 2^-24 relative each) divided by h
        diff = (8 * (val[0][0] - val[1][0]) - (val[2][0] - val[3][0])) / (12 * h)
        size = max(v[1] for v in val)
        assert abs(diff - ref) <= 4 * size * (h ** 4 * 64 + 2.0 ** -24 * 16 / h), (diff, ref)


def test_captured_replays_and_other_stream():
    """Route, tokens and gradient captured on a side stream in one graph, replayed on new inputs in the same
    buffers, beside an eager call on the default stream with buffers of its own."""
    T, k, e, d, R = 3, 2, 64, 256, 2_000
    m, W = make("bf16", T, e, d, 41)
    ev = torch.randn(R, e, device="cuda").bfloat16()
    types, wt = make_types("skewed", R, k, T, 42), torch.randn(R, k, device="cuda")
    dy = torch.randn(R, d, device="cuda").bfloat16()

    def buffers():
        grads = {f: [torch.empty(tuple(x.shape), device="cuda") for x in W[f]] for f in ("Wb1", "bb1", "Wb2", "bb2")}
        grads["type_emb"] = torch.empty(T, d, device="cuda")
        return dict(plan=m.input_workspace(ot.OP_ROUTE, R, k), ws=m.input_workspace(ot.OP_ROUTED, R, k),
                    wsb=m.input_workspace(ot.OP_ROUTED_BACKWARD, R, k), tok=torch.empty(R, d, device="cuda", dtype=torch.bfloat16),
                    de=torch.empty_like(ev), dw=torch.empty(R, k, device="cuda"), grads=grads)

    def step(b):
        ot.onetrans_route_events(m, types, b["plan"])
        ot.onetrans_tokenize_routed(m, ev, types, wt, b["plan"], b["tok"], b["ws"])
        ot.onetrans_tokenize_routed_backward(m, ev, types, wt, b["plan"], dy, b["de"], b["dw"], b["grads"], b["wsb"])

    def flat(b):
        return [b["tok"], b["de"], b["dw"], b["grads"]["type_emb"]] + [x for f in ("Wb1", "bb1", "Wb2", "bb2") for x in b["grads"][f]]

    one, two = buffers(), buffers()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(one)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(one)
    for seed in (43, 44):
        types.copy_(make_types("uniform" if seed == 43 else "skewed", R, k, T, seed))
        ev.copy_(torch.randn(R, e, device="cuda").bfloat16())
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        step(two)                                         # at the same time, on the default stream
        torch.cuda.synchronize()
        for a, b in zip(flat(one), flat(two)):
            assert torch.equal(a, b)
    assert ot.onetrans_device_status() == 0


def test_no_events():
    m, W = make("bf16", 2, 16, 64, 51)
    types = torch.empty(0, device="cuda", dtype=torch.int32)
    ev, tok = torch.empty(0, 16, device="cuda", dtype=torch.bfloat16), torch.empty(0, 64, device="cuda", dtype=torch.bfloat16)
    plan = m.input_workspace(ot.OP_ROUTE, 0, 1)
    ot.onetrans_route_events(m, types, plan)
    ot.onetrans_tokenize_routed(m, ev, types, None, plan, tok, m.input_workspace(ot.OP_ROUTED, 0, 1))
    grads = {f: [torch.full(tuple(x.shape), 9.0, device="cuda") for x in W[f]] for f in ("Wb1", "bb1", "Wb2", "bb2")}
    grads["type_emb"] = torch.full((2, 64), 9.0, device="cuda")
    ot.onetrans_tokenize_routed_backward(m, ev, types, None, plan, tok, None, None, grads, m.input_workspace(ot.OP_ROUTED_BACKWARD, 0, 1))
    assert all((x == 0).all() for f in ("Wb1", "bb1", "Wb2", "bb2") for x in grads[f]) and (grads["type_emb"] == 0).all()


def test_more_slot_tiles_than_a_grid_dimension():
    """4.2 million choices, 65552 tiles of 64 slots on CUDA cores: tokens and event gradient of every row."""
    R, d, e = 64 * 65536 + 1000, 16, 1
    m, W = make("fp32", 1, e, d, 71)
    g = torch.Generator(device="cuda").manual_seed(72)
    ev = torch.randn(R, e, device="cuda", generator=g)
    types = torch.zeros(R, device="cuda", dtype=torch.int32)
    wt = torch.ones(R, 1, device="cuda")
    plan = m.input_workspace(ot.OP_ROUTE, R, 1)
    ot.onetrans_route_events(m, types, plan)
    tok = torch.empty(R, d, device="cuda")
    ot.onetrans_tokenize_routed(m, ev, types, None, plan, tok, m.input_workspace(ot.OP_ROUTED, R, 1))
    ref, tol = forward_ref(W, ev, types[:, None], wt, "fp32")
    close(tok, ref, tol, "tokens")
    del ref, tol
    dy = torch.randn(R, d, device="cuda", generator=g)
    de = torch.empty_like(ev)
    grads = {f: [torch.empty(tuple(x.shape), device="cuda") for x in W[f]] for f in ("Wb1", "bb1", "Wb2", "bb2")}
    grads["type_emb"] = torch.empty(1, d, device="cuda")
    ot.onetrans_tokenize_routed_backward(m, ev, types, None, plan, dy, de, None, grads,
                                         m.input_workspace(ot.OP_ROUTED_BACKWARD, R, 1))
    ref, tol = backward_ref(W, ev, types[:, None], wt, dy, dy, "fp32")
    close(de, ref["devents"], tol["devents"], "devents")
    for f in ("Wb1", "bb1", "Wb2", "bb2"):
        close(torch.stack(grads[f]), ref[f], tol[f], f)
    assert ot.onetrans_device_status() == 0


@pytest.mark.parametrize("d,k", [(128, 1), (256, 1), (256, 2), (384, 2)])
def test_choice_weights_reach_every_sum_exactly(d, k):
    """Small whole choice weights through operands that make every product a whole number: W1 = 0 and b1 = 16 give
    z = 16 and a slope of 1, W2 the identity gives dz = dtoken = 1.  Every gradient is then a sum of whole numbers
    below 2^24 and has to be exact: one choice whose weight was read from another step would change it."""
    T, e, R = 3, 64, 40_001
    m, W = make("bf16", T, e, d, 91)
    for t in range(T):
        W["Wb1"][t].zero_()
        W["bb1"][t].fill_(16.0)
        W["Wb2"][t].copy_(torch.eye(d))
        W["bb2"][t].zero_()
    W["type_emb"].zero_()
    g = torch.Generator(device="cuda").manual_seed(92)
    ev = torch.ones(R, e, device="cuda", dtype=torch.bfloat16)
    dy = torch.ones(R, d, device="cuda", dtype=torch.bfloat16)
    plan, ws = m.input_workspace(ot.OP_ROUTE, R, k), m.input_workspace(ot.OP_ROUTED_BACKWARD, R, k)
    for seed in range(6):
        types = make_types("skewed", R, k, T, 93 + seed)
        wt = torch.randint(1, 10, (R, k), device="cuda", generator=g).float()
        ot.onetrans_route_events(m, types, plan)
        grads = {f: [torch.full(tuple(x.shape), float("nan"), device="cuda") for x in W[f]] for f in ("Wb1", "bb1", "Wb2", "bb2")}
        grads["type_emb"] = torch.full((T, d), float("nan"), device="cuda")
        de, dw = torch.full_like(ev, float("nan")), torch.full((R, k), float("nan"), device="cuda")
        ot.onetrans_tokenize_routed_backward(m, ev, types, wt, plan, dy, de, dw, grads, ws)
        assert ot.onetrans_device_status() == 0
        for t in range(T):
            n = float(wt[types == t].sum())
            assert 16 * n < 2 ** 24
            for f, scale in (("Wb1", 1), ("bb1", 1), ("Wb2", 16), ("bb2", 1)):
                assert (grads[f][t] == scale * n).all(), (seed, t, f)
            assert (grads["type_emb"][t] == n).all()
        assert (dw[types >= 0] == 16 * d).all() and (dw[types < 0] == 0).all() and (de == 0).all()


@pytest.mark.parametrize("mode,d,k", [("bf16", 256, 1), ("bf16", 128, 2), ("fp32", 64, 2)])
def test_the_stride_of_a_lone_sample_changes_nothing(mode, d, k):
    """With rows_per_sample >= R the sample stride is unused: whatever it is, the same kernels run and give the same
    bits, forward and backward (an odd one once sent a bf16 call to the CUDA-core kernels, which round less)."""
    R, T, e = 333, 3, 64
    m, W, ev, types, wt, plan, g = inputs(mode, R, T, k, e, d, True, "skewed")
    ot.onetrans_route_events(m, types, plan)
    ws, wsb = m.input_workspace(ot.OP_ROUTED, R, k), m.input_workspace(ot.OP_ROUTED_BACKWARD, R, k)
    st = torch.cuda.current_stream().cuda_stream
    dy = torch.randn(R, d, device="cuda", generator=g)
    out = []
    for per, ld in ((R, R * d), (R, 0), (R, 1), (R + 1, 12_345), (2 ** 40, -7)):
        tok = torch.empty(R, d, device="cuda", dtype=DT[mode])
        ot._check("tokens", ot.lib.onetrans_tokenize_routed(m.handle, ev.data_ptr(), wt.data_ptr(), R, k, plan.data_ptr(),
                                                            plan.numel(), tok.data_ptr(), per, ld, ws.data_ptr(), ws.numel(), st))
        grads = {f: [torch.empty(tuple(x.shape), device="cuda") for x in W[f]] for f in ("Wb1", "bb1", "Wb2", "bb2")}
        emb, de, dw = torch.empty(T, d, device="cuda"), torch.empty_like(ev), torch.empty(R, k, device="cuda")
        s, keep = ot.EventGrads(), []
        for f in ("Wb1", "bb1", "Wb2", "bb2"):
            keep.append((ot.P * T)(*[x.data_ptr() for x in grads[f]]))
            setattr(s, f, ot.ctypes.cast(keep[-1], ot.PP))
        s.type_emb = emb.data_ptr()
        ot._check("gradient", ot.lib.onetrans_tokenize_routed_backward(
            m.handle, ev.data_ptr(), wt.data_ptr(), R, k, plan.data_ptr(), plan.numel(), dy.data_ptr(), ot.FP32, per, ld,
            de.data_ptr(), dw.data_ptr(), ot.ctypes.byref(s), wsb.data_ptr(), wsb.numel(), st))
        out.append([tok, de, dw, emb] + [x for f in ("Wb1", "bb1", "Wb2", "bb2") for x in grads[f]])
    for other in out[1:]:
        assert all(torch.equal(a, b) for a, b in zip(out[0], other))
    assert ot.onetrans_device_status() == 0


@pytest.mark.parametrize("mode,d,e", [("fp32", 64, 24), ("bf16", 96, 20), ("bf16", 128, 64)])
def test_hidden_units_whose_squares_overflow_keep_a_finite_slope(mode, d, e):
    """Events of 1e19 and more give u whose square is past float32: GELU's slope there is 0 or 1, and the event's
    gradient W1^T (w dz slope) an ordinary number (the polynomial factor of the slope, inf, times its 0 once made NaN).
    Off by the float32 sums, in bf16 mode by du's and the event gradient's roundings (2^-8 each)."""
    T, R = 2, 200
    m, W = make(mode, T, e, d, 121)
    g = torch.Generator(device="cuda").manual_seed(122)
    ev = torch.randn(R, e, device="cuda", generator=g)
    ev[::3] *= 2.0 ** 66
    ev = ev.to(DT[mode])
    types = make_types("uniform", R, 1, T, 123)
    wt, dy = torch.rand(R, 1, device="cuda", generator=g) + 0.5, torch.randn(R, d, device="cuda", generator=g).to(DT[mode])
    plan = m.input_workspace(ot.OP_ROUTE, R, 1)
    ot.onetrans_route_events(m, types, plan)
    de, dw = torch.empty_like(ev), torch.empty(R, 1, device="cuda")
    grads = {f: [torch.empty(tuple(x.shape), device="cuda") for x in W[f]] for f in ("Wb1", "bb1", "Wb2", "bb2")}
    grads["type_emb"] = torch.empty(T, d, device="cuda")
    ot.onetrans_tokenize_routed_backward(m, ev, types, wt, plan, dy, de, dw, grads, m.input_workspace(ot.OP_ROUTED_BACKWARD, R, 1))
    assert ot.onetrans_device_status() == 0
    for f in grads:
        assert all(torch.isfinite(x).all() for x in grads[f]), f
    assert torch.isfinite(dw).all()
    u23, one = 2.0 ** -23, 2.0 ** -8 * 1.01 if mode == "bf16" else 2.0 ** -24
    big = torch.arange(R, device="cuda") % 3 == 0
    for t in range(T):
        r = torch.nonzero((types[:, 0] == t) & big)[:, 0]
        W1, W2 = W["Wb1"][t].double(), W["Wb2"][t].double()
        u, _, slope = parts(W, t, ev[r].double())
        assert (u.abs() > 1e10).all() and ((slope == 0) | (slope == 1)).all()
        y = dy[r].double()
        du = wt[r].double() * (y @ W2) * slope
        edu = wt[r].double() * (y.abs() @ W2.abs()) * ((d + 2) * u23) + du.abs() * (one + 4 * u23)
        ref = du @ W1
        tol = edu @ W1.abs() + (du.abs() @ W1.abs()) * ((2 * d + 2) * u23)
        close(de[r], ref, tol + (ref.abs() + tol) * one, "devents")


@pytest.mark.parametrize("R,T,k,e,d", [(30_000, 3, 1, 64, 256), (20_011, 8, 2, 64, 384)])
def test_weight_gradients_of_many_events_norm_wise(R, T, k, e, d):
    """The element bounds above grow with the number of events, past what a lost low term of z or du would cost; the
    norm does not.  dtokens are random and independent of z, so the terms of a sum and their errors both add up as
    random walks: the two bf16 terms' rounding (2^-16 at most, 2^-16.8 in the mean square), and the tensor cores'
    truncated float32 sums (about 126 additions of a piece, 2^-24 each in the mean, all of one sign: 2^-17) make about
    2^-15.5 of the norm.  The bar is 2^-12.  With one term (2^-8 at most, 2^-9.3 in the mean square) the oracle itself
    is twice past it and more."""
    m, W, ev, types, wt, plan, g = inputs("bf16", R, T, k, e, d, True, "skewed")
    dy = torch.randn(R, d, device="cuda", generator=g).bfloat16()
    ot.onetrans_route_events(m, types, plan)
    grads = {f: [torch.empty(tuple(x.shape), device="cuda") for x in W[f]] for f in ("Wb1", "bb1", "Wb2", "bb2")}
    grads["type_emb"] = torch.empty(T, d, device="cuda")
    ot.onetrans_tokenize_routed_backward(m, ev, types, wt, plan, dy, None, None, grads, m.input_workspace(ot.OP_ROUTED_BACKWARD, R, k))
    assert ot.onetrans_device_status() == 0
    ref, _ = backward_ref(W, ev, types, wt, dy, dy, "bf16")

    def off(got, want):
        return float((got.double() - want).norm() / want.norm())

    for f in ("Wb1", "bb1", "Wb2", "bb2"):
        for t in range(T):
            assert off(grads[f][t], ref[f][t]) <= 2.0 ** -12, (f, t)
    Wc = {f: ([x.cpu() for x in W[f]] if isinstance(W[f], list) else W[f].cpu()) for f in W}   # the planted mistake
    r = torch.nonzero(types[:, 0].cpu() == 0)[:, 0]
    x, w, y = ev.cpu()[r].double(), wt.cpu()[r, 0].double()[:, None], dy.cpu()[r].double()
    _, z, slope = parts(Wc, 0, x)
    z, du = w * z, w * (y @ Wc["Wb2"][0].double()) * slope
    assert off(y.t() @ z.bfloat16().double(), y.t() @ z) > 2.0 ** -11
    assert off(du.bfloat16().double().t() @ x, du.t() @ x) > 2.0 ** -11


@pytest.mark.parametrize("mode,positive", [("bf16", False), ("bf16", True), ("fp32", True)])
def test_weight_gradients_of_millions_of_events(mode, positive):
    """A weight gradient's float32 sums are cut into pieces of at most 8192 events.  On tensor cores a piece is 1024
    additions (16 slots each, two terms) that truncate by 2^-23 of the partial sum at most; a term is in half of the
    partial sums on average: within 1024 / 2 * 2^-23 = 2^-14 of the norm, and the two terms' rounding (2^-16) is of
    either sign.  One CTA's sum over a share of all events grew with their number (here past 1e-4)."""
    R, T, e, d = 4_000_000, 1, 16, 64
    m, W, ev, types, wt, plan, g = inputs(mode, R, T, 1, e, d, True, "last")
    dy = torch.randn(R, d, device="cuda", generator=g).to(DT[mode])
    if positive:
        wt, dy = wt.abs(), dy.abs()
    ot.onetrans_route_events(m, types, plan)
    grads = {f: [torch.empty(tuple(x.shape), device="cuda") for x in W[f]] for f in ("Wb1", "bb1", "Wb2", "bb2")}
    grads["type_emb"] = torch.empty(T, d, device="cuda")
    ot.onetrans_tokenize_routed_backward(m, ev, types, wt, plan, dy, None, None, grads, m.input_workspace(ot.OP_ROUTED_BACKWARD, R, 1))
    assert ot.onetrans_device_status() == 0
    ref = {f: torch.zeros(tuple(W[f][0].shape), device="cuda", dtype=torch.float64) for f in ("Wb1", "bb1", "Wb2", "bb2")}
    for r in torch.arange(R, device="cuda").split(1 << 19):
        x, w, y = ev[r].double(), wt[r].double(), dy[r].double()
        _, z, slope = parts(W, 0, x)
        du = w * (y @ W["Wb2"][0].double()) * slope
        for f, v in (("Wb1", du.t() @ x), ("bb1", du.sum(0)), ("Wb2", (w * y).t() @ z), ("bb2", (w * y).sum(0))):
            ref[f] += v
    for f in ref:
        assert float((grads[f][0].double() - ref[f]).norm() / ref[f].norm()) <= 2.0 ** -14, f
