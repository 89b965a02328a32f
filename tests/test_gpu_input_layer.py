"""The input layer's operators as they are used together: item ids -> embedding
lookup -> routed tokenizer, written into x0 -> the block stack's training step
-> dx0 -> the tokenizer's gradient -> the table's gradient.  Against the fp64
oracle of the stack and plain float64 code for the rest.  Norm-wise bars, as
for the stack's own training step: 1e-4 in float32 mode; 2e-2 in bf16 mode
(each step rounds its operands and stored values to bf16, 2^-8 at most and
about 2^-9.3 in the mean: a chain of a dozen adds up to well below 1e-2)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from onetrans_synth import gen_normal
from oracle import onetrans as O
from helpers import EPS, attn_std, build, shape, tdt, to_dev, to_np
from test_gpu_routed import backward_ref, close

import unified_transformer_recommender_b200 as ot  # noqa: E402

KEYS = ("g_attn", "g_ffn", "Wqkv_S", "Wqkv_NS", "Wo", "W1_S", "b1_S", "W2_S", "b2_S", "W1_NS", "b1_NS", "W2_NS", "b2_NS")


def gelu(u):
    c, a = np.sqrt(2 / np.pi), 0.044715
    th = np.tanh(c * (u + a * u ** 3))
    return 0.5 * u * (1 + th), 0.5 * (1 + th) + 0.5 * u * (1 - th * th) * c * (1 + 3 * a * u * u)


def nerr(got, ref):
    return float(np.linalg.norm(np.asarray(got, np.float64) - ref) / np.linalg.norm(ref))


@pytest.mark.parametrize("dtype,k", [("bf16", 1), ("bf16", 2), ("fp32", 2)])
def test_ids_to_table_gradient(dtype, k):
    B, L, V, e, T = 3, 90, 400, 64, 3
    sh = shape(n_layers=2, L_NS=12)
    b = build(sh, 61, dtype, event_dim=e, std=attn_std(sh.d), pyramid=[L + 12, 12])
    m, W, d, R, dt = b.model, b.W, sh.d, B * L, tdt(dtype)
    g = np.random.default_rng(62)
    ids = g.integers(0, V, R)
    ids[g.random(R) < 0.05] = -1
    types = g.integers(0, T, (R, k)).astype(np.int32)
    if k > 1:
        types[g.random((R, k)) < 0.3] = -1
    wt = (g.random((R, k)) + 0.25).astype(np.float32)
    table = gen_normal(63, (V, e), dtype)
    NS = gen_normal(64, (B, 12, d), dtype)
    dY = gen_normal(65, (B, 12, d), "fp32")
    scale = 1.25

    # the framework
    ids_d = torch.from_numpy(ids).cuda()
    ty_d, wt_d = torch.from_numpy(types).cuda(), torch.from_numpy(wt).cuda()
    ev = torch.empty(R, e, device="cuda", dtype=dt)
    x0 = torch.empty(B, L + 12, d, device="cuda", dtype=dt)
    x0[:, L:] = to_dev(NS, dt)
    plan = m.input_workspace(ot.OP_ROUTE, R, k)
    ot.onetrans_embedding_lookup(m, to_dev(table, dt), ids_d, ev, scale=scale)
    ot.onetrans_route_events(m, ty_d, plan)
    ot.onetrans_tokenize_routed(m, ev, ty_d, wt_d, plan, x0[:, :L], m.input_workspace(ot.OP_ROUTED, R, k))
    out, dx0 = torch.empty(B, 12, d, device="cuda"), torch.empty(B, L + 12, d, device="cuda")
    sg = {f: [torch.empty(np.shape(W[f][n]), device="cuda") for n in range(2)] for f in KEYS}
    ot.onetrans_forward_backward(m, x0, torch.from_numpy(dY).cuda(), out, dx0, sg, m.workspace(ot.OP_TRAIN, B, L))
    grads = {f: [torch.empty(np.shape(W[f][t]), device="cuda") for t in range(T)] for f in ("Wb1", "bb1", "Wb2", "bb2")}
    grads["type_emb"] = torch.empty(T, d, device="cuda")
    de, dw = torch.empty_like(ev), torch.empty(R, k, device="cuda")
    ot.onetrans_tokenize_routed_backward(m, ev, ty_d, wt_d, plan, dx0[:, :L], de, dw, grads,
                                         m.input_workspace(ot.OP_ROUTED_BACKWARD, R, k))
    uniq, rows = torch.zeros(V, device="cuda", dtype=torch.int64), torch.zeros(V, e, device="cuda")
    n = torch.zeros(1, device="cuda", dtype=torch.int32)
    ot.onetrans_embedding_backward_sparse(m, de, ids_d, V, uniq, rows, n, m.input_workspace(ot.OP_EMBEDDING_BACKWARD, R, e),
                                          scale=scale)
    torch.cuda.synchronize()
    assert ot.onetrans_device_status() == 0

    # float64
    E = np.where((ids >= 0)[:, None], table[np.maximum(ids, 0)].astype(np.float64) * scale, 0.0)
    tok = np.zeros((R, d))
    for t in range(T):
        for j in range(k):
            r = np.nonzero(types[:, j] == t)[0]
            z, _ = gelu(E[r] @ W["Wb1"][t].T.astype(np.float64) + W["bb1"][t])
            tok[r] += wt[r, j, None] * (z @ W["Wb2"][t].T.astype(np.float64) + W["bb2"][t] + W["type_emb"][t])
    X0 = np.concatenate([tok.reshape(B, L, d), NS], axis=1)
    Y, dX, dW = O.forward_backward(X0, W, 12, sh.n_heads, EPS, [L + 12, 12], dY)
    dtok = dX[:, :L].reshape(R, d)
    gE, gw, tn = np.zeros((R, e)), np.zeros((R, k)), np.zeros((R, k))   # tn: |t| of each choice
    G = {"Wb1": [0.0] * T, "bb1": [0.0] * T, "Wb2": [0.0] * T, "bb2": [0.0] * T}
    for t in range(T):
        W1, W2 = W["Wb1"][t].astype(np.float64), W["Wb2"][t].astype(np.float64)
        for j in range(k):
            r = np.nonzero(types[:, j] == t)[0]
            z, slope = gelu(E[r] @ W1.T + W["bb1"][t])
            y, w = dtok[r], wt[r, j, None].astype(np.float64)
            dz = y @ W2
            du = w * dz * slope
            gE[r] += du @ W1
            tn[r, j] = np.linalg.norm(z @ W2.T + W["bb2"][t] + W["type_emb"][t], axis=1)
            gw[r, j] = (dz * z).sum(1) + y @ (W["bb2"][t] + W["type_emb"][t]).astype(np.float64)
            G["Wb1"][t] = G["Wb1"][t] + du.T @ E[r]
            G["bb1"][t] = G["bb1"][t] + du.sum(0)
            G["Wb2"][t] = G["Wb2"][t] + (w * y).T @ z
            G["bb2"][t] = G["bb2"][t] + (w * y).sum(0)
    tab = np.zeros((V, e))
    np.add.at(tab, ids[ids >= 0], scale * gE[ids >= 0])

    bar = 2e-2 if dtype == "bf16" else 1e-4
    assert nerr(to_np(out), Y) <= bar
    assert nerr(to_np(x0[:, :L]).reshape(R, d), tok) <= bar
    assert nerr(to_np(dx0), dX) <= bar
    assert nerr(to_np(de), gE) <= bar
    # dw = <y, t> (y: the row of dx0, t: the MLP's token before its weight) and
    # y is nearly normal to t, as the stack reads x0 through RMSNorm: relative
    # to dw itself the inherited errors have no bound.  They have one relative
    # to the factors: |dw' - dw| <= |y' - y| |t| + |y| |t' - t| in each row, so
    # over the rows at most max|t| ||y' - y|| + max|y| ||t' - t||, and both
    # differences are within the bar.  The operator's own error is bounded
    # element by element, against float64 on the dx0 and events it was given.
    rn = lambda a: np.linalg.norm(a, axis=1)
    assert np.linalg.norm(to_np(dw) - gw) <= bar * (tn.max() * np.linalg.norm(dtok) + rn(dtok).max() * np.sqrt((tn ** 2).sum()))
    Wt = {f: [to_dev(np.asarray(W[f][t]), dt) for t in range(T)] for f in ("Wb1", "bb1", "Wb2", "bb2")}
    Wt["type_emb"] = to_dev(np.asarray(W["type_emb"]), dt)
    y_in = dx0[:, :L].reshape(R, d)
    ref, tol = backward_ref(Wt, ev, ty_d, wt_d, y_in.to(dt), y_in, dtype)
    close(dw, ref["dweights"], tol["dweights"], "dweights")
    close(de, ref["devents"], tol["devents"], "devents")
    for f in G:
        assert nerr(np.stack([to_np(x) for x in grads[f]]), np.stack(G[f])) <= bar, f
    assert nerr(to_np(grads["type_emb"]), np.stack(G["bb2"])) <= bar
    U = int(n.item())
    touched = np.unique(ids[ids >= 0])
    assert (uniq[:U].cpu().numpy() == touched).all()
    assert nerr(to_np(rows[:U]), tab[touched]) <= bar


def test_refusals_of_the_binding():
    """Arguments the binding refuses before any call: other devices, types, shapes and strides."""
    b = build(shape(n_layers=1, d=64, H=1, dff=64, L_NS=1, F=16), 5, "bf16", event_dim=64)
    m = b.model
    table, ids = torch.zeros(10, 8, device="cuda"), torch.zeros(4, device="cuda", dtype=torch.int32)
    out = torch.zeros(4, 8, device="cuda", dtype=torch.bfloat16)
    good = dict(table=table, ids=ids, out=out)
    for kw in (dict(table=table.cpu()), dict(ids=ids.cpu()), dict(out=out.cpu()), dict(ids=ids.short()), dict(table=table.half()),
               dict(out=out.float()), dict(out=out[:3]), dict(out=out.t()), dict(table=table[:, :4]), dict(table=table.t()),
               dict(ids=ids[None]), dict(out=torch.zeros(4, device="cuda", dtype=torch.bfloat16)[:, None].expand(4, 8))):
        a = dict(good, **kw)
        with pytest.raises(ValueError):
            ot.onetrans_embedding_lookup(m, a["table"], a["ids"], a["out"])
    ws = m.input_workspace(ot.OP_EMBEDDING_BACKWARD, 4, 8)
    for d in (torch.zeros(10, 9, device="cuda"), torch.zeros(10, 8, device="cuda", dtype=torch.bfloat16), torch.zeros(10, 8)):
        with pytest.raises(ValueError):
            ot.onetrans_embedding_backward(m, out, ids, d, ws)
    rows, n = torch.zeros(4, 8, device="cuda"), torch.zeros(1, device="cuda", dtype=torch.int32)
    for u, r in ((ids.long(), rows), (ids[:3].contiguous(), rows), (ids, rows[:3])):
        with pytest.raises(ValueError):
            ot.onetrans_embedding_backward_sparse(m, out, ids, 10, u, r, n, ws)
    ev, types = torch.zeros(4, 64, device="cuda", dtype=torch.bfloat16), ids
    plan, wsr = m.input_workspace(ot.OP_ROUTE, 4, 1), m.input_workspace(ot.OP_ROUTED, 4, 1)
    tok = torch.zeros(4, 64, device="cuda", dtype=torch.bfloat16)
    for kw in (dict(types=types.long()), dict(ev=ev[:3]), dict(ev=ev.float()), dict(tok=tok[:3]), dict(tok=tok.float()),
               dict(tok=tok.view(2, 2, 64)[:, :1]), dict(wt=torch.zeros(3, device="cuda")), dict(wt=torch.zeros(4)),
               dict(plan=plan.cpu())):
        a = dict(dict(ev=ev, types=types, wt=None, plan=plan, tok=tok), **kw)
        with pytest.raises(ValueError):
            ot.onetrans_tokenize_routed(m, a["ev"], a["types"], a["wt"], a["plan"], a["tok"], wsr)
    with pytest.raises(ot.OneTransError):
        ot.onetrans_route_events(m, types, plan[:256])


def test_values_per_choice_and_gradients_of_another_shape_are_refused():
    """A buffer of the right number of elements but another shape (the transpose's) would be read or written in the
    wrong order: refused.  The shape itself and a flat view of it are taken."""
    e, d, R, k = 32, 64, 6, 3
    e, d, R, k = 32, 64, 6, 3
    b = build(shape(n_layers=1, d=d, H=1, dff=64, L_NS=1, F=16), 5, "bf16", event_dim=e)
    m, T = b.model, b.model.cfg.n_behaviors
    ev, types = torch.randn(R, e, device="cuda").bfloat16(), torch.zeros(R, k, device="cuda", dtype=torch.int32)
    plan, ws, wsb = (m.input_workspace(op, R, k) for op in (ot.OP_ROUTE, ot.OP_ROUTED, ot.OP_ROUTED_BACKWARD))
    ot.onetrans_route_events(m, types, plan)
    wt, tok = torch.rand(R, k, device="cuda"), torch.zeros(R, d, device="cuda", dtype=torch.bfloat16)

    def grads(**other):
        g = {"Wb1": (d, e), "bb1": (d,), "Wb2": (d, d), "bb2": (d,)}
        out = {f: [torch.zeros(other.get(f, s), device="cuda") for _ in range(T)] for f, s in g.items()}
        return dict(out, type_emb=torch.zeros(other.get("type_emb", (T, d)), device="cuda"))

    def back(weights=wt, dw=None, **other):
        ot.onetrans_tokenize_routed_backward(m, ev, types, weights, plan, tok, None, dw, grads(**other), wsb)

    for good in (wt, wt.view(-1)):
        ot.onetrans_tokenize_routed(m, ev, types, good, plan, tok, ws)
        back(good, torch.empty_like(good))
    back(Wb1=(d * e,), Wb2=(d * d,), type_emb=(T * d,))
    for bad in (wt.view(k, R), wt.view(1, R, k), wt.view(R * k, 1)):
        with pytest.raises(ValueError):
            ot.onetrans_tokenize_routed(m, ev, types, bad, plan, tok, ws)
        with pytest.raises(ValueError):
            back(bad)
        with pytest.raises(ValueError):
            back(dw=torch.empty_like(bad))
    for other in (dict(Wb1=(e, d)), dict(Wb1=(d, e, 1)), dict(bb1=(1, d)), dict(type_emb=(d, T))):
        with pytest.raises(ValueError):
            back(**other)
    assert ot.onetrans_device_status() == 0
