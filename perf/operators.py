"""What is measured of the input layer's operators: embedding lookup, its gradient by sorted ids, the routed
event tokenizer (events sorted by behaviour, each through its behaviour's MLP, weighted and put back) and its
gradient.  `run` computes them in elementary torch operations, or, with `own`, calls the framework."""
import math

import numpy as np
import torch

own = False

BF16, FP32 = "bf16", "fp32"
TYPES = {BF16: torch.bfloat16, FP32: torch.float32}
SIZE = {BF16: 2, FP32: 4}
GELU_C, GELU_A = math.sqrt(2.0 / math.pi), 0.044715


def listed():
    return [
        # 16 users' 16 appended events: the latency of one call
        dict(name="lookup append", op="lookup", R=256, V=100_000, w=64, table=BF16, out=BF16, wide=False, skew=1),
        # non-sequential features of a batch of candidates: a float32 table of an odd width, 64-bit ids
        dict(name="lookup candidates", op="lookup", R=8_191, V=20_011, w=50, table=FP32, out=BF16, wide=True, skew=0),
        # every event of a large batch of long behaviour sequences
        dict(name="lookup sequences", op="lookup", R=524_288, V=2_000_000, w=64, table=BF16, out=BF16, wide=False, skew=1),
        # one user's sequence, as an online update sees it
        dict(name="table grad user", op="grad", R=1_178, V=100_000, w=64, dout=BF16, wide=False, skew=1, dense=False),
        # a training batch's events (64 samples x 1178), popular items repeated thousands of times
        dict(name="table grad batch", op="grad", R=75_392, V=1_000_000, w=64, dout=BF16, wide=False, skew=1, dense=False),
        # a dense table gradient from float32 rows, as a dense optimizer takes it
        dict(name="table grad dense", op="grad", R=262_147, V=200_003, w=128, dout=FP32, wide=True, skew=0, dense=True),
        # cross-request append: 16 users x 16 events of 3 behaviours
        dict(name="tokens append", op="tokens", R=256, T=3, k=1, e=64, d=256, mode=BF16, weighted=False),
        # a training batch's events
        dict(name="tokens batch", op="tokens", R=75_392, T=3, k=1, e=64, d=256, mode=BF16, weighted=False),
        # events that stand for up to two of eight behaviours, weighted; odd row count, the wider model
        dict(name="tokens mixed", op="tokens", R=20_011, T=8, k=2, e=64, d=384, mode=BF16, weighted=True),
        # the float32 mode on one user's sequence
        dict(name="tokens grad fp32", op="tokens_grad", R=1_178, T=3, k=1, e=64, d=256, mode=FP32, weighted=True),
        # the gradient of a training batch's tokens
        dict(name="tokens grad batch", op="tokens_grad", R=75_392, T=3, k=1, e=64, d=256, mode=BF16, weighted=False),
        # the gradient of weighted mixtures, odd row count, the wider model
        dict(name="tokens grad mixed", op="tokens_grad", R=9_973, T=8, k=2, e=64, d=384, mode=BF16, weighted=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["lookup", "grad", "tokens", "tokens_grad"])
    if op in ("lookup", "grad"):
        w = rng.choice([16, 24, 32, 50, 64, 100, 128, 200, 256])
        R = _log_int(rng, 1, 524_288 * 64 // max(64, w))
        V = _log_int(rng, 100, 2_000_000)
        wide, skew = rng.random() < 0.5, rng.choice([0, 1])
        if op == "lookup":
            return dict(op=op, R=R, V=V, w=w, table=rng.choice([BF16, FP32]), out=rng.choice([BF16, FP32]), wide=wide, skew=skew)
        dense = rng.random() < 0.5
        if dense:
            V = min(V, 200_003 * 128 // w)
        return dict(op=op, R=min(R, 524_288 * 64 // (2 * w)), V=V, w=w, dout=rng.choice([BF16, FP32]), wide=wide, skew=skew, dense=dense)
    mode = FP32 if rng.random() < 0.2 else BF16
    T, k = rng.randint(1, 8), rng.choice([1, 1, 2, 3])
    e, d = rng.choice([16, 32, 64, 96, 128]), rng.choice([128, 256, 384])
    most = 75_392 * 3 * 256 // (max(T, 3) * d)
    return dict(op=op, R=_log_int(rng, 1, min(most, 4_096) if mode == FP32 else most), T=T, k=k, e=e, d=d, mode=mode,
                weighted=k > 1 or rng.random() < 0.5)


# ------------------------------------------------------------------ inputs

def _ids(case, g):
    """Item ids: uniform, or by popularity (the i-th item about as often as 1 / i); one in fifty is padding (-1)."""
    R, V = case["R"], case["V"]
    u = torch.rand(R, generator=g, device="cuda", dtype=torch.float64)
    ids = ((V + 1.0) ** u - 1.0 if case["skew"] else u * V).long().clamp_(0, V - 1)
    ids = ids * 2_654_435_761 % V
    ids = torch.where(torch.rand(R, generator=g, device="cuda") < 0.02, torch.full_like(ids, -1), ids)
    return ids if case["wide"] else ids.int()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape, t=torch.float32, std=1.0):
        return torch.empty(shape, device="cuda", dtype=torch.float32).normal_(0.0, std, generator=g).to(t)

    s = {"op": case["op"]}
    if case["op"] in ("lookup", "grad"):
        R, V, w = case["R"], case["V"], case["w"]
        s |= {"ids": _ids(case, g), "V": V, "scale": math.sqrt(w)}
        if case["op"] == "lookup":
            s |= {"table": normal(V, w, t=TYPES[case["table"]], std=0.02)}
            s |= {"out": torch.zeros(R, w, device="cuda", dtype=TYPES[case["out"]])}
        else:
            s |= {"dout": normal(R, w, t=TYPES[case["dout"]], std=0.01), "dense": case["dense"]}
            if case["dense"]:
                s |= {"dtable": torch.zeros(V, w, device="cuda")}
            else:
                s |= {"uniq": torch.zeros(R, device="cuda", dtype=s["ids"].dtype), "rows": torch.zeros(R, w, device="cuda"),
                      "n": torch.zeros(1, device="cuda", dtype=torch.int32)}
    else:
        R, T, k, e, d, t = case["R"], case["T"], case["k"], case["e"], case["d"], TYPES[case["mode"]]
        s |= {"W1": normal(T, d, e, t=t, std=e ** -0.5), "b1": normal(T, d, t=t, std=0.02),
              "W2": normal(T, d, d, t=t, std=d ** -0.5), "b2": normal(T, d, t=t, std=0.02), "emb": normal(T, d, t=t, std=0.1)}
        s |= {"events": normal(R, e, t=t)}
        # behaviours are unequally frequent; a mixed event's further choices are often empty (-1)
        p = 1.0 / torch.arange(1, T + 1, device="cuda", dtype=torch.float32)
        types = torch.multinomial(p, R * k, replacement=True, generator=g).view(R, k).int()
        if k > 1:
            none = torch.rand(R, k, generator=g, device="cuda") < 0.3
            none[:, 0] &= torch.rand(R, generator=g, device="cuda") < 0.1
            types = torch.where(none, torch.full_like(types, -1), types)
        s |= {"types": types}
        s |= {"weights": torch.rand(R, k, generator=g, device="cuda") + 0.25 if case["weighted"] else None}
        if case["op"] == "tokens":
            s |= {"tokens": torch.zeros(R, d, device="cuda", dtype=t)}
        else:
            s |= {"dtokens": normal(R, d, t=t, std=0.01), "devents": torch.zeros(R, e, device="cuda", dtype=t),
                  "dweights": torch.zeros(R, k, device="cuda") if case["weighted"] else None,
                  "grads": {f: torch.zeros(s[f].shape, device="cuda") for f in ("W1", "b1", "W2", "b2", "emb")}}
    if own:
        _handle(case, s)
    return s


def _handle(case, s):
    """The model handle and the workspaces that a user's program keeps."""
    import unified_transformer_recommender_b200 as ot
    mode, d = case.get("mode", case.get("out", BF16)), case.get("d", 256)
    t = TYPES[mode]
    shapes = {"g_attn": (d,), "g_ffn": (d,), "Wqkv_S": (3 * d, d), "Wqkv_NS": (1, 3 * d, d), "Wo": (d, d), "W1_S": (d, d), "b1_S": (d,),
              "W2_S": (d, d), "b2_S": (d,), "W1_NS": (1, d, d), "b1_NS": (1, d), "W2_NS": (1, d, d), "b2_NS": (1, d)}
    stack = {f: [torch.zeros(n, device="cuda", dtype=t)] for f, n in shapes.items()}
    if "W1" in s:
        stack |= {"Wb1": list(s["W1"]), "bb1": list(s["b1"]), "Wb2": list(s["W2"]), "bb2": list(s["b2"]), "type_emb": s["emb"]}
    m = ot.Model(n_layers=1, d_model=d, n_heads=d // 64, d_ff=d, L_NS=1, weights=stack, mode=ot.BF16 if mode == BF16 else ot.FP32,
                 n_behaviors=case.get("T", 0), event_dim=case.get("e", 0))
    s["model"] = m
    if case["op"] == "grad":
        s["ws"] = m.input_workspace(ot.OP_EMBEDDING_BACKWARD, case["R"], case["w"])
    elif case["op"] != "lookup":
        s["plan"] = m.input_workspace(ot.OP_ROUTE, case["R"], case["k"])
        s["ws"] = m.input_workspace(ot.OP_ROUTED if case["op"] == "tokens" else ot.OP_ROUTED_BACKWARD, case["R"], case["k"])
    if case["op"] == "tokens_grad":
        s["lists"] = {"Wb1": list(s["grads"]["W1"]), "bb1": list(s["grads"]["b1"]), "Wb2": list(s["grads"]["W2"]),
                      "bb2": list(s["grads"]["b2"]), "type_emb": s["grads"]["emb"]}


# --------------------------------------------------------------------- run

def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import unified_transformer_recommender_b200 as ot
    m = s["model"]
    if s["op"] == "lookup":
        ot.onetrans_embedding_lookup(m, s["table"], s["ids"], s["out"], scale=s["scale"])
        return s["out"]
    if s["op"] == "grad" and s["dense"]:
        ot.onetrans_embedding_backward(m, s["dout"], s["ids"], s["dtable"], s["ws"], scale=s["scale"])
        return s["dtable"]
    if s["op"] == "grad":
        ot.onetrans_embedding_backward_sparse(m, s["dout"], s["ids"], s["V"], s["uniq"], s["rows"], s["n"], s["ws"], scale=s["scale"])
        return s["uniq"], s["rows"], s["n"]
    ot.onetrans_route_events(m, s["types"], s["plan"])
    if s["op"] == "tokens":
        ot.onetrans_tokenize_routed(m, s["events"], s["types"], s["weights"], s["plan"], s["tokens"], s["ws"])
        return s["tokens"]
    ot.onetrans_tokenize_routed_backward(m, s["events"], s["types"], s["weights"], s["plan"], s["dtokens"], s["devents"],
                                         s["dweights"], s["lists"], s["ws"])
    return {"devents": s["devents"], "dweights": s["dweights"], **s["grads"]}


def _plain(s):
    return {"lookup": _plain_lookup, "grad": _plain_grad, "tokens": _plain_tokens, "tokens_grad": _plain_tokens_grad}[s["op"]](s)


def _plain_lookup(s):
    ids, V = s["ids"], s["V"]
    valid = (ids >= 0) & (ids < V)
    rows = s["table"][ids.clamp(0, V - 1)].float() * s["scale"]
    return torch.where(valid[:, None], rows, 0.0).to(s["out"].dtype)


def _plain_grad(s):
    ids, V = s["ids"], s["V"]
    R, w = s["dout"].shape
    valid = (ids >= 0) & (ids < V)
    rows = torch.where(valid[:, None], s["dout"].float() * s["scale"], 0.0)
    if s["dense"]:
        return torch.zeros(V, w, device="cuda").index_add_(0, ids.clamp(0, V - 1), rows)
    key, order = torch.sort(torch.where(valid, ids, V), stable=True)
    head = key < V
    head[1:] &= key[1:] != key[:-1]
    at = torch.cumsum(head, 0) - 1
    at = torch.where(key < V, at, R)
    out = torch.zeros(R + 1, w, device="cuda").index_add_(0, at, rows[order])
    uniq = torch.zeros(R + 1, device="cuda", dtype=ids.dtype).scatter_(0, at, torch.where(key < V, key, 0))
    return uniq[:R], out[:R], head.sum(dtype=torch.int32)[None]


def _mixture(s):
    """C [T, R]: the weight with which event r takes part in behaviour t."""
    types, T = s["types"], s["W1"].shape[0]
    valid = (types >= 0) & (types < T)
    at = torch.where(valid, types, T).long()
    w = s["weights"] if s["weights"] is not None else torch.ones(types.shape, device="cuda")
    C = torch.zeros(types.shape[0], T + 1, device="cuda").scatter_add_(1, at, w)[:, :T].t().contiguous()
    return C, at, valid


def _hidden(s):
    """Pre-activation u, GELU(u) and GELU'(u) [T, R, d] of every event in every behaviour's MLP."""
    u = s["events"].float()[None] @ s["W1"].float().transpose(1, 2) + s["b1"].float()[:, None]
    th = torch.tanh(GELU_C * (u + GELU_A * u * u * u))
    return u, 0.5 * u * (1.0 + th), th


def _plain_tokens(s):
    C, _, _ = _mixture(s)
    _, z, _ = _hidden(s)
    y = z @ s["W2"].float().transpose(1, 2) + (s["b2"].float() + s["emb"].float())[:, None]
    return (C[:, :, None] * y).sum(0).to(s["tokens"].dtype)


def _plain_tokens_grad(s):
    C, at, valid = _mixture(s)
    u, z, th = _hidden(s)
    dy, W1, W2 = s["dtokens"].float(), s["W1"].float(), s["W2"].float()
    dz = dy[None] @ W2
    slope = 0.5 * (1.0 + th) + 0.5 * u * (1.0 - th * th) * GELU_C * (1.0 + 3.0 * GELU_A * u * u)
    du = C[:, :, None] * dz * slope
    cdy = C[:, :, None] * dy[None]
    out = {"devents": (du @ W1).sum(0).to(s["devents"].dtype), "dweights": None}
    if s["weights"] is not None:
        dot = (dz * z).sum(2) + (s["b2"].float() + s["emb"].float()) @ dy.t()
        each = torch.cat([dot.t(), torch.zeros(dy.shape[0], 1, device="cuda")], 1).gather(1, at)
        out["dweights"] = torch.where(valid, each, 0.0)
    db2 = cdy.sum(1)
    return {**out, "W1": du.transpose(1, 2) @ s["events"].float()[None], "b1": du.sum(1), "W2": cdy.transpose(1, 2) @ z, "b2": db2, "emb": db2}


# ------------------------------------------------------------ work, exact

def _touched(case):
    """Expected number of distinct rows that the ids name."""
    R, V = 0.98 * case["R"], case["V"]
    if not case["skew"]:
        return V * -math.expm1(R * math.log1p(-1.0 / V))
    r = np.arange(V, dtype=np.float64)
    p = (np.log(r + 2.0) - np.log(r + 1.0)) / math.log(V + 1.0)
    return float(-np.expm1(R * np.log1p(-np.minimum(p, 1 - 1e-12))).sum())


def work(case):
    R = case["R"]
    if case["op"] in ("lookup", "grad"):
        w, idb, n = case["w"], 8 if case["wide"] else 4, _touched(case)
        if case["op"] == "lookup":
            return {"bytes": R * idb + n * w * SIZE[case["table"]] + R * w * SIZE[case["out"]], "flops": R * w}
        out = case["V"] * w * 4 if case["dense"] else n * (w * 4 + idb) + 4
        return {"bytes": R * (idb + w * SIZE[case["dout"]]) + out, "flops": R * w}
    T, k, e, d, es = case["T"], case["k"], case["e"], case["d"], SIZE[case["mode"]]
    mlp = T * (d * e + d * d + 3 * d)
    ins = R * e * es + R * k * (4 + (4 if case["weighted"] else 0)) + mlp * es
    rows = R * k * (0.7 if k > 1 else 1.0)  # choices that are not empty, about
    if case["op"] == "tokens":
        return {"bytes": ins + R * d * es, "flops": 2 * rows * (e * d + d * d)}
    return {"bytes": ins + R * d * es + R * e * es + (R * k * 4 if case["weighted"] else 0) + mlp * 4, "flops": 2 * rows * (3 * e * d + 2 * d * d)}


def exact(case, seed):
    """The same outputs from the definitions in 64 bits: sums over the occurrences of an id, and behaviour by behaviour over its own events."""
    s = prepare(case, seed)
    if case["op"] == "lookup":
        out = torch.zeros(case["R"], case["w"], device="cuda", dtype=torch.float64)
        at = torch.nonzero((s["ids"] >= 0) & (s["ids"] < case["V"]))[:, 0]
        out[at] = s["table"][s["ids"][at].long()].double() * s["scale"]
        return out
    if case["op"] == "grad":
        at = torch.nonzero((s["ids"] >= 0) & (s["ids"] < case["V"]))[:, 0]
        uniq, which = torch.unique(s["ids"][at].long(), sorted=True, return_inverse=True)
        rows = torch.zeros(uniq.numel(), case["w"], device="cuda", dtype=torch.float64)
        rows.index_add_(0, which, s["dout"][at].double() * s["scale"])
        if case["dense"]:
            full = torch.zeros(case["V"], case["w"], device="cuda", dtype=torch.float64)
            full[uniq] = rows
            return full
        full = torch.zeros(case["R"], case["w"], device="cuda", dtype=torch.float64)
        full[: uniq.numel()] = rows
        ids = torch.zeros(case["R"], device="cuda", dtype=s["ids"].dtype)
        ids[: uniq.numel()] = uniq.to(ids.dtype)
        return ids, full, torch.tensor([uniq.numel()], device="cuda", dtype=torch.int32)
    R, T, k, e, d = (case[f] for f in ("R", "T", "k", "e", "d"))
    wt = s["weights"].double() if s["weights"] is not None else torch.ones(R, k, device="cuda", dtype=torch.float64)
    W1, b1, W2 = s["W1"].double(), s["b1"].double(), s["W2"].double()
    shift = s["b2"].double() + s["emb"].double()
    zeros = lambda *n: torch.zeros(*n, device="cuda", dtype=torch.float64)  # noqa: E731
    tok, de, dw = zeros(R, d), zeros(R, e), zeros(R, k)
    g = {"W1": zeros(T, d, e), "b1": zeros(T, d), "W2": zeros(T, d, d), "b2": zeros(T, d), "emb": zeros(T, d)}
    for t in range(T):
        for j in range(k):
            r = torch.nonzero(s["types"][:, j] == t)[:, 0]
            x, c = s["events"][r].double(), wt[r, j][:, None]
            u = x @ W1[t].t() + b1[t]
            v = GELU_C * (u + GELU_A * u ** 3)
            z = 0.5 * u * (1 + torch.tanh(v))
            y = z @ W2[t].t() + shift[t]
            if case["op"] == "tokens":
                tok.index_add_(0, r, c * y)
                continue
            dy = s["dtokens"][r].double()
            dz = (c * dy) @ W2[t]
            du = dz * (0.5 * (1 + torch.tanh(v)) + 0.5 * u * GELU_C * (1 + 3 * GELU_A * u * u) / torch.cosh(v) ** 2)
            de.index_add_(0, r, du @ W1[t])
            dw[r, j] = (dy * y).sum(1)
            g["W1"][t] += du.t() @ x
            g["b1"][t] += du.sum(0)
            g["W2"][t] += (c * dy).t() @ z
            g["b2"][t] += (c * dy).sum(0)
    if case["op"] == "tokens":
        return tok
    g["emb"] = g["b2"]
    return {"devents": de, "dweights": dw if case["weighted"] else None, **g}
