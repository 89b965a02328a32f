"""Embedding lookup with scaling and its gradient by sorted ids, through the C
ABI against plain float64 implementations.

Tolerances.  A lookup is one float32 product rounded once: float32 output
within half a step (2^-24 of the value, the product itself; a bf16 or float32
table entry is exact in float32), bf16 output 2^-8 of the value plus the
product's own 2^-24.  A gradient entry is a float32 sum of n terms: every
addition is off by at most 2^-24 of its partial sum, which sum |terms| bounds,
and a term passes through fewer than n additions, so the error is at most
n * 2^-24 * sum |terms|, plus one rounding for the scale."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from helpers import build, shape

import unified_transformer_recommender_b200 as ot  # noqa: E402

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}
_models = {}


def model(mode):
    if mode not in _models:
        _models[mode] = build(shape(n_layers=1, d=64, H=1, dff=64, L_NS=1, F=16), 5, mode).model
    return _models[mode]


def make_ids(kind, R, V, seed, dtype=torch.int32):
    g = np.random.default_rng(seed)
    if kind == "uniform":
        ids = g.integers(0, V, R)
    elif kind == "popular":
        ids = ((V + 1.0) ** g.random(R) - 1).astype(np.int64).clip(0, V - 1)
    elif kind == "one":
        ids = np.full(R, V - 1)
    elif kind == "padding":
        ids = np.full(R, -1)
    else:                                    # every id once, descending
        ids = np.arange(R)[::-1] % V
    if kind in ("uniform", "popular"):
        ids[g.random(R) < 0.1] = -1
    return torch.from_numpy(ids.copy()).to("cuda", dtype)


@pytest.mark.parametrize("mode,table_t,ids_t,R,V,w,pad", [
    ("bf16", "bf16", torch.int32, 1, 1, 1, 0),
    ("bf16", "bf16", torch.int32, 1000, 501, 64, 0),
    ("bf16", "fp32", torch.int64, 777, 333, 50, 14),     # a field inside a wider feature row
    ("fp32", "bf16", torch.int64, 129, 70, 7, 2),
    ("fp32", "fp32", torch.int32, 2049, 100, 300, 0),
    ("bf16", "bf16", torch.int32, 70001, 5003, 16, 0),
    ("fp32", "fp32", torch.int64, 37, 20, 5000, 0),      # rows wider than a CTA
    ("bf16", "fp32", torch.int32, 100_001, 77, 12, 4),   # many rows, each CTA walking
    ("bf16", "bf16", torch.int64, 300_001, 5003, 64, 0),
])
def test_lookup(mode, table_t, ids_t, R, V, w, pad):
    g = torch.Generator(device="cuda").manual_seed(R)
    table = torch.randn(V, w, device="cuda", generator=g).to(DT[table_t])
    ids = make_ids("uniform", R, V, R + 1, ids_t)
    buf = torch.full((R, w + pad), 7.0, device="cuda", dtype=DT[mode])
    off = 8 if pad >= 8 else 0                # a column offset that keeps 16-byte alignment
    out = buf[:, off:off + w]
    ot.onetrans_embedding_lookup(model(mode), table, ids, out, scale=1.7)
    torch.cuda.synchronize()
    assert ot.onetrans_device_status() == 0
    scale = float(np.float32(1.7))
    ref = torch.where((ids >= 0)[:, None], table[ids.clamp(min=0).long()].double() * scale, 0.0)
    err = (out.double() - ref).abs()
    assert (err <= ref.abs() * (HALF[mode] * (1 + 2.0 ** -8) + 2.0 ** -24)).all()
    rest = torch.ones(w + pad, dtype=torch.bool)
    rest[off:off + w] = False
    assert (buf[:, rest.cuda()] == 7.0).all()     # what lies between two rows is left as it was


def test_lookup_flags_ids_out_of_range():
    table = torch.ones(10, 8, device="cuda", dtype=torch.bfloat16)
    for bad in (10, -2, 2 ** 31 - 1):
        ids = torch.tensor([3, bad, -1], device="cuda", dtype=torch.int32)
        out = torch.full((3, 8), 5.0, device="cuda", dtype=torch.bfloat16)
        ot.onetrans_embedding_lookup(model("bf16"), table, ids, out)
        assert ot.onetrans_device_status() == 3
        assert (out[0] == 1).all() and (out[1:] == 0).all()
    ids = torch.tensor([2 ** 40 + 1, 9], device="cuda")
    out = torch.full((2, 8), 5.0, device="cuda", dtype=torch.bfloat16)
    ot.onetrans_embedding_lookup(model("bf16"), table, ids, out)
    assert ot.onetrans_device_status() == 3
    assert (out[0] == 0).all() and (out[1] == 1).all()


def test_lookup_offsets_past_32_bits():
    V, w = 40_000_000, 64                          # 2.56e9 elements
    table = torch.empty(V, w, device="cuda", dtype=torch.bfloat16)
    rows = torch.tensor([0, V // 2, V - 1, 33_554_433], device="cuda")
    for i, r in enumerate(rows.tolist()):
        table[r] = i + 1
    out = torch.zeros(4, w, device="cuda", dtype=torch.bfloat16)
    ot.onetrans_embedding_lookup(model("bf16"), table, rows, out)
    assert torch.equal(out, torch.arange(1, 5, device="cuda", dtype=torch.bfloat16)[:, None].expand(4, w))


def reference(dout, ids, V, scale):
    """float64 sums [V, w], sums of absolute values, occurrences [V]."""
    ok = torch.nonzero((ids >= 0) & (ids < V))[:, 0]
    at = ids[ok].long()
    x = dout[ok].double()
    s = torch.zeros(V, dout.shape[1], device="cuda", dtype=torch.float64)
    m = torch.zeros_like(s)
    s.index_add_(0, at, x)
    m.index_add_(0, at, x.abs())
    n = torch.bincount(at, minlength=V)
    return s * scale, m * abs(scale), n


def check_rows(got, s, m, n):
    err = (got.double() - s).abs()
    bound = m * ((n[:, None] + 1) * 2.0 ** -24)
    assert (err <= bound).all(), float((err - bound).max())


GRADS = [
    # kind, dout type, ids type, R, V, w
    ("uniform", "bf16", torch.int32, 1, 1, 1),
    ("uniform", "fp32", torch.int64, 31, 5, 3),
    ("popular", "bf16", torch.int32, 256, 1000, 64),
    ("popular", "bf16", torch.int32, 257, 3, 64),          # runs across the warps' and chunks' borders
    ("one", "fp32", torch.int32, 4096, 2, 40),             # one run through every chunk
    ("padding", "bf16", torch.int32, 700, 50, 16),         # nothing to add
    ("each", "bf16", torch.int64, 5000, 5000, 24),         # every id once
    ("uniform", "bf16", torch.int32, 4097, 7, 300),        # two tiles, several column blocks
    ("popular", "fp32", torch.int64, 20011, 2_000_000, 50),
    ("one", "bf16", torch.int64, 30000, 100_000, 128),
    ("popular", "bf16", torch.int32, 75_392, 1_000_000, 64),
    ("uniform", "fp32", torch.int32, 270_001, 60_000, 20),  # more tiles than a pass adds up itself
    ("popular", "bf16", torch.int32, 300_000, 2_147_483_647, 8),   # three passes
    ("popular", "bf16", torch.int32, 1_100_000, 5_000, 16),        # chunks of more rows
    ("uniform", "bf16", torch.int64, 100_003, 50_000, 12),         # four items a thread, counts added up by the passes
    ("popular", "fp32", torch.int32, 400_000, 3_000, 8),           # the same with scanned counts
    ("uniform", "bf16", torch.int32, 1 << 26, 1_000, 1),           # the most ids a call takes
]


@pytest.mark.parametrize("kind,dout_t,ids_t,R,V,w", GRADS)
def test_gradient_sparse(kind, dout_t, ids_t, R, V, w):
    g = torch.Generator(device="cuda").manual_seed(R)
    dout = torch.randn(R, w, device="cuda", generator=g).to(DT[dout_t])
    ids = make_ids(kind, R, V, R + 2, ids_t)
    m = model("bf16")
    room = min(R, V)
    uniq = torch.full((room,), -7, device="cuda", dtype=ids_t)
    rows = torch.full((room, w), 7.0, device="cuda")
    n = torch.full((1,), -1, device="cuda", dtype=torch.int32)
    ws = m.input_workspace(ot.OP_EMBEDDING_BACKWARD, R, w)
    ot.onetrans_embedding_backward_sparse(m, dout, ids, V, uniq, rows, n, ws, scale=0.3)
    torch.cuda.synchronize()
    assert ot.onetrans_device_status() == 0
    ref = torch.unique(ids[ids >= 0])
    U = int(n.item())
    assert U == ref.numel()
    assert torch.equal(uniq[:U], ref)
    assert (uniq[U:] == -7).all() and (rows[U:] == 7.0).all()     # rows behind the last stay as they were
    scale = float(np.float32(0.3))
    pos = torch.where(ids >= 0, torch.searchsorted(ref, ids), torch.full_like(ids, -1))
    if U:
        check_rows(rows[:U], *reference(dout, pos, U, scale))
    again = torch.zeros_like(rows)
    ot.onetrans_embedding_backward_sparse(m, dout, ids, V, uniq, again, n, ws, scale=0.3)
    assert torch.equal(again[:U], rows[:U])                       # a fixed order of additions


@pytest.mark.parametrize("R,V,w", [(200, 37, 9), (9000, 4000, 48), (30_000, 50, 20), (70_000, 300, 200)])
def test_gradient_writes_nothing_past_its_outputs(R, V, w):
    """Widths that leave lanes without a column, scale 1: elements behind the last row stay as they were."""
    m = model("fp32")
    dout = torch.randn(R, w, device="cuda")
    ids = make_ids("popular", R, V, R + 5)
    ws = m.input_workspace(ot.OP_EMBEDDING_BACKWARD, R, w)
    buf = torch.full((V * w + 4096,), 7.0, device="cuda")
    ot.onetrans_embedding_backward(m, dout, ids, buf[:V * w].view(V, w), ws)
    assert (buf[V * w:] == 7.0).all()
    check_rows(buf[:V * w].view(V, w), *reference(dout, ids, V, 1.0))
    rows = torch.full((V * w + 4096,), 7.0, device="cuda")
    uniq, n = torch.zeros(V, device="cuda", dtype=torch.int32), torch.zeros(1, device="cuda", dtype=torch.int32)
    ot.onetrans_embedding_backward_sparse(m, dout, ids, V, uniq, rows[:V * w].view(V, w), n, ws)
    assert (rows[int(n.item()) * w:] == 7.0).all()


@pytest.mark.parametrize("kind,dout_t,ids_t,R,V,w", [c for c in GRADS if c[4] <= 2_000_000])
def test_gradient_dense(kind, dout_t, ids_t, R, V, w):
    g = torch.Generator(device="cuda").manual_seed(R)
    wide = torch.randn(R, w + 8, device="cuda", generator=g).to(DT[dout_t])
    dout = wide[:, :w]                                            # rows of a wider gradient
    ids = make_ids(kind, R, V, R + 3, ids_t)
    m = model("fp32")
    dtable = torch.full((V, w), float("nan"), device="cuda")
    ws = m.input_workspace(ot.OP_EMBEDDING_BACKWARD, R, w)
    ot.onetrans_embedding_backward(m, dout, ids, dtable, ws, scale=-2.5)
    torch.cuda.synchronize()
    assert ot.onetrans_device_status() == 0
    s, mag, n = reference(dout, ids, V, -2.5)
    check_rows(dtable, s, mag, n)
    assert (dtable[n == 0] == 0).all()


def test_gradient_flags_and_skips_ids_out_of_range():
    ids = torch.tensor([4, 1, 9, -3, 1, -1], device="cuda", dtype=torch.int32)
    dout = torch.arange(1, 7, device="cuda", dtype=torch.float32)[:, None].expand(6, 4).contiguous()
    dtable = torch.full((5, 4), float("nan"), device="cuda")
    m = model("fp32")
    ws = m.input_workspace(ot.OP_EMBEDDING_BACKWARD, 6, 4)
    ot.onetrans_embedding_backward(m, dout, ids, dtable, ws)
    assert ot.onetrans_device_status() == 3
    ref = torch.tensor([0.0, 7.0, 0.0, 0.0, 1.0], device="cuda")[:, None].expand(5, 4)
    assert torch.equal(dtable, ref)


def test_gradient_keeps_infinities_and_nan_in_their_rows():
    R, V, w = 3000, 50, 64
    ids = make_ids("uniform", R, V, 9)
    dout = torch.randn(R, w, device="cuda")
    hit = int(torch.nonzero(ids == 3)[0])
    nan = int(torch.nonzero(ids == 7)[0])
    dout[hit, 5], dout[nan, 6] = float("inf"), float("nan")
    dout[ids == -1] = float("nan")                                # padding rows are not read into any sum
    m = model("bf16")
    dtable = torch.zeros(V, w, device="cuda")
    ot.onetrans_embedding_backward(m, dout, ids, dtable, m.input_workspace(ot.OP_EMBEDDING_BACKWARD, R, w))
    bad = ~torch.isfinite(dtable)
    assert bad[3, 5] and bad[7, 6] and int(bad.sum()) == 2


def test_no_ids():
    m = model("bf16")
    none = torch.empty(0, device="cuda", dtype=torch.int32)
    ws = m.input_workspace(ot.OP_EMBEDDING_BACKWARD, 0, 8)
    n = torch.full((1,), 5, device="cuda", dtype=torch.int32)
    e = torch.empty(0, 8, device="cuda")
    ot.onetrans_embedding_backward_sparse(m, e, none, 10, none, e, n, ws)
    assert int(n.item()) == 0
    dtable = torch.full((10, 8), 3.0, device="cuda")
    ot.onetrans_embedding_backward(m, e, none, dtable, ws)
    assert (dtable == 0).all()
    ot.onetrans_embedding_lookup(m, torch.zeros(3, 8, device="cuda"), none, torch.empty(0, 8, device="cuda", dtype=torch.bfloat16))


def test_captured_and_on_another_stream():
    """A lookup and both gradients captured on a side stream, replayed on new inputs in the same buffers."""
    m = model("fp32")
    R, V, w = 9000, 4000, 48
    table = torch.randn(V, w, device="cuda")
    ids = make_ids("popular", R, V, 21)
    out, dtable = torch.empty(R, w, device="cuda"), torch.empty(V, w, device="cuda")
    uniq, rows = torch.empty(V, device="cuda", dtype=torch.int32), torch.empty(V, w, device="cuda")
    n = torch.empty(1, device="cuda", dtype=torch.int32)
    ws = [m.input_workspace(ot.OP_EMBEDDING_BACKWARD, R, w) for _ in range(2)]

    def step():
        ot.onetrans_embedding_lookup(m, table, ids, out, scale=2.0)
        ot.onetrans_embedding_backward(m, out, ids, dtable, ws[0])
        ot.onetrans_embedding_backward_sparse(m, out, ids, V, uniq, rows, n, ws[1])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (22, 23):
        ids.copy_(make_ids("popular", R, V, seed))
        graph.replay()
        torch.cuda.synchronize()
        s, mag, cnt = reference(out, ids, V, 1.0)
        check_rows(dtable, s, mag, cnt)
        U = int(n.item())
        assert torch.equal(uniq[:U].long(), torch.nonzero(cnt)[:, 0])
        assert torch.equal(rows[:U], dtable[cnt > 0])
    assert ot.onetrans_device_status() == 0


def test_finite_differences():
    """The gradient of f(table) = sum(c * lookup(table)) against central differences of the lookup itself."""
    m = model("fp32")
    R, V, w = 200, 37, 9
    g = torch.Generator(device="cuda").manual_seed(3)
    table = torch.randn(V, w, device="cuda", generator=g)
    c = torch.randn(R, w, device="cuda", generator=g)
    ids = make_ids("uniform", R, V, 31)
    dtable = torch.empty(V, w, device="cuda")
    ot.onetrans_embedding_backward(m, c, ids, dtable, m.input_workspace(ot.OP_EMBEDDING_BACKWARD, R, w), scale=1.5)

    def f(t):
        out = torch.empty(R, w, device="cuda")
        ot.onetrans_embedding_lookup(m, t, ids, out, scale=1.5)
        return float((out.double() * c.double()).sum())

    for seed in range(4):
        v = torch.randn(V, w, device="cuda", generator=g)
        # the lookup is linear: a unit step has no truncation error, only the lookups' own
        # roundings (2^-24 of about 2 * 1.5 * (|t| + |v|) per entry, and of the sum table + v)
        diff = (f(table + v) - f(table - v)) / 2
        ref = float((dtable.double() * v.double()).sum())
        size = float((c.double().abs() * 1.5 * (table.abs() + v.abs())[ids.clamp(min=0).long()].double()).sum())
        assert abs(diff - ref) <= size * 8 * 2.0 ** -24


@pytest.mark.parametrize("R,V", [(1500, 100), (2500, 256), (9_000, 255), (300_000, 257), (300_000, 1000), (1_100_000, 3)])
def test_zero_rows_among_popular_ids(R, V):
    """Tables much smaller than R in which two rows of three are named by no id: many repeats of the ids on either
    side of a row that has to be zero, in spans of 256 rows with few and with many ids."""
    m, w = model("fp32"), 8
    ids = make_ids("uniform", R, V, R + 41)
    ids = torch.where(ids % 3 == 1, ids, torch.full_like(ids, -1)) if V > 3 else torch.where(ids >= 0, 1, ids).int()
    dout = torch.randn(R, w, device="cuda")
    dtable = torch.full((V, w), float("nan"), device="cuda")
    ot.onetrans_embedding_backward(m, dout, ids, dtable, m.input_workspace(ot.OP_EMBEDDING_BACKWARD, R, w), scale=0.5)
    s, mag, n = reference(dout, ids, V, 0.5)
    assert (n > 0).sum() <= V // 3 + 1
    check_rows(dtable, s, mag, n)
    assert (dtable[n == 0] == 0).all()
    assert ot.onetrans_device_status() == 0


def test_dense_gradient_into_a_small_table_takes_about_the_sparse_ones_time():
    """The dense form does what the sparse one does and writes the rows that no id names.  With 2^22 ids of 256 rows
    there are none, so finding that out must not cost more than the sums did (it once took one CTA's walk over all
    ids: 17 times the sparse form's time)."""
    m, R, V, w = model("bf16"), 1 << 22, 256, 16
    dout, ids = torch.randn(R, w, device="cuda").bfloat16(), make_ids("uniform", R, V, 47)
    ws = m.input_workspace(ot.OP_EMBEDDING_BACKWARD, R, w)
    dtable, rows = torch.empty(V, w, device="cuda"), torch.empty(V, w, device="cuda")
    uniq, n = torch.empty(V, device="cuda", dtype=torch.int32), torch.empty(1, device="cuda", dtype=torch.int32)

    def best(f):
        t = []
        for _ in range(7):
            e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            e0.record()
            f()
            e1.record()
            e1.synchronize()
            t.append(e0.elapsed_time(e1))
        return min(t)

    dense = best(lambda: ot.onetrans_embedding_backward(m, dout, ids, dtable, ws))
    sparse = best(lambda: ot.onetrans_embedding_backward_sparse(m, dout, ids, V, uniq, rows, n, ws))
    assert torch.equal(rows[:int(n.item())], dtable[:int(n.item())])
    assert dense <= 2 * sparse, (dense, sparse)


# fields of one feature row, side by side: widths, the first one's column
FIELDS = [("bf16", (50, 14, 6, 64, 2), 0), ("bf16", (8, 16, 24), 4), ("fp32", (50, 7, 1, 3, 64), 0), ("fp32", (4, 8), 1)]


@pytest.mark.parametrize("mode,widths,first", FIELDS)
@pytest.mark.parametrize("R", [300, 40_000])
def test_fields_of_a_feature_row_are_looked_up_side_by_side(mode, widths, first, R):
    """Each field's rows go to its columns of one wide row, whose starts are 4-byte aligned and no more."""
    m = model(mode)
    total = first + sum(widths) + 4
    row = torch.full((R, total), 7.0, device="cuda", dtype=DT[mode])
    want = row.double()
    col = first
    for i, w in enumerate(widths):
        for table_t in ("bf16", "fp32"):          # the last one stays
            V = 40 + i
            table, ids = torch.randn(V, w, device="cuda").to(DT[table_t]), make_ids("uniform", R, V, 50 + i)
            ot.onetrans_embedding_lookup(m, table, ids, row[:, col:col + w], scale=2.0)
        want[:, col:col + w] = torch.where((ids >= 0)[:, None], table[ids.clamp(min=0).long()].double() * 2.0, 0.0)
        col += w
    err = (row.double() - want).abs()
    assert (err <= want.abs() * HALF[mode]).all()             # the product by 2 is exact
    assert (row[:, :first] == 7.0).all() and (row[:, col:] == 7.0).all()
    assert ot.onetrans_device_status() == 0


def test_a_field_at_an_odd_bf16_column_is_refused():
    row = torch.zeros(10, 20, device="cuda", dtype=torch.bfloat16)
    ids = torch.zeros(10, device="cuda", dtype=torch.int32)
    with pytest.raises(ot.OneTransError) as e:
        ot.onetrans_embedding_lookup(model("bf16"), torch.zeros(5, 8, device="cuda"), ids, row[:, 3:11])
    assert e.value.status == ot.ERR_INVALID_ARG


@pytest.mark.parametrize("dout_t,widths,first", FIELDS)
@pytest.mark.parametrize("R", [300, 40_000])
def test_gradients_of_the_fields_of_a_feature_row(dout_t, widths, first, R):
    """Each field's gradient is read from its columns of the wide row's gradient, whose starts are 4-byte aligned."""
    m = model("bf16")
    row = torch.randn(R, first + sum(widths) + 4, device="cuda").to(DT[dout_t])
    col = first
    for i, w in enumerate(widths):
        V = 40 + i
        dout, ids = row[:, col:col + w], make_ids("popular", R, V, 60 + i)
        ws = m.input_workspace(ot.OP_EMBEDDING_BACKWARD, R, w)
        dtable, rows = torch.full((V, w), float("nan"), device="cuda"), torch.full((V, w), float("nan"), device="cuda")
        uniq, n = torch.empty(V, device="cuda", dtype=torch.int32), torch.empty(1, device="cuda", dtype=torch.int32)
        ot.onetrans_embedding_backward(m, dout, ids, dtable, ws, scale=0.75)
        ot.onetrans_embedding_backward_sparse(m, dout, ids, V, uniq, rows, n, ws, scale=0.75)
        s, mag, cnt = reference(dout, ids, V, 0.75)
        check_rows(dtable, s, mag, cnt)
        assert torch.equal(rows[:int(n.item())], dtable[cnt > 0])
        col += w
    assert ot.onetrans_device_status() == 0


def test_a_gradient_field_at_an_odd_bf16_column_is_refused():
    row = torch.zeros(10, 20, device="cuda", dtype=torch.bfloat16)
    ids, m = torch.zeros(10, device="cuda", dtype=torch.int32), model("bf16")
    with pytest.raises(ot.OneTransError) as e:
        ot.onetrans_embedding_backward(m, row[:, 3:11], ids, torch.zeros(5, 8, device="cuda"),
                                       m.input_workspace(ot.OP_EMBEDDING_BACKWARD, 10, 8))
    assert e.value.status == ot.ERR_INVALID_ARG


@pytest.mark.parametrize("R", [4096, 4097, 37_888, 37_889, 77_824, 77_825, 81_920, 81_921, 155_648, 155_649, 327_680, 327_681])
@pytest.mark.parametrize("V", [90, 1_000_003])
def test_gradient_on_both_sides_of_the_size_rules(R, V):
    """Counted and sorted ids, tiles of two and of four items a thread, each with counts added up by the passes and
    scanned, chunks of 64, 128 and 256 positions."""
    m, w = model("bf16"), 8
    dout, ids = torch.randn(R, w, device="cuda").bfloat16(), make_ids("popular", R, V, R + 71)
    ws = m.input_workspace(ot.OP_EMBEDDING_BACKWARD, R, w)
    room = min(R, V)
    dtable, rows = torch.full((V, w), float("nan"), device="cuda"), torch.full((room, w), 7.0, device="cuda")
    uniq, n = torch.full((room,), -7, device="cuda", dtype=torch.int32), torch.zeros(1, device="cuda", dtype=torch.int32)
    ot.onetrans_embedding_backward(m, dout, ids, dtable, ws)
    ot.onetrans_embedding_backward_sparse(m, dout, ids, V, uniq, rows, n, ws)
    s, mag, cnt = reference(dout, ids, V, 1.0)
    check_rows(dtable, s, mag, cnt)
    U = int(n.item())
    assert torch.equal(uniq[:U].long(), torch.nonzero(cnt)[:, 0]) and (uniq[U:] == -7).all()
    assert torch.equal(rows[:U], dtable[cnt > 0]) and (rows[U:] == 7.0).all()
    assert ot.onetrans_device_status() == 0
