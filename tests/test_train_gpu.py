"""The training operators on the GPU against their formulas in 64 bits.

Tolerances. A bf16 result may differ from the exact value by its own rounding, at most 2^-8 of its
size (half a unit in the last of 8 significant bits; about 2^-9 in the mean), plus the error of the fp32 sum before it: a sum
of m products in fp32, each addition off by at most 2^-23 of the running magnitude (truncation;
rounding is half that), is off by at most m 2^-23 S with S the sum of the products' magnitudes.
The products of two bf16 values are exact in fp32.
"""
import dataclasses

import pytest
import torch

import synth

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module")
def moe():
    import combine_grouped_gemm_gb300 as m
    return m


def normal(seed, *shape, std=1.0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(BF)


def spread(rows, E, kind, seed=0):
    """Rows per group: even, one group with all, every second empty, or random."""
    gen = torch.Generator()
    gen.manual_seed(seed + 17 * rows + E)
    if kind == "one":
        c = [0] * E
        c[E // 2] = rows
    elif kind == "gaps":
        live = max(1, E // 2)
        c = [rows // live if e % 2 == 0 and e // 2 < live else 0 for e in range(E)]
        c[0] += rows - sum(c)
    elif kind == "even":
        c = [rows // E + (e < rows % E) for e in range(E)]
    else:
        p = torch.rand(E, generator=gen) ** 3
        at = torch.multinomial(p + 1e-6, rows, replacement=True, generator=gen) if rows else []
        c = torch.bincount(torch.as_tensor(at, dtype=torch.long), minlength=E).tolist()
    assert sum(c) == rows
    return c


def workspace(moe, g):
    return torch.zeros(moe.grouped_ws_bytes(g), dtype=torch.uint8, device="cuda")


def check(got, ref, slack, what):
    """|got - ref| <= 2^-8 |ref| (a bf16 result) + slack, element by element; NaN never."""
    got = got.double()
    own = ref.abs() * 2.0 ** -8 if what != "fp32" else ref.abs() * 2.0 ** -24
    over = (got - ref).abs() - (own + slack + 1e-37)
    assert bool(torch.isfinite(got).all())
    assert float(over.max() if over.numel() else -1.0) <= 0.0


def grouped_reference(kind, a, b, counts):
    """(result, sum of the magnitudes, additions) in 64 bits."""
    out, mag, first = [], [], 0
    for e, c in enumerate(counts):
        r = slice(first, first + c)
        first += c
        if kind == "mm":
            u, v = a[r].double(), b[e].double().t()
        elif kind == "dx":
            u, v = a[r].double(), b[e].double()
        else:
            u, v = a[r].double().t(), b[r].double()
        out.append(u @ v)
        mag.append(u.abs() @ v.abs())
    join = torch.stack if kind == "dw" else torch.cat
    return join(out), join(mag)


SHAPES = [
    # rows, E, n, k, how the rows lie
    (1, 1, 8, 8, "even"), (1, 3, 64, 128, "one"), (5, 8, 72, 40, "random"),
    (33, 4, 136, 264, "gaps"), (64, 2, 128, 64, "even"), (129, 3, 256, 512, "random"),
    (300, 5, 520, 328, "gaps"), (257, 1, 1032, 136, "one"), (513, 2, 264, 1000, "random"),
    (2000, 7, 384, 256, "random"), (96, 1024, 64, 64, "random"), (8, 256, 512, 1024, "random"),
    (700, 1, 8, 2048, "one"), (777, 2, 2048, 16, "even"), (4100, 3, 256, 192, "gaps"),
    # few units and long reductions: split, with parts of unequal length and groups without any
    (64, 1, 512, 4096, "one"), (2, 2, 1096, 3272, "even"), (40, 5, 264, 2056, "gaps"),
    (9000, 1, 256, 264, "one"), (3001, 4, 128, 512, "random"),
]


@pytest.mark.parametrize("rows,E,n,k,kind", SHAPES)
def test_grouped_mm_and_dx(moe, rows, E, n, k, kind):
    counts = spread(rows, E, kind)
    c = torch.tensor(counts, dtype=torch.int32, device="cuda")
    g = moe.GroupCfg(rows=rows, E=E, n=n, k=k)
    ws = workspace(moe, g)
    x, w = normal(1, rows, k), normal(2, E, n, k, std=0.05)
    y = torch.full((rows, n), float("nan"), dtype=BF, device="cuda")
    moe.grouped_mm(g, x, c, w, y, ws)
    ref, mag = grouped_reference("mm", x, w, counts)
    check(y, ref, k * 2.0 ** -23 * mag, "bf16")
    dy = normal(3, rows, n)
    dx = torch.full((rows, k), float("nan"), dtype=BF, device="cuda")
    moe.grouped_mm_dx(g, dy, c, w, dx, ws)
    ref, mag = grouped_reference("dx", dy, w, counts)
    check(dx, ref, n * 2.0 ** -23 * mag, "bf16")
    # once more in the same workspace: the same bits
    y2, dx2 = torch.empty_like(y), torch.empty_like(dx)
    moe.grouped_mm(g, x, c, w, y2, ws)
    moe.grouped_mm_dx(g, dy, c, w, dx2, ws)
    assert torch.equal(y, y2) and torch.equal(dx, dx2)
    assert moe.read_status(ws) == 0


@pytest.mark.parametrize("rows,E,n,k,kind", SHAPES)
def test_grouped_mm_dw(moe, rows, E, n, k, kind):
    counts = spread(rows, E, kind)
    c = torch.tensor(counts, dtype=torch.int32, device="cuda")
    g = moe.GroupCfg(rows=rows, E=E, n=n, k=k)
    ws = workspace(moe, g)
    x, dy = normal(1, rows, k), normal(3, rows, n)
    ref, mag = grouped_reference("dw", dy, x, counts)
    slack = max(1, max(counts)) * 2.0 ** -23 * mag
    nan = float("nan")
    f32 = torch.full((E, n, k), nan, device="cuda")
    moe.grouped_mm_dw(g, dy, x, c, f32, ws)
    check(f32, ref, slack, "fp32")
    bf = torch.full((E, n, k), nan, dtype=BF, device="cuda")
    moe.grouped_mm_dw(g, dy, x, c, bf, ws)
    check(bf, ref, slack, "bf16")
    empty = torch.tensor([v == 0 for v in counts], device="cuda")
    assert float(f32[empty].abs().sum()) == 0.0 and float(bf[empty].float().abs().sum()) == 0.0
    # added to what is there: one more rounding of an fp32 sum
    base = torch.randn((E, n, k), device="cuda")
    acc = base.clone()
    moe.grouped_mm_dw(g, dy, x, c, acc, ws, accumulate=True)
    check(acc, ref + base.double(), slack + 2.0 ** -23 * (ref.abs() + base.double().abs()), "fp32")
    again = torch.empty_like(f32)
    moe.grouped_mm_dw(g, dy, x, c, again, ws)
    assert torch.equal(f32, again)
    assert moe.read_status(ws) == 0


def test_fp32_weight_gradient_of_a_long_group_keeps_its_precision(moe):
    """20000 rows of one group: the relative error stays at that of fp32 sums of at most 512 rows
    joined in fp32, 512 x 2^-24 in the mean of truncated sums, not growing with the rows."""
    g = moe.GroupCfg(rows=20000, E=2, n=128, k=128)
    c = torch.tensor([19999, 1], dtype=torch.int32, device="cuda")
    x, dy = normal(1, g.rows, g.k), normal(2, g.rows, g.n)
    dw = torch.empty((2, g.n, g.k), device="cuda")
    moe.grouped_mm_dw(g, dy, x, c, dw, workspace(moe, g))
    ref, _ = grouped_reference("dw", dy, x, c.tolist())
    assert float((dw.double() - ref).norm() / ref.norm()) < 512 * 2.0 ** -24


def test_gradients_against_differences(moe):
    """<dy, mm(x + h v) - mm(x - h v)> / 2h = <dx, v>, and the same for the weights: the products
    are linear, so the central difference of the 64-bit formula is the derivative itself."""
    counts = [3, 0, 40, 21]
    g = moe.GroupCfg(rows=64, E=4, n=72, k=136)
    c = torch.tensor(counts, dtype=torch.int32, device="cuda")
    ws = workspace(moe, g)
    x, w, dy = normal(1, 64, 136), normal(2, 4, 72, 136), normal(3, 64, 72)
    dx = torch.empty((64, 136), dtype=BF, device="cuda")
    dw = torch.empty((4, 72, 136), device="cuda")
    moe.grouped_mm_dx(g, dy, c, w, dx, ws)
    moe.grouped_mm_dw(g, dy, x, c, dw, ws)

    def loss(xx, ww):
        at, s = 0, 0.0
        for e, n in enumerate(counts):
            s = s + (dy[at:at + n].double() * (xx[at:at + n] @ ww[e].t())).sum()
            at += n
        return s
    X, W = x.double(), w.double()
    for seed in range(4):
        v, u = normal(10 + seed, 64, 136).double(), normal(20 + seed, 4, 72, 136).double()
        h = 1e-3
        d = (loss(X + h * v, W) - loss(X - h * v, W)) / (2 * h)
        assert abs(float(d - (dx.double() * v).sum())) <= 2.0 ** -8 * float((dx.double() * v).abs().sum())
        d = (loss(X, W + h * u) - loss(X, W - h * u)) / (2 * h)
        assert abs(float(d - (dw.double() * u).sum())) <= 2.0 ** -16 * float((dw.double() * u).abs().sum())


def test_grouped_rows_without_a_group(moe):
    """Rows past the groups' are not read into a result and not written; NaN there, in another
    group's rows or in another group's weights goes nowhere else."""
    counts = [70, 0, 3, 130]
    own = sum(counts)
    g = moe.GroupCfg(rows=own + 61, E=4, n=72, k=200)   # neither size a whole number of tiles
    c = torch.tensor(counts, dtype=torch.int32, device="cuda")
    ws = workspace(moe, g)
    x, w, dy = normal(1, g.rows, g.k), normal(2, 4, g.n, g.k), normal(3, g.rows, g.n)
    nan = float("nan")
    for t in (x, dy):
        t[own:] = nan
        t[70:73] = nan                       # group 2
    w[1] = nan                               # no rows
    w[2] = float("inf")
    for fn, src, width in (("mm", x, g.n), ("dx", dy, g.k)):
        out = torch.full((g.rows, width), 7.0, dtype=BF, device="cuda")
        (moe.grouped_mm if fn == "mm" else moe.grouped_mm_dx)(g, src, c, w, out, ws)
        assert bool((out[own:] == 7.0).all())
        ok = torch.ones(own, dtype=torch.bool)
        ok[70:73] = False
        ref, mag = grouped_reference(fn, src[:own], w, counts)
        check(out[:own][ok], ref[ok], 256 * 2.0 ** -23 * mag[ok], "bf16")
        assert bool(out[70:73].isnan().all())
    dw = torch.empty((4, g.n, g.k), device="cuda")
    moe.grouped_mm_dw(g, dy, x, c, dw, ws)
    assert bool(dw[2].isnan().all()) and float(dw[1].abs().sum()) == 0.0
    ref, mag = grouped_reference("dw", dy[:own], x[:own], counts)
    for e in (0, 3):
        check(dw[e], ref[e], 256 * 2.0 ** -23 * mag[e], "fp32")
    assert moe.read_status(ws) == 0


@pytest.mark.parametrize("counts,owned", [([5, -3, 6], [5, 0, 6]), ([10, 20, 5], [10, 6, 0]),
                                          ([2 ** 31 - 1, 2 ** 31 - 1, 1], [16, 0, 0])])
def test_wrong_counts_are_reported_and_cut(moe, counts, owned):
    g = moe.GroupCfg(rows=16, E=3, n=64, k=64)
    c = torch.tensor(counts, dtype=torch.int32, device="cuda")
    x, w, dy = normal(1, 16, 64), normal(2, 3, 64, 64), normal(3, 16, 64)
    own = sum(owned)
    for fn in ("mm", "dx", "dw"):
        ws = workspace(moe, g)
        if fn == "dw":
            out = torch.empty((3, 64, 64), device="cuda")
            moe.grouped_mm_dw(g, dy, x, c, out, ws)
            ref, mag = grouped_reference("dw", dy, x, owned)
            check(out, ref, 64 * 2.0 ** -23 * mag, "fp32")
        else:
            out = torch.zeros((16, 64), dtype=BF, device="cuda")
            src = x if fn == "mm" else dy
            (moe.grouped_mm if fn == "mm" else moe.grouped_mm_dx)(g, src, c, w, out, ws)
            ref, mag = grouped_reference(fn, src, w, owned)
            check(out[:own], ref, 64 * 2.0 ** -23 * mag, "bf16")
            assert float(out[own:].float().abs().sum()) == 0.0
        assert moe.read_status(ws) == moe.MOE_DEV_BOUNDS


def test_no_rows_zero_the_weight_gradient(moe):
    g = moe.GroupCfg(rows=0, E=3, n=72, k=40)
    c = torch.zeros(3, dtype=torch.int32, device="cuda")
    ws = workspace(moe, g)
    none = torch.empty((0, 72), dtype=BF, device="cuda"), torch.empty((0, 40), dtype=BF, device="cuda")
    dw = torch.full((3, 72, 40), 5.0, device="cuda")
    moe.grouped_mm_dw(g, *none, c, dw, ws, accumulate=True)
    assert bool((dw == 5.0).all())
    moe.grouped_mm_dw(g, *none, c, dw, ws)
    assert float(dw.abs().sum()) == 0.0
    b = torch.full((3, 72, 40), 5.0, dtype=BF, device="cuda")
    moe.grouped_mm_dw(g, *none, c, b, ws)
    assert float(b.float().abs().sum()) == 0.0


def test_groups_without_any_row(moe):
    """Rows that no group owns at all: nothing is written, and the weight gradient is zero."""
    g = moe.GroupCfg(rows=50, E=5, n=264, k=136)
    c = torch.zeros(5, dtype=torch.int32, device="cuda")
    ws = workspace(moe, g)
    x = torch.full((50, 136), float("nan"), dtype=BF, device="cuda")
    dy = torch.full((50, 264), float("nan"), dtype=BF, device="cuda")
    w = normal(1, 5, 264, 136)
    y = torch.full((50, 264), 3.0, dtype=BF, device="cuda")
    dx = torch.full((50, 136), 3.0, dtype=BF, device="cuda")
    moe.grouped_mm(g, x, c, w, y, ws)
    moe.grouped_mm_dx(g, dy, c, w, dx, ws)
    assert bool((y == 3.0).all()) and bool((dx == 3.0).all())
    for dtype in (torch.float32, BF):
        dw = torch.full((5, 264, 136), float("nan"), dtype=dtype, device="cuda")
        moe.grouped_mm_dw(g, dy, x, c, dw, ws)
        assert float(dw.float().abs().sum()) == 0.0
    dw = torch.full((5, 264, 136), 3.0, device="cuda")
    moe.grouped_mm_dw(g, dy, x, c, dw, ws, accumulate=True)
    assert bool((dw == 3.0).all())
    assert moe.read_status(ws) == 0


def test_one_workspace_for_many_shapes(moe):
    """Calls of several shapes and directions one after the other in the largest one's workspace:
    each leaves it as the next needs it."""
    shapes = [(300, 3, 264, 520), (64, 1, 512, 4096), (9000, 1, 256, 264), (5, 40, 64, 64)]
    cfgs = [moe.GroupCfg(rows=r, E=E, n=n, k=k) for r, E, n, k in shapes]
    ws = torch.zeros(max(moe.grouped_ws_bytes(g) for g in cfgs), dtype=torch.uint8, device="cuda")
    for turn in range(2):
        for g in cfgs:
            counts = spread(g.rows, g.E, "random", turn)
            c = torch.tensor(counts, dtype=torch.int32, device="cuda")
            x, w, dy = normal(turn, g.rows, g.k), normal(2, g.E, g.n, g.k), normal(3, g.rows, g.n)
            y, dx = torch.empty_like(dy), torch.empty_like(x)
            dw = torch.empty((g.E, g.n, g.k), device="cuda")
            moe.grouped_mm(g, x, c, w, y, ws)
            moe.grouped_mm_dw(g, dy, x, c, dw, ws)
            moe.grouped_mm_dx(g, dy, c, w, dx, ws)
            for out, kind, a, b, m, t in ((y, "mm", x, w, g.k, "bf16"), (dx, "dx", dy, w, g.n, "bf16"),
                                          (dw, "dw", dy, x, max(counts), "fp32")):
                ref, mag = grouped_reference(kind, a, b, counts)
                check(out, ref, m * 2.0 ** -23 * mag, t)
    assert moe.read_status(ws) == 0


def test_offsets_past_32_bits(moe):
    """The last group's weights and gradient start past 2^31 elements."""
    g = moe.GroupCfg(rows=40, E=75, n=4096, k=7168)
    counts = [0] * 75
    counts[0], counts[74] = 1, 39
    c = torch.tensor(counts, dtype=torch.int32, device="cuda")
    ws = workspace(moe, g)
    w = torch.zeros((75, g.n, g.k), dtype=BF, device="cuda")
    w[74] = normal(5, g.n, g.k, std=0.05)
    x, dy = normal(1, 40, g.k), normal(3, 40, g.n)
    y, dx = torch.empty((40, g.n), dtype=BF, device="cuda"), torch.empty((40, g.k), dtype=BF, device="cuda")
    moe.grouped_mm(g, x, c, w, y, ws)
    moe.grouped_mm_dx(g, dy, c, w, dx, ws)
    W = w[74].double()
    check(y[1:], x[1:].double() @ W.t(), g.k * 2.0 ** -23 * (x[1:].double().abs() @ W.t().abs()), "bf16")
    check(dx[1:], dy[1:].double() @ W, g.n * 2.0 ** -23 * (dy[1:].double().abs() @ W.abs()), "bf16")
    moe.grouped_mm_dw(g, dy, x, c, w, ws)
    A, B = dy[1:].double().t(), x[1:].double()
    check(w[74], A @ B, 39 * 2.0 ** -23 * (A.abs() @ B.abs()), "bf16")
    assert float(w[1:74].abs().amax()) == 0.0


def test_grouped_on_another_stream(moe):
    g = moe.GroupCfg(rows=500, E=3, n=256, k=512)
    counts = spread(500, 3, "random")
    c = torch.tensor(counts, dtype=torch.int32, device="cuda")
    ws, s = workspace(moe, g), torch.cuda.Stream()
    x, w = normal(1, 500, 512), normal(2, 3, 256, 512)
    y, y2 = torch.empty((500, 256), dtype=BF, device="cuda"), torch.empty((500, 256), dtype=BF, device="cuda")
    moe.grouped_mm(g, x, c, w, y, ws)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        x2 = x * 1
        moe.grouped_mm(g, x2, c, w, y2, ws)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y, y2)


def test_grouped_in_a_graph(moe):
    g = moe.GroupCfg(rows=300, E=4, n=128, k=256)
    c = torch.tensor([100, 0, 150, 50], dtype=torch.int32, device="cuda")
    ws = workspace(moe, g)
    x, w, dy = normal(1, 300, 256), normal(2, 4, 128, 256), normal(3, 300, 128)
    y = torch.empty((300, 128), dtype=BF, device="cuda")
    dw = torch.empty((4, 128, 256), device="cuda")

    def step():
        moe.grouped_mm(g, x, c, w, y, ws)
        moe.grouped_mm_dw(g, dy, x, c, dw, ws)
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    x.copy_(normal(9, 300, 256))
    c.copy_(torch.tensor([0, 17, 3, 280], dtype=torch.int32))
    graph.replay()
    ref, mag = grouped_reference("mm", x, w, c.tolist())
    check(y, ref, 256 * 2.0 ** -23 * mag, "bf16")
    ref, mag = grouped_reference("dw", dy, x, c.tolist())
    check(dw, ref, 300 * 2.0 ** -23 * mag, "fp32")


# -------------------------------------- 8-bit checkpoints --------------------------------------
def quantise(x):
    """The dispatch's rule on the host in fp32, step by step (IEEE divisions, nearest even)."""
    b = x.float().cpu().view(x.shape[0], -1, 128)
    amax = b.abs().amax(-1, keepdim=True)
    s = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
    q = (b / s).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).view(x.shape)
    return q, s.squeeze(-1).t().contiguous()


def values(q, s):
    v = q.cpu().view(torch.float8_e4m3fn).double()
    return (v.view(v.shape[0], -1, 128) * s.cpu().double().t().unsqueeze(-1)).view(v.shape)


def awkward(seed, rows, cols):
    """Normal values over many magnitudes, with zero blocks, single spikes and tiny blocks."""
    x = normal(seed, rows, cols)
    x[0, :128] = 0
    x[-1, -128:] = 0
    x[-1, -5] = -3e-39          # a subnormal alone in its block
    x[rows // 2] *= 1e-30
    x[rows // 3, 7] = 3e4
    x[:, ::9] *= 0.01
    return x


@pytest.mark.parametrize("rows,d", [(1, 128), (3, 384), (17, 256), (250, 1152), (1000, 2048)])
def test_act_save_and_load(moe, rows, d):
    x = awkward(4, rows, d)
    q = torch.empty((rows, d), dtype=torch.uint8, device="cuda")
    s = torch.empty((d // 128, rows), device="cuda")
    moe.act_save(x, q, s)
    rq, rs = quantise(x)
    assert torch.equal(q.cpu(), rq) and torch.equal(s.cpu(), rs)
    out = torch.empty((rows, d), dtype=BF, device="cuda")
    moe.act_load(q, s, None, out)
    exact = values(rq, rs).float().to(BF)     # code * scale rounds to fp32, then to bf16
    assert torch.equal(out.cpu(), exact)
    # every row twice, backwards, with empty rows between
    idx = torch.stack([torch.arange(rows).flip(0), torch.full((rows,), -1),
                       torch.arange(rows)], 1).flatten().to(torch.int32).cuda()
    wide = torch.full((3 * rows, d), 5.0, dtype=BF, device="cuda")
    st = torch.zeros(4, dtype=torch.int32, device="cuda")
    moe.act_load(q, s, idx, wide, status=st)
    assert torch.equal(wide[0::3].cpu(), exact.flip(0)) and torch.equal(wide[2::3].cpu(), exact)
    assert float(wide[1::3].float().abs().sum()) == 0.0
    assert int(st[0]) == 0


@pytest.mark.parametrize("amax", [1.0, 1.9921875, 448.0, 0.0131, 3.3e38, 3.1e-20, 1e-37])
def test_codes_of_every_bf16_value(moe, amax):
    """Every finite bf16 value up to the block's largest against the IEEE quotient."""
    v = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(BF)
    top = torch.tensor(amax).to(BF)
    v = v[v.float().isfinite() & (v.float().abs() <= top.float())]
    pad = -v.numel() % 127
    v = torch.cat([v, torch.zeros(pad, dtype=BF)]).view(-1, 127)
    x = torch.cat([v, top.expand(v.shape[0], 1)], 1).contiguous().cuda()
    q = torch.empty(x.shape, dtype=torch.uint8, device="cuda")
    s = torch.empty((1, x.shape[0]), device="cuda")
    moe.act_save(x, q, s)
    rq, rs = quantise(x)
    assert torch.equal(q.cpu(), rq) and torch.equal(s.cpu(), rs)


def test_act_load_reports_wrong_rows(moe):
    x = normal(1, 4, 128)
    q, s = torch.empty((4, 128), dtype=torch.uint8, device="cuda"), torch.empty((1, 4), device="cuda")
    moe.act_save(x, q, s)
    idx = torch.tensor([3, 4, -2, 0, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    out = torch.full((5, 128), 5.0, dtype=BF, device="cuda")
    st = torch.zeros(4, dtype=torch.int32, device="cuda")
    moe.act_load(q, s, idx, out, status=st)
    assert int(st[0]) == moe.MOE_DEV_BOUNDS
    assert float(out[[1, 2, 4]].float().abs().sum()) == 0.0
    assert bool((out[0] != 0).any()) and bool((out[3] != 0).any())


def test_what_is_not_finite_reads_back_as_nan(moe):
    x = normal(1, 3, 256)
    x[0, 5], x[1, 130] = float("nan"), float("inf")
    q, s = torch.empty((3, 256), dtype=torch.uint8, device="cuda"), torch.empty((2, 3), device="cuda")
    out = torch.empty((3, 256), dtype=BF, device="cuda")
    moe.act_save(x, q, s)
    moe.act_load(q, s, None, out)
    bad = torch.zeros((3, 256), dtype=torch.bool, device="cuda")
    bad[0, 5] = True
    bad[1, 128:] = True
    assert torch.equal(out.isnan(), bad)


@pytest.mark.parametrize("rows,f", [(1, 128), (7, 384), (130, 256), (999, 2048), (2500, 128)])
def test_swiglu_save(moe, rows, f):
    gu = awkward(6, rows, 2 * f)
    gu[0, 1], gu[0, 2] = 100.0, -100.0      # exp runs out of range on one side
    a = torch.empty((rows, f), dtype=BF, device="cuda")
    q = torch.empty((rows, 2 * f), dtype=torch.uint8, device="cuda")
    s = torch.empty((2 * f // 128, rows), device="cuda")
    moe.swiglu_save(gu, a, q, s)
    rq, rs = quantise(gu)
    assert torch.equal(q.cpu(), rq) and torch.equal(s.cpu(), rs)
    g, u = gu.double().chunk(2, 1)
    ref = g * torch.sigmoid(g) * u
    # the exponential is off by 2^-21 + 2^-24 |g| of its size; where it passes the fp32 range
    # (g < -88) the result is 0 instead of at most 88 e^-88 |u|
    check(a, ref, 2.0 ** -16 * ref.abs() + 1e-36 * u.abs(), "bf16")


@pytest.mark.parametrize("rows,f", [(1, 128), (7, 384), (130, 256), (999, 2048)])
def test_swiglu_grad(moe, rows, f):
    gu, da = awkward(7, rows, 2 * f) * 3, normal(8, rows, f)
    q, s = (t.cuda() for t in quantise(gu))
    dgu = torch.empty((rows, 2 * f), dtype=BF, device="cuda")
    a = torch.empty((rows, f), dtype=BF, device="cuda")
    moe.swiglu_grad(q, s, da, dgu, a)
    v = values(q, s).cuda()
    g, u = v.chunk(2, 1)
    d, sig = da.double(), torch.sigmoid(g)
    dg = d * u * sig * (1 + g * (1 - sig))
    du, ra = d * g * sig, g * sig * u
    # each factor is off by a few units of 2^-24 and the exponential by 2^-16 at most: of the two
    # terms of dg each by 2^-15 of its own size; e^-88 as in the forward
    tiny = 1e-36 * (d.abs() + u.abs()) * (1 + u.abs() + d.abs())
    check(dgu[:, :f], dg, 2.0 ** -15 * (d * u * sig).abs() * (1 + g.abs() * (1 - sig)) + tiny, "bf16")
    check(dgu[:, f:], du, 2.0 ** -15 * du.abs() + tiny, "bf16")
    check(a, ra, 2.0 ** -15 * ra.abs() + tiny, "bf16")
    # against central differences of the 64-bit forward at the saved values: their own error is
    # of the order of h^2
    h = 1e-5
    num = (((g + h) * torch.sigmoid(g + h) - (g - h) * torch.sigmoid(g - h)) / (2 * h)) * u * d
    check(dgu[:, :f], num, (2.0 ** -15 + 1e-7) * (d * u).abs() * (1 + g.abs()) + tiny, "bf16")
    # without the product again
    dgu2 = torch.empty_like(dgu)
    moe.swiglu_grad(q, s, da, dgu2)
    assert torch.equal(dgu, dgu2)


# ------------------------------------- the combine's gradient -------------------------------------
@pytest.mark.parametrize("T,k,d", [(1, 1, 128), (1, 8, 7168), (3, 32, 256), (37, 5, 640),
                                   (64, 8, 7168), (500, 2, 1024), (5000, 2, 1152)])
def test_combine_grad(moe, T, k, d):
    rows = T * k + 9                                   # rows that no choice names
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    row_of = torch.randperm(rows, generator=gen, device="cuda")[:T * k].to(torch.int32).view(T, k)
    row_of[T // 2, k - 1] = -1                         # a choice that the dispatch skipped
    w = torch.rand((T, k), generator=gen, device="cuda")
    ebuf, dy = normal(1, rows, d), normal(2, T, d)
    de = torch.full((rows, d), 7.0, dtype=BF, device="cuda")
    dw = torch.full((T, k), float("nan"), device="cuda")
    st = torch.zeros(4, dtype=torch.int32, device="cuda")
    moe.combine_grad(ebuf, row_of, w, dy, de, dw, status=st)
    assert int(st[0]) == 0
    named = row_of >= 0
    at = row_of[named].long()
    tok = torch.arange(T, device="cuda").view(T, 1).expand(T, k)[named]
    assert torch.equal(de[at], (w[named].unsqueeze(1) * dy[tok].float()).to(BF))
    rest = torch.ones(rows, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert bool((de[rest] == 7.0).all())
    prod = dy[tok].double() * ebuf[at].double()
    check(dw[named], prod.sum(1), d * 2.0 ** -24 * prod.abs().sum(1), "fp32")
    assert float(dw[~named].abs().sum()) == 0.0
    dw2 = torch.empty_like(dw)
    moe.combine_grad(ebuf, row_of, w, dy, de, dw2)
    assert torch.equal(dw, dw2)


def test_combine_grad_against_differences(moe):
    """The combine y[t] = sum_i w[t][i] e[row_of[t][i]] is linear in w and in e, so its central
    difference in 64 bits is the derivative itself; dtopk_w is off by the fp32 sum (d 2^-24 of the
    products' magnitudes), debuf by its rounding to bf16."""
    T, k, d, rows = 9, 3, 256, 40
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    row_of = torch.randperm(rows, generator=gen, device="cuda")[:T * k].to(torch.int32).view(T, k)
    w = torch.rand((T, k), generator=gen, device="cuda")
    ebuf, dy = normal(1, rows, d), normal(2, T, d)
    de, dw = torch.zeros_like(ebuf), torch.empty((T, k), device="cuda")
    moe.combine_grad(ebuf, row_of, w, dy, de, dw)

    def loss(ww, ee):
        return ((ww.unsqueeze(-1) * ee[row_of.long()]).sum(1) * dy.double()).sum()
    W, E, h = w.double(), ebuf.double(), 1e-3
    for seed in range(3):
        v = torch.randn((T, k), generator=gen, device="cuda", dtype=torch.float64)
        u = torch.randn((rows, d), generator=gen, device="cuda", dtype=torch.float64)
        diff = float((loss(W + h * v, E) - loss(W - h * v, E)) / (2 * h))
        mag = (dy.double().unsqueeze(1) * E[row_of.long()]).abs().sum(-1)
        assert abs(diff - float((dw.double() * v).sum())) <= d * 2.0 ** -24 * float((mag * v.abs()).sum()) + 1e-9
        diff = float((loss(W, E + h * u) - loss(W, E - h * u)) / (2 * h))
        assert abs(diff - float((de.double() * u).sum())) <= 2.0 ** -8 * float((de.double() * u).abs().sum())


def test_combine_grad_reports_wrong_rows(moe):
    ebuf, dy = normal(1, 6, 256), normal(2, 2, 256)
    row_of = torch.tensor([[0, 6], [-5, 2 ** 31 - 1]], dtype=torch.int32, device="cuda")
    w = torch.ones((2, 2), device="cuda")
    de, dw = torch.zeros_like(ebuf), torch.full((2, 2), 9.0, device="cuda")
    st = torch.zeros(4, dtype=torch.int32, device="cuda")
    moe.combine_grad(ebuf, row_of, w, dy, de, dw, status=st)
    assert int(st[0]) == moe.MOE_DEV_BOUNDS
    assert torch.equal(de[0], dy[0]) and float(de[1:].float().abs().sum()) == 0.0
    assert dw.flatten()[1:].tolist() == [0.0, 0.0, 0.0]


# ------------------------------------------ the step ------------------------------------------
@pytest.mark.parametrize("T,shared", [(1, 0), (37, 128), (200, 128)])
def test_training_step(moe, T, shared):
    """The layer's forward equals moe_layer's but for the order of sums, and its gradients are
    those of the 64-bit layer at the values the backward pass holds: the saved codes."""
    from combine_grouped_gemm_gb300.train import MoETrainLayer
    cfg = dataclasses.replace(synth.CONFIGS["tiny"], T=T, d_ff_shared=shared, R=1)
    inp, W = synth.make_router_inputs(cfg, "cuda"), synth.make_expert_weights(cfg, "cuda")
    if not shared:
        W = {n: v for n, v in W.items() if v is not None}
    layer = MoETrainLayer(cfg, inp["w_gate"], inp["bias"], W)
    x = inp["x"]
    y = layer.forward(x)
    serve = moe.MoELayer(cfg, inp["w_gate"], inp["bias"], W)
    ys = serve(x)
    rel = lambda a, b: float((a.double() - b.double()).norm() / b.double().norm())   # noqa: E731
    # each side rounds the expert outputs and the result to bf16 (2^-9 each) and, before the
    # down product, the gate/up product here and the activation on both
    assert rel(y, ys) < 6 * 2.0 ** -9
    dy = normal(11, T, cfg.d)
    grads = {n: v.clone() for n, v in layer.backward(dy).items()}

    b = layer.bufs
    idx, w = b["topk_idx"].long(), b["topk_w"].double()
    xv = values(layer.xq, layer.x_scales).cuda()
    f = cfg.d_ff

    def expert(xr, gu, dyr, w13, w2):
        """dx, dw13, dw2 of one expert's rows, gate/up values given."""
        g, u = gu.chunk(2, 1)
        s = torch.sigmoid(g)
        da = dyr @ w2
        dgu = torch.cat([da * u * s * (1 + g * (1 - s)), da * g * s], 1)
        return dgu @ w13, dgu.t() @ xr, dyr.t() @ (g * s * u)

    guv = values(layer.routed.q, layer.routed.scales).cuda()
    dx = torch.zeros((T, cfg.d), dtype=torch.float64, device="cuda")
    dw13 = torch.zeros((cfg.E, 2 * f, cfg.d), dtype=torch.float64, device="cuda")
    dw2 = torch.zeros((cfg.E, cfg.d, f), dtype=torch.float64, device="cuda")
    for e in range(cfg.E):
        t, i = (idx == e).nonzero(as_tuple=True)
        if not t.numel():
            continue
        rows = b["row_of"][t, i].long()
        r, p, o = expert(xv[t], guv[rows], w[t, i].unsqueeze(1) * dy[t].double(),
                         W["w13"][e].double(), W["w2"][e].double())
        dx.index_add_(0, t, r)
        dw13[e], dw2[e] = p, o
    if shared:
        gs = values(layer.shared.q, layer.shared.scales).cuda()
        r, p, o = expert(xv, gs, dy.double(), W["ws13"].double(), W["ws2"].double())
        dx += r
        assert rel(grads["dws13"][0], p) < 8 * 2.0 ** -9 and rel(grads["dws2"][0], o) < 8 * 2.0 ** -9
    # up to eight roundings to bf16 on the way (d_ebuf, da, dgu, the rows, their gradient, dx)
    assert rel(grads["dx"], dx) < 8 * 2.0 ** -9
    assert rel(grads["dw13"], dw13) < 8 * 2.0 ** -9
    assert rel(grads["dw2"], dw2) < 8 * 2.0 ** -9
    # the routing weights' gradient, from the whole forward in 64 bits
    xd = x.double()
    eo = torch.stack([torch.stack([(lambda g, u: (g * torch.sigmoid(g) * u))(
        *(xd[t] @ W["w13"][e].double().t()).chunk(2)) @ W["w2"][e].double().t()
        for e in idx[t].tolist()]) for t in range(T)])
    assert rel(grads["dtopk_w"], (eo * dy.double().unsqueeze(1)).sum(-1)) < 8 * 2.0 ** -9
    # micro-batches: the same gradient added to itself
    layer.forward(x)
    g2 = layer.backward(dy, accumulate=True)
    assert rel(g2["dw13"], 2 * grads["dw13"].double()) < 1e-6
    assert torch.equal(g2["dx"], grads["dx"])
    assert moe.read_status(b["ws"]) == 0 and moe.read_status(layer.routed.ws) == 0
