"""The grouped products where a CTA pair works through many units: the load ring wraps, units come
from the counter through the scheduler's ring, both accumulator buffers are used again.

The references are 64-bit products of the same bf16 values. A bf16 result is off by its own rounding
(at most 2^-8 of its size) and by the fp32 sum before it: m products, each addition truncated to
2^-23 of the running magnitude, are off by at most m 2^-23 of the products' magnitudes in all.
"""
import pytest
import torch

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


def uneven(rows, E, seed, empty=0.0):
    """Rows dealt over E groups of random popularity, a share of them without any."""
    gen = torch.Generator()
    gen.manual_seed(seed)
    p = torch.rand(E, generator=gen) + 0.05
    p[torch.rand(E, generator=gen) < empty] = 0.0
    p[E // 2] += 1e-3
    at = torch.multinomial(p, rows, replacement=True, generator=gen)
    return torch.bincount(at, minlength=E).tolist()


def within(got, ref, mag, m):
    """Element by element: the result's own rounding and the sum of m products."""
    own = 2.0 ** -8 if got.dtype is BF else 2.0 ** -24
    assert bool(torch.isfinite(got).all())
    over = (got.double() - ref).abs() - (own * ref.abs() + m * 2.0 ** -23 * mag + 1e-37)
    assert float(over.max()) <= 0.0


def check_rows(out, src, w, counts, transposed, m):
    first = 0
    for e, c in enumerate(counts):
        if c:
            a = src[first:first + c].double()
            b = w[e].double().t() if transposed else w[e].double()
            within(out[first:first + c], a @ b, a.abs() @ b.abs(), m)
        first += c


def check_dw(dw, dy, x, counts):
    first = 0
    for e, c in enumerate(counts):
        a, b = dy[first:first + c].double().t(), x[first:first + c].double()
        within(dw[e], a @ b, a.abs() @ b.abs(), max(1, c))
        first += c


# rows, E, n, k, share of empty groups: row tile, units (at most) and k-steps of fwd; of dx
SHAPES = [
    (6000, 5, 2056, 1096, 0.0),     # 256 rows, 252 units of 18 steps; 140 of 33
    (4001, 40, 2056, 1096, 0.0),    # 128 rows, 630 units of 18; 350 of 33
    (3333, 40, 1288, 904, 0.5),     # the same tile, about half of the groups empty
    (500, 40, 2056, 1096, 0.1),     # 64 rows, 423 units of 18; 235 of 33
    (2000, 1000, 2056, 64, 0.3),    # 64 rows, up to 9135 units of one step: a hundred a pair
]


@pytest.mark.parametrize("rows,E,n,k,empty", SHAPES)
def test_rows_over_many_units_a_pair(moe, rows, E, n, k, empty):
    counts = uneven(rows, E, rows, empty)
    c = torch.tensor(counts, dtype=torch.int32, device="cuda")
    g = moe.GroupCfg(rows=rows, E=E, n=n, k=k)
    ws = torch.zeros(moe.grouped_ws_bytes(g), dtype=torch.uint8, device="cuda")
    x, w, dy = normal(1, rows, k), normal(2, E, n, k, std=0.05), normal(3, rows, n)
    y = torch.full((rows, n), float("nan"), dtype=BF, device="cuda")
    dx = torch.full((rows, k), float("nan"), dtype=BF, device="cuda")
    moe.grouped_mm(g, x, c, w, y, ws)
    moe.grouped_mm_dx(g, dy, c, w, dx, ws)
    check_rows(y, x, w, counts, True, k)
    check_rows(dx, dy, w, counts, False, n)
    again = torch.empty_like(y), torch.empty_like(dx)
    for _ in range(20):   # the units are taken by other pairs each time: the bits stay
        moe.grouped_mm(g, x, c, w, again[0], ws)
        moe.grouped_mm_dx(g, dy, c, w, again[1], ws)
        assert torch.equal(again[0], y) and torch.equal(again[1], dx)
    assert moe.read_status(ws) == 0


@pytest.mark.parametrize("rows,E,n,k,empty", [
    (6000, 5, 2056, 1096, 0.0),     # 225 units of up to about 30 steps: three to four fp32 sums
    (9000, 6, 2056, 1096, 0.4),
    (2000, 1000, 264, 264, 0.3),    # 4000 units of one step, a third of them without rows
])
def test_weight_gradients_over_many_units_a_pair(moe, rows, E, n, k, empty):
    counts = uneven(rows, E, rows, empty)
    c = torch.tensor(counts, dtype=torch.int32, device="cuda")
    g = moe.GroupCfg(rows=rows, E=E, n=n, k=k)
    ws = torch.zeros(moe.grouped_ws_bytes(g), dtype=torch.uint8, device="cuda")
    x, dy = normal(1, rows, k), normal(3, rows, n)
    for dtype in (torch.float32, BF):
        dw = torch.full((E, n, k), float("nan"), dtype=dtype, device="cuda")
        moe.grouped_mm_dw(g, dy, x, c, dw, ws)
        check_dw(dw, dy, x, counts)
        again = torch.empty_like(dw)
        for _ in range(10):
            moe.grouped_mm_dw(g, dy, x, c, again, ws)
            assert torch.equal(again, dw)
        if dtype is torch.float32:   # added to itself: the doubled value is exact in fp32
            moe.grouped_mm_dw(g, dy, x, c, again, ws, accumulate=True)
            assert torch.equal(again, 2 * dw)
    assert moe.read_status(ws) == 0


def test_groups_near_the_end_of_the_row_range(moe):
    """One group of nearly 2^31 rows: all rows are written and read, and the weight gradient's sum
    keeps its precision. It adds 2^31 products in parts of at most 512; each addition of those sums
    rounds by at most 2^-24 of a partial sum no larger than the result, with random signs, 2^25
    additions in all: 2^-24 2^12.5 of it, at most."""
    g = moe.GroupCfg(rows=2 ** 31 - 520, E=2, n=8, k=8)
    counts = [g.rows - 3, 3]
    c = torch.tensor(counts, dtype=torch.int32, device="cuda")
    ws = torch.zeros(moe.grouped_ws_bytes(g), dtype=torch.uint8, device="cuda")
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    x = torch.empty((g.rows, 8), dtype=BF, device="cuda").normal_(0.25, 1.0, generator=gen)
    w = normal(2, 2, 8, 8)
    y = torch.full((g.rows, 8), float("nan"), dtype=BF, device="cuda")
    moe.grouped_mm(g, x, c, w, y, ws)
    at = torch.randint(0, counts[0], (200000,), generator=gen, device="cuda")
    at[:3] = torch.tensor([0, 2 ** 30, counts[0] - 1])

    def check(out, src, mats):
        for first in range(0, g.rows, 1 << 27):
            assert bool(torch.isfinite(out[first:first + (1 << 27)]).all())
        for s, o, m in ((src[at], out[at], mats[0]), (src[-3:], out[-3:], mats[1])):
            within(o, s.double() @ m, s.double().abs() @ m.abs(), 8)
    check(y, x, [w[e].double().t() for e in range(2)])
    dx = torch.full((g.rows, 8), float("nan"), dtype=BF, device="cuda")
    moe.grouped_mm_dx(g, y, c, w, dx, ws)
    check(dx, y, [w[e].double() for e in range(2)])
    del dx
    dw = torch.empty((2, 8, 8), device="cuda")
    moe.grouped_mm_dw(g, y, x, c, dw, ws)
    ref = torch.zeros((8, 8), dtype=torch.float64, device="cuda")
    for first in range(0, counts[0], 1 << 25):
        r = slice(first, min(first + (1 << 25), counts[0]))
        ref += y[r].double().t() @ x[r].double()
    assert float((dw[0].double() - ref).norm() / ref.norm()) < 2.0 ** -11.5
    last = y[-3:].double().t(), x[-3:].double()
    within(dw[1], last[0] @ last[1], last[0].abs() @ last[1].abs(), 3)
    assert moe.read_status(ws) == 0
