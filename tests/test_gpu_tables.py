"""Weight-table operators on the GPU against plain implementations in 64 bits.

Three kinds of comparison:
- exact: small whole numbers, scales of powers of two.  Every product and every
  partial sum is a whole number (times one power of two) below 2^24, so fp32
  sums are exact in any order and the result must be equal, bit for bit.
- moved or rounded values (builders, lookups): equal to the definition.
- random values: within the bound of fp32 summation, derived at `sum_bound`.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import spmv_storage_formats_amd as spmv  # noqa: E402

F = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spmv.load_library()
    return torch.device("cuda:0")


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


# ------------------------------------------------------------ 4-bit matrices

class Packed:
    """A random 4-bit matrix, and its values in 64 bits (numpy)."""

    def __init__(self, R, C, group, zeros, scale_dtype, seed, exact=False):
        rng = np.random.default_rng(seed)
        G = -(-C // group)
        q = rng.integers(0, 16, (R, C))
        self.q = q
        if exact:
            s = 2.0 ** rng.integers(-2, 3, (R, G))
        else:
            s = rng.uniform(0.5, 1.5, (R, G)) * 0.01
        self.scales = torch.from_numpy(s).to(F[scale_dtype])
        self.z = rng.integers(0, 16, (R, G)) if zeros else np.full((R, G), 8)
        full = np.zeros((R, C + (C & 1)), np.uint8)
        full[:, :C] = q
        self.codes = torch.from_numpy(full[:, 0::2] | (full[:, 1::2] << 4))
        self.s64 = self.scales.double().numpy()
        c = np.arange(C) // group
        self.w = self.s64[:, c] * (q - self.z[:, c])
        self.R, self.C, self.group, self.G = R, C, group, G
        # largest |code| + |zero| a kernel may form while it removes an offset
        self.wide = self.s64[:, c] * 64.0
        self.zeros = torch.from_numpy(self.z.astype(np.uint8)) if zeros else None

    def build(self, dev):
        return spmv.build_quant_packed(
            self.codes.to(dev), self.scales.to(dev), self.C, group_size=self.group,
            zero_points=None if self.zeros is None else self.zeros.to(dev))


def sum_bound(p, x):
    """Bound of an fp32 dot product of row r with x: each of its at most C + C/32 + 64
    roundings (C products' sums, one scaling and its addition per 32 columns, the join of
    parts) is off by at most 2^-24 of a partial sum, and no partial sum is larger than
    sum |s| * 64 * |x|: codes and zero points are moved by at most 16, so no factor that a
    kernel sums exceeds 31 + 31 < 64."""
    return (p.C + p.C / 32 + 64) * 2.0 ** -24 * (p.wide @ np.abs(x).T).T


# matrix heights at which the kernel's shape changes: few rows, and odd ones past each bound
HEIGHTS = [48, 4097, 8193, 16390]

SHAPES = [(1, 1, 32), (1, 7, 32), (3, 32, 32), (16, 128, 32), (17, 130, 64), (15, 255, 128),
          (33, 256, 64), (64, 257, 32), (100, 1000, 128), (48, 4096, 128), (31, 2750, 32),
          (130, 777, 256), (20, 5000, 384), (300, 515, 64), (5, 3000, 4096)]


@pytest.mark.parametrize("x_dtype,y_dtype", [("fp32", "fp32"), ("fp16", "fp16"),
                                             ("fp16", "fp32"), ("bf16", "bf16"),
                                             ("bf16", "fp32")])
@pytest.mark.parametrize("R,C,group", SHAPES)
def test_product_exact(dev, R, C, group, x_dtype, y_dtype):
    """Whole numbers: |q - z| <= 15 < 2^4, scales 2^-2..2^2, |x| <= 4; moved by 16 the factors
    stay below 2^5, so in units of 2^-2 a sum of C terms is below 2^5 * 2^4 * 2^2 * C <= 2^24
    for C <= 2^13, as is y.  A rounded 16-bit result is the exact one's rounding."""
    seed = R * 7919 + C
    rng = np.random.default_rng(seed)
    for zeros, scale_dtype, n, accumulate in ((False, "bf16", 1, False), (True, "fp32", 2, True),
                                              (True, "fp16", 5, False), (False, "fp32", 16, True),
                                              (True, "bf16", 17, True), (False, "fp16", 33, False),
                                              (True, "fp16", 70, True)):
        p = Packed(R, C, group, zeros, scale_dtype, seed, exact=True)
        x = rng.integers(-4, 5, (n, C)).astype(np.float64)
        y0 = rng.integers(-8, 9, (n, R)).astype(np.float64)
        q = p.build(dev)
        y = torch.from_numpy(y0).to(F[y_dtype]).to(dev)
        if not accumulate:
            y.fill_(float("nan"))     # what y held must not matter
        q.run(torch.from_numpy(x).to(F[x_dtype]).to(dev), y, accumulate=accumulate)
        want = x @ p.w.T + (y0 if accumulate else 0)
        want = torch.from_numpy(want).to(torch.float32).to(F[y_dtype])
        assert torch.equal(y.cpu(), want), (zeros, scale_dtype, n, accumulate)
        q.close()


@pytest.mark.parametrize("x_dtype,y_dtype", [("fp32", "fp32"), ("fp16", "fp16"),
                                             ("bf16", "fp32"), ("bf16", "bf16")])
@pytest.mark.parametrize("R,C,group,zeros,scale_dtype,n", [
    (40, 96, 32, True, "fp32", 1), (257, 4096, 128, False, "bf16", 1),
    (100, 2750, 32, True, "fp16", 3), (64, 1111, 64, True, "fp32", 21),
    (33, 8192, 256, False, "fp16", 64)])
def test_product_random(dev, R, C, group, zeros, scale_dtype, n, x_dtype, y_dtype):
    rng = np.random.default_rng(R + C + n)
    p = Packed(R, C, group, zeros, scale_dtype, R + C)
    spread = np.exp(rng.uniform(-3, 3, (n, C)))
    xt = torch.from_numpy(rng.standard_normal((n, C)) * spread).to(F[x_dtype])
    yt = torch.from_numpy(rng.standard_normal((n, R))).to(F[y_dtype])
    x, y0 = xt.double().numpy(), yt.double().numpy()
    q = p.build(dev)
    y = q.run(xt.to(dev), yt.to(dev)).double().cpu().numpy()
    want = x @ p.w.T + y0
    tol = sum_bound(p, x) + 2.0 ** -23 * np.abs(y0)
    if y_dtype != "fp32":
        tol = tol + half_step(F[y_dtype]) * (np.abs(want) + tol) + 2.0 ** -24
    assert np.all(np.abs(y - want) <= tol), np.max(np.abs(y - want) / tol)
    # two runs are the same, bit for bit
    a = q.run(xt.to(dev), yt.to(dev))
    assert torch.equal(a.double().cpu(), torch.from_numpy(y))


def test_product_fp32_keeps_all_bits_of_x(dev):
    """One nonzero per vector: y is a single product, w * x with |w| a power of two."""
    R, C = 48, 700
    p = Packed(R, C, 32, False, "fp32", 3, exact=True)
    p.q[:] = 9
    full = np.full((R, C), 9, np.uint8)
    p.codes = torch.from_numpy(full[:, 0::2] | (full[:, 1::2] << 4))
    rng = np.random.default_rng(1)
    x = np.zeros((9, C), np.float32)
    at = [0, 1, 31, 32, 255, 256, 511, 512, 699]
    # exponents far apart, all 24 bits in use
    val = (1 + rng.random(9)) * 2.0 ** np.array([0, 20, -20, 60, -60, 100, -90, 3, 1])
    val = val.astype(np.float32) * np.array([1, -1, 1, -1, 1, -1, 1, -1, 1], np.float32)
    for i, c in enumerate(at):
        x[i, c] = val[i]
    q = p.build(dev)
    y = torch.zeros(9, R, device=dev)
    q.run(torch.from_numpy(x).to(dev), y)
    want = np.stack([val[i].astype(np.float64) * p.s64[:, c // 32] for i, c in enumerate(at)])
    assert np.array_equal(y.double().cpu().numpy(), want)


@pytest.mark.parametrize("n", [1, 3, 5])
@pytest.mark.parametrize("R", HEIGHTS)
def test_product_fp32_keeps_all_bits_of_few_vectors(dev, R, n):
    """As above, for the numbers of vectors whose parts are 3, 9 and 15 columns of one pass, at
    the matrix heights of every kernel shape."""
    C = 420
    p = Packed(R, C, 32, False, "bf16", 3, exact=True)
    p.codes = torch.full((R, C // 2), 0x99, dtype=torch.uint8)
    q = p.build(dev)
    rng = np.random.default_rng(R + n)
    for turn in range(6):
        at = rng.integers(0, C, n)
        val = (1 + rng.random(n)) * 2.0 ** rng.integers(-80, 81, n) * rng.choice([-1, 1], n)
        x = np.zeros((n, C), np.float32)
        x[np.arange(n), at] = val
        y = q.run(torch.from_numpy(x).to(dev), torch.zeros(n, R, device=dev))
        want = x[np.arange(n), at].astype(np.float64)[:, None] * p.s64[:, at // 32].T
        assert np.array_equal(y.double().cpu().numpy(), want), (turn, at)


@pytest.mark.parametrize("n", [1, 3, 5, 6, 16, 17])
@pytest.mark.parametrize("R", HEIGHTS)
def test_product_fp32_of_24_bit_vectors(dev, R, n):
    """Dense vectors of all 24 bits, with only the join of their parts rounded.  |x| = 2^23 +
    2^16 a + 2^15 + b, a < 2^7, b < 2^15: the parts are whole multiples below 2^8 of 2^16, 2^8
    and 1.  In those units a group's moved sums are below 31 * 2^8 * 128 < 2^20, and in a
    quarter of them (scales 2^-2..2^2) every sum over the columns is below 16 * 15 * 2^8 * C <=
    2^24 for C <= 273: exact.  What is left are the additions of the second to the third part
    (together below 2^-7 |x|) and of both to the first, 2^-24 of their results each."""
    C, u = 270, 2.0 ** -24
    rng = np.random.default_rng(R + n)
    for group, zeros in ((32, True), (64, False), (128, True)):
        p = Packed(R, C, group, zeros, "fp32", R + group, exact=True)
        x = (2.0 ** 23 + 2.0 ** 16 * rng.integers(0, 2 ** 7, (n, C)) + 2 ** 15
             + rng.integers(0, 2 ** 15, (n, C))) * rng.choice([-1, 1], (n, C))
        q = p.build(dev)
        y = torch.full((n, R), float("nan"), device=dev)
        q.run(torch.from_numpy(x).float().to(dev), y, accumulate=False)
        want = x @ p.w.T
        tol = u * (np.abs(want) + 2.0 ** -7 * (np.abs(x) @ np.abs(p.w).T)) * (1 + 2 * u)
        err = np.abs(y.double().cpu().numpy() - want)
        assert np.all(err <= tol), (group, np.max(err / tol))
        q.close()


@pytest.mark.parametrize("n", [1, 4, 16, 17, 33, 48])
@pytest.mark.parametrize("R", HEIGHTS)
def test_product_exact_with_all_bits_of_16_bit_vectors(dev, R, n):
    """Whole numbers of all 8 bits (bf16) and 11 bits (fp16), scales of 1: a group's moved sums
    are below 31 * 2047 * 128 < 2^23, y below 15 * 2047 * C < 2^24 for C <= 546."""
    C = 530
    rng = np.random.default_rng(R + n)
    for dtype, low in (("bf16", 128), ("fp16", 1024)):
        for group, zeros in ((32, False), (64, True), (128, True)):
            p = Packed(R, C, group, zeros, "fp16", R + group, exact=True)
            p.scales = torch.ones_like(p.scales)
            x = rng.integers(low, 2 * low, (n, C)) * rng.choice([-1.0, 1.0], (n, C))
            q = p.build(dev)
            y = torch.full((n, R), float("nan"), device=dev)
            q.run(torch.from_numpy(x).to(F[dtype]).to(dev), y, accumulate=False)
            want = x @ (p.q - p.z[:, np.arange(C) // group]).T.astype(np.float64)
            assert np.array_equal(y.double().cpu().numpy(), want), (dtype, group)
            q.close()


@pytest.mark.parametrize("x_dtype", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("R,C,group", [(50, 33, 32), (70, 1000, 64), (4100, 640, 128),
                                       (30, 5000, 384)])
def test_product_of_codes_equal_to_their_zero_points(dev, R, C, group, x_dtype):
    """W = 0: the moved codes' sums and the moved zero points' cancel.  Exactly where they are
    whole numbers below 2^24; else up to the roundings (as many as at sum_bound) of sums of
    |s| (32 + code + zero) |x|.  A row whose codes differ in one column is that column's."""
    rng = np.random.default_rng(R + C)
    p = Packed(R, C, group, True, "fp32", R + C)
    cols = np.arange(C) // group
    q = p.z[:, cols].copy()
    q[3, C // 2] = (q[3, C // 2] + 5) % 16
    w3 = p.s64[3, C // 2 // group] * (q[3, C // 2] - p.z[3, C // 2 // group])
    full = np.zeros((R, C + (C & 1)), np.uint8)
    full[:, :C] = q
    p.codes = torch.from_numpy(full[:, 0::2] | (full[:, 1::2] << 4))
    h = p.build(dev)
    for n in (1, 5, 16, 20, 40):
        x = torch.from_numpy(rng.integers(-4, 5, (n, C))).to(F[x_dtype])
        y = h.run(x.to(dev), torch.full((n, R), float("nan"), device=dev), accumulate=False)
        y[:, 3] = 0
        assert (y == 0).all()
        x = torch.from_numpy(rng.standard_normal((n, C))).to(F[x_dtype])
        y = h.run(x.to(dev), y, accumulate=False).double().cpu().numpy()
        x = x.double().numpy()
        moved = p.s64[:, cols] * (32 + q + p.z[:, cols])
        tol = (C + C / 32 + 64) * 2.0 ** -24 * (np.abs(x) @ moved.T)
        y[:, 3] -= w3 * x[:, C // 2]
        assert np.all(np.abs(y) <= tol), np.max(np.abs(y) / tol)


@pytest.mark.parametrize("x_dtype", ["fp32", "fp16", "bf16"])
def test_product_infinities_and_nan(dev, x_dtype):
    """An infinity in x gives rows +-inf by its weight's sign, NaN where the weight is zero; a
    NaN gives NaN; the other vectors do not see them; nor do overflowing moved codes (31 * x)
    where the result is finite."""
    R, C = 50, 300
    p = Packed(R, C, 64, True, "fp32", 5, exact=True)
    rng = np.random.default_rng(2)
    x = rng.integers(-4, 5, (6, C)).astype(np.float64)
    big = float(torch.finfo(F[x_dtype]).max)
    x[1, 17] = np.inf
    x[2, 299] = -np.inf
    x[3, 64] = np.nan
    x[4, :] = 0
    x[4, 100] = big
    x[5, 3], x[5, 4] = np.inf, -np.inf
    q = p.build(dev)
    y = torch.zeros(6, R, device=dev)
    q.run(torch.from_numpy(x).to(F[x_dtype]).to(dev), y, accumulate=False)
    with np.errstate(all="ignore"):
        want = np.stack([(p.w * v).sum(1) for v in x])
        want = want.astype(np.float32).astype(np.float64)
    # (p.w * v) * s can pass fp32's range only in vector 4, as single products
    got = y.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(want))
    ok = ~np.isnan(want)
    assert np.array_equal(got[ok], want[ok])


@pytest.mark.parametrize("R", [4096, 4097, 5001, 8192, 8193, 9999, 16384, 16390])
def test_product_exact_over_heights(dev, R):
    """Whole numbers as in test_product_exact, over matrices of few and many row tiles, odd
    ones among them, for one vector up to several passes of them."""
    rng = np.random.default_rng(R)
    for C, group, zeros, dtype, n in ((300, 32, True, "fp32", 1), (131, 64, False, "bf16", 3),
                                      (640, 128, True, "fp16", 9), (1030, 32, False, "fp32", 5),
                                      (257, 32, True, "bf16", 40), (2100, 64, True, "fp32", 19)):
        p = Packed(R, C, group, zeros, "bf16", R + C, exact=True)
        x = rng.integers(-4, 5, (n, C)).astype(np.float64)
        y0 = rng.integers(-8, 9, (n, R)).astype(np.float64)
        y = torch.from_numpy(y0).float().to(dev)
        q = p.build(dev)
        q.run(torch.from_numpy(x).to(F[dtype]).to(dev), y)
        assert np.array_equal(y.double().cpu().numpy(), x @ p.w.T + y0), (C, dtype, n)
        q.close()


@pytest.mark.parametrize("n", [1, 20])
@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
def test_product_subnormal_vectors(dev, dtype, n):
    """Vectors of whole multiples (up to 100) of the type's smallest number keep their bits:
    in those units every sum is a whole number below 31 * 100 * 130 < 2^24, and for the wide
    types (smallest 2^-133, 2^-149) the scale of 2^4 keeps y among fp32's own numbers."""
    R, C = 70, 130
    unit = {"fp16": 2.0 ** -24, "bf16": 2.0 ** -133, "fp32": 2.0 ** -149}[dtype]
    p = Packed(R, C, 32, True, "fp32", 4, exact=True)
    p.scales = torch.full((R, p.G), 16.0)
    w = 16.0 * (p.q - p.z[:, np.arange(C) // 32])
    rng = np.random.default_rng(5)
    k = rng.integers(-100, 101, (n, C)).astype(np.float64)
    xt = torch.from_numpy(k * unit).to(F[dtype])
    assert np.array_equal(xt.double().numpy(), k * unit)
    q = p.build(dev)
    y = torch.full((n, R), float("nan"), device=dev)
    q.run(xt.to(dev), y, accumulate=False)
    assert np.array_equal(y.double().cpu().numpy(), (k @ w.T) * unit)


def test_product_nowhere_finite(dev):
    """Every result infinite or NaN, by one vector and by many."""
    p = Packed(300, 700, 64, True, "fp16", 6, exact=True)
    q = p.build(dev)
    for dtype in ("fp32", "fp16", "bf16"):
        for n in (1, 33):
            x = torch.ones(n, 700, dtype=F[dtype])
            x[:, 5], x[n // 2, 9] = float("inf"), float("nan")
            y = torch.zeros(n, 300, dtype=F[dtype], device=dev)
            q.run(x.to(dev), y)
            with np.errstate(all="ignore"):
                want = np.stack([(p.w * v).sum(1) for v in x.double().numpy()])
            assert np.array_equal(y.double().cpu().numpy(), want, equal_nan=True)


def test_product_strides_and_rows_behind(dev):
    """Row strides beyond the row, bases at odd elements; what lies between rows stays."""
    p = Packed(37, 301, 32, True, "fp16", 8, exact=True)
    q = p.build(dev)
    rng = np.random.default_rng(8)
    for dtype in ("fp32", "fp16", "bf16"):
        xb = torch.full((6, 311), float("nan"), dtype=F[dtype], device=dev)
        yb = torch.full((6, 45), 77.0, dtype=F[dtype], device=dev)
        xv = rng.integers(-4, 5, (6, 301)).astype(np.float64)
        xb[:, 3:304] = torch.from_numpy(xv).to(F[dtype]).to(dev)
        q.run(xb[:, 3:304], yb[:, 5:42], accumulate=False)
        want = torch.from_numpy(xv @ p.w.T).float().to(F[dtype])
        assert torch.equal(yb[:, 5:42].cpu(), want)
        assert (yb[:, :5] == 77).all() and (yb[:, 42:] == 77).all()
    # no vectors, and one-dimensional arguments
    e = torch.empty(0, 37, device=dev)
    assert q.run(torch.empty(0, 301, device=dev), e) is e
    x1 = torch.from_numpy(xv[2]).float().to(dev)
    y1 = q.run(x1, torch.ones(37, device=dev))
    assert np.array_equal(y1.cpu().numpy(), (p.w @ xv[2] + 1).astype(np.float32))


def test_product_workspace(dev):
    """Many vectors over few rows: the columns are split and the parts' sums meet in the
    workspace, given or allocated; it may hold anything before, and is needed whole."""
    p = Packed(90, 6000, 64, True, "bf16", 21, exact=True)
    q = p.build(dev)
    rng = np.random.default_rng(21)
    x = rng.integers(-4, 5, (40, 6000)).astype(np.float64)
    want = torch.from_numpy(x @ p.w.T).float()
    xt = torch.from_numpy(x).bfloat16().to(dev)
    assert q.run_workspace(1, torch.bfloat16) == 0
    need = q.run_workspace(40, torch.bfloat16)
    assert need >= 2 * 40 * 90 * 4
    ws = torch.full((need + 64,), 255, dtype=torch.uint8, device=dev)     # NaN as fp32
    for w in (ws, ws[16:], None):
        y = torch.full((40, 90), float("nan"), device=dev)
        q.run(xt, y, accumulate=False, workspace=w)
        assert torch.equal(y.cpu(), want)
    assert (ws[need + 16:] == 255).all()          # nothing behind what is needed
    for bad in (ws[:need - 1], ws[8:], ws.float(), ws[:0]):
        with pytest.raises((ValueError, TypeError)):
            q.run(xt, y, workspace=bad)
    side = torch.cuda.Stream()
    for _ in range(3):
        y = torch.zeros(40, 90, device=dev)
        torch.cuda.synchronize()
        q.run(xt, y, stream=side)
        junk = torch.full((need // 4,), 9.0, device=dev)      # would reuse a freed workspace
        torch.cuda.synchronize()
        assert torch.equal(y.cpu(), want)
        del junk


def test_empty_matrices(dev):
    for R, C in ((0, 64), (5, 0), (0, 0)):
        q = spmv.build_quant(torch.zeros(R, C, device=dev), group_size=32)
        y = torch.full((2, R), 3.0, device=dev)
        q.run(torch.zeros(2, C, device=dev), y)
        assert (y == 3).all()
        q.run(torch.zeros(2, C, device=dev), y, accumulate=False)
        assert (y == 0).all()
        out = q.lookup(torch.tensor([0, 1], device=dev))
        assert out.shape == (2, C) and (out == 0).all()
        assert q.array("codes").size == 0
        q.close()


# ------------------------------------------------------------------ builders

def quantise64(w, group, zeros, scale_dtype):
    """The builder's definition: fp32 scales, quotients rounded exactly (in 64 bits the
    quotient of two fp32 numbers lies on a half only if it is one)."""
    R, C = w.shape
    G = -(-C // group)
    q = np.zeros((R, C), np.int64)
    s = np.zeros((R, G), np.float32)
    z = np.full((R, G), 8, np.int64)
    for g in range(G):
        v = w[:, g * group:(g + 1) * group].astype(np.float32)
        lo, hi = np.minimum(v.min(1), 0), np.maximum(v.max(1), 0)
        sg = (hi - lo) / np.float32(15) if zeros else np.maximum(hi, -lo) / np.float32(7)
        sg = torch.from_numpy(sg).to(F[scale_dtype]).float().numpy()
        s[:, g] = sg
        safe = np.where(sg > 0, sg, 1).astype(np.float64)
        if zeros:
            z[:, g] = np.where(sg > 0, np.clip(np.rint(-lo.astype(np.float64) / safe), 0, 15), 0)
        k = np.where(sg[:, None] > 0, np.rint(v.astype(np.float64) / safe[:, None]), 0)
        q[:, g * group:(g + 1) * group] = np.clip(k + z[:, g:g + 1], 0, 15)
    return q, s, z


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("weight_dtype", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("R,C,group", [(1, 1, 32), (5, 33, 32), (17, 300, 64), (9, 1000, 128),
                                       (20, 513, 256), (3, 2000, 640)])
def test_build_matches_definition(dev, R, C, group, weight_dtype, zeros):
    rng = np.random.default_rng(C + R)
    w = rng.standard_normal((R, C)) * np.exp(rng.uniform(-8, 4, (R, 1)))
    w[0] = 0                                    # a row whose scales are zero
    if R > 4:
        w[1] = np.rint(w[1] * 3) / 2            # many ties
        w[2] = np.abs(w[2])
        w[3] = -np.abs(w[3])
    wt = torch.from_numpy(w).to(F[weight_dtype])
    for scale_dtype in ("fp32", "fp16", "bf16"):
        q = spmv.build_quant(wt.to(dev), group_size=group, zero_points=zeros,
                             scale_dtype=F[scale_dtype])
        codes, s, z = quantise64(wt.float().numpy(), group, zeros, scale_dtype)
        full = np.zeros((R, C + (C & 1)), np.int64)
        full[:, :C] = codes
        assert np.array_equal(q.array("codes"), (full[:, 0::2] | full[:, 1::2] << 4))
        assert np.array_equal(q.array("scales"), s)
        if zeros:
            assert np.array_equal(q.array("zero_points"), z)
        else:
            assert q.array("zero_points").size == 0
        assert q.info["num_groups"] == -(-C // group)
        q.close()


def test_build_strided_weights_and_packed_round_trip(dev):
    w = torch.randn(21, 400, device=dev)
    q = spmv.build_quant(w[:, 7:300], group_size=64, zero_points=True, scale_dtype=torch.bfloat16)
    q2 = spmv.build_quant(w[:, 7:300].contiguous(), group_size=64, zero_points=True,
                          scale_dtype=torch.bfloat16)
    for name in ("codes", "scales", "zero_points"):
        assert np.array_equal(q.array(name), q2.array(name))
    q3 = spmv.build_quant_packed(torch.from_numpy(q.array("codes")).to(dev),
                                 torch.from_numpy(q.array("scales")).bfloat16().to(dev), 293,
                                 group_size=64,
                                 zero_points=torch.from_numpy(q.array("zero_points")).to(dev))
    for name in ("codes", "scales", "zero_points"):
        assert np.array_equal(q.array(name), q3.array(name))


def test_build_refuses_bad_values(dev):
    for bad in (float("nan"), float("inf"), float("-inf")):
        w = torch.randn(9, 200, device=dev)
        w[8, 199] = bad
        with pytest.raises(spmv.SpmvError) as e:
            spmv.build_quant(w, group_size=32)
        assert e.value.name == "SPMV_ERR_BAD_VALUE"
    w = torch.full((2, 64), 1e6, device=dev)      # 1e6 / 7 > 65504
    with pytest.raises(spmv.SpmvError):
        spmv.build_quant(w, group_size=64, scale_dtype=torch.float16)
    assert spmv.build_quant(w, group_size=64, scale_dtype=torch.bfloat16).num_rows == 2
    w[0, 0], w[0, 1] = 3e38, -3e38                # hi - lo passes fp32's range
    with pytest.raises(spmv.SpmvError):
        spmv.build_quant(w, group_size=64, zero_points=True)
    codes = torch.zeros(2, 32, dtype=torch.uint8, device=dev)
    s = torch.ones(2, 2, device=dev)
    z = torch.tensor([[0, 15], [16, 3]], dtype=torch.uint8, device=dev)
    with pytest.raises(spmv.SpmvError) as e:
        spmv.build_quant_packed(codes, s, 64, group_size=32, zero_points=z)
    assert e.value.name == "SPMV_ERR_BAD_VALUE"
    kept = spmv.build_quant_packed(codes, s, 64, group_size=32, zero_points=z, validate=False)
    assert kept.array("zero_points").tolist() == [[0, 15], [0, 3]]
    s[1, 0] = float("inf")
    with pytest.raises(spmv.SpmvError):
        spmv.build_quant_packed(codes, s, 64, group_size=32)


def test_binding_refusals(dev):
    p = Packed(10, 64, 32, False, "fp32", 1)
    q = p.build(dev)
    x, y = torch.zeros(2, 64, device=dev), torch.zeros(2, 10, device=dev)
    with pytest.raises(ValueError):
        q.run(x[:, :63], y)
    with pytest.raises(ValueError):
        q.run(x[:1], y)
    with pytest.raises(TypeError):
        q.run(x.half(), y.bfloat16())
    with pytest.raises(TypeError):
        q.run(x.double(), y)
    with pytest.raises(ValueError):
        q.run(x.t().contiguous().t(), y)
    with pytest.raises(ValueError):
        q.run(x[:1].expand(2, 64), y[:1].expand(2, 10))   # rows of y on one another
    buf = torch.zeros(2, 64, device=dev)
    with pytest.raises(ValueError):
        q.run(buf, buf[:, :10])
    with pytest.raises(TypeError):
        q.lookup(torch.zeros(3, device=dev))
    with pytest.raises(ValueError):
        q.lookup(torch.zeros(3, dtype=torch.int64, device=dev), torch.zeros(3, 63, device=dev))
    with pytest.raises(TypeError):
        q.lookup(torch.zeros(3, dtype=torch.int64, device=dev), torch.zeros(3, 64, device=dev),
                 dtype=torch.float16)
    with pytest.raises(ValueError):
        spmv.build_quant_packed(p.codes.to(dev), p.scales.to(dev), 63, group_size=64)
    with pytest.raises(spmv.SpmvError):
        spmv.build_quant(torch.zeros(4, 64, device=dev), group_size=48)
    ids = torch.zeros(4, dtype=torch.int32, device=dev)
    g = torch.zeros(4, 8, device=dev)
    with pytest.raises(ValueError):
        spmv.lookup_grad(g[:3], ids, 5)
    with pytest.raises(ValueError):
        spmv.lookup_grad(g, ids, 5, accumulate=True)
    with pytest.raises(ValueError):
        spmv.lookup_grad(g, ids, 5, torch.zeros(4, 8, device=dev))
    with pytest.raises(ValueError):
        spmv.lookup_grad(g, ids, 5, workspace=torch.zeros(8, dtype=torch.uint8, device=dev))
    with pytest.raises(ValueError):
        spmv.lookup_grad(g, ids, 4, g)
    with pytest.raises(TypeError):
        spmv.lookup_grad(g, ids.float(), 5)
    with pytest.raises(ValueError):
        spmv.lookup(g, ids[::2])
    with pytest.raises(ValueError):
        spmv.lookup(g, ids, g)
    q.close()
    with pytest.raises(RuntimeError):
        q.run(x, y)


def test_binding_refuses_what_is_no_tensor(dev):
    """Outputs and workspaces that are no cuda tensors are of a wrong type, as inputs are."""
    p = Packed(90, 6000, 64, True, "bf16", 21)
    q = p.build(dev)
    x = torch.zeros(40, 6000, dtype=torch.bfloat16, device=dev)
    y = torch.zeros(40, 90, device=dev)
    ids = torch.zeros(4, dtype=torch.int32, device=dev)
    g = torch.zeros(4, 8, device=dev)
    need = spmv.lookup_grad_workspace(4, 5, 8)
    for call in (lambda: q.run(x, y, workspace=bytearray(1 << 20)),
                 lambda: q.run(x, y, workspace=torch.zeros(1 << 20, dtype=torch.uint8)),
                 lambda: q.run(x, y.cpu()),
                 lambda: q.run(x, None),
                 lambda: spmv.lookup_grad(g, ids, 5, [0.0], dtype=torch.float32),
                 lambda: spmv.lookup_grad(g, ids, 5, torch.zeros(5, 8)),
                 lambda: spmv.lookup_grad(g, ids, 5, workspace=bytearray(need)),
                 lambda: spmv.lookup_grad(g, None, 5),
                 lambda: spmv.lookup(g, [0, 1])):
        with pytest.raises(TypeError):
            call()


def test_binding_refuses_sizes_beyond_int32(dev):
    """2^32 + 5 rows, which an int32 argument would take for 5."""
    wrap = 2 ** 32 + 5
    q = Packed(10, 64, 32, False, "fp32", 1).build(dev)
    ids = torch.zeros(3, dtype=torch.int64, device=dev)
    one = torch.zeros(1, dtype=torch.bfloat16, device=dev)
    many = one.as_strided((wrap, 1), (0, 1))
    for call in (lambda: spmv.lookup(many, ids),
                 lambda: spmv.lookup_grad(torch.zeros(3, 1, device=dev), ids, wrap),
                 lambda: spmv.build_quant(many),
                 lambda: q.run_workspace(wrap, torch.float32)):
        with pytest.raises(spmv.SpmvError) as e:
            call()
        assert e.value.name == "SPMV_ERR_TOO_LARGE"


# ------------------------------------------------------------------- lookups

IDS = {"int32": torch.int32, "int64": torch.int64}


def some_ids(rng, V, n, dtype):
    """Rows of [0, V) with repeats, the first and last, and some that name no row."""
    ids = rng.integers(0, max(V, 1), n)
    if n > 5:
        ids[0], ids[1], ids[2], ids[3] = V - 1, -1, V, 0
        ids[4] = np.iinfo(np.int32).min if dtype == "int32" else np.iinfo(np.int64).max
    return torch.from_numpy(ids).to(IDS[dtype])


@pytest.mark.parametrize("ids_dtype", ["int32", "int64"])
@pytest.mark.parametrize("V,D,n", [(1, 1, 1), (5, 3, 9), (100, 8, 64), (1000, 100, 33),
                                   (77, 2048, 50), (300, 1001, 500), (50, 12345, 7)])
def test_lookup_is_the_rounded_product(dev, V, D, n, ids_dtype):
    rng = np.random.default_rng(V + D)
    for a in ("fp32", "fp16", "bf16"):
        for b in ("fp32", "fp16", "bf16"):
            table = torch.from_numpy(rng.standard_normal((V, D))).to(F[a])
            ids = some_ids(rng, V, n, ids_dtype)
            scale = 1.0 if a == b else 22.627417
            got = spmv.lookup(table.to(dev), ids.to(dev), scale=scale, dtype=F[b]).cpu()
            ok = (ids >= 0) & (ids.long() < V)
            rows = table[ids.long().clamp(0, V - 1)].float() * torch.tensor(scale)
            want = torch.where(ok[:, None], rows, 0.0).to(F[b])
            assert torch.equal(got, want), (a, b)


@pytest.mark.parametrize("R,C,group,n", [(1, 1, 32, 1), (40, 31, 32, 9), (33, 256, 64, 40),
                                         (100, 1000, 128, 65), (20, 2750, 384, 30)])
def test_quant_lookup_is_the_rounded_product(dev, R, C, group, n):
    rng = np.random.default_rng(R * 3 + C)
    for zeros, sd, out, idd in ((False, "bf16", "bf16", "int64"), (True, "fp16", "fp32", "int32"),
                                (True, "fp32", "fp16", "int64"), (False, "fp32", "fp32", "int32")):
        p = Packed(R, C, group, zeros, sd, R + C)
        q = p.build(dev)
        ids = some_ids(rng, R, n, idd)
        got = q.lookup(ids.to(dev), scale=5.5, dtype=F[out]).cpu()
        c = np.arange(C) // group
        w = (torch.from_numpy((p.q - p.z[:, c]).astype(np.float32))
             * p.scales.float()[:, torch.from_numpy(c)]) * torch.tensor(5.5)
        ok = (ids >= 0) & (ids.long() < R)
        want = torch.where(ok[:, None], w[ids.long().clamp(0, R - 1)], 0.0).to(F[out])
        assert torch.equal(got, want), (zeros, sd, out)


def test_lookup_shapes_strides_and_rows_behind(dev):
    table = torch.randn(50, 90, device=dev)[:, 5:82]
    ids = torch.randint(0, 50, (3, 4), device=dev)
    out = spmv.lookup(table, ids)
    assert out.shape == (3, 4, 77)
    assert torch.equal(out, table[ids])
    buf = torch.full((14, 80), 9.0, device=dev)
    spmv.lookup(table, ids.view(-1), buf[1:13, 1:78])
    assert torch.equal(buf[1:13, 1:78], table[ids.view(-1)])
    assert (buf[0] == 9).all() and (buf[13] == 9).all()
    assert (buf[:, 0] == 9).all() and (buf[:, 78:] == 9).all()
    assert spmv.lookup(table, ids[:0]).shape == (0, 4, 77)
    assert spmv.lookup(table[:, :0], ids).shape == (3, 4, 0)
    assert (spmv.lookup(table[:0], ids) == 0).all()
    one = torch.tensor(7, device=dev)              # a scalar token
    assert torch.equal(spmv.lookup(table, one), table[7])


def test_lookup_padding_ignores_the_table(dev):
    """A padded position is zero whatever the rows hold (no product with them)."""
    table = torch.full((4, 40), float("nan"), device=dev)
    ids = torch.tensor([-1, 4, 2], device=dev)
    out = spmv.lookup(table, ids)
    assert (out[:2] == 0).all() and out[2].isnan().all()


# ------------------------------------------------------------------ gradient

def grad64(g, ids, V, scale):
    out = np.zeros((V, g.shape[1]))
    mag = np.zeros((V, g.shape[1]))
    cnt = np.zeros(V)
    for t, v in enumerate(ids):
        if 0 <= v < V:
            out[v] += g[t]
            mag[v] += np.abs(g[t])
            cnt[v] += 1
    return out * scale, mag * abs(scale), cnt


def skewed_ids(rng, V, n, kind):
    if kind == "uniform":
        return rng.integers(0, V, n)
    if kind == "one":
        return np.full(n, V // 2)
    if kind == "none":
        return np.full(n, -1)
    if kind == "runs":                           # long runs next to single tokens
        ids = rng.integers(0, V, n)
        ids[: n // 2] = V - 1
        ids[n // 2: n // 2 + n // 4] = 0
        return rng.permutation(ids)
    ids = (V ** rng.random(n)).astype(np.int64) - 1     # frequency ~ 1 / rank
    ids[rng.random(n) < 0.1] = -1
    ids[rng.random(n) < 0.05] = V
    return ids


@pytest.mark.parametrize("kind", ["uniform", "one", "none", "runs", "language"])
@pytest.mark.parametrize("V,D,n", [(1, 1, 1), (3, 5, 31), (40, 8, 32), (10, 64, 33),
                                   (1000, 100, 257), (5000, 33, 4096), (700, 16, 4097),
                                   (70000, 9, 9000), (300, 2500, 700)])
def test_gradient_exact(dev, V, D, n, kind):
    """Whole numbers |g| <= 8, so a sum of n <= 2^16 of them is exact in fp32; scale 0.5."""
    rng = np.random.default_rng(V + D + n)
    ids = skewed_ids(rng, V, n, kind)
    g = rng.integers(-8, 9, (n, D)).astype(np.float64)
    want, _, cnt = grad64(g, ids, V, 0.5)
    for gd, od, idd, acc in (("fp32", "fp32", "int64", False), ("bf16", "fp32", "int32", True),
                             ("fp16", "fp16", "int64", True), ("bf16", "bf16", "int32", False)):
        gt = torch.from_numpy(g).to(F[gd]).to(dev)
        it = torch.from_numpy(ids).to(IDS[idd]).to(dev)
        base = torch.full((V, D), 3.0, dtype=F[od], device=dev)
        if not acc:
            base.fill_(float("nan"))
        out = spmv.lookup_grad(gt, it, V, base, scale=0.5, accumulate=acc)
        assert out is base
        w = torch.from_numpy(want + (3.0 if acc else 0.0)).float().to(F[od])
        assert torch.equal(out.cpu(), w), (gd, od, idd, acc)


@pytest.mark.parametrize("V,D,n,kind", [(50, 300, 3000, "language"), (9, 40, 5000, "uniform"),
                                        (2000, 70, 20000, "language"), (3, 130, 70000, "runs")])
def test_gradient_random(dev, V, D, n, kind):
    """Each row's sum of m gradients takes m + 2 roundings (its additions, the scaling) of at
    most 2^-24 of the sum of sizes, in whatever parts it is taken; then the output's half step."""
    rng = np.random.default_rng(n)
    ids = skewed_ids(rng, V, n, kind)
    for gd, od in (("fp32", "fp32"), ("bf16", "fp32"), ("fp16", "fp16"), ("bf16", "bf16")):
        gt = torch.from_numpy(rng.standard_normal((n, D))).to(F[gd])
        want, mag, cnt = grad64(gt.double().numpy(), ids, V, 1.25)
        it = torch.from_numpy(ids).to(dev)
        out = spmv.lookup_grad(gt.to(dev), it, V, scale=1.25, dtype=F[od])
        got = out.double().cpu().numpy()
        tol = (cnt[:, None] + 2) * 2.0 ** -24 * mag
        if od != "fp32":
            tol = tol + half_step(F[od]) * (np.abs(want) + tol) + 2.0 ** -24
        assert np.all(np.abs(got - want) <= tol), (gd, od)
        again = spmv.lookup_grad(gt.to(dev), it, V, scale=1.25, dtype=F[od])
        assert torch.equal(again, out)          # the same from run to run


@pytest.mark.parametrize("V,D,n", [(9, 40, 500), (50, 301, 3000), (2000, 70, 20000),
                                   (700, 12, 70000)])
def test_gradient_order_does_not_depend_on_types_or_strides(dev, V, D, n):
    """Values that all three types hold, whose fp32 sums are rounded: the sums are equal bit for
    bit whatever the types of gradients and ids, the strides, and what the workspace held."""
    rng = np.random.default_rng(n)
    h = skewed_ids(rng, V, n, "language")
    ids = torch.from_numpy(h).to(dev)
    # 8 bits, exponents far apart: in bf16, fp16 (2^-14 and above) and fp32 alike
    g = (rng.integers(128, 256, (n, D)) * 2.0 ** rng.integers(-21, 5, (n, D))
         * rng.choice([-1, 1], (n, D)))
    first = spmv.lookup_grad(torch.from_numpy(g).float().to(dev), ids, V)
    want, mag, cnt = grad64(g, h, V, 1.0)
    assert np.all(np.abs(first.double().cpu().numpy() - want)
                  <= (cnt[:, None] + 2) * 2.0 ** -24 * mag)
    need = spmv.lookup_grad_workspace(n, V, D)
    for gd, idd, fill, pad in (("fp16", "int32", 255, 0), ("bf16", "int64", 1, 3),
                               ("fp32", "int32", 7, 5)):
        buf = torch.zeros(n, D + 2 * pad, dtype=F[gd], device=dev)
        gt = buf[:, pad:pad + D]
        gt.copy_(torch.from_numpy(g))
        assert torch.equal(gt.double().cpu(), torch.from_numpy(g))
        out = torch.empty(V, D + pad, device=dev)[:, :D]
        ws = torch.full((need,), fill, dtype=torch.uint8, device=dev)
        spmv.lookup_grad(gt, ids.to(IDS[idd]), V, out, workspace=ws)
        assert torch.equal(out, first), gd


def test_gradient_many_tokens_and_large_tables(dev):
    """Merged tiles up to 65,536 tokens (16,384 for up to 1023 rows); radix passes beyond, in
    one segment of tiles and in several; three passes with 2^20 + 1 rows and more; ids at the
    top of the range."""
    rng = np.random.default_rng(0)
    for V, D, n in ((2 ** 20 + 1, 4, 150_000), (2 ** 21, 3, 50_000), (131072, 8, 300_001),
                    (70, 2, 16_384), (70, 2, 16_385), (1023, 2, 20_000), (1024, 2, 20_000),
                    (5000, 2, 65_536), (5000, 2, 65_537), (2 ** 25, 1, 1_000_000)):
        ids = skewed_ids(rng, V, n, "language")
        ids[::7] = V - 1
        g = rng.integers(-4, 5, (n, D)).astype(np.float32)
        want = np.zeros((V, D))
        ok = (ids >= 0) & (ids < V)
        np.add.at(want, ids[ok], g[ok])
        out = spmv.lookup_grad(torch.from_numpy(g).to(dev), torch.from_numpy(ids).to(dev), V)
        assert np.array_equal(out.cpu().numpy(), want.astype(np.float32))


def test_gradient_strides_shapes_and_untouched_rows(dev):
    rng = np.random.default_rng(4)
    ids = torch.from_numpy(rng.integers(0, 30, (4, 25))).to(dev)
    buf = torch.from_numpy(rng.integers(-8, 9, (100, 50)).astype(np.float32)).to(dev)
    g = buf[:, 3:40]
    want, _, cnt = grad64(g.double().cpu().numpy(), ids.view(-1).tolist(), 33, 1.0)
    ob = torch.full((33, 41), 5.0, device=dev)
    spmv.lookup_grad(g, ids.view(-1), 33, ob[:, 2:39])
    assert np.array_equal(ob[:, 2:39].cpu().numpy(), want.astype(np.float32))
    assert (ob[:, :2] == 5).all() and (ob[:, 39:] == 5).all()
    # three-dimensional, as a batch has it
    out = spmv.lookup_grad(g.contiguous().view(4, 25, 37), ids, 33)
    assert np.array_equal(out.cpu().numpy(), want.astype(np.float32))
    # accumulate leaves rows without tokens untouched, NaN among them
    base = torch.full((33, 37), float("nan"), device=dev)
    hit = torch.from_numpy(cnt > 0).to(dev)
    base[hit] = 1.0
    spmv.lookup_grad(g, ids.view(-1), 33, base, accumulate=True)
    assert base[~hit].isnan().all()
    assert np.array_equal(base[hit].cpu().numpy(), (want[cnt > 0] + 1).astype(np.float32))
    # no tokens
    none = torch.empty(0, dtype=torch.int64, device=dev)
    z = spmv.lookup_grad(torch.empty(0, 6, device=dev), none, 4)
    assert z.shape == (4, 6) and (z == 0).all()
    keep = torch.ones(4, 6, device=dev)
    spmv.lookup_grad(torch.empty(0, 6, device=dev), none, 4, keep, accumulate=True)
    assert (keep == 1).all()


def test_gradient_padding_ignores_its_rows(dev):
    """Gradients of padded positions may hold anything."""
    g = torch.ones(6, 20, device=dev)
    ids = torch.tensor([2, -1, 0, 5, 2, 9], device=dev)
    g[1], g[5] = float("nan"), float("inf")
    out = spmv.lookup_grad(g, ids, 6)
    assert out[:, 0].tolist() == [1, 0, 2, 0, 0, 1]


def test_gradient_is_the_difference_of_the_lookup(dev):
    """L(table) = sum(r * lookup(table)) is linear: with whole numbers a step of 1 in one
    weight changes L by exactly the gradient there."""
    rng = np.random.default_rng(6)
    V, D, n = 7, 5, 40
    table = torch.from_numpy(rng.integers(-9, 10, (V, D)).astype(np.float32)).to(dev)
    ids = torch.from_numpy(rng.integers(-1, V, n)).to(dev)
    r = torch.from_numpy(rng.integers(-9, 10, (n, D)).astype(np.float32)).to(dev)

    def loss(t):
        return (spmv.lookup(t, ids, scale=4.0).double() * r.double()).sum().item()

    d = spmv.lookup_grad(r, ids, V, scale=4.0).cpu()
    for v in range(V):
        for c in range(D):
            step = table.clone()
            step[v, c] += 1
            assert loss(step) - loss(table) == d[v, c].item()


# ------------------------------------------------- together, streams, graphs

def token_step(table, q, ids, y, out, ws):
    """One step as a program runs it: rows in, logits out, the loss's gradient at the rows
    (a fixed linear head here), and the table's gradient."""
    rows = spmv.lookup(table, ids, scale=2.0)
    q.run(rows, y, accumulate=False)
    back = rows.mul(0.5)
    spmv.lookup_grad(back, ids, table.shape[0], out, workspace=ws)
    return rows


def test_token_step_together(dev):
    """Lookup, 4-bit logits and gradient in one run, against 64 bits."""
    rng = np.random.default_rng(12)
    V, D, n = 400, 96, 50
    p = Packed(V, D, 32, True, "fp16", 12, exact=True)
    q = p.build(dev)
    table = torch.from_numpy(rng.integers(-2, 3, (V, D)).astype(np.float32)).to(dev)
    ids_h = skewed_ids(rng, V, n, "language")
    ids = torch.from_numpy(ids_h).to(dev)
    y, out = torch.empty(n, V, device=dev), torch.empty(V, D, device=dev)
    ws = torch.empty(spmv.lookup_grad_workspace(n, V, D), dtype=torch.uint8, device=dev)
    rows = token_step(table, q, ids, y, out, ws)
    ok = (ids_h >= 0) & (ids_h < V)
    r = np.where(ok[:, None], table.double().cpu().numpy()[np.clip(ids_h, 0, V - 1)] * 2, 0)
    assert np.array_equal(rows.cpu().numpy(), r)
    assert np.array_equal(y.cpu().numpy(), (r @ p.w.T).astype(np.float32))
    want, _, _ = grad64(r * 0.5, ids_h, V, 1.0)
    assert np.array_equal(out.cpu().numpy(), want.astype(np.float32))
    # the tied 4-bit table's rows
    got = q.lookup(ids, scale=1.0)
    want = np.where(ok[:, None], p.w[np.clip(ids_h, 0, V - 1)], 0)
    assert np.array_equal(got.cpu().numpy(), want)


def test_step_captured_and_replayed(dev):
    """Two graphs of the same step (many tokens and few), replayed in turn with eager work
    between; every replay equals the eager result on its inputs."""
    rng = np.random.default_rng(13)
    V, D = 3000, 72
    p = Packed(V, D, 32, False, "bf16", 13, exact=True)
    q = p.build(dev)
    table = torch.from_numpy(rng.integers(-2, 3, (V, D)).astype(np.float32)).to(dev)
    sets = []
    for n in (6000, 40):
        ids = torch.from_numpy(skewed_ids(rng, V, n, "language")).to(dev)
        y, out = torch.empty(n, V, device=dev), torch.empty(V, D, device=dev)
        ws = torch.empty(spmv.lookup_grad_workspace(n, V, D), dtype=torch.uint8, device=dev)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            token_step(table, q, ids, y, out, ws)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            rows = token_step(table, q, ids, y, out, ws)
        sets.append((n, ids, y, out, graph, rows))
    for turn in range(3):
        for n, ids, y, out, graph, rows in sets:
            ids.copy_(torch.from_numpy(skewed_ids(rng, V, n, "language")).to(dev))
            y.fill_(float("nan"))
            out.fill_(float("nan"))
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            y2, out2 = torch.empty_like(y), torch.empty_like(out)
            ws = torch.empty(spmv.lookup_grad_workspace(n, V, D), dtype=torch.uint8, device=dev)
            r2 = token_step(table, q, ids, y2, out2, ws)
            assert torch.equal(rows, r2) and torch.equal(y, y2) and torch.equal(out, out2)


def test_split_products_captured_and_at_once(dev):
    """Products whose columns are split: two streams at once with workspaces of their own, and
    two graphs with theirs (one allocated while it is captured), replayed in turn with eager
    products between."""
    rng = np.random.default_rng(31)
    p = Packed(150, 9000, 128, True, "bf16", 31, exact=True)
    q = p.build(dev)
    assert q.run_workspace(24, torch.bfloat16) > 0
    xs = [torch.empty(24, 9000, dtype=torch.bfloat16, device=dev) for _ in range(2)]
    ys = [torch.empty(24, 150, device=dev) for _ in range(2)]
    ws = [torch.empty(q.run_workspace(24, torch.bfloat16), dtype=torch.uint8, device=dev), None]

    def renew():
        want = []
        for x, y in zip(xs, ys):
            v = rng.integers(-4, 5, (24, 9000)).astype(np.float64)
            x.copy_(torch.from_numpy(v))
            y.fill_(float("nan"))
            want.append(torch.from_numpy(v @ p.w.T).float().to(dev))
        torch.cuda.synchronize()
        return want

    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        want = renew()
        for x, y, w, s in zip(xs, ys, ws, streams):
            q.run(x, y, accumulate=False, workspace=w, stream=s)
        torch.cuda.synchronize()
        assert all(torch.equal(y, w) for y, w in zip(ys, want))
    graphs = []
    for x, y, w in zip(xs, ys, ws):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            q.run(x, y, accumulate=False, workspace=w)
        graphs.append(g)
    for _ in range(3):
        want = renew()
        for g in graphs:
            g.replay()
            eager = torch.zeros(24, 150, device=dev)
            q.run(xs[0], eager)
            torch.cuda.synchronize()
            assert torch.equal(eager, want[0])
        assert all(torch.equal(y, w) for y, w in zip(ys, want))


def test_gradient_of_many_tokens_captured(dev):
    """The sort's passes over several segments of tiles, replayed on other tokens."""
    rng = np.random.default_rng(32)
    V, D, n = 60_000, 3, 300_000
    ids = torch.empty(n, dtype=torch.int64, device=dev)
    g = torch.from_numpy(rng.integers(-3, 4, (n, D)).astype(np.float32)).to(dev)
    out = torch.empty(V, D, device=dev)
    ws = torch.empty(spmv.lookup_grad_workspace(n, V, D), dtype=torch.uint8, device=dev)
    ids.copy_(torch.from_numpy(rng.integers(0, V, n)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        spmv.lookup_grad(g, ids, V, out, workspace=ws)
    for kind in ("uniform", "language", "runs"):
        h = skewed_ids(rng, V, n, kind)
        ids.copy_(torch.from_numpy(h))
        out.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        ok = (h >= 0) & (h < V)
        want = np.zeros((V, D))
        np.add.at(want, h[ok], g.double().cpu().numpy()[ok])
        assert np.array_equal(out.double().cpu().numpy(), want)
        assert torch.equal(spmv.lookup_grad(g, ids, V), out)


def test_streams(dev):
    """Two steps at once on streams of their own, given as streams and as raw handles; the
    memory that a call allocates for itself lives until its work is done."""
    rng = np.random.default_rng(14)
    V, D, n = 5000, 200, 6000
    g = torch.from_numpy(rng.integers(-8, 9, (n, D)).astype(np.float32)).to(dev)
    ids = [torch.from_numpy(skewed_ids(rng, V, n, k)).to(dev) for k in ("language", "runs")]
    want = [spmv.lookup_grad(g, i, V) for i in ids]
    rows = [spmv.lookup(w, i) for w, i in zip(want, ids)]
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        got = [spmv.lookup_grad(g, ids[0], V, stream=a),
               spmv.lookup_grad(g, ids[1], V, stream=b.cuda_stream)]
        junk = torch.full((4 * n * D,), 7.0, device=dev)     # reuses freed memory, if any
        back = [spmv.lookup(want[0], ids[0], stream=b), spmv.lookup(want[1], ids[1], stream=a)]
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert torch.equal(back[0], rows[0]) and torch.equal(back[1], rows[1])
        del junk


def test_handles_free_their_memory(dev):
    w = torch.randn(2000, 2000, device=dev)
    spmv.build_quant(w).close()
    torch.cuda.synchronize()
    free0, _ = torch.cuda.mem_get_info()
    for _ in range(10):
        with spmv.build_quant(w, zero_points=True) as q:
            assert q.info["device_bytes"] >= 2000 * 1000
    torch.cuda.synchronize()
    assert torch.cuda.mem_get_info()[0] == free0


def test_long_offsets(dev):
    """Rows whose bytes and elements lie past 2^31 and 2^32: the last rows of a table, of the
    outputs and of the gradients."""
    V, D = 1_100_000, 4096                       # 4.5e9 elements of bf16, 9 GB
    table = torch.empty(V, D, dtype=torch.bfloat16, device=dev)
    for r in range(0, V, 100_000):
        table[r:r + 100_000] = torch.arange(r, min(V, r + 100_000), device=dev)[:, None] % 251
    ids = torch.tensor([V - 1, 0, V - 2, 524_288, 1_048_577], device=dev)
    out = spmv.lookup(table, ids)
    assert out[:, 0].tolist() == [float(int(i) % 251) for i in ids]
    assert (out == out[:, :1]).all()
    back = spmv.lookup_grad(out, ids, V, table)   # every row written, most of them zero
    assert back is table
    assert torch.equal(table[ids], out)
    table[ids] = 0
    for r in range(0, V, 100_000):
        assert not table[r:r + 100_000].any()
    del table, back
    torch.cuda.empty_cache()
    # many tokens: the last output rows and gradient rows lie past 2^32 elements
    n, D = 1_050_000, 4100
    t = torch.arange(97, device=dev)[:, None].expand(97, D).to(torch.bfloat16).contiguous()
    ids = torch.arange(n, device=dev, dtype=torch.int32) % 97
    rows = spmv.lookup(t, ids)
    assert torch.equal(rows[-500:], t[ids[-500:].long()])
    d = spmv.lookup_grad(rows, ids, 97, dtype=torch.float32)
    cnt = torch.bincount(ids.long(), minlength=97)
    assert torch.equal(d[:, 0].double(), cnt.double() * torch.arange(97, device=dev))
    assert (d == d[:, :1]).all()


def test_quant_long_offsets(dev):
    """A 4-bit matrix whose words pass 2^31 bytes and whose rows' codes pass 2^32 of them."""
    R, C = 1_100_000, 4096
    codes = torch.empty(R, C // 2, dtype=torch.uint8, device=dev)
    for r in range(0, R, 100_000):
        codes[r:r + 100_000] = ((torch.arange(r, min(R, r + 100_000), device=dev) % 16) * 17
                                ).to(torch.uint8)[:, None]
    scales = torch.ones(R, C // 128, dtype=torch.bfloat16, device=dev)
    q = spmv.build_quant_packed(codes, scales, C)
    x = torch.ones(1, C, dtype=torch.bfloat16, device=dev)
    y = q.run(x, torch.empty(1, R, device=dev), accumulate=False)
    want = (torch.arange(R, device=dev) % 16 - 8).float() * C
    assert torch.equal(y[0], want)
    ids = torch.tensor([R - 1, 524_289, 0], device=dev)
    assert torch.equal(q.lookup(ids)[:, 7], want[ids] / C)
