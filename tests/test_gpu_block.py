"""The operators of include/moe_block.h on the GPU against float64 references
(tests/block_ref.py).

Tolerances are worst-case bounds of the kernels' float32 arithmetic, derived
from the formulas: half a step of the output type relative to the value (bf16
2^-8, f16 2^-11, f32 2^-24), plus a count of float32 roundings times 2^-24 times
the size of the terms that are added.  Outputs lie between guard bytes that
have to survive.
"""

from __future__ import annotations

import ctypes

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import block_ref as ref  # noqa: E402
import w4_dequant_expert_amd as moe  # noqa: E402

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
GUARD = 256
E32 = ref.EPS32


class Out:
    """Output buffers with guard bytes on both sides, filled with a pattern."""

    def __init__(self):
        self.bufs = []

    def __call__(self, shape, dtype):
        n = int(np.prod(shape)) * torch.empty((), dtype=dtype).element_size()
        raw = torch.full((n + 2 * GUARD,), 0x5A, dtype=torch.uint8, device="cuda")
        self.bufs.append((raw, n))
        return raw[GUARD:GUARD + n].view(dtype).view(shape)

    def check(self):
        torch.cuda.synchronize()
        for raw, n in self.bufs:
            assert bool((raw[:GUARD] == 0x5A).all()) and bool((raw[GUARD + n:] == 0x5A).all()), \
                "a kernel wrote outside an output"


def rows_of(rng, shape, typ, scale=1.0):
    """Device rows of a type and the values they hold, in float64."""
    t = torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(TYPES[typ])
    return t.cuda(), t.double().numpy()


def f64(t):
    return t.double().cpu().numpy()


def f32(rng, shape, lo=0.5, hi=1.5):
    a = rng.uniform(lo, hi, shape).astype(np.float32)
    return torch.from_numpy(a).cuda(), a


def within(got, want, bound, what):
    err = np.abs(got - want)
    bad = ~(err <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} outside; worst error "
                           f"{float(np.nanmax(err[bad])):.3e} against {float(bound[bad].min()) if np.ndim(bound) else bound:.3e}")


def tiny(typ):
    """Half the smallest step of the type's subnormal range."""
    return 2.0 ** -25 if typ == "f16" else 2.0 ** -134


# ----------------------------------------------------------------------------------- the norm

# one wave, four and sixteen waves a row; rows that do not fill the last lane; one element group
NORM_SIZES = [(1, 8), (3, 64), (8, 2048), (9, 2048), (1, 2048), (5, 2040), (2049, 520), (2050, 2048), (7, 2056), (3, 4096),
              (2, 8192), (2, 8200), (3, 16384), (333, 1032)]


@pytest.mark.parametrize("typ", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,H", NORM_SIZES)
def test_norm(T, H, typ):
    print(f"norm {T} {H} {typ}", flush=True)
    rng = np.random.default_rng(T * 7 + H)
    x, xv = rows_of(rng, (T, H), typ)
    r, rv = rows_of(rng, (T, H), typ, 2.0)
    w, wv = f32(rng, H)
    eps = 1e-5
    d = moe.NormDims(T, H, moe.ELEM[TYPES[typ]], eps)
    out = Out()
    s, y = out((T, H), TYPES[typ]), out((T, H), TYPES[typ])
    q, qs = out((T, H), torch.int8), out((T,), torch.float32)
    moe.moe_add_rmsnorm(d, x, r, w, s, y, q, qs)
    out.check()
    sv, yv = ref.norm(xv, rv, wv, np.float32(eps))
    u = ref.HALF_STEP[typ]
    within(f64(s), sv, (u + E32) * np.abs(sv) * (1 + 1e-6) + tiny(typ), "sum")
    # rho: a sum of squares of at most 32 terms in a lane, 6 steps across lanes, up to 16 waves, then
    # mean, eps, root, quotient (60 roundings, halved by the root where they belong to the sum), and
    # two products; s itself one rounding
    c = 64
    within(f64(y), yv, (u + c * E32) * np.abs(yv) * (1 + 1e-6) + tiny(typ), "y")
    a = np.abs(yv).max(axis=1)
    within(f64(qs), a / 127, (c + 2) * E32 * a / 127, "scale")
    # half a step, and the roundings of y, of its largest and of three products, on at most 127 steps
    codes = f64(q)
    within(codes, yv * (127 / a)[:, None], np.full((T, H), 0.5 + 127 * (2 * c + 4) * E32), "codes")
    assert np.abs(codes).max() == 127
    # the rows alone, the codes alone, and no residual give the same bits
    s2, y2 = out((T, H), TYPES[typ]), out((T, H), TYPES[typ])
    q2, qs2 = out((T, H), torch.int8), out((T,), torch.float32)
    moe.moe_add_rmsnorm(d, x, r, w, s2, y2)
    moe.moe_add_rmsnorm(d, x, r, w, None, None, q2, qs2)
    out.check()
    assert torch.equal(s, s2) and torch.equal(y, y2) and torch.equal(q, q2) and torch.equal(qs, qs2)
    moe.moe_add_rmsnorm(d, x, None, w, s2, y2)
    out.check()
    assert torch.equal(s2, x)
    within(f64(y2), ref.norm(xv, None, wv, np.float32(eps))[1],
           (u + c * E32) * np.abs(ref.norm(xv, None, wv, np.float32(eps))[1]) * (1 + 1e-6) + tiny(typ), "y alone")


def test_norm_in_place():
    """sum over the residual and y over x."""
    rng = np.random.default_rng(1)
    for T, H in ((3, 2048), (2100, 256), (2, 9000)):
        x, _ = rows_of(rng, (T, H), "bf16")
        r, _ = rows_of(rng, (T, H), "bf16")
        w, _ = f32(rng, H)
        d = moe.NormDims(T, H, moe.ELEM_BF16, 1e-6)
        s, y = torch.empty_like(x), torch.empty_like(x)
        moe.moe_add_rmsnorm(d, x, r, w, s, y)
        moe.moe_add_rmsnorm(d, x, r, w, r, x)
        torch.cuda.synchronize()
        assert torch.equal(r, s) and torch.equal(x, y)


def test_norm_of_more_rows_than_one_grid_row_holds():
    """Four rows a workgroup and 2^20 workgroups along x: the rows past 2^22 come along y."""
    T, H = (1 << 22) + 9, 8
    x = torch.arange(T * H, device="cuda", dtype=torch.float32).remainder_(97.0).sub_(48.5).to(torch.bfloat16).reshape(T, H)
    w = torch.ones(H, device="cuda")
    y, q, qs = torch.empty_like(x), torch.empty((T, H), dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    moe.moe_add_rmsnorm(moe.NormDims(T, H, moe.ELEM_BF16, 1e-6), x, None, w, None, y, q, qs)
    for rows in (slice(0, 4096), slice(T - 4096, T)):
        xv = f64(x[rows])
        want = ref.norm(xv, None, np.ones(H), np.float32(1e-6))[1]
        within(f64(y[rows]), want, (2.0 ** -8 + 64 * E32) * np.abs(want) * (1 + 1e-6), "y")
        within(f64(q[rows]) * f64(qs[rows])[:, None], want, 0.501 * np.abs(want).max(axis=1, keepdims=True) / 127 + 0 * want,
               "values")
    dx, dw = torch.empty_like(x), torch.empty(H, device="cuda")
    d = moe.NormDims(T, H, moe.ELEM_BF16, 1e-6)
    n = moe.moe_add_rmsnorm_backward_ws_bytes(d)
    moe.moe_add_rmsnorm_backward(d, x, w, y, None, dx, dw, torch.empty(n, dtype=torch.uint8, device="cuda"), n)
    xd, yd = x.double(), y.double()
    rho = torch.rsqrt((xd * xd).mean(1, keepdim=True) + np.float64(np.float32(1e-6)))
    terms = yd * xd * rho
    # a lane adds T / (8 * 256) rows one after the other, then the folds and the partial sums
    bound = (64 + T / 2048 + 1 + 3 + 80) * E32 * terms.abs().sum(0)
    assert bool(((dw.double() - terms.sum(0)).abs() <= bound).all())


def test_empty_batches():
    """No rows: every entry point accepts empty tensors and writes nothing."""
    e = dict(device="cuda")
    x, q, s = torch.empty((0, 64), **e), torch.empty((0, 64), dtype=torch.int8, **e), torch.empty(0, **e)
    w, dw = torch.ones(64, **e), torch.full((64,), 5.0, **e)
    d, nd = moe.make_dims(0, 64, 64, 4, 2, 1), moe.NormDims(0, 64, moe.ELEM_F32, 1e-6)
    tab = Tables(ref.routing(np.random.default_rng(0), 1, 4, 2, 128, 16, 1), 1)
    moe.moe_add_rmsnorm(nd, x, x, w, x, x.clone(), q, s)
    moe.moe_q8_quantize(nd, x, q, s)
    moe.moe_q8_matmul(moe.Q8Dims(0, 64, 64, 0), q, s, torch.zeros((64, 64), dtype=torch.int8, **e), w, x)
    moe.moe_q8_gate_up(d, q, s, tab.c, moe.Q8Bank(), None, x)
    moe.moe_q8_down(d, tab.c, moe.Q8Bank(), None, q, s, x)
    moe.moe_dispatch_rows(d, 0, x, tab.c, x)
    moe.moe_combine_rows(d, 0, x, tab.c, x)
    moe.moe_dispatch_rows_backward(d, 0, x, tab.c, x)
    moe.moe_combine_rows_backward(d, 0, x, x, tab.c, x, s)
    moe.moe_add_rmsnorm_backward(nd, x, w, x, None, x, dw, None, 0)
    torch.cuda.synchronize()
    assert bool((dw == 0).all()) and int(tab.status.item()) == 0


def test_norm_rows_of_zeros_infinities_and_nans():
    """A row of zeros, one of the smallest values, one with an infinity, one with a NaN: each row's
    8-bit form stands on its own, and the others are as without them."""
    T, H = 6, 256
    rng = np.random.default_rng(2)
    x = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32))
    clean = x.clone()
    x[1] = 0.0
    x[2] = 1e-38 * torch.arange(H)
    x[3, 5] = float("inf")
    x[4, 200] = float("nan")
    w = torch.ones(H).cuda()
    for eps in (0.0, 1e-6):
        d = moe.NormDims(T, H, moe.ELEM_F32, eps)
        y, q, qs = torch.empty((T, H)).cuda(), torch.empty((T, H), dtype=torch.int8).cuda(), torch.empty(T).cuda()
        yc, qc, qsc = torch.empty_like(y), torch.empty_like(q), torch.empty_like(qs)
        moe.moe_add_rmsnorm(d, x.cuda(), None, w, None, y, q, qs)
        moe.moe_add_rmsnorm(d, clean.cuda(), None, w, None, yc, qc, qsc)
        torch.cuda.synchronize()
        for row in (0, 5):
            assert torch.equal(y[row], yc[row]) and torch.equal(q[row], qc[row]) and qs[row] == qsc[row]
        if not eps:
            assert bool(torch.isnan(y[1]).all()) and torch.isnan(qs[1]) and bool((q[1] == 0).all())
        else:
            assert bool((y[1] == 0).all()) and qs[1] == 0 and bool((q[1] == 0).all())
        for row in (3, 4):
            assert torch.isnan(qs[row]) and bool((q[row] == 0).all())
    # the quantiser alone: the smallest values keep their codes, zeros give zero
    d = moe.NormDims(T, H, moe.ELEM_F32, 0.0)
    moe.moe_q8_quantize(d, x.cuda(), q, qs)
    torch.cuda.synchronize()
    v = f64(x)
    for row in (0, 2, 5):
        a = np.abs(v[row]).max()
        # the scale of a row this small is itself subnormal: one step of 2^-149 on it
        assert abs(float(qs[row]) - a / 127) <= 2 * E32 * a / 127 + 2.0 ** -149
        assert np.abs(f64(q[row]) - v[row] * 127 / a).max() <= 0.5 + 127 * 4 * E32
    assert qs[1] == 0 and bool((q[1] == 0).all())
    for row in (3, 4):
        assert torch.isnan(qs[row]) and bool((q[row] == 0).all())


@pytest.mark.parametrize("typ", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,K", [(1, 8), (2049, 64), (5, 512), (3, 2048), (2, 16384)])
def test_quantize(rows, K, typ):
    print(f"quantize {rows} {K} {typ}", flush=True)
    rng = np.random.default_rng(rows + K)
    x, xv = rows_of(rng, (rows, K), typ)
    out = Out()
    q, s = out((rows, K), torch.int8), out((rows,), torch.float32)
    moe.moe_q8_quantize(moe.NormDims(rows, K, moe.ELEM[TYPES[typ]], 0.0), x, q, s)
    out.check()
    a = np.abs(xv).max(axis=1)
    within(f64(s), a / 127, E32 * a / 127, "scale")
    within(f64(q), xv * (127 / a)[:, None], np.full((rows, K), 0.5 + 127 * 3 * E32), "codes")


# --------------------------------------------------------------------------- the norm's gradient

@pytest.mark.parametrize("typ", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,H", NORM_SIZES)
def test_norm_backward(T, H, typ):
    print(f"norm backward {T} {H} {typ}", flush=True)
    rng = np.random.default_rng(T + 3 * H)
    s, sv = rows_of(rng, (T, H), typ, 2.0)
    dy, dyv = rows_of(rng, (T, H), typ)
    ds, dsv = rows_of(rng, (T, H), typ)
    w, wv = f32(rng, H)
    eps = 1e-5
    d = moe.NormDims(T, H, moe.ELEM[TYPES[typ]], eps)
    n = moe.moe_add_rmsnorm_backward_ws_bytes(d)
    out = Out()
    dx, dw, ws = out((T, H), TYPES[typ]), out((H,), torch.float32), out((n,), torch.uint8)
    u = ref.HALF_STEP[typ]
    for resid, residv in ((ds, dsv), (None, None)):
        moe.moe_add_rmsnorm_backward(d, s, w, dy, resid, dx, dw, ws, n)
        out.check()
        want, wantw, size, sizew = ref.norm_backward(sv, wv, dyv, residv, np.float32(eps))
        # as for y, with a second row sum (two roundings a term) and four more operations
        within(f64(dx), want, u * np.abs(want) * (1 + 1e-6) + 160 * E32 * size + tiny(typ), "dx")
        # rows of one lane (at most T / 512 + 1), 3 folds or none, partial sums (at most 64 + 16)
        within(f64(dw), wantw, (64 + T / 512 + 1 + 3 + 80) * E32 * sizew, "dweight")
    # a dweight off the 16-byte grid (one workgroup writes an aligned one itself): the same bits
    off = torch.empty(H + 1, device="cuda")[1:]
    moe.moe_add_rmsnorm_backward(d, s, w, dy, None, dx, off, ws, n)
    torch.cuda.synchronize()
    assert torch.equal(off, dw)
    # without dweight: the same dx; over dy and over dsum: the same dx
    first, firstw = dx.clone(), dw.clone()
    dx.zero_()
    moe.moe_add_rmsnorm_backward(d, s, w, dy, None, dx, None, None, 0)
    out.check()
    assert torch.equal(dx, first) and torch.equal(dw, firstw)
    moe.moe_add_rmsnorm_backward(d, s, w, dy, ds, dx, dw, ws, n)
    over = ds.clone()
    moe.moe_add_rmsnorm_backward(d, s, w, dy, over, over, None, None, 0)
    moe.moe_add_rmsnorm_backward(d, s, w, dy, ds, dy, None, None, 0)
    torch.cuda.synchronize()
    assert torch.equal(over, dx) and torch.equal(dy, dx)


def test_norm_backward_of_no_rows():
    dw = torch.full((64,), 7.0, device="cuda")
    d = moe.NormDims(0, 64, moe.ELEM_BF16, 1e-6)
    e = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    raw = 0x10000
    moe.moe_add_rmsnorm_backward(d, raw, torch.ones(64, device="cuda"), raw, None, raw, dw, None, 0)
    torch.cuda.synchronize()
    assert e.numel() == 0 and bool((dw == 0).all())


def test_norm_gradient_against_differences():
    """The kernels' own gradient against differences of the kernels' forward pass, in float32."""
    rng = np.random.default_rng(11)
    T, H, eps = 2, 64, 1e-3
    s, sv = rows_of(rng, (T, H), "f32")
    dy, dyv = rows_of(rng, (T, H), "f32")
    w, wv = f32(rng, H)
    d = moe.NormDims(T, H, moe.ELEM_F32, eps)
    n = moe.moe_add_rmsnorm_backward_ws_bytes(d)
    dx, dw, ws = torch.empty_like(s), torch.empty_like(w), torch.empty(n, dtype=torch.uint8, device="cuda")
    moe.moe_add_rmsnorm_backward(d, s, w, dy, None, dx, dw, ws, n)

    def loss(s, w):
        y = torch.empty_like(s)
        moe.moe_add_rmsnorm(d, s, None, w, None, y)
        return float((y.double() * dy.double()).sum())

    h = 2.0 ** -6
    # each loss carries y's float32 roundings (64 E32 |y| |dy| summed, see test_norm); the quotient
    # divides their difference by 2h, and a third derivative of order one adds h^2
    y = ref.norm(sv, None, wv, eps)[1]
    noise = 2 * 64 * E32 * float((np.abs(y) * np.abs(dyv)).sum()) / (2 * h)
    bound = noise + 2 * h * h
    for i, j in ((0, 0), (1, 63), (0, 17)):
        e = torch.zeros_like(s)
        e[i, j] = h
        assert abs((loss(s + e, w) - loss(s - e, w)) / (2 * h) - float(dx[i, j])) <= bound * max(1, abs(dyv).max())
    for j in (0, 40):
        e = torch.zeros_like(w)
        e[j] = h
        assert abs((loss(s, w + e) - loss(s, w - e)) / (2 * h) - float(dw[j])) <= bound * max(1, abs(dyv).max())


# ------------------------------------------------------------------------------ 8-bit products

def codes(rng, shape):
    a = rng.integers(-127, 128, size=shape, dtype=np.int64)
    return torch.from_numpy(a.astype(np.int8)).cuda(), a


PRODUCT_SIZES = [(1, 8, 64), (1, 8192, 2048), (2, 40, 64), (15, 136, 192), (16, 2048, 128), (17, 72, 320),
                 (32, 1000, 256), (33, 200, 64), (65, 264, 192), (127, 520, 576), (128, 128, 128),
                 (200, 2056, 512), (333, 8192, 320), (513, 1032, 192), (2000, 8200, 128), (4097, 4104, 64),
                 (4000, 4360, 320), (4000, 4360, 512), (3900, 4360, 704)]


@pytest.mark.parametrize("typ", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,N,K", PRODUCT_SIZES)
def test_product(M, N, K, typ):
    print(f"product {M} {N} {K} {typ}", flush=True)
    rng = np.random.default_rng(M + N + K)
    xq, xv = codes(rng, (M, K))
    wq, wv = codes(rng, (N, K))
    xs, xsv = f32(rng, M, 0.001, 0.01)
    ws, wsv = f32(rng, N, 0.001, 0.01)
    out = Out()
    y = out((M, N), TYPES[typ])
    moe.moe_q8_matmul(moe.Q8Dims(M, N, K, moe.ELEM[TYPES[typ]]), xq, xs, wq, ws, y)
    out.check()
    want = ref.product(xv, xsv, wv, wsv)
    # the integer sum is exact: one conversion, two products, one rounding to the type
    within(f64(y), want, (ref.HALF_STEP[typ] + 3 * E32) * np.abs(want) * (1 + 1e-6) + tiny(typ), "product")


def test_product_of_the_largest_values():
    """-128 times -128 over the longest K: the sum is 2^30, and exact."""
    M, N, K = 3, 16, 65536
    xq = torch.full((M, K), -128, dtype=torch.int8, device="cuda")
    wq = torch.full((N, K), -128, dtype=torch.int8, device="cuda")
    wq[1, 7] = 127
    one = torch.ones(N, device="cuda")
    y = torch.empty((M, N), device="cuda")
    moe.moe_q8_matmul(moe.Q8Dims(M, N, K, moe.ELEM_F32), xq, one, wq, one, y)
    torch.cuda.synchronize()
    assert float(y[0, 0]) == 2.0 ** 30 and float(y[2, 15]) == 2.0 ** 30
    assert float(y[0, 1]) == float(np.float32(2 ** 30 - 128 * 255))


def test_product_rows_do_not_depend_on_the_batch():
    rng = np.random.default_rng(5)
    N, K, M = 264, 320, 300
    xq, _ = codes(rng, (M, K))
    wq, _ = codes(rng, (N, K))
    xs, _ = f32(rng, M, 0.001, 0.01)
    ws, _ = f32(rng, N, 0.001, 0.01)

    def rows(n):
        y = torch.empty((n, N), dtype=torch.bfloat16, device="cuda")
        moe.moe_q8_matmul(moe.Q8Dims(n, N, K, moe.ELEM_BF16), xq, xs, wq, ws, y)
        return y

    full = rows(M)
    for n in (1, 16, 17, 32, 33, 128, 129):
        assert torch.equal(rows(n), full[:n]), n


def test_product_with_a_nan_scale():
    """The scale of a row that held a NaN poisons that row alone."""
    M, N, K = 5, 64, 128
    rng = np.random.default_rng(6)
    xq, _ = codes(rng, (M, K))
    wq, _ = codes(rng, (N, K))
    xs, _ = f32(rng, M)
    ws, _ = f32(rng, N)
    xs[2] = float("nan")
    y = torch.empty((M, N), device="cuda")
    moe.moe_q8_matmul(moe.Q8Dims(M, N, K, moe.ELEM_F32), xq, xs, wq, ws, y)
    bad = torch.isnan(y).all(dim=1).cpu().tolist()
    assert bad == [False, False, True, False, False] and not bool(torch.isnan(y[[0, 1, 3, 4]]).any())


# --------------------------------------------------------------------------- tables on the device

class Tables:
    def __init__(self, r, T):
        self.t = {n: torch.from_numpy(np.ascontiguousarray(v)).cuda() for n, v in r.items()}
        if self.t["blocks"].numel() == 0:
            self.t["blocks"] = torch.zeros((1, 4), dtype=torch.int32, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.c = moe.RouteOut(*[self.t[n].data_ptr() for n in
                                ("topk_idx", "topk_w", "counts", "offsets", "sorted_slot", "slot_pos",
                                 "blocks", "n_blocks")], None, self.status.data_ptr(), None, 0)


# T, H, I, E, k, n_shared, tile_m_max, tile_gran
EXPERT_SIZES = [(1, 64, 64, 4, 1, 0, 16, 16), (1, 2048, 512, 256, 8, 1, 32, 16), (3, 128, 192, 5, 2, 1, 16, 16),
                (16, 256, 128, 8, 2, 1, 128, 16), (37, 320, 64, 300, 8, 0, 32, 32), (100, 192, 320, 6, 3, 1, 256, 16),
                (200, 128, 128, 3, 2, 1, 48, 16), (600, 64, 192, 4, 2, 1, 128, 16), (513, 576, 128, 9, 4, 0, 64, 32),
                (1500, 128, 64, 5, 2, 1, 256, 16), (300, 128, 64, 1, 1, 1, 240, 16), (64, 128, 64, 1024, 4, 1, 16, 16)]
# few rows an expert, but every token in the shared one, whose blocks take several passes
EXPERT_SIZES += [(17, 128, 64, 64, 1, 1, 64, 16), (40, 192, 64, 64, 1, 1, 64, 16), (300, 128, 128, 300, 2, 1, 256, 16),
                 (1294, 192, 320, 105, 1, 1, 128, 16), (4096, 64, 512, 512, 1, 1, 256, 16),
                 (8192, 64, 1024, 1024, 1, 1, 256, 32)]
# hundreds of rows an expert over several steps of inputs, an odd number of halves among them
EXPERT_SIZES += [(1300, 448, 320, 4, 2, 1, 256, 16), (1100, 704, 512, 3, 1, 0, 256, 32)]


def bank(rng, n, rows, K):
    q, qv = codes(rng, (n, rows, K))
    s, sv = f32(rng, (n, rows), 0.001, 0.004)
    return q, s, qv, sv


def expert_products(rows_q, rows_s, groups, qv, sv):
    out = np.empty((rows_q.shape[0], qv.shape[1]))
    for g in np.unique(groups):
        m = groups == g
        out[m] = ref.product(rows_q[m], rows_s[m], qv[g], sv[g])
    return out


@pytest.mark.parametrize("T,H,I,E,k,n_shared,tile,gran", EXPERT_SIZES)
@pytest.mark.parametrize("skew", [False, True])
def test_expert_products(T, H, I, E, k, n_shared, tile, gran, skew):
    """Both products over every block of the map; skew: most tokens take the same experts, others
    stay empty."""
    print(f"experts {T} {H} {I} {E} {k} {n_shared} {tile} skew={skew}", flush=True)
    rng = np.random.default_rng(T + H + E)
    idx = None
    if skew:
        idx = np.stack([np.arange(k) if t % 5 else np.arange(E - k, E) for t in range(T)])
    r = ref.routing(rng, T, E, k, tile, gran, n_shared, idx)
    tab = Tables(r, T)
    d = moe.make_dims(T, H, I, E, k, n_shared, tile, gran)
    assert len(r["blocks"]) <= moe.moe_max_blocks(d)
    n = E + n_shared
    tok, grp = ref.row_tokens(r, T, k, n_shared), ref.row_groups(r, T, E, k, n_shared)
    rows = len(tok)
    out = Out()

    gq, gs, gqv, gsv = bank(rng, n, 2 * I, H)
    xq, xv = codes(rng, (T, H))
    xs, xsv = f32(rng, T, 0.0005, 0.002)
    h = out((rows, I), torch.bfloat16)
    routed = moe.Q8Bank(gu=gq.data_ptr(), gu_s=gs.data_ptr())
    shared = moe.Q8Bank(gu=gq[E].data_ptr(), gu_s=gs[E].data_ptr()) if n_shared else None
    moe.moe_q8_gate_up(d, xq, xs, tab.c, routed, shared, h)
    out.check()
    gu = expert_products(xv[tok], xsv[tok], grp, gqv, gsv)
    g, u = gu[:, :I], gu[:, I:]
    want = ref.silu(g) * u
    # g and u carry three roundings; silu'(g) g / silu(g) is at most 1 + |g|; the exponential and the
    # reciprocal add a few units in the last place (the exponential |g| / ln 2 more for its argument)
    bound = (2.0 ** -8 + (16 + 6 * np.abs(g)) * E32) * np.abs(want) * (1 + 1e-6) + 1e-37
    within(f64(h), want, bound, "h")

    dq, dsc, dqv, dsv = bank(rng, n, H, I)
    hq, hv = codes(rng, (rows, I))
    hs, hsv = f32(rng, rows, 0.0005, 0.002)
    y = out((rows, H), torch.bfloat16)
    routed = moe.Q8Bank(dn=dq.data_ptr(), dn_s=dsc.data_ptr())
    shared = moe.Q8Bank(dn=dq[E].data_ptr(), dn_s=dsc[E].data_ptr()) if n_shared else None
    moe.moe_q8_down(d, tab.c, routed, shared, hq, hs, y)
    out.check()
    want = expert_products(hv, hsv, grp, dqv, dsv)
    within(f64(y), want, (2.0 ** -8 + 3 * E32) * np.abs(want) * (1 + 1e-6) + 1e-37, "y_slots")
    assert int(tab.status.item()) == 0


def test_expert_products_with_bad_tables():
    """Entries out of range are skipped with the status bit; the other rows are as before."""
    T, H, I, E, k = 40, 128, 64, 6, 2
    rng = np.random.default_rng(8)
    r = ref.routing(rng, T, E, k, 32, 16, 1)
    d = moe.make_dims(T, H, I, E, k, 1, 32, 16)
    gq, gs, _, _ = bank(rng, E + 1, 2 * I, H)
    xq, _ = codes(rng, (T, H))
    xs, _ = f32(rng, T)
    routed = moe.Q8Bank(gu=gq.data_ptr(), gu_s=gs.data_ptr())
    shared = moe.Q8Bank(gu=gq[E].data_ptr(), gu_s=gs[E].data_ptr())

    def run(r):
        tab = Tables(r, T)
        h = torch.zeros((T * 3, I), dtype=torch.bfloat16, device="cuda")
        moe.moe_q8_gate_up(d, xq, xs, tab.c, routed, shared, h)
        torch.cuda.synchronize()
        return h, int(tab.status.item())

    good, status = run(r)
    assert status == 0
    for what in ("group", "row", "rows", "negative", "slot"):
        b = {n: v.copy() for n, v in r.items()}
        first = b["blocks"][0].copy()
        lost = slice(first[1], first[1] + first[2])
        if what == "group":
            b["blocks"][0, 0] = E + 1
        elif what == "row":
            b["blocks"][0, 1] = -1
        elif what == "rows":
            b["blocks"][0, 2] = T * 3 + 1
        elif what == "negative":
            b["blocks"][0, 0] = -2
        else:
            b["sorted_slot"][3] = T * k
            lost = slice(3, 4)
        h, status = run(b)
        assert status & moe.STATUS_BAD_INDEX, what
        keep = torch.ones(T * 3, dtype=torch.bool)
        keep[lost] = False
        assert torch.equal(h[keep.cuda()], good[keep.cuda()]), what
        assert bool((h[~keep.cuda()] == 0).all()), what


# ------------------------------------------------------------------------- rows sorted and back

ROW_SIZES = [(1, 64, 4, 1, 0), (1, 2048, 256, 8, 1), (5, 64, 8, 8, 1), (37, 320, 300, 9, 0),
             (130, 2112, 16, 2, 1), (33, 4160, 40, 32, 1), (511, 256, 64, 6, 1)]


@pytest.mark.parametrize("typ", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,H,E,k,n_shared", ROW_SIZES)
def test_rows(T, H, E, k, n_shared, typ):
    print(f"rows {T} {H} {E} {k} {n_shared} {typ}", flush=True)
    rng = np.random.default_rng(T + H + k)
    r = ref.routing(rng, T, E, k, 128, 16, n_shared)
    tab = Tables(r, T)
    d = moe.make_dims(T, H, 64, E, k, n_shared)
    elem, dt, u = moe.ELEM[TYPES[typ]], TYPES[typ], ref.HALF_STEP[typ]
    n = T * (k + n_shared)
    pos, w = r["slot_pos"], r["topk_w"]
    x, xv = rows_of(rng, (T, H), typ)
    dy, dyv = rows_of(rng, (T, H), typ)
    ys, ysv = rows_of(rng, (n, H), typ)
    out = Out()

    rows = out((n, H), dt)
    moe.moe_dispatch_rows(d, elem, x, tab.c, rows)
    out.check()
    assert np.array_equal(f64(rows), xv[ref.row_tokens(r, T, k, n_shared)])

    y = out((T, H), dt)
    moe.moe_combine_rows(d, elem, ys, tab.c, y)
    out.check()
    want, size = ref.combine(ysv, w, pos, n_shared)
    within(f64(y), want, u * np.abs(want) * (1 + 1e-6) + (k + 1) * E32 * size * (1 + 1e-6) + tiny(typ), "y")
    if typ == "bf16":
        y2 = out((T, H), dt)
        moe.moe_combine(d, tab.c, ys, y2)
        out.check()
        assert torch.equal(y, y2)

    dx = out((T, H), dt)
    moe.moe_dispatch_rows_backward(d, elem, ys, tab.c, dx)
    out.check()
    want, size = ref.combine(ysv, None, pos, n_shared)
    within(f64(dx), want, u * np.abs(want) * (1 + 1e-6) + (k + 1) * E32 * size * (1 + 1e-6) + tiny(typ), "dx")

    drows, dw = out((n, H), dt), out((T, k), torch.float32)
    moe.moe_combine_rows_backward(d, elem, dy, ys, tab.c, drows, dw)
    out.check()
    want, wantw, sizew = ref.combine_backward(dyv, ysv, w, pos, n_shared)
    within(f64(drows), want, (u + E32) * np.abs(want) * (1 + 1e-6) + tiny(typ), "drows")
    # a lane adds at most H / 256 + 8 products one after the other, then ten steps of the tree
    within(f64(dw), wantw, (H / 256 + 8 + 10) * E32 * sizew, "dtopk_w")
    # without the weights' gradient, and over the rows themselves
    only = out((n, H), dt)
    moe.moe_combine_rows_backward(d, elem, dy, None, tab.c, only, None)
    over, dw2 = ys.clone(), out((T, k), torch.float32)
    moe.moe_combine_rows_backward(d, elem, dy, over, tab.c, over, dw2)
    out.check()
    assert torch.equal(only, drows) and torch.equal(over, drows) and torch.equal(dw, dw2)
    assert int(tab.status.item()) == 0


def test_rows_with_a_bad_position():
    """A slot position out of range: the status bit, its slot skipped, everything else as before."""
    T, H, E, k = 9, 64, 5, 3
    rng = np.random.default_rng(9)
    r = ref.routing(rng, T, E, k, 16, 16, 1)
    d = moe.make_dims(T, H, 64, E, k, 1)
    x, xv = rows_of(rng, (T, H), "f32")
    ys, ysv = rows_of(rng, (T * 4, H), "f32")
    for bad in (-1, T * k):
        b = {n: v.copy() for n, v in r.items()}
        was = int(b["slot_pos"][4, 1])
        b["slot_pos"][4, 1] = bad
        w = r["topk_w"].copy()
        w[4, 1] = 0
        for call in ("dispatch", "combine", "backward"):
            tab = Tables(b, T)
            if call == "dispatch":
                rows = torch.full((T * 4, H), 7.0, device="cuda")
                moe.moe_dispatch_rows(d, 0, x, tab.c, rows)
                want = xv[ref.row_tokens(r, T, k, 1)]
                want[was] = 7.0
                assert np.array_equal(f64(rows), want)
            elif call == "combine":
                y = torch.empty((T, H), device="cuda")
                moe.moe_combine_rows(d, 0, ys, tab.c, y)
                want, size = ref.combine(ysv, w, r["slot_pos"], 1)
                within(f64(y), want, 8 * E32 * size, "y")
            else:
                drows, dw = torch.full((T * 4, H), 7.0, device="cuda"), torch.empty((T, k), device="cuda")
                moe.moe_combine_rows_backward(d, 0, x, ys, tab.c, drows, dw)
                assert float(dw[4, 1]) == 0 and bool((drows[was] == 7.0).all())
            torch.cuda.synchronize()
            assert int(tab.status.item()) & moe.STATUS_BAD_INDEX, call


def test_binding_refuses_strided_and_short_tensors():
    d = moe.NormDims(4, 64, moe.ELEM_F32, 1e-6)
    x, w, y = torch.zeros((4, 128), device="cuda"), torch.ones(64, device="cuda"), torch.empty((4, 64), device="cuda")
    with pytest.raises(ValueError):
        moe.moe_add_rmsnorm(d, x[:, :64], None, w, None, y)
    with pytest.raises(ValueError):
        moe.moe_add_rmsnorm(d, x, None, w, None, y[:3])
    with pytest.raises(ValueError):
        moe.moe_add_rmsnorm(d, x, None, w.cpu(), None, y)
    with pytest.raises(moe.MoeError):
        moe.moe_add_rmsnorm(moe.NormDims(4, 60, 0, 1e-6), x, None, w, None, y)


# ------------------------------------------------------------------------ together, as they are used

def layer_inputs(rng, T, H, I, E):
    gu = rng.standard_normal((E + 1, 2 * I, H)) / np.sqrt(H)
    dn = rng.standard_normal((E + 1, H, I)) / np.sqrt(I)
    wr = (rng.standard_normal((H, E)) / np.sqrt(H)).astype(np.float32)
    w = rng.uniform(0.5, 1.5, H).astype(np.float32)
    return gu, dn, wr, w


def quantised(v):
    a = np.abs(v).max(axis=-1, keepdims=True)
    return np.rint(v * (127 / a)) * (a / 127)


@pytest.mark.parametrize("T", [1, 7, 96, 600])
def test_layer_in_8_bits(T):
    """norm, routing, both 8-bit products and the combine, against the same steps in float64 with the
    layer's own routing."""
    print(f"8-bit layer {T}", flush=True)
    H, I, E, k = 256, 128, 8, 2
    rng = np.random.default_rng(T)
    gu, dn, wr, w = layer_inputs(rng, T, H, I, E)
    gu_t, dn_t = (torch.from_numpy(a.astype(np.float32)).cuda() for a in (gu, dn))
    layer = moe.Q8MoeLayer(H, I, E, k, 1, moe.DeviceBankQ8(gu_t[:E], dn_t[:E]), moe.DeviceBankQ8(gu_t[E:], dn_t[E:]),
                           wr, None, T_max=600, tile_m_max=32)
    x, xv = rows_of(rng, (T, H), "bf16")
    res, rv = rows_of(rng, (T, H), "bf16", 2.0)
    y = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    layer.forward_residual(x, res, torch.from_numpy(w).cuda(), y)
    torch.cuda.synchronize()
    sv, yn = ref.norm(xv, rv, w, 1e-6)
    within(f64(res), sv, (2.0 ** -8 + E32) * np.abs(sv) * (1 + 1e-6), "residual")
    idx = layer.rt.topk_idx[:T].cpu().numpy()
    tw = layer.rt.topk_w[:T].cpu().numpy().astype(np.float64)
    assert int(layer.rt.status.item()) == 0
    guq, dnq, xq = quantised(gu), quantised(dn), quantised(yn)
    want = np.zeros((T, H))
    for t in range(T):
        for e, weight in list(zip(idx[t], tw[t])) + [(E, 1.0)]:
            p = guq[e] @ xq[t]
            hv = quantised(ref.silu(p[:I]) * p[I:])
            want[t] += weight * (dnq[e] @ hv)
    # each of the three outputs that a slot goes through rounds to bf16 (h, y_slots, y); h's rounding can
    # move a code by one step, 1/127 of the row's largest: on the norm of a row that is at most
    # sqrt(I) / 127 of its largest, spread over I random signs by the down product
    err = np.linalg.norm(f64(y) - want, axis=1) / np.linalg.norm(want, axis=1)
    assert err.max() <= 3 * 2.0 ** -8 + 1.0 / 127 * 4, err.max()
    # forward() on the normed rows: its tokens are quantised after their rounding to bf16
    y2 = torch.empty_like(y)
    layer.forward(layer.xn[:T].clone(), y2)
    torch.cuda.synchronize()
    err = np.linalg.norm(f64(y2) - want, axis=1) / np.linalg.norm(want, axis=1)
    assert err.max() <= 4 * 2.0 ** -8 + 2.0 / 127 * 4, err.max()
    # the stages on their own: the same bits
    h, ys, xn = layer.h.clone(), layer.y_slots.clone(), layer.xn[:T].clone()
    layer.h.zero_()
    layer.xq.zero_()
    d = layer.route(xn)
    layer.gate_up(d, xn)
    layer.down(d)
    y3 = torch.empty_like(y)
    layer.combine(d, y3)
    torch.cuda.synchronize()
    rows = T * (k + 1)
    assert torch.equal(layer.h[:rows], h[:rows]) and torch.equal(layer.y_slots[:rows], ys[:rows]) and torch.equal(y3, y2)
    with pytest.raises(NotImplementedError):
        layer.shared_ffn(d, xn)


def test_layer_in_4_bits_behind_the_norm():
    """MoeLayer.forward_residual is the norm, then the layer, bit for bit; and an 8-bit bank made from the
    same 4-bit checkpoint stays near it."""
    from synth import build_config
    c = build_config("tiny16")
    sh, T = c["shape"], c["T"]
    args = (sh.H, sh.I, sh.E, sh.k, sh.n_shared)
    layer = moe.MoeLayer(*args, moe.DeviceBank(c["routed"]), moe.DeviceBank(c["shared"]), c["wr"], None, T_max=T)
    x = torch.from_numpy(c["x"].view(np.int16)).cuda()
    res = torch.roll(x, 1, 0).contiguous()
    w = torch.linspace(0.5, 1.5, sh.H, device="cuda")
    y, y2, xn, s = (torch.empty_like(x) for _ in range(4))
    before = res.clone()
    layer.forward_residual(x, res, w, y)
    d = moe.NormDims(T, sh.H, moe.ELEM_BF16, 1e-6)
    moe.moe_add_rmsnorm(d, x, before, w, s, xn)
    layer.forward(xn, y2)
    torch.cuda.synchronize()
    assert torch.equal(res, s) and torch.equal(y, y2)
    q8 = moe.Q8MoeLayer(*args, moe.DeviceBankQ8.from_w4(c["routed"]), moe.DeviceBankQ8.from_w4(c["shared"]),
                        c["wr"], None, T_max=T)
    y8, res8 = torch.empty_like(x), before.clone()
    q8.forward_residual(x, res8, w, y8)
    torch.cuda.synchronize()
    a, b = (f64(t.view(torch.bfloat16)) for t in (y, y8))
    # tokens, weights and h in 8 bits: a step is 1/127 of a row's largest value, about 4 of its rms, and
    # its rounding has an rms of 1 / sqrt(12): 4 / 127 / 3.46 for each of the four, under 2.5 % together
    err = np.linalg.norm(a - b, axis=1) / np.linalg.norm(a, axis=1)
    assert err.max() <= 0.025, err.max()
    assert torch.equal(q8.rt.topk_idx, layer.rt.topk_idx)


def test_training_step():
    """norm, routing, dispatch, the experts in torch, combine, and the whole way back, against float64
    autograd with the same routing."""
    T, H, I, E, k = 48, 64, 64, 4, 2
    rng = np.random.default_rng(21)
    gu, dn, wr, w = layer_inputs(rng, T, H, I, E)
    gu_t, dn_t = (torch.from_numpy(a.astype(np.float32)).cuda() for a in (gu, dn))
    x, xv = rows_of(rng, (T, H), "f32")
    res, rv = rows_of(rng, (T, H), "f32")
    dout, doutv = rows_of(rng, (T, H), "f32")
    w_t = torch.from_numpy(w).cuda()
    d = moe.make_dims(T, H, I, E, k, 1, 32, 16)
    nd = moe.NormDims(T, H, moe.ELEM_F32, 1e-6)
    rt = moe.RouteTables(d, export_logits=False)
    s, xn = torch.empty_like(x), torch.empty_like(x)
    moe.moe_add_rmsnorm(nd, x, res, w_t, s, xn)
    moe.moe_route(d, xn.to(torch.bfloat16), torch.from_numpy(wr).cuda(), None, rt.c)
    F = moe.ELEM_F32
    rows = torch.empty((T * (k + 1), H), device="cuda")
    moe.moe_dispatch_rows(d, F, xn, rt.c, rows)
    edges = rt.offsets.tolist() + [T * (k + 1)]
    leaf = rows.clone().requires_grad_()
    parts = []
    for e in range(E + 1):
        g, u = (leaf[edges[e]:edges[e + 1]] @ gu_t[e].t()).chunk(2, dim=1)
        parts.append((torch.nn.functional.silu(g) * u) @ dn_t[e].t())
    ys = torch.cat(parts)
    y = torch.empty_like(x)
    moe.moe_combine_rows(d, F, ys.detach(), rt.c, y)
    # back: the loss is <y + s, dout>
    dys, dtw = torch.empty_like(rows), torch.empty((T, k), device="cuda")
    moe.moe_combine_rows_backward(d, F, dout, ys.detach(), rt.c, dys, dtw)
    ys.backward(dys)
    dxn = torch.empty_like(x)
    moe.moe_dispatch_rows_backward(d, F, leaf.grad, rt.c, dxn)
    n = moe.moe_add_rmsnorm_backward_ws_bytes(nd)
    dx, dw, ws = torch.empty_like(x), torch.empty_like(w_t), torch.empty(n, dtype=torch.uint8, device="cuda")
    moe.moe_add_rmsnorm_backward(nd, s, w_t, dxn, dout, dx, dw, ws, n)
    torch.cuda.synchronize()

    idx, tw = rt.topk_idx.cpu().numpy(), rt.topk_w.cpu().double().requires_grad_()
    X, W = torch.from_numpy(xv).requires_grad_(), torch.from_numpy(w).double().requires_grad_()
    S = X + torch.from_numpy(rv)
    XN = S * torch.rsqrt((S * S).mean(1, keepdim=True) + np.float64(np.float32(1e-6))) * W
    GU, DN = torch.from_numpy(gu.astype(np.float32)).double(), torch.from_numpy(dn.astype(np.float32)).double()

    def expert(e, v):
        g, u = (v @ GU[e].t()).chunk(2, dim=-1)
        return (torch.nn.functional.silu(g) * u) @ DN[e].t()

    Y = torch.stack([sum(tw[t, j] * expert(int(idx[t, j]), XN[t]) for j in range(k)) + expert(E, XN[t])
                     for t in range(T)])
    ((Y + S) * torch.from_numpy(doutv)).sum().backward()
    # float32 throughout, sums of at most 2 H + I terms at each of six stages: a relative 1e-5 of each
    # output's largest value is over ten times that
    for name, got, want in (("y", y, Y.detach()), ("dx", dx, X.grad), ("dw", dw, W.grad), ("dtopk_w", dtw, tw.grad)):
        want = want.numpy()
        assert np.abs(f64(got) - want).max() <= 1e-5 * np.abs(want).max(), name


# ------------------------------------------------------------------------ streams and captured graphs

def test_graph_replays_match_eager():
    """Every operator captured once and replayed, with eager calls of the same operators (their own
    workspace) and synchronisations between the replays."""
    T, H, I, E, k = 40, 256, 128, 8, 2
    rng = np.random.default_rng(31)
    r = ref.routing(rng, T, E, k, 32, 16, 1)
    tab = Tables(r, T)
    d = moe.make_dims(T, H, I, E, k, 1, 32, 16)
    nd = moe.NormDims(T, H, moe.ELEM_BF16, 1e-6)
    w, _ = f32(rng, H)
    gu, dn, _, _ = layer_inputs(rng, T, H, I, E)
    b = moe.DeviceBankQ8(*(torch.from_numpy(a.astype(np.float32)).cuda() for a in (gu, dn)))
    shared = moe.Q8Bank(b.t["gu"][E].data_ptr(), b.t["gu_s"][E].data_ptr(), b.t["dn"][E].data_ptr(), b.t["dn_s"][E].data_ptr())
    n = moe.moe_add_rmsnorm_backward_ws_bytes(nd)
    rows = T * (k + 1)
    bf = dict(dtype=torch.bfloat16, device="cuda")

    def buffers():
        return dict(s=torch.empty((T, H), **bf), xn=torch.empty((T, H), **bf),
                    xq=torch.empty((T, H), dtype=torch.int8, device="cuda"), xs=torch.empty(T, device="cuda"),
                    h=torch.empty((rows, I), **bf), hq=torch.empty((rows, I), dtype=torch.int8, device="cuda"),
                    hs=torch.empty(rows, device="cuda"), ys=torch.empty((rows, H), **bf), y=torch.empty((T, H), **bf),
                    sorted=torch.empty((rows, H), **bf), dys=torch.empty((rows, H), **bf),
                    dtw=torch.empty((T, k), device="cuda"), dxn=torch.empty((T, H), **bf),
                    dx=torch.empty((T, H), **bf), dw=torch.empty(H, device="cuda"),
                    ws=torch.empty(n, dtype=torch.uint8, device="cuda"))

    def run(x, res, o, stream=None):
        B = moe.ELEM_BF16
        kw = dict(stream=stream)
        moe.moe_add_rmsnorm(nd, x, res, w, o["s"], o["xn"], o["xq"], o["xs"], **kw)
        moe.moe_q8_gate_up(d, o["xq"], o["xs"], tab.c, b.c, shared, o["h"], **kw)
        moe.moe_q8_quantize(moe.NormDims(rows, I, B, 0.0), o["h"], o["hq"], o["hs"], **kw)
        moe.moe_q8_down(d, tab.c, b.c, shared, o["hq"], o["hs"], o["ys"], **kw)
        moe.moe_combine_rows(d, B, o["ys"], tab.c, o["y"], **kw)
        moe.moe_dispatch_rows(d, B, o["xn"], tab.c, o["sorted"], **kw)
        moe.moe_combine_rows_backward(d, B, o["y"], o["ys"], tab.c, o["dys"], o["dtw"], **kw)
        moe.moe_dispatch_rows_backward(d, B, o["dys"], tab.c, o["dxn"], **kw)
        moe.moe_add_rmsnorm_backward(nd, o["s"], w, o["dxn"], o["y"], o["dx"], o["dw"], o["ws"], n, **kw)

    names = [m for m in buffers() if m != "ws"]
    ins = [(rows_of(rng, (T, H), "bf16")[0], rows_of(rng, (T, H), "bf16")[0]) for _ in range(3)]
    want = []
    for x, res in ins:
        o = buffers()
        run(x, res, o)
        torch.cuda.synchronize()
        want.append({m: o[m].clone() for m in names})
    x_buf, r_buf, og, oe = torch.empty_like(ins[0][0]), torch.empty_like(ins[0][0]), buffers(), buffers()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        run(x_buf, r_buf, og)
    for rep in range(3):
        for i, (x, res) in enumerate(ins):
            x_buf.copy_(x)
            r_buf.copy_(res)
            g.replay()
            torch.cuda.synchronize()
            for m in names:
                assert torch.equal(og[m], want[i][m]), (rep, i, m)
            j = (i + 1) % 3
            run(*ins[j], oe)
            torch.cuda.synchronize()
            for m in names:
                assert torch.equal(oe[m], want[j][m]), (rep, j, m, "eager")
    # on a stream of its own, named by the argument, next to work on the current one
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    on_side = buffers()
    run(*ins[0], on_side, stream=side)
    run(*ins[1], oe)
    torch.cuda.synchronize()
    for m in names:
        assert torch.equal(on_side[m], want[0][m]) and torch.equal(oe[m], want[1][m]), m
    assert int(tab.status.item()) == 0


def test_rows_past_32_bit_offsets():
    """Sorted rows that reach past 2^32 bytes: the last token's rows land where they belong."""
    T, H, k, E = 8200, 16384, 15, 16
    idx = np.stack([np.roll(np.arange(E), t)[:k] for t in range(T)])
    r = ref.routing(np.random.default_rng(1), T, E, k, 128, 16, 1, idx)
    tab = Tables(r, T)
    d = moe.make_dims(T, H, 64, E, k, 1)
    n = T * (k + 1)
    assert n * H * 2 > 2 ** 32
    x = torch.arange(T, device="cuda", dtype=torch.float32)[:, None].expand(T, H).to(torch.bfloat16).contiguous()
    rows = torch.zeros((n, H), dtype=torch.bfloat16, device="cuda")
    moe.moe_dispatch_rows(d, moe.ELEM_BF16, x, tab.c, rows)
    tok = torch.from_numpy(ref.row_tokens(r, T, k, 1)).cuda()
    assert torch.equal(rows[:, 0], x[tok, 0]) and torch.equal(rows[:, H - 1], x[tok, 0])
    y, y2 = torch.empty_like(x), torch.empty_like(x)
    moe.moe_combine_rows(d, moe.ELEM_BF16, rows, tab.c, y)
    moe.moe_combine(d, tab.c, rows, y2)
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and int(tab.status.item()) == 0
    # every row of a token holds the token's value v, and its weights sum to one: y is near 2 v
    v = x[:, 0].double()
    assert bool(((y[:, 5].double() - 2 * v).abs() <= (2.0 ** -8 + 20 * E32) * 2 * v + 1e-30).all())
