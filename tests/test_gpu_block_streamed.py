"""The forms of the operators of include/moe_block.h that go past the caches:
stores of arrays above 32 MiB and loads of arrays above 64 MiB.  References in
float64 on the device by elementary operations; bounds as in test_gpu_block.py."""

from __future__ import annotations

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import block_ref as ref  # noqa: E402
import w4_dequant_expert_amd as moe  # noqa: E402
from test_gpu_block import E32, Out, TYPES, Tables, tiny  # noqa: E402

STORE, LOAD = 32 << 20, 64 << 20
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


def rand(g, shape, typ="f32", scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(TYPES[typ])


def codes(g, shape):
    return torch.randint(-127, 128, shape, generator=g, device="cuda", dtype=torch.int32).to(torch.int8)


def scales(g, shape):
    return torch.rand(shape, generator=g, device="cuda") * 0.0015 + 0.0005


def within(got, want, bound, what):
    """|got - want| <= bound in float64, in runs of rows; a NaN is outside."""
    for lo in range(0, got.shape[0], 4096):
        a, w = got[lo:lo + 4096].double(), want[lo:lo + 4096]
        b = bound(lo, w) if callable(bound) else bound[lo:lo + 4096]
        bad = ~((a - w).abs() <= b)
        assert not bool(bad.any()), f"{what}: {int(bad.sum())} outside from row {lo}"


# one wave a row (one to four chunks a lane), four waves, sixteen
NORM = [(40000, 512, "bf16"), (17000, 1024, "bf16"), (11000, 1536, "f16"), (9000, 2048, "bf16"), (9000, 2040, "f16"),
        (4200, 2048, "f32"), (2200, 4096, "f32"), (8200, 2056, "bf16"), (3000, 6000, "f16"), (2100, 8192, "bf16"),
        (1100, 16384, "bf16"), (600, 16384, "f32"), (2050, 8200, "f16")]


@pytest.mark.parametrize("T,H,typ", NORM)
def test_norm(T, H, typ):
    print(f"streamed norm {T} {H} {typ}", flush=True)
    assert T * H * SIZE[typ] > STORE
    g = torch.Generator("cuda").manual_seed(T + H)
    x, r, w = rand(g, (T, H), typ), rand(g, (T, H), typ, 2.0), torch.rand(H, generator=g, device="cuda") + 0.5
    d = moe.NormDims(T, H, moe.ELEM[TYPES[typ]], 1e-5)
    eps, u = float(np.float32(1e-5)), ref.HALF_STEP[typ]
    out = Out()
    s, y = out((T, H), TYPES[typ]), out((T, H), TYPES[typ])
    q, qs = out((T, H), torch.int8), out((T,), torch.float32)
    moe.moe_add_rmsnorm(d, x, r, w, s, y, q, qs)
    out.check()
    for lo in range(0, T, 4096):
        rows = slice(lo, lo + 4096)
        sv = x[rows].double() + r[rows].double()
        yv = sv / torch.sqrt((sv * sv).mean(1, keepdim=True) + eps) * w.double()
        a = yv.abs().amax(1, keepdim=True)
        for what, got, want, bound in (
                ("sum", s, sv, (u + E32) * sv.abs() * (1 + 1e-6) + tiny(typ)),
                ("y", y, yv, (u + 64 * E32) * yv.abs() * (1 + 1e-6) + tiny(typ)),
                ("scale", qs[:, None], a / 127, 66 * E32 * a / 127),
                ("codes", q, yv * (127 / a), 0.5 + 127 * 132 * E32 + 0 * yv)):
            bad = ~((got[rows].double() - want).abs() <= bound)
            assert not bool(bad.any()), (what, lo, int(bad.sum()))
    # the sum over the residual and y over x: the same bits
    moe.moe_add_rmsnorm(d, x, r, w, r, x)
    torch.cuda.synchronize()
    assert torch.equal(r, s) and torch.equal(x, y)
    # the quantiser alone
    moe.moe_q8_quantize(d, x, q, qs)
    out.check()
    a = x.double().abs().amax(1)
    assert bool(((qs.double() - a / 127).abs() <= E32 * a / 127).all())
    within(q, x.double() * (127 / a)[:, None], lambda lo, v: 0.5 + 127 * 3 * E32 + 0 * v, "codes alone")


@pytest.mark.parametrize("T,H,typ", NORM)
def test_norm_backward(T, H, typ):
    print(f"streamed norm backward {T} {H} {typ}", flush=True)
    g = torch.Generator("cuda").manual_seed(T + 3 * H)
    s, dy, ds = rand(g, (T, H), typ, 2.0), rand(g, (T, H), typ), rand(g, (T, H), typ)
    w = torch.rand(H, generator=g, device="cuda") + 0.5
    d = moe.NormDims(T, H, moe.ELEM[TYPES[typ]], 1e-5)
    eps, u = float(np.float32(1e-5)), ref.HALF_STEP[typ]
    n = moe.moe_add_rmsnorm_backward_ws_bytes(d)
    out = Out()
    dx, dw, ws = out((T, H), TYPES[typ]), out((H,), torch.float32), out((n,), torch.uint8)
    for resid in (ds, None):
        moe.moe_add_rmsnorm_backward(d, s, w, dy, resid, dx, dw, ws, n)
        out.check()
        wantw, sizew = torch.zeros(H, device="cuda").double(), torch.zeros(H, device="cuda").double()
        for lo in range(0, T, 4096):
            rows = slice(lo, lo + 4096)
            sv, dv = s[rows].double(), dy[rows].double()
            rho = 1 / torch.sqrt((sv * sv).mean(1, keepdim=True) + eps)
            gv = dv * w.double()
            want = rho * gv - sv * rho ** 3 * (gv * sv).mean(1, keepdim=True)
            size = (rho * gv).abs() + sv.abs() * rho ** 3 * (gv * sv).abs().mean(1, keepdim=True)
            if resid is not None:
                want, size = want + resid[rows].double(), size + resid[rows].double().abs()
            bad = ~((dx[rows].double() - want).abs() <= u * want.abs() * (1 + 1e-6) + 160 * E32 * size + tiny(typ))
            assert not bool(bad.any()), ("dx", lo, int(bad.sum()))
            t = dv * sv * rho
            wantw, sizew = wantw + t.sum(0), sizew + t.abs().sum(0)
        # rows of one lane (at most T / 256 + 1), 3 folds or none, partial sums (at most 64 + 16)
        assert bool(((dw.double() - wantw).abs() <= (64 + T / 256 + 1 + 3 + 80) * E32 * sizew).all()), "dweight"
    # over dy and over dsum: the same bits
    moe.moe_add_rmsnorm_backward(d, s, w, dy, ds, dx, None, None, 0)
    over = ds.clone()
    moe.moe_add_rmsnorm_backward(d, s, w, dy, over, over, None, None, 0)
    moe.moe_add_rmsnorm_backward(d, s, w, dy, ds, dy, None, None, 0)
    torch.cuda.synchronize()
    assert torch.equal(over, dx) and torch.equal(dy, dx)


# T, H, E, k, n_shared, type: streamed stores alone, then streamed loads too
ROWS = [(1000, 2048, 64, 8, 1, "bf16"), (1000, 2048, 64, 8, 1, "f16"), (500, 2048, 64, 8, 1, "f32"),
        (2000, 2048, 64, 8, 1, "bf16"), (2000, 2048, 64, 8, 1, "f16"), (1000, 2048, 64, 8, 1, "f32"),
        (2001, 2112, 40, 9, 0, "bf16"), (300, 6208, 40, 11, 1, "f32")]


def test_rows_cover_both_limits():
    """Each type with stores past the caches alone and with loads too."""
    for typ in TYPES:
        sizes = [T * (k + n) * H * SIZE[t] for T, H, _, k, n, t in ROWS if t == typ]
        assert any(STORE < b <= LOAD for b in sizes) and any(b > LOAD for b in sizes), typ


@pytest.mark.parametrize("T,H,E,k,n_shared,typ", ROWS)
def test_rows(T, H, E, k, n_shared, typ):
    print(f"streamed rows {T} {H} {E} {k} {n_shared} {typ}", flush=True)
    r = ref.routing(np.random.default_rng(T + H + k), T, E, k, 128, 16, n_shared)
    tab = Tables(r, T)
    d = moe.make_dims(T, H, 64, E, k, n_shared)
    elem, dt, u = moe.ELEM[TYPES[typ]], TYPES[typ], ref.HALF_STEP[typ]
    n, S = T * (k + n_shared), T * k
    g = torch.Generator("cuda").manual_seed(T)
    x, dy, ys = rand(g, (T, H), typ), rand(g, (T, H), typ), rand(g, (n, H), typ)
    pos, w = torch.from_numpy(r["slot_pos"]).cuda().long(), torch.from_numpy(r["topk_w"]).cuda().double()
    tok = torch.from_numpy(ref.row_tokens(r, T, k, n_shared)).cuda().long()
    out = Out()
    rows = out((n, H), dt)
    moe.moe_dispatch_rows(d, elem, x, tab.c, rows)
    out.check()
    assert torch.equal(rows, x[tok])

    y, dx = out((T, H), dt), out((T, H), dt)
    moe.moe_combine_rows(d, elem, ys, tab.c, y)
    moe.moe_dispatch_rows_backward(d, elem, ys, tab.c, dx)
    out.check()
    for what, got, weight in (("y", y, w), ("dx", dx, torch.ones_like(w))):
        want, size = torch.zeros((T, H), device="cuda").double(), torch.zeros((T, H), device="cuda").double()
        for j in range(k):
            t = ys[pos[:, j]].double() * weight[:, j:j + 1]
            want, size = want + t, size + t.abs()
        if n_shared:
            want, size = want + ys[S:].double(), size + ys[S:].double().abs()
        bound = u * want.abs() * (1 + 1e-6) + (k + 1) * E32 * size * (1 + 1e-6) + tiny(typ)
        within(got, want, bound, what)
    if typ == "bf16":
        y2 = out((T, H), dt)
        moe.moe_combine(d, tab.c, ys, y2)
        out.check()
        assert torch.equal(y, y2)

    drows, dw = out((n, H), dt), out((T, k), torch.float32)
    moe.moe_combine_rows_backward(d, elem, dy, ys, tab.c, drows, dw)
    out.check()
    for j in range(k):
        want = dy.double() * w[:, j:j + 1]
        within(drows[pos[:, j]], want, (u + E32) * want.abs() * (1 + 1e-6) + tiny(typ), "drows")
        t = ys[pos[:, j]].double() * dy.double()
        # a lane adds at most H / 256 + 8 products one after the other, then ten steps of the tree
        assert bool(((dw[:, j].double() - t.sum(1)).abs() <= (H / 256 + 18) * E32 * t.abs().sum(1)).all()), "dtopk_w"
    if n_shared:
        assert torch.equal(drows[S:], dy)
    # without the weights' gradient, and over the rows themselves
    only, over, dw2 = out((n, H), dt), ys.clone(), out((T, k), torch.float32)
    moe.moe_combine_rows_backward(d, elem, dy, None, tab.c, only, None)
    moe.moe_combine_rows_backward(d, elem, dy, over, tab.c, over, dw2)
    out.check()
    assert torch.equal(only, drows) and torch.equal(over, drows) and torch.equal(dw, dw2)
    assert int(tab.status.item()) == 0


# T, E, k, tile_m_max: the kernels of the grouped products whose outputs can be this large
EXPERTS = [(9000, 16, 3, 32), (9000, 16, 3, 64), (8300, 1024, 3, 256), (9000, 16, 3, 128), (9001, 16, 3, 256)]


def expert_rows(x, xs, wq, ws, edges):
    return torch.cat([(x[lo:hi].double() @ wq[e].double().t()) * xs[lo:hi].double()[:, None] * ws[e].double()
                      for e, (lo, hi) in enumerate(zip(edges[:-1], edges[1:]))])


@pytest.mark.parametrize("T,E,k,tile", EXPERTS)
@pytest.mark.parametrize("skew", [False, True])
def test_expert_products(T, E, k, tile, skew):
    print(f"streamed experts {T} {E} {k} {tile} skew={skew}", flush=True)
    wide, narrow, rows = 512, 64, T * (k + 1)
    assert rows * wide * 2 > STORE
    rng = np.random.default_rng(T + E + tile)
    idx = np.stack([np.arange(k) if t % 5 else np.arange(E - k, E) for t in range(T)]) if skew else None
    r = ref.routing(rng, T, E, k, tile, 16, 1, idx)
    tab = Tables(r, T)
    tok = torch.from_numpy(ref.row_tokens(r, T, k, 1)).cuda().long()
    edges = r["offsets"].tolist() + [rows]
    g = torch.Generator("cuda").manual_seed(T)
    out = Out()
    # gate/up: narrow inputs, wide hidden rows
    d = moe.make_dims(T, narrow, wide, E, k, 1, tile, 16)
    assert len(r["blocks"]) <= moe.moe_max_blocks(d)
    wq, ws = codes(g, (E + 1, 2 * wide, narrow)), scales(g, (E + 1, 2 * wide))
    xq, xs = codes(g, (T, narrow)), scales(g, (T,))
    h = out((rows, wide), torch.bfloat16)
    moe.moe_q8_gate_up(d, xq, xs, tab.c, moe.Q8Bank(gu=wq.data_ptr(), gu_s=ws.data_ptr()),
                       moe.Q8Bank(gu=wq[E].data_ptr(), gu_s=ws[E].data_ptr()), h)
    out.check()
    gu = expert_rows(xq[tok], xs[tok], wq, ws, edges)
    a = gu[:, :wide]
    want = a * torch.sigmoid(a) * gu[:, wide:]
    within(h, want, (2.0 ** -8 + (16 + 6 * a.abs()) * E32) * want.abs() * (1 + 1e-6) + 1e-37, "h")
    del gu, a, want
    # down: narrow hidden rows, wide outputs
    d = moe.make_dims(T, wide, narrow, E, k, 1, tile, 16)
    wq, ws = codes(g, (E + 1, wide, narrow)), scales(g, (E + 1, wide))
    hq, hs = codes(g, (rows, narrow)), scales(g, (rows,))
    y = out((rows, wide), torch.bfloat16)
    moe.moe_q8_down(d, tab.c, moe.Q8Bank(dn=wq.data_ptr(), dn_s=ws.data_ptr()),
                    moe.Q8Bank(dn=wq[E].data_ptr(), dn_s=ws[E].data_ptr()), hq, hs, y)
    out.check()
    want = expert_rows(hq, hs, wq, ws, edges)
    within(y, want, (2.0 ** -8 + 3 * E32) * want.abs() * (1 + 1e-6) + 1e-37, "y_slots")
    assert int(tab.status.item()) == 0


@pytest.mark.parametrize("M,N,K,typ", [(3800, 4096, 192, "f32"), (2900, 4360, 320, "f32"), (4100, 4360, 192, "f16"),
                                       (4500, 8200, 64, "bf16")])
def test_product(M, N, K, typ):
    print(f"streamed product {M} {N} {K} {typ}", flush=True)
    assert M * N * SIZE[typ] > STORE
    g = torch.Generator("cuda").manual_seed(M)
    xq, xs, wq, ws = codes(g, (M, K)), scales(g, (M,)), codes(g, (N, K)), scales(g, (N,))
    out = Out()
    y = out((M, N), TYPES[typ])
    moe.moe_q8_matmul(moe.Q8Dims(M, N, K, moe.ELEM[TYPES[typ]]), xq, xs, wq, ws, y)
    out.check()
    want = (xq.double() @ wq.double().t()) * xs.double()[:, None] * ws.double()
    within(y, want, (ref.HALF_STEP[typ] + 3 * E32) * want.abs() * (1 + 1e-6) + tiny(typ), "product")
