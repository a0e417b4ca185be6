"""The entry points of include/moe_block.h on the CPU: bad arguments come back
with the documented codes before any launch, empty batches are accepted, and
the binding refuses tensors the C side could not check.  The float64 references
are pinned against hand-worked values and differences."""

import ctypes

import numpy as np
import pytest

import block_ref as ref
import w4_dequant_expert_amd as moe

torch = pytest.importorskip("torch")

P = [0x10000 * (i + 1) for i in range(12)]   # distinct aligned addresses, never read


def norm_dims(T=4, H=64, type=moe.ELEM_BF16, eps=1e-6):
    return moe.NormDims(T, H, type, eps)


BAD_NORM = [dict(T=-1), dict(T=(1 << 24) + 1), dict(H=0), dict(H=12), dict(H=16392), dict(type=3),
            dict(type=-1), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf"))]


@pytest.mark.parametrize("bad", BAD_NORM)
def test_norm_dims_refused(bad):
    L, d = moe.lib(), norm_dims(**bad)
    b = ctypes.byref(d)
    assert L.moe_add_rmsnorm(b, *P[:5], None, None, None) == -1
    assert L.moe_q8_quantize(b, *P[:3], None) == -1
    assert L.moe_add_rmsnorm_backward(b, *P[:7], 1 << 30, None) == -1
    assert L.moe_add_rmsnorm_backward_ws_bytes(b) == 0


def call_norm(d=None, **kw):
    a = dict(x=P[0], res=P[1], w=P[2], sum=P[3], y=P[4], yq=P[5], ys=P[6])
    a.update(kw)
    d = d or norm_dims()
    return moe.lib().moe_add_rmsnorm(ctypes.byref(d), a["x"], a["res"], a["w"], a["sum"], a["y"],
                                     a["yq"], a["ys"], None)


def test_norm_refusals():
    for name in ("x", "w"):
        assert call_norm(**{name: None}) == -1, name
    assert call_norm(y=None, yq=None, ys=None) == -1
    assert call_norm(ys=None) == -1 and call_norm(yq=None) == -1
    assert call_norm(y=P[3]) == -1                       # y over sum
    for name in ("x", "res", "w", "sum", "y", "yq"):
        assert call_norm(**{name: P[7] + 8}) == -2, name
    assert call_norm(ys=P[7] + 2) == -2
    assert moe.lib().moe_add_rmsnorm(None, *P[:7], None) == -1
    for kw in (dict(), dict(res=None, sum=None), dict(y=None), dict(yq=None, ys=None),
               dict(sum=P[0]), dict(y=P[1])):
        assert call_norm(norm_dims(T=0), **kw) == 0, kw


def call_backward(d=None, ws_bytes=None, **kw):
    a = dict(sum=P[0], w=P[1], dy=P[2], dsum=P[3], dx=P[4], dw=P[5], ws=P[6])
    a.update(kw)
    d = d or norm_dims()
    need = moe.moe_add_rmsnorm_backward_ws_bytes(d)
    return moe.lib().moe_add_rmsnorm_backward(
        ctypes.byref(d), a["sum"], a["w"], a["dy"], a["dsum"], a["dx"], a["dw"], a["ws"],
        need if ws_bytes is None else ws_bytes, None)


def test_norm_backward_refusals():
    d = norm_dims(T=300, H=256)
    need = moe.moe_add_rmsnorm_backward_ws_bytes(d)
    assert need > 0 and need % (256 * 4) == 0
    for name in ("sum", "w", "dy", "dx", "ws"):
        assert call_backward(d, **{name: None}) == -1, name
    for name in ("sum", "w", "dy", "dsum", "dx", "ws"):
        assert call_backward(d, **{name: P[8] + 8}) == -2, name
    assert call_backward(d, dw=P[8] + 2) == -2
    assert call_backward(d, ws_bytes=need - 1) == -3
    # no rows and no weight gradient: nothing to do, no workspace either
    d0 = norm_dims(T=0)
    assert moe.moe_add_rmsnorm_backward_ws_bytes(d0) == 0
    assert call_backward(d0, dw=None, ws=None, ws_bytes=0) == 0


@pytest.mark.parametrize("bad", [dict(M=-1), dict(M=(1 << 24) + 1), dict(N=0), dict(N=12),
                                 dict(N=(1 << 20) + 8), dict(K=0), dict(K=96), dict(K=65600),
                                 dict(type=3)])
def test_product_dims_refused(bad):
    a = dict(M=4, N=64, K=128, type=moe.ELEM_BF16)
    a.update(bad)
    d = moe.Q8Dims(*[a[n] for n in ("M", "N", "K", "type")])
    assert moe.lib().moe_q8_matmul(ctypes.byref(d), *P[:5], None) == -1


def test_product_refusals():
    L = moe.lib()
    d = moe.Q8Dims(4, 64, 128, moe.ELEM_BF16)
    for i in range(5):
        a = list(P[:5])
        a[i] = None
        assert L.moe_q8_matmul(ctypes.byref(d), *a, None) == -1, i
        a[i] = P[6] + (2 if i == 1 else 8)
        assert L.moe_q8_matmul(ctypes.byref(d), *a, None) == -2, i
    assert L.moe_q8_matmul(None, *P[:5], None) == -1
    assert L.moe_q8_matmul(ctypes.byref(moe.Q8Dims(0, 64, 128, 0)), *P[:5], None) == 0
    q = norm_dims()
    for i in range(3):
        a = list(P[:3])
        a[i] = None
        assert L.moe_q8_quantize(ctypes.byref(q), *a, None) == -1
        a[i] = P[6] + (2 if i == 2 else 8)
        assert L.moe_q8_quantize(ctypes.byref(q), *a, None) == -2
    assert L.moe_q8_quantize(ctypes.byref(norm_dims(T=0)), *P[:3], None) == 0


def tables():
    return moe.RouteOut(*[0x100000 + 256 * i for i in range(11)], 0)


def test_expert_product_refusals():
    L, r = moe.lib(), tables()
    d = moe.make_dims(4, 128, 64, 8, 2, 1)
    full = moe.Q8Bank(P[0], P[1], P[2], P[3])
    ref_ = ctypes.byref

    def gate_up(d=d, x=P[4], xs=P[5], r=r, routed=full, shared=full, h=P[6]):
        return L.moe_q8_gate_up(ref_(d), x, xs, ref_(r) if r else None, ref_(routed) if routed else None,
                                ref_(shared) if shared else None, h, None)

    def down(d=d, x=P[4], xs=P[5], r=r, routed=full, shared=full, h=P[6]):
        return L.moe_q8_down(ref_(d), ref_(r) if r else None, ref_(routed) if routed else None,
                             ref_(shared) if shared else None, x, xs, h, None)

    for call, halves in ((gate_up, ("gu", "gu_s")), (down, ("dn", "dn_s"))):
        for name in ("x", "xs", "r", "routed", "shared", "h"):
            assert call(**{name: None}) == -1, name
        assert call(x=P[4] + 8) == -2 and call(xs=P[5] + 2) == -2 and call(h=P[6] + 8) == -2
        for half in halves:
            for which in ("routed", "shared"):
                b = moe.Q8Bank(P[0], P[1], P[2], P[3])
                setattr(b, half, None)
                assert call(**{which: b}) == -1, (which, half)
                setattr(b, half, P[7] + 8)
                assert call(**{which: b}) == -2, (which, half)
        assert call(d=moe.make_dims(4, 128, 96, 8, 2, 1)) == -1
        assert call(d=moe.make_dims(0, 128, 64, 8, 2, 1)) == 0
        # the other half of the bank is not looked at
        only = moe.Q8Bank(**{h: P[i] for i, h in enumerate(halves)})
        assert call(d=moe.make_dims(0, 128, 64, 8, 2, 1), routed=only, shared=only) == 0


def test_row_refusals():
    L, r = moe.lib(), tables()
    d, d0 = moe.make_dims(4, 128, 64, 8, 2, 1), moe.make_dims(0, 128, 64, 8, 2, 1)
    b = ctypes.byref
    for f in (L.moe_dispatch_rows, L.moe_dispatch_rows_backward, L.moe_combine_rows):
        assert f(b(d), 3, P[0], b(r), P[1], None) == -1
        assert f(b(d), 1, None, b(r), P[1], None) == -1
        assert f(b(d), 1, P[0], None, P[1], None) == -1
        assert f(b(d), 1, P[0], b(r), None, None) == -1
        assert f(b(d), 1, P[0] + 8, b(r), P[1], None) == -2
        assert f(b(d), 1, P[0], b(r), P[1] + 8, None) == -2
        assert f(None, 1, P[0], b(r), P[1], None) == -1
        assert f(b(d0), 1, P[0], b(r), P[1], None) == 0
        for name in ("slot_pos", "status"):
            bad = tables()
            setattr(bad, name, None)
            assert f(b(d), 1, P[0], b(bad), P[1], None) == -1, name
            setattr(bad, name, 0x5002)
            assert f(b(d), 1, P[0], b(bad), P[1], None) == -2, name
    g = L.moe_combine_rows_backward
    assert g(b(d), 1, None, P[1], b(r), P[2], P[3], None) == -1
    assert g(b(d), 1, P[0], None, b(r), P[2], P[3], None) == -1      # rows, for dtopk_w
    assert g(b(d0), 1, P[0], None, b(r), P[2], None, None) == 0      # not for drows alone
    assert g(b(d), 1, P[0], P[1], b(r), None, P[3], None) == -1
    assert g(b(d), 1, P[0], P[1], b(r), P[2], P[3] + 2, None) == -2
    assert g(b(d), 1, P[0], P[1], b(r), P[2] + 8, P[3], None) == -2
    assert g(b(d), 3, P[0], P[1], b(r), P[2], P[3], None) == -1


def test_binding_refuses_host_strided_and_short_tensors():
    """What the C side could not see never reaches a kernel."""
    _arg = moe.moe._arg
    assert _arg(None, 16, "x", 0) is None and _arg(4096, 16, "x", 0) == 4096
    x = torch.zeros((4, 4))
    host = x.get_device()   # -1
    assert _arg(x, 64, "x", host) == x.data_ptr()
    for t, n, dev in ((x, 64, 0), (x, 65, host), (x.t(), 64, host), (x[:, :2], 32, host)):
        with pytest.raises(ValueError):
            _arg(t, n, "x", dev)


# ------------------------------------------------------------------ the references themselves

def test_reference_norm_by_hand():
    s, y = ref.norm(np.array([[3.0, 4.0]]), np.array([[0.0, 0.0]]), np.array([1.0, 2.0]), 0.0)
    rms = np.sqrt(12.5)
    assert np.allclose(s, [[3.0, 4.0]]) and np.allclose(y, [[3 / rms, 8 / rms]], rtol=1e-15)


def test_reference_norm_gradient_by_differences():
    rng = np.random.default_rng(3)
    s, w, dy, ds = (rng.standard_normal(n) for n in ((3, 16), (16,), (3, 16), (3, 16)))

    def loss(s, w):
        return (ref.norm(s, None, w, 1e-3)[1] * dy).sum() + (s * ds).sum()

    dx, dw, _, _ = ref.norm_backward(s, w, dy, ds, 1e-3)
    h = 1e-6
    for i in range(3):
        for j in range(16):
            e = np.zeros_like(s)
            e[i, j] = h
            assert abs((loss(s + e, w) - loss(s - e, w)) / (2 * h) - dx[i, j]) < 1e-7
    for j in range(16):
        e = np.zeros_like(w)
        e[j] = h
        assert abs((loss(s, w + e) - loss(s, w - e)) / (2 * h) - dw[j]) < 1e-7


def test_reference_combine_gradient_by_differences():
    rng = np.random.default_rng(4)
    T, E, k, H = 5, 4, 2, 3
    r = ref.routing(rng, T, E, k, 16, 16, 1)
    rows, dy = rng.standard_normal((T * 3, H)), rng.standard_normal((T, H))
    w, pos = r["topk_w"].astype(np.float64), r["slot_pos"]

    def loss(rows, w):
        return (ref.combine(rows, w, pos, 1)[0] * dy).sum()

    drows, dw, _ = ref.combine_backward(dy, rows, w, pos, 1)
    h = 1e-6
    for i in range(T * 3):
        for j in range(H):
            e = np.zeros_like(rows)
            e[i, j] = h
            assert abs((loss(rows + e, w) - loss(rows - e, w)) / (2 * h) - drows[i, j]) < 1e-8
    for t in range(T):
        for j in range(k):
            e = np.zeros_like(w)
            e[t, j] = h
            assert abs((loss(rows, w + e) - loss(rows, w - e)) / (2 * h) - dw[t, j]) < 1e-8
    # the dispatch's gradient is the combine with weights of one: <x sorted, g> = <x, gradient of g>
    x, g = rng.standard_normal((T, H)), rng.standard_normal((T * 3, H))
    sorted_x = x[ref.row_tokens(r, T, k, 1)]
    assert np.isclose((sorted_x * g).sum(), (x * ref.combine(g, None, pos, 1)[0]).sum(), rtol=1e-12)


def test_reference_routing_matches_the_oracle(orc):
    import oracle
    from synth import build_config
    c = build_config("tiny16")
    sh = c["shape"]
    o = oracle.route(c["x"], c["wr"], None, sh.k, sh.n_shared, 32, 16)
    r = ref.routing(np.random.default_rng(0), c["T"], sh.E, sh.k, 32, 16, sh.n_shared, idx=np.asarray(o["topk_idx"]))
    for name in ("counts", "offsets", "sorted_slot", "blocks"):
        assert np.array_equal(np.asarray(o[name]).reshape(-1), r[name].reshape(-1)), name
    assert np.array_equal(np.asarray(o["slot_pos"]).reshape(-1), r["slot_pos"].reshape(-1))


def test_reference_silu():
    g = np.array([-800.0, -1.0, 0.0, 1.0, 800.0])
    want = [0.0, -1 / (1 + np.e), 0.0, 1 / (1 + 1 / np.e), 800.0]
    assert np.allclose(ref.silu(g), want, rtol=1e-14, atol=1e-300)
