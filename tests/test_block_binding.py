"""The binding's own checks for the operators of include/moe_block.h, on the CPU: host tensors stand
for device ones and a stub for the library, so nothing is launched."""

import numpy as np
import pytest

import w4_dequant_expert_amd as moe

torch = pytest.importorskip("torch")

F32, BF16, F16, I8 = torch.float32, torch.bfloat16, torch.float16, torch.int8


class Stub:
    """A library that only records which functions were called."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append(name)
            return 0
        return call


@pytest.fixture
def stub(monkeypatch):
    s = Stub()
    monkeypatch.setattr(moe.moe, "_lib", s)
    monkeypatch.setattr(moe.moe, "_device", lambda: torch.zeros(1).get_device())
    return s


T, H, I, E, K = 3, 64, 64, 4, 2
ROWS = T * (K + 1)


def calls():
    """Every entry point: its name, the row type of the call, and its arrays (name, shape, type; None:
    the row type)."""
    d = moe.make_dims(T, H, I, E, K, 1)
    r, b = moe.RouteOut(), moe.Q8Bank()
    out = []
    for elem in (moe.ELEM_F32, moe.ELEM_BF16, moe.ELEM_F16):
        n = moe.NormDims(T, H, elem, 1e-6)
        out += [
            ("moe_add_rmsnorm", elem, lambda a, n=n: moe.moe_add_rmsnorm(n, *a, stream=0),
             [("x", (T, H), None), ("res", (T, H), None), ("weight", (H,), F32), ("sum", (T, H), None),
              ("y", (T, H), None), ("yq", (T, H), I8), ("ys", (T,), F32)]),
            ("moe_add_rmsnorm_backward", elem, lambda a, n=n: moe.moe_add_rmsnorm_backward(n, *a, None, 0, stream=0),
             [("sum", (T, H), None), ("weight", (H,), F32), ("dy", (T, H), None), ("dsum", (T, H), None),
              ("dx", (T, H), None), ("dweight", (H,), F32)]),
            ("moe_q8_quantize", elem, lambda a, n=n: moe.moe_q8_quantize(n, *a, stream=0),
             [("x", (T, H), None), ("xq", (T, H), I8), ("xs", (T,), F32)]),
            ("moe_q8_matmul", elem, lambda a, elem=elem: moe.moe_q8_matmul(moe.Q8Dims(T, I, H, elem), *a, stream=0),
             [("xq", (T, H), I8), ("xs", (T,), F32), ("wq", (I, H), I8), ("ws", (I,), F32), ("out", (T, I), None)]),
            ("moe_dispatch_rows", elem, lambda a, e=elem: moe.moe_dispatch_rows(d, e, a[0], r, a[1], stream=0),
             [("x", (T, H), None), ("rows", (ROWS, H), None)]),
            ("moe_dispatch_rows_backward", elem,
             lambda a, e=elem: moe.moe_dispatch_rows_backward(d, e, a[0], r, a[1], stream=0),
             [("drows", (ROWS, H), None), ("dx", (T, H), None)]),
            ("moe_combine_rows", elem, lambda a, e=elem: moe.moe_combine_rows(d, e, a[0], r, a[1], stream=0),
             [("rows", (ROWS, H), None), ("y", (T, H), None)]),
            ("moe_combine_rows_backward", elem,
             lambda a, e=elem: moe.moe_combine_rows_backward(d, e, a[0], a[1], r, a[2], a[3], stream=0),
             [("dy", (T, H), None), ("rows", (ROWS, H), None), ("drows", (ROWS, H), None), ("dtopk_w", (T, K), F32)]),
        ]
    out += [
        ("moe_q8_gate_up", None, lambda a: moe.moe_q8_gate_up(d, a[0], a[1], r, b, b, a[2], stream=0),
         [("xq", (T, H), I8), ("xs", (T,), F32), ("h", (ROWS, I), BF16)]),
        ("moe_q8_down", None, lambda a: moe.moe_q8_down(d, r, b, b, *a, stream=0),
         [("hq", (ROWS, I), I8), ("hs", (ROWS,), F32), ("y_slots", (ROWS, H), BF16)]),
    ]
    return out


ROW = {moe.ELEM_F32: F32, moe.ELEM_BF16: BF16, moe.ELEM_F16: F16}
# enough bytes whatever is asked for, but another type
WRONG = {F32: (torch.float64, torch.int32, BF16), I8: (torch.uint8, torch.int16, F32),
         BF16: (F16, F32, I8), F16: (BF16, F32, I8)}


def test_arrays_of_another_type_are_refused(stub):
    for name, elem, call, arrays in calls():
        types = [ROW[elem] if t is None else t for _, _, t in arrays]
        good = [torch.zeros(shape, dtype=t) for (_, shape, _), t in zip(arrays, types)]
        stub.calls.clear()
        call(good)
        assert stub.calls == [name]
        for i, (arg, shape, _) in enumerate(arrays):
            for wrong in WRONG[types[i]]:
                bad = list(good)
                bad[i] = torch.zeros((shape[0] * 4, *shape[1:]), dtype=wrong)
                with pytest.raises(ValueError, match=f"^{arg}: "):
                    call(bad)
        assert stub.calls == [name]
        # 16-bit rows as the integers of their bits
        if elem in (moe.ELEM_BF16, moe.ELEM_F16):
            call([t.view(torch.int16) if t.dtype == ROW[elem] else t for t in good])
            call([t.view(torch.uint16) if t.dtype == ROW[elem] else t for t in good])
            assert stub.calls == [name] * 3


def test_arrays_that_are_not_looked_at_have_any_type(stub):
    e = torch.empty(0, dtype=torch.float64)
    moe.moe_q8_matmul(moe.Q8Dims(0, I, H, moe.ELEM_F32), e, e, torch.zeros((I, H), dtype=I8), torch.zeros(I), e, stream=0)
    assert stub.calls == ["moe_q8_matmul"]


# ------------------------------------------------------------------------------- the 8-bit layer

def q8_bank(n, h=H, i=I):
    """A bank on the host, made without the quantiser."""
    b = moe.DeviceBankQ8.__new__(moe.DeviceBankQ8)
    b.n, b.H, b.I = n, h, i
    b.t = {"gu": torch.zeros((n, 2 * i, h), dtype=I8), "gu_s": torch.zeros((n, 2 * i)),
           "dn": torch.zeros((n, h, i), dtype=I8), "dn_s": torch.zeros((n, h))}
    b.c = moe.Q8Bank(*[b.t[k].data_ptr() for k in ("gu", "gu_s", "dn", "dn_s")])
    return b


def q8_layer(routed, shared, n_shared=1, **kw):
    return moe.Q8MoeLayer(H, I, E, K, n_shared, routed, shared, np.zeros((H, E), np.float32), T_max=8, device="cpu", **kw)


def test_layer_refuses_banks_that_are_not_its_own_size(stub):
    layer = q8_layer(q8_bank(E), q8_bank(1))
    x, y = torch.zeros((T, H), dtype=BF16), torch.zeros((T, H), dtype=BF16)
    layer.forward(x, y, stream=0)
    layer.forward(x, y, routed=q8_bank(E + 1), shared=q8_bank(2), stream=0)   # more experts than are read
    assert stub.calls.count("moe_q8_gate_up") == 2 and stub.calls.count("moe_q8_down") == 2
    stub.calls.clear()
    d = layer.dims(T)
    w4 = moe.DeviceBank.from_tensors({"gu": torch.zeros(1), "dn": torch.zeros(1)}, E, H, I)
    for routed in (q8_bank(E - 1), q8_bank(E, h=H + 64), q8_bank(E, i=I - 32), q8_bank(E, h=H // 2), w4):
        with pytest.raises(ValueError, match="^routed: "):
            q8_layer(routed, q8_bank(1))
        with pytest.raises(ValueError, match="^routed: "):
            layer.gate_up(d, x, routed=routed, stream=0)
        with pytest.raises(ValueError, match="^routed: "):
            layer.down(d, routed=routed, stream=0)
    for shared in (q8_bank(0), q8_bank(1, h=H + 64), q8_bank(1, i=2 * I)):
        with pytest.raises(ValueError, match="^shared: "):
            q8_layer(q8_bank(E), shared)
        with pytest.raises(ValueError, match="^shared: "):
            layer.down(d, shared=shared, stream=0)
    assert not {"moe_q8_gate_up", "moe_q8_down"} & set(stub.calls)
    # without a shared expert none is read, whatever is at hand
    q8_layer(q8_bank(E), None, n_shared=0)
    q8_layer(q8_bank(E), q8_bank(1, h=H + 64), n_shared=0).down(d, shared=q8_bank(0), stream=0)
    stub.calls.clear()
    # replaced on the layer itself
    layer.routed = q8_bank(1)
    with pytest.raises(ValueError, match="^routed: "):
        layer.forward(x, y, stream=0)
    with pytest.raises(ValueError, match="^routed: "):
        layer.forward_residual(x, x.clone(), torch.ones(H), y, stream=0)
    assert "moe_add_rmsnorm" not in stub.calls


def test_bank_refuses_an_odd_count_of_gate_and_up_rows(stub):
    with pytest.raises(ValueError):
        moe.DeviceBankQ8(torch.zeros((2, 129, 64)), torch.zeros((2, 64, 64)))
    assert not stub.calls


def checkpoint(n=2):
    z = lambda rows, k, t: np.zeros((n, rows, k), t)
    return dict(gu_q=z(2 * I, H // 2, np.uint8), gu_s=z(2 * I, H // 64, np.uint16), gu_b=z(2 * I, H // 64, np.uint16),
                dn_q=z(H, I // 2, np.uint8), dn_s=z(H, I // 64, np.uint16), dn_b=z(H, I // 64, np.uint16))


def test_bank_from_4_bits_checks_what_the_dequantiser_gets(stub, monkeypatch):
    """Arrays off the current device, with too few scales or of another type never reach it."""
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: type("S", (), dict(cuda_stream=0, synchronize=lambda s: None))())
    monkeypatch.setattr(moe.moe, "_raw_stream", lambda device: 0)
    moe.DeviceBankQ8.from_w4(checkpoint(), device="cpu")
    assert stub.calls == ["moe_w4_dequant"] * 2 + ["moe_q8_quantize"] * 2
    stub.calls.clear()
    bad = []
    for half, field in (("gu", "s"), ("gu", "b"), ("dn", "s"), ("dn", "b")):
        c = checkpoint()
        c[f"{half}_{field}"] = c[f"{half}_{field}"][:1]
        bad.append((f"{half}_{field}", c))
        c = checkpoint()
        c[f"{half}_{field}"] = c[f"{half}_{field}"].astype(np.float32)
        bad.append((f"{half}_{field}", c))
    for what, c in bad:
        with pytest.raises(ValueError, match=f"^{what}: "):
            moe.DeviceBankQ8.from_w4(c, device="cpu")
    monkeypatch.setattr(moe.moe, "_device", lambda: 0)
    with pytest.raises(ValueError, match="^gu_q: "):
        moe.DeviceBankQ8.from_w4(checkpoint(), device="cpu")
    assert stub.calls.count("moe_w4_dequant") == 4    # the gate/up half of the four whose down half was wrong


def test_widths_that_the_quantiser_does_not_take_are_refused_at_construction(stub):
    wide = moe.NORM_MAX_H + 64
    for h, i in ((wide, I), (H, wide)):
        with pytest.raises(ValueError, match="quantised at up to"):
            moe.DeviceBankQ8(torch.zeros((1, 2 * i, h)), torch.zeros((1, h, i)))
        with pytest.raises(ValueError, match="quantised at up to"):
            moe.Q8MoeLayer(h, i, E, K, 0, None, None, None, T_max=8, device="cpu")
    assert not stub.calls


def test_layer_quantises_more_rows_than_one_call_takes(stub, monkeypatch):
    """h goes to the quantiser in runs of at most its row limit (a small one here)."""
    monkeypatch.setattr(moe.moe, "NORM_MAX_T", 7)
    seen = []
    monkeypatch.setattr(moe.moe, "moe_q8_quantize", lambda d, x, q, s, stream=None: seen.append(
        (d.T, x.data_ptr(), q.data_ptr(), s.data_ptr())))
    layer = q8_layer(q8_bank(E), q8_bank(1))
    for t in (0, 1, 2, 3, 5, 7, 8):
        seen.clear()
        layer.down(layer.dims(t), stream=0)
        rows = t * (K + 1)
        assert [n for n, *_ in seen] == ([7] * (rows // 7) + [rows % 7] * (rows % 7 > 0) or [0])
        for j, (_, x, q, s) in enumerate(seen):
            assert (x, q, s) == (layer.h.data_ptr() + 14 * j * I, layer.hq.data_ptr() + 7 * j * I,
                                 layer.hs.data_ptr() + 28 * j)


def test_banks_of_more_rows_than_one_call_takes_go_in_pieces(stub, monkeypatch):
    """2^24 rows for the quantiser, 2^32 groups of eight weights for the dequantiser; and a checkpoint in
    pieces gets the addresses of its pieces."""
    pieces = moe.moe._pieces
    for n, rows, k in ((256, 1024, 2048), (256, 2 ** 17, 64), (1024, 2 ** 15 + 128, 64), (5, 2 ** 17, 16384),
                       (256, 4096, 16384), (1, 64, 64), (0, 64, 64)):
        p = pieces(n, rows, k)
        assert [e for s in p for e in range(s.start, s.stop)] == list(range(n))
        for s in p:
            m = s.stop - s.start
            assert m >= 1 and m * rows <= 2 ** 24 and (m * rows * (k // 8) + 255) // 256 * 256 < 2 ** 32
    assert len(pieces(256, 1024, 2048)) == 1 and len(pieces(256, 2 ** 17, 64)) == 2
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: type("S", (), dict(synchronize=lambda s: None))())
    monkeypatch.setattr(moe.moe, "NORM_MAX_T", 2 * 2 * I)   # two experts' gate and up rows
    seen = []
    monkeypatch.setattr(moe.moe, "moe_w4_dequant", lambda r, k, q, s, b, w: seen.append((r, q.shape, s.shape, w.shape)))
    monkeypatch.setattr(moe.moe, "moe_q8_quantize", lambda d, w, q, s: seen.append((d.T, w.shape, q.shape, s.shape)))
    moe.DeviceBankQ8.from_w4(checkpoint(5), device="cpu")
    two_i = 2 * I
    want = [(m * two_i, (m, two_i, H // 2), (m, two_i, 1), (m, two_i, H)) for m in (2, 2, 1)]
    want += [(m * H, (m, H, I // 2), (m, H, 1), (m, H, I)) for m in (4, 1)]
    want += [(m * two_i, (m, two_i, H), (m, two_i, H), (m, two_i)) for m in (2, 2, 1)]
    want += [(m * H, (m, H, I), (m, H, I), (m, H)) for m in (4, 1)]
    assert seen == want


def test_the_4_bit_layer_holds_no_buffer_for_the_norm(stub):
    """Who calls forward alone pays nothing for forward_residual."""
    bank = moe.DeviceBank.from_tensors({"gu": torch.zeros(1), "dn": torch.zeros(1)}, E, H, I)
    layer = moe.MoeLayer(H, I, E, K, 1, bank, bank, np.zeros((H, E), np.float32), T_max=8, device="cpu")
    held = {v.untyped_storage().data_ptr(): v.untyped_storage().nbytes() for v in vars(layer).values()
            if isinstance(v, torch.Tensor)}
    assert sum(held.values()) == 4 * H * E + 2 * 8 * (K + 1) * (H + I)   # the router, y_slots and h


def test_residual_layer_checks_its_output_first(stub):
    w4 = moe.DeviceBank.from_tensors({"gu": torch.zeros(1), "dn": torch.zeros(1)}, E, H, I)
    for layer in (q8_layer(q8_bank(E), q8_bank(1)),
                  moe.MoeLayer(H, I, E, K, 1, w4, w4, np.zeros((H, E), np.float32), T_max=8, device="cpu")):
        stub.calls.clear()
        x, res, w = torch.zeros((T, H), dtype=BF16), torch.zeros((T, H), dtype=BF16), torch.ones(H)
        for y in (torch.zeros((T - 1, H), dtype=BF16), torch.zeros((T, H)), torch.zeros((T, 2 * H), dtype=BF16)[:, ::2]):
            with pytest.raises(ValueError, match="^y: "):
                layer.forward_residual(x, res, w, y, stream=0)
        with pytest.raises(ValueError, match="exceeds"):
            layer.forward_residual(torch.zeros((9, H), dtype=BF16), res, w, x, stream=0)
        assert not stub.calls
        layer.forward_residual(x, res, w, torch.zeros((T, H), dtype=torch.int16), stream=0)
        assert stub.calls[0] == "moe_add_rmsnorm"
