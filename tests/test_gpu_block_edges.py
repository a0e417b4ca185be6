"""Edges of the operators of include/moe_block.h on the GPU: table entries that
only some kernels would take, launches and batches past a limit, the streamed
forms, and the layer's checks.  References and bounds as in test_gpu_block.py."""

from __future__ import annotations

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import block_ref as ref  # noqa: E402
import w4_dequant_expert_amd as moe  # noqa: E402
from test_gpu_block import Tables, bank, codes, f32  # noqa: E402


# tokens, experts, tile_m_max: one for each kernel of the grouped products
@pytest.mark.parametrize("T,E,tile", [(8, 8, 16), (40, 6, 32), (100, 6, 64), (300, 4, 128), (600, 4, 256)])
def test_a_block_taller_than_the_map_allows_is_refused_by_every_kernel(T, E, tile):
    print(f"tall block {T} {E} {tile}", flush=True)
    H, I, k = 128, 64, 2
    rng = np.random.default_rng(T)
    r = ref.routing(rng, T, E, k, tile, 16, 1)
    d = moe.make_dims(T, H, I, E, k, 1, tile, 16)
    rows = T * (k + 1)
    gq, gs, _, _ = bank(rng, E + 1, 2 * I, H)
    dq, ds, _, _ = bank(rng, E + 1, H, I)
    xq, _ = codes(rng, (T, H))
    xs, _ = f32(rng, T, 0.0005, 0.002)
    hq, _ = codes(rng, (rows, I))
    hs, _ = f32(rng, rows, 0.0005, 0.002)
    routed = moe.Q8Bank(gq.data_ptr(), gs.data_ptr(), dq.data_ptr(), ds.data_ptr())
    shared = moe.Q8Bank(gq[E].data_ptr(), gs[E].data_ptr(), dq[E].data_ptr(), ds[E].data_ptr())

    def run(r):
        tab = Tables(r, T)
        h = torch.zeros((rows, I), dtype=torch.bfloat16, device="cuda")
        y = torch.zeros((rows, H), dtype=torch.bfloat16, device="cuda")
        moe.moe_q8_gate_up(d, xq, xs, tab.c, routed, shared, h)
        up = int(tab.status.item())
        tab.status.zero_()
        moe.moe_q8_down(d, tab.c, routed, shared, hq, hs, y)
        torch.cuda.synchronize()
        return h, y, up, int(tab.status.item())

    h, y, up, down = run(r)
    assert up == 0 and down == 0
    b = {n: v.copy() for n, v in r.items()}
    lost = slice(0, int(b["blocks"][0, 2]))
    b["blocks"][0, 2] = tile + 1
    h2, y2, up, down = run(b)
    assert up & moe.STATUS_BAD_INDEX and down & moe.STATUS_BAD_INDEX
    for got, want in ((h2, h), (y2, y)):
        assert bool((got[lost] == 0).all()) and torch.equal(got[lost.stop:], want[lost.stop:])


def test_a_launch_of_more_than_2_32_threads():
    """A million tokens in blocks of 16 rows: more workgroups than a launch holds along x.  The map here
    ends after a few blocks, and the arrays hold those blocks' rows alone."""
    T, H, I, E, k = 1 << 20, 8192, 64, 64, 8
    d = moe.make_dims(T, H, I, E, k, 0, 16, 16)
    S = T * k
    assert moe.moe_max_blocks(d) * (H // 128) * 128 >= 2 ** 32
    rng = np.random.default_rng(12)
    n = 2000
    at = np.arange(0, n, 16)
    blocks = np.zeros((moe.moe_max_blocks(d), 4), np.int32)
    blocks[:len(at)] = [[i % E, a, min(16, n - a), 16] for i, a in enumerate(at)]
    tab = dict(topk_idx=np.zeros(1, np.int32), topk_w=np.zeros(1, np.float32), counts=np.zeros(E, np.int32),
               offsets=np.zeros(E + 1, np.int32), sorted_slot=np.zeros(1, np.int32), slot_pos=np.zeros(1, np.int32),
               blocks=blocks, n_blocks=np.array([len(at)], np.int32))
    tab = Tables(tab, T)
    q, s, qv, sv = bank(rng, E, H, I)
    hq, hv = codes(rng, (n, I))
    hs, hsv = f32(rng, n, 0.0005, 0.002)
    y = torch.zeros((n, H), dtype=torch.bfloat16, device="cuda")
    assert S > n   # the binding would ask for all rows: raw addresses
    moe.moe_q8_down(d, tab.c, moe.Q8Bank(dn=q.data_ptr(), dn_s=s.data_ptr()), None, hq.data_ptr(), hs.data_ptr(),
                    y.data_ptr())
    torch.cuda.synchronize()
    group = np.arange(n) // 16 % E
    for g in np.unique(group):
        m = group == g
        want = ref.product(hv[m], hsv[m], qv[g], sv[g])
        got = y[torch.from_numpy(m).cuda()].double().cpu().numpy()
        assert (np.abs(got - want) <= (2.0 ** -8 + 3 * ref.EPS32) * np.abs(want) * (1 + 1e-6) + 1e-37).all()
    assert int(tab.status.item()) == 0


# ------------------------------------------------------------------------------------- the 8-bit bank

def test_a_bank_is_complete_when_it_is_made():
    """Its weights may be used on any stream from then on, as those of a 4-bit bank."""
    from synth import build_config
    c = build_config("tiny16")
    a = torch.randn((4096, 4096), device="cuda")
    gu, dn = torch.randn((8, 1024, 2048), device="cuda"), torch.randn((8, 2048, 512), device="cuda")
    for make in (lambda: moe.DeviceBankQ8(gu, dn), lambda: moe.DeviceBankQ8.from_w4(c["routed"]),
                 lambda: moe.DeviceBank(c["routed"])):
        for _ in range(8):
            a = torch.mm(a, a).mul_(1e-3)   # work that the bank's own waits behind
        make()
        assert torch.cuda.current_stream().query()


def test_layer_of_more_rows_than_the_quantiser_takes_at_once():
    """A million tokens with sixteen experts and a shared one each: 17 * 2^20 rows between the products.
    Tokens repeat with a period, so every period has the first one's outputs."""
    H, I, E, k, T, period = 64, 64, 16, 16, 1 << 20, 1 << 14
    print(f"layer of {T * (k + 1)} rows", flush=True)
    rng = np.random.default_rng(17)
    gu = torch.from_numpy((rng.standard_normal((E + 1, 2 * I, H)) / 8).astype(np.float32)).cuda()
    dn = torch.from_numpy((rng.standard_normal((E + 1, H, I)) / 8).astype(np.float32)).cuda()
    wr = rng.standard_normal((H, E)).astype(np.float32)
    routed, shared = moe.DeviceBankQ8(gu[:E], dn[:E]), moe.DeviceBankQ8(gu[E:], dn[E:])
    x = torch.from_numpy(rng.standard_normal((period, H)).astype(np.float32)).cuda().to(torch.bfloat16)
    small = moe.Q8MoeLayer(H, I, E, k, 1, routed, shared, wr, None, T_max=period, tile_m_max=256)
    want = torch.empty_like(x)
    small.forward(x, want)
    layer = moe.Q8MoeLayer(H, I, E, k, 1, routed, shared, wr, None, T_max=T, tile_m_max=256)
    assert T * (k + 1) > moe.NORM_MAX_T
    y = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    layer.forward(x.repeat(T // period, 1), y)
    torch.cuda.synchronize()
    assert int(layer.rt.status.item()) == 0 and int(small.rt.status.item()) == 0
    assert bool(torch.isfinite(want.float()).all()) and float(want.abs().max()) > 0
    # the router scores, and so every weight and output, are defined bit for bit
    assert bool((y.view(T // period, period, H) == want).all())


def test_bank_of_more_rows_than_the_quantiser_takes_at_once():
    """Three experts of 2^23 gate and up rows: two calls, and every row as by itself."""
    n, rows, H = 3, 1 << 23, 8
    gu = torch.randn((n, rows, H), device="cuda", generator=torch.Generator("cuda").manual_seed(3)).to(torch.bfloat16)
    q, s = moe.DeviceBankQ8._quantize(gu)
    one, ones = torch.empty_like(q[0]), torch.empty_like(s[0])
    for e in range(n):
        moe.moe_q8_quantize(moe.NormDims(rows, H, moe.ELEM_BF16, 0.0), gu[e], one, ones)
        assert torch.equal(q[e], one) and torch.equal(s[e], ones)


# ------------------------------------------------------------------------- the 4-bit layer and the norm

@pytest.mark.parametrize("T,tile", [(1, 32), (5, 32), (40, 16), (300, 128), (700, 256)])
def test_residual_layer_in_4_bits_over_its_kernels(T, tile):
    """The norm's rows lie in the layer's own buffers: the bits of the separate calls, twice in a row."""
    from synth import build_config
    c = build_config("tiny16")
    sh = c["shape"]
    layer = moe.MoeLayer(sh.H, sh.I, sh.E, sh.k, sh.n_shared, moe.DeviceBank(c["routed"]), moe.DeviceBank(c["shared"]),
                         c["wr"], None, T_max=T, tile_m_max=tile)
    g = torch.Generator("cuda").manual_seed(T)
    x, res = (torch.randn((T, sh.H), device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
    w = torch.linspace(0.5, 1.5, sh.H, device="cuda")
    s, xn, want, y = (torch.empty_like(x) for _ in range(4))
    moe.moe_add_rmsnorm(moe.NormDims(T, sh.H, moe.ELEM_BF16, 1e-6), x, res, w, s, xn)
    layer.forward(xn, want)
    for _ in range(2):
        r = res.clone()
        layer.forward_residual(x, r, w, y)
        torch.cuda.synchronize()
        assert torch.equal(r, s) and torch.equal(y, want) and int(layer.rt.status.item()) == 0
