"""The operators around the expert layer, as measured calls: the residual addition with its RMS norm
(forward, with an 8-bit output, and backward), products of 8-bit integers (dense, and grouped by
expert), and the sort of tokens by expert and back with its gradient.

Each case can run in two forms on the same inputs.  With `own` false, `run` computes the operator
from elementary torch operations in float32, rounded once at the end; with `own` true it makes the
calls of include/moe_block.h through the package's binding.  `exact` evaluates the definition in
float64.
"""

from __future__ import annotations

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-6
DEV = "cuda"


# ------------------------------------------------------------------------------------------ cases

def listed():
    full = dict(H=2048, I=512, E=256, k=8)
    return [
        # the norm in front of the layer for one decoded token
        dict(name="norm, one token", op="norm", q8=False, T=1, H=2048, type="bf16"),
        # a prompt chunk: bf16 rows for the router and int8 rows for the 8-bit products, in one pass
        dict(name="norm, chunk, 8 bits", op="norm", q8=True, T=2048, H=2048, type="bf16"),
        # gradients of a short odd batch held in float32
        dict(name="norm gradient, short", op="norm_grad", T=333, H=2048, type="f32"),
        # gradients of a long training batch
        dict(name="norm gradient, long", op="norm_grad", T=16384, H=2048, type="bf16"),
        # one token through the linear-attention layer's joint q, k, v projection
        dict(name="linear, one token", op="linear", M=1, N=8192, K=2048, type="bf16"),
        # a ragged mid-size batch through the same projection
        dict(name="linear, odd batch", op="linear", M=333, N=8192, K=2048, type="bf16"),
        # a long prompt through the same projection
        dict(name="linear, long", op="linear", M=16384, N=8192, K=2048, type="bf16"),
        # gate and up products of one decoded token: nine experts' rows
        dict(name="gate_up, one token", op="gate_up", T=1, tile=32, **full),
        # down products of a 512-token prompt: every expert holds a few rows
        dict(name="down, 512 tokens", op="down", T=512, tile=32, **full),
        # gate and up products of a long prompt in one call: hundreds of rows an expert
        dict(name="gate_up, long", op="gate_up", T=16384, tile=256, **full),
        # dispatch, combine and both gradients of a training step: odd token count, float32 rows
        dict(name="sort, short", op="sort", T=511, H=2048, E=256, k=8, type="f32"),
        # the same for a long batch in bfloat16
        dict(name="sort, long", op="sort", T=8192, H=2048, E=256, k=8, type="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "linear", "gate_up", "down", "sort"])
    typ = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op in ("norm", "norm_grad"):
        H = 8 * _log(rng, 8, 1024)
        T = _log(rng, 1, max(1, min(16384, 16384 * 2048 * 2 // (H * SIZE[typ]))))
        if op == "norm":
            return dict(op=op, q8=rng.random() < 0.5, T=T, H=H, type=typ)
        return dict(op=op, T=T, H=H, type=typ)
    if op == "linear":
        return dict(op=op, M=_log(rng, 1, 16384), N=8 * _log(rng, 8, 1024), K=64 * _log(rng, 1, 32), type=typ)
    if op == "sort":
        E = _log(rng, 4, 512)
        return dict(op=op, T=_log(rng, 1, 16384 // SIZE[typ]), H=64 * _log(rng, 1, 32), E=E,
                    k=rng.randint(1, min(E, 8)), type=typ)
    # expert products: the token count stays where the expert sizes keep the padded plain form small
    E = _log(rng, 8, 256)
    return dict(op=op, T=_log(rng, 1, 8192), H=64 * _log(rng, 2, 32), I=64 * _log(rng, 1, 8), E=E,
                k=rng.randint(1, min(E, 8)), tile=rng.choice([16, 32, 64, 128, 256]))


# ----------------------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _rows(g, rows, width, typ, scale=1.0):
    return (torch.randn((rows, width), generator=g, device=DEV) * scale).to(TYPES[typ])


def _weights8(g, n, rows, K):
    """int8 weights with a normal distribution and positive channel scales, [n][rows][K] and [n][rows]."""
    w = torch.empty((n, rows, K), dtype=torch.int8, device=DEV)
    for i in range(0, n, 32):
        part = torch.randn((min(32, n - i), rows, K), generator=g, device=DEV)
        w[i:i + 32] = part.mul_(32.0).round_().clamp_(-127, 127).to(torch.int8)
    s = (0.5 + torch.rand((n, rows), generator=g, device=DEV)) * (1.5 / (32 * K ** 0.5))
    return w, s


def _tokens8(g, rows, K):
    """int8 rows and their scales, as the norm's 8-bit output gives them."""
    x = torch.randn((rows, K), generator=g, device=DEV)
    a = x.abs().amax(1, keepdim=True)
    return torch.round(x * (127.0 / a)).to(torch.int8), (a / 127.0).reshape(-1)


def _routing(g, T, E, k, tile, n_shared=1):
    """Routing tables as moe_route writes them, for scores with a mild preference among experts."""
    scores = torch.randn((T, E), generator=g, device=DEV)
    scores += 0.5 * torch.randn((1, E), generator=g, device=DEV)
    top, idx = scores.topk(k, dim=1)
    w = torch.softmax(top, dim=1)
    flat = idx.reshape(-1)
    order = torch.argsort(flat, stable=True)
    pos = torch.empty_like(order)
    pos[order] = torch.arange(T * k, device=DEV)
    counts = torch.bincount(flat, minlength=E)
    blocks, row = [], 0
    for e, c in enumerate(counts.tolist() + [T] * n_shared):
        nb = -(-c // tile)
        for b in range(nb):
            lo, hi = c * b // nb, c * (b + 1) // nb
            blocks.append([e, row + lo, hi - lo, -(-(-(-c // nb)) // 16) * 16])
        row += c
    n_blocks = len(blocks)
    # the table holds moe_max_blocks entries, as the calls ask for; those behind the map stay empty
    S, cut = T * k, -(-T // tile)
    blocks += [[0, 0, 0, 0]] * (S // tile + min(S, E) + n_shared * cut - n_blocks)
    i32 = dict(dtype=torch.int32, device=DEV)
    offsets = torch.zeros(E + 1, **i32)
    offsets[1:] = counts.cumsum(0)
    return dict(topk_idx=idx.to(torch.int32), topk_w=w.contiguous(), counts=counts.to(torch.int32),
                offsets=offsets, sorted_slot=order.to(torch.int32), slot_pos=pos.to(torch.int32),
                blocks=torch.tensor(blocks, **i32).reshape(-1, 4), n_blocks=torch.tensor([n_blocks], **i32),
                status=torch.zeros(1, **i32), cmax=int(counts.max()) if T else 0)


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    op = case["op"]
    if op in ("norm", "norm_grad"):
        T, H, typ = case["T"], case["H"], case["type"]
        s["w"] = 1.0 + 0.1 * torch.randn((H,), generator=g, device=DEV)
        if op == "norm":
            s["x"], s["res"] = _rows(g, T, H, typ), _rows(g, T, H, typ, 2.0)
            s["sum"], s["y"] = torch.empty_like(s["x"]), torch.empty_like(s["x"])
            if case["q8"]:
                s["yq"] = torch.empty((T, H), dtype=torch.int8, device=DEV)
                s["ys"] = torch.empty((T, 1), dtype=torch.float32, device=DEV)
                s["values"] = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
        else:
            s["sum"], s["dy"], s["dsum"] = _rows(g, T, H, typ, 2.0), _rows(g, T, H, typ), _rows(g, T, H, typ)
            s["dx"] = torch.empty_like(s["sum"])
            s["dw"] = torch.empty((H,), dtype=torch.float32, device=DEV)
    elif op == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        w, ws = _weights8(g, 1, N, K)
        s["wq"], s["ws"] = w[0], ws[0]
        s["xq"], s["xs"] = _tokens8(g, M, K)
        s["out"] = torch.empty((M, N), dtype=TYPES[case["type"]], device=DEV)
    elif op in ("gate_up", "down"):
        T, H, I, E, k = case["T"], case["H"], case["I"], case["E"], case["k"]
        s["r"] = _routing(g, T, E, k, case["tile"])
        n, K = (2 * I, H) if op == "gate_up" else (H, I)
        # the last matrix is the shared expert's
        s["wq"], s["ws"] = _weights8(g, E + 1, n, K)
        rows = T * (k + 1)
        s["xq"], s["xs"] = _tokens8(g, T if op == "gate_up" else rows, K)
        s["out"] = torch.empty((rows, I if op == "gate_up" else H), dtype=torch.bfloat16, device=DEV)
    else:
        T, H, E, k, typ = case["T"], case["H"], case["E"], case["k"], case["type"]
        s["r"] = _routing(g, T, E, k, 128)
        rows = T * (k + 1)
        s["x"], s["dy"] = _rows(g, T, H, typ), _rows(g, T, H, typ)
        s["ys"], s["dxs"] = _rows(g, rows, H, typ), _rows(g, rows, H, typ)
        s["rows"], s["dys"] = torch.empty_like(s["ys"]), torch.empty_like(s["ys"])
        s["y"], s["dx"] = torch.empty_like(s["x"]), torch.empty_like(s["x"])
        s["dw"] = torch.empty((T, k), dtype=torch.float32, device=DEV)
    if own:  # the argument structs, banks and workspaces that a user's program keeps
        _handles(s)
    return s


def _handles(s):
    import w4_dequant_expert_amd as moe
    op = s["op"]
    if op in ("norm", "norm_grad"):
        s["d"] = moe.NormDims(s["T"], s["H"], moe.ELEM[TYPES[s["type"]]], EPS)
        if op == "norm_grad":
            s["wsb"] = moe.moe_add_rmsnorm_backward_ws_bytes(s["d"])
            s["wsp"] = torch.empty((max(s["wsb"], 1),), dtype=torch.uint8, device=DEV)
    elif op == "linear":
        s["d"] = moe.Q8Dims(s["M"], s["N"], s["K"], moe.ELEM[TYPES[s["type"]]])
    else:
        r = s["r"]
        s["d"] = moe.make_dims(s["T"], s["H"], s.get("I", 64), s["E"], s["k"], 1, s.get("tile", 128), 16)
        s["route"] = moe.RouteOut(*[r[n].data_ptr() for n in ("topk_idx", "topk_w", "counts", "offsets", "sorted_slot",
                                                             "slot_pos", "blocks", "n_blocks")],
                                  None, r["status"].data_ptr(), None, 0)
        if op != "sort":
            E, q, c = s["E"], s["wq"], s["ws"]
            half = {"gate_up": ("gu", "gu_s"), "down": ("dn", "dn_s")}[op]
            s["routed"] = moe.Q8Bank(**{half[0]: q.data_ptr(), half[1]: c.data_ptr()})
            s["shared"] = moe.Q8Bank(**{half[0]: q[E].data_ptr(), half[1]: c[E].data_ptr()})
        else:
            s["elem"] = moe.ELEM[TYPES[s["type"]]]


# ------------------------------------------------------------------------------------- one pass

def run(state):
    return _run_own(state) if own else PLAIN[state["op"]](state)


def _run_own(s):
    import w4_dequant_expert_amd as moe
    op = s["op"]
    if op == "norm":
        moe.moe_add_rmsnorm(s["d"], s["x"], s["res"], s["w"], s["sum"], s["y"], s.get("yq"), s.get("ys"))
        if s["q8"]:  # the 8-bit rows as the values they stand for
            return s["sum"], s["y"], torch.mul(s["yq"], s["ys"], out=s["values"])
        return s["sum"], s["y"]
    if op == "norm_grad":
        moe.moe_add_rmsnorm_backward(s["d"], s["sum"], s["w"], s["dy"], s["dsum"], s["dx"], s["dw"], s["wsp"], s["wsb"])
        return s["dx"], s["dw"]
    if op == "linear":
        moe.moe_q8_matmul(s["d"], s["xq"], s["xs"], s["wq"], s["ws"], s["out"])
        return s["out"]
    if op == "gate_up":
        moe.moe_q8_gate_up(s["d"], s["xq"], s["xs"], s["route"], s["routed"], s["shared"], s["out"])
        return s["out"]
    if op == "down":
        moe.moe_q8_down(s["d"], s["route"], s["routed"], s["shared"], s["xq"], s["xs"], s["out"])
        return s["out"]
    d, r, e = s["d"], s["route"], s["elem"]
    moe.moe_dispatch_rows(d, e, s["x"], r, s["rows"])
    moe.moe_combine_rows(d, e, s["ys"], r, s["y"])
    moe.moe_combine_rows_backward(d, e, s["dy"], s["ys"], r, s["dys"], s["dw"])
    moe.moe_dispatch_rows_backward(d, e, s["dxs"], r, s["dx"])
    return s["rows"], s["y"], s["dys"], s["dw"], s["dx"]


def _norm(s):
    t = s["x"].float() + s["res"].float()
    y = t * torch.rsqrt(t.square().mean(1, keepdim=True) + EPS) * s["w"]
    if not s["q8"]:
        return t.to(s["x"].dtype), y.to(s["x"].dtype)
    a = y.abs().amax(1, keepdim=True)
    q = torch.round(y * (127.0 / a)).to(torch.int8)
    return t.to(s["x"].dtype), y.to(s["x"].dtype), (q.float() * (a / 127.0)).to(torch.bfloat16)


def _norm_grad(s):
    t, dy = s["sum"].float(), s["dy"].float()
    rho = torch.rsqrt(t.square().mean(1, keepdim=True) + EPS)
    xh = t * rho
    g = dy * s["w"]
    dx = rho * (g - xh * (g * xh).mean(1, keepdim=True)) + s["dsum"].float()
    return dx.to(s["sum"].dtype), (dy * xh).sum(0)


def _linear(s):
    y = torch.mm(s["xq"].float(), s["wq"].float().t())
    return (y * s["xs"][:, None] * s["ws"]).to(s["out"].dtype)


def _products(s, x, xs):
    """Products of all rows (expert order, then the shared expert's).  With fewer routed rows than
    experts each row takes its expert's matrix; otherwise the experts' rows are padded to the largest
    group, for one batched product."""
    r, T, k, E = s["r"], s["T"], s["k"], s["E"]
    n = s["wq"].shape[1]
    S = T * k
    group = torch.repeat_interleave(torch.arange(E, device=DEV), r["counts"].long(), output_size=S)
    out = torch.empty((S + T, n), device=DEV)
    if S <= E:
        y = torch.bmm(s["wq"][group].float(), x[:S].float()[:, :, None])[:, :, 0]
    else:
        at = torch.arange(S, device=DEV) - r["offsets"].long()[group]
        pad = torch.zeros((E, r["cmax"], x.shape[1]), device=DEV)
        pad[group, at] = x[:S].float()
        y = torch.bmm(s["wq"][:E].float(), pad.transpose(1, 2).contiguous()).transpose(1, 2)[group, at]
    out[:S] = y * s["ws"][group]
    out[S:] = torch.mm(x[S:].float(), s["wq"][E].float().t()) * s["ws"][E]
    return out * xs[:, None]


def _tokens(s):
    """The token of each row."""
    return torch.cat([s["r"]["sorted_slot"].long() // s["k"], torch.arange(s["T"], device=DEV)])


def _gate_up(s):
    tok = _tokens(s)
    y = _products(s, s["xq"][tok], s["xs"][tok])
    I = s["I"]
    g, u = y[:, :I], y[:, I:]
    return (g / (1.0 + torch.exp(-g)) * u).to(torch.bfloat16)


def _down(s):
    return _products(s, s["xq"], s["xs"]).to(torch.bfloat16)


def _sort(s):
    r, T, k, H = s["r"], s["T"], s["k"], s["H"]
    S, typ = T * k, s["x"].dtype
    pos, w = r["slot_pos"].long(), r["topk_w"]
    rows = s["x"][_tokens(s)]
    picked = s["ys"][pos].float().reshape(T, k, H)
    y = (picked * w[:, :, None]).sum(1) + s["ys"][S:].float()
    dy = s["dy"].float()
    dys = torch.empty_like(s["ys"])
    dys[pos] = (dy[:, None] * w[:, :, None]).reshape(S, H).to(typ)
    dys[S:] = s["dy"]
    dw = (picked * dy[:, None]).sum(2)
    dx = s["dxs"][pos].float().reshape(T, k, H).sum(1) + s["dxs"][S:].float()
    return rows, y.to(typ), dys, dw, dx.to(typ)


PLAIN = dict(norm=_norm, norm_grad=_norm_grad, linear=_linear, gate_up=_gate_up, down=_down, sort=_sort)


# ------------------------------------------------------------------------- what a pass has to do

def work(case):
    op = case["op"]
    if op == "norm":
        n, e = case["T"] * case["H"], SIZE[case["type"]]
        q = 3 * n + 4 * case["T"] if case["q8"] else 0
        return dict(bytes=4 * n * e + q + 4 * case["H"], flops=(12 if case["q8"] else 6) * n)
    if op == "norm_grad":
        n, e = case["T"] * case["H"], SIZE[case["type"]]
        return dict(bytes=4 * n * e + 8 * case["H"], flops=14 * n)
    if op == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        return dict(bytes=M * K + N * K + M * N * SIZE[case["type"]] + 4 * (M + N), flops=2 * M * N * K)
    T, H, E, k = case["T"], case["H"], case["E"], case["k"]
    rows = T * (k + 1)
    if op == "sort":
        e = SIZE[case["type"]]
        return dict(bytes=(4 * T + 4 * rows) * H * e + 12 * T * k, flops=6 * rows * H)
    n, K, width = (2 * case["I"], H, case["I"]) if op == "gate_up" else (H, case["I"], H)
    touched = E * (1.0 - (1.0 - k / E) ** T) + 1  # experts that hold a row, in the mean of even routing
    inputs = T if op == "gate_up" else rows
    return dict(bytes=int(touched * n * (K + 4)) + inputs * (K + 4) + rows * width * 2, flops=2 * rows * n * K)


# --------------------------------------------------------------------- the definitions in float64

def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    with torch.no_grad():
        return EXACT[case["op"]](s)


def _exact_norm(s):
    t = torch.add(s["x"].double(), s["res"].double())
    size = torch.sqrt(torch.sum(t ** 2, dim=-1, keepdim=True) / s["H"] + EPS)
    y = (t / size) * s["w"].double()
    if not s["q8"]:
        return t, y
    step = torch.amax(torch.abs(y), dim=-1, keepdim=True) / 127
    return t, y, torch.round(y / step) * step


def _exact_norm_grad(s):
    """From the Jacobian of t / |t|: the part of the incoming gradient along t is removed."""
    t, dy, w, H = s["sum"].double(), s["dy"].double(), s["w"].double(), s["H"]
    square = (t ** 2).sum(-1, keepdim=True) / H + EPS
    along = (dy * w * t).sum(-1, keepdim=True) / (H * square)
    dx = (dy * w - along * t) / square.sqrt() + s["dsum"].double()
    return dx, torch.sum(dy * (t / square.sqrt()), dim=0)


def _exact_linear(s):
    out = []
    for lo in range(0, s["M"], 4096):
        x = s["xq"][lo:lo + 4096].double() * s["xs"][lo:lo + 4096].double()[:, None]
        out.append(x @ (s["wq"].double() * s["ws"].double()[:, None]).t())
    return torch.cat(out)


def _exact_products(s, x, xs):
    """Expert by expert."""
    r, S = s["r"], s["T"] * s["k"]
    edges = r["offsets"].tolist() + [S + s["T"]]
    out = []
    for e in range(s["E"] + 1):
        lo, hi = edges[e], edges[e + 1]
        out.append((x[lo:hi].double() @ s["wq"][e].double().t()) * s["ws"][e].double() * xs[lo:hi].double()[:, None])
    return torch.cat(out)


def _exact_gate_up(s):
    tok = torch.cat([torch.div(s["r"]["sorted_slot"], s["k"], rounding_mode="floor").long(), torch.arange(s["T"], device=DEV)])
    y = _exact_products(s, s["xq"][tok], s["xs"][tok])
    gate, up = y.chunk(2, dim=1)
    return gate * torch.sigmoid(gate) * up


def _exact_down(s):
    return _exact_products(s, s["xq"], s["xs"])


def _exact_sort(s):
    """Rank by rank, each rank's rows gathered or scattered on their own."""
    r, T, k = s["r"], s["T"], s["k"]
    S = T * k
    pos = r["slot_pos"].long().reshape(T, k)
    w = r["topk_w"].double()
    x, dy = s["x"].double(), s["dy"].double()
    rows, dys = torch.empty_like(s["ys"], dtype=torch.float64), torch.empty_like(s["ys"], dtype=torch.float64)
    y, dx = s["ys"][S:].double(), s["dxs"][S:].double()
    rows[S:], dys[S:] = x, dy
    dw = torch.empty((T, k), dtype=torch.float64, device=DEV)
    for j in range(k):
        p = pos[:, j]
        mine = s["ys"][p].double()
        rows[p] = x
        dys[p] = dy * w[:, j:j + 1]
        y = y + mine * w[:, j:j + 1]
        dw[:, j] = (mine * dy).sum(1)
        dx = dx + s["dxs"][p].double()
    return rows, y, dys, dw, dx


EXACT = dict(norm=_exact_norm, norm_grad=_exact_norm_grad, linear=_exact_linear, gate_up=_exact_gate_up,
             down=_exact_down, sort=_exact_sort)
