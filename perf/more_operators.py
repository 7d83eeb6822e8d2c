"""Cases of the experts held in 8 bits and of the grouped products of any width.

Every case is one pass of one operator, in its plain form (elementary torch operations in
32 bits) or, where ``own`` is true, through the calls a user makes of the library:

* ``i8``: one projection with experts in 8-bit integers, a scale for each token and one for each
  output channel of each expert. ``first``: tokens are quantised and sent to their expert-grouped
  rows, and multiplied. ``second``: the gated activation of the first projection's output is
  quantised and multiplied.
* ``ragged``: products of rows grouped by expert with each expert's own matrix, of widths that need
  not be multiples of a tile (low-rank adapters beside an expert's projection, odd layers):
  y = alpha x W, on top of another projection's output where ``add`` is true; in training also
  the gradients of the rows (again on top) and of the matrices.

A value v of a row (or channel) whose largest magnitude is m is held as the integer 127 v / m,
rounded to nearest with ties to even; the scale is m / 127.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------------------ cases
def listed():
    return [
        # one token on each of 8 ranks: a decode step that streams the weights of the experts it hits
        dict(name="i8_decode", op="i8", stage="first", R=8, S=1, E=384, K=8, H=7168, Hp=2048, zipf=0.2),
        # a decode batch through the second projection (1024 activations back to 7168)
        dict(name="i8_decode_second", op="i8", stage="second", R=8, S=12, E=384, K=8, H=1024, Hp=7168, zipf=0.2),
        # odd sizes: 3 ranks, rows of 1088, 576 outputs, short ragged segments
        dict(name="i8_ragged", op="i8", stage="first", R=3, S=211, E=48, K=6, H=1088, Hp=576, zipf=0.5),
        # the inference batch over 384 experts: 32,768 rows, about 85 a segment, every weight read
        dict(name="i8_infer", op="i8", stage="first", R=8, S=512, E=384, K=8, H=7168, Hp=2048, zipf=0.3),
        # the same batch's second projection
        dict(name="i8_infer_second", op="i8", stage="second", R=8, S=512, E=384, K=8, H=1024, Hp=7168, zipf=0.3),
        # the largest: 524,288 rows, long segments, bound by the products
        dict(name="i8_bench", op="i8", stage="first", R=8, S=8192, E=384, K=8, H=7168, Hp=2048, zipf=0.2),
        # adapters of rank 16 in a decode step: into the rank, and from it on top of the projection
        dict(name="ragged_decode_in", op="ragged", R=8, S=1, E=384, K=8, H=7168, Hp=16, alpha=1.0, add=False,
             strided=False, train=False, zipf=0.2),
        dict(name="ragged_decode_out", op="ragged", R=8, S=1, E=384, K=8, H=16, Hp=2048, alpha=2.0, add=True,
             strided=False, train=False, zipf=0.2),
        # training of a small odd layer on one half of a wider buffer
        dict(name="ragged_odd", op="ragged", R=3, S=1237, E=90, K=3, H=328, Hp=1000, alpha=1.0, add=False,
             strided=True, train=True, zipf=0.6),
        # training of adapters: 131,072 rows into rank 16
        dict(name="ragged_train_in", op="ragged", R=8, S=2048, E=384, K=8, H=7168, Hp=16, alpha=1.0, add=False,
             strided=False, train=True, zipf=0.2),
        # and from rank 64 on top of the projection's output
        dict(name="ragged_train_out", op="ragged", R=8, S=2048, E=384, K=8, H=64, Hp=2048, alpha=0.5, add=True,
             strided=False, train=True, zipf=0.2),
        # a layer of widths between the tiles, bound by its products
        dict(name="ragged_train_wide", op="ragged", R=8, S=2048, E=64, K=4, H=1096, Hp=1544, alpha=1.0, add=False,
             strided=False, train=True, zipf=0.3),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    zipf = rng.choice((0.0, 0.2, 0.5))
    if rng.random() < 0.5:
        R = rng.choice((1, 2, 3, 4, 8))
        E = R * _log(rng, 2, 384 // R)
        K = rng.randint(1, min(8, E))
        stage = rng.choice(("first", "second"))
        H, Hp = 64 * _log(rng, 1, 112), 64 * _log(rng, 1, 112)
        while E * H * Hp > 384 * 7168 * 2048:
            H, Hp = 64 * _log(rng, 1, 112), 64 * _log(rng, 1, 112)
        # no more products than the largest listed case, nor more rows than the plain form can hold in 32 bits
        rows = min(65536 * K, int(7e12 / (2 * H * Hp)), int((5e8 if stage == "second" else 2e9) / max(H, Hp)))
        return dict(op="i8", stage=stage, R=R, S=_log(rng, 1, min(8192, rows // (R * K))), E=E, K=K, H=H, Hp=Hp, zipf=zipf)
    R = rng.choice((1, 2, 3, 4, 8))
    E = R * _log(rng, 2, 384 // R)
    K = rng.randint(1, min(8, E))
    wide, narrow = 8 * _log(rng, 8, 896), 8 * _log(rng, 1, 16)
    kind = rng.choice(("in", "out", "both"))
    if kind == "both":
        H, Hp = 8 * _log(rng, 4, 256), 8 * _log(rng, 4, 256)
    else:
        H, Hp = (wide, narrow) if kind == "in" else (narrow, wide)
    while E * H * Hp > 5e8:
        E = R * max(2, E // (2 * R))
        if E == 2 * R:
            break
    K = min(K, E)
    rows = min(131072, int(5e11 / (H * Hp)), int(9e8 / max(H, Hp)))
    return dict(op="ragged", R=R, S=_log(rng, 1, min(8192, max(1, rows // (R * K)))), E=E, K=K, H=H, Hp=Hp,
                alpha=rng.choice((1.0, 0.5, 2.0)), add=rng.random() < 0.5, strided=rng.random() < 0.3,
                train=rng.random() < 0.6, zipf=zipf)


# ------------------------------------------------------------------------------ work
def work(case):
    c = case
    H, Hp, E = c["H"], c["Hp"], c["E"]
    T = c["R"] * c["S"]
    rows = T * c["K"]
    # the matrices of the experts that some token chose
    hit = sum(1.0 - (1.0 - min(1.0, q * c["K"])) ** T for q in _zipf(E, c["zipf"]))
    if c["op"] == "i8":
        # tokens, or gate and up of every row; integers and scales of the weights; outputs
        rows_in = T * H * 2 + rows * 4 if c["stage"] == "first" else rows * H * 4
        return dict(bytes=hit * Hp * (H + 4) + rows_in + rows * Hp * 2, flops=2 * rows * H * Hp)
    nbytes = 2 * (rows * H + rows * Hp * (2 if c["add"] else 1) + hit * H * Hp)
    flops = 2 * rows * H * Hp
    if c["train"]:
        nbytes += 2 * (rows * Hp + rows * H * (2 if c["add"] else 1)) + 4 * E * H * Hp
        flops *= 3
    return dict(bytes=nbytes, flops=flops)


# ------------------------------------------------------------------------------ inputs
def _zipf(E, s):
    p = [(e + 1) ** -s for e in range(E)]
    z = sum(p)
    return [q / z for q in p]


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 1000003 + 24680)
    return g


def _normal(g, shape, std=1.0):
    return torch.empty(shape, dtype=torch.bfloat16, device=DEV).normal_(std=std, generator=g)


def _groups(c, g):
    """K different experts of each token by perturbed popularity, and the rows in expert order, cut into
    R equal ranks whose segments all read home matrices."""
    R, S, K, E = c["R"], c["S"], c["K"], c["E"]
    T = R * S
    s = {}
    logp = torch.tensor(_zipf(E, c["zipf"]), device=DEV).log()
    u = torch.rand(T, E, device=DEV, generator=g).clamp_(1e-12, 1.0)
    topk = (logp - (-u.log()).log()).sort(dim=-1, descending=True).indices[:, :K]
    order = topk.reshape(-1).sort(stable=True)
    s["row_expert"] = order.values
    s["row_token"] = order.indices // K
    dest = torch.empty(T * K, dtype=torch.int32, device=DEV)
    dest[order.indices] = torch.arange(T * K, dtype=torch.int32, device=DEV)
    s["dest"] = dest.view(R, S, K)
    rank = torch.arange(T * K, device=DEV) // (S * K)
    counts = torch.zeros(R * E, dtype=torch.int64, device=DEV)
    counts.index_add_(0, rank * E + order.values, torch.ones_like(rank))
    counts = counts.view(R, E)
    cu = torch.zeros(R, E + 2, dtype=torch.int32, device=DEV)
    cu[:, 1:E + 1] = counts.cumsum(1)
    cu[:, E + 1] = cu[:, E]
    s["cu"] = cu
    s["slot_expert"] = torch.full((R, 1), -1, dtype=torch.int32, device=DEV)
    total = counts.sum(0)
    s["cap"] = int(total.max())                                   # longest expert: a plan's number
    s["place"] = torch.arange(T * K, device=DEV) - (total.cumsum(0) - total)[order.values]
    return s


def _inputs(c, seed):
    g = _gen(seed)
    s = _groups(c, g)
    R, S, E, H, Hp = c["R"], c["S"], c["E"], c["H"], c["Hp"]
    rows = R * S * c["K"]
    s["case"] = c
    s["w"] = _normal(g, (E, H, Hp), 0.02 if c["op"] == "i8" else H ** -0.5)
    if c["op"] == "i8":
        if c["stage"] == "first":
            s["x"] = _normal(g, (R, S, H))
        else:
            s["h"] = _normal(g, (rows, 2 * H))
        return s
    s["x"] = _normal(g, (rows, 2 * H))[:, H:] if c["strided"] else _normal(g, (rows, H))
    s["add"] = _normal(g, (rows, Hp)) if c["add"] else None
    if c["train"]:
        s["dy"] = _normal(g, (rows, Hp), 0.02)
        s["dx_add"] = _normal(g, (rows, H), 0.02) if c["add"] else None
    return s


def _i8(x):
    """Integers and scales of the rows of fp32 x."""
    top = x.abs().amax(-1, keepdim=True)
    q = torch.where(top > 0, x * 127.0 / top, 0.0)
    return torch.round(q).to(torch.int8), (top / 127.0).squeeze(-1)


def prepare(case, seed):
    c = case
    s = _inputs(c, seed)
    R, S, E, K, H, Hp = (c[n] for n in ("R", "S", "E", "K", "H", "Hp"))
    rows = R * S * K
    if own:
        import moe_expert_dispatch_online_gb300 as bep
        s["bep"] = bep
        pad = 64 if c["op"] == "ragged" else 1    # a context's own widths: the products' come with their tensors
        s["ctx"] = bep.Context(bep.Config(R, E, 1, K, S, max(H, pad) // pad * pad, max(Hp, pad) // pad * pad, bep.BEP_INFER))
        s["y"] = torch.empty(rows, Hp, dtype=torch.bfloat16, device=DEV)
        if c["op"] == "i8":
            w = s.pop("w")
            s["w"] = bep.IntWeight(s["ctx"])
            bep.bep_int_quantize_weight(s["ctx"], w, s["w"].codes, s["w"].scales)
            s["rows"] = bep.IntRows(rows, H)
        elif c["train"]:
            s["dx"] = torch.empty(rows, H, dtype=torch.bfloat16, device=DEV)
            s["dw"] = torch.empty(E, H, Hp, dtype=torch.float32, device=DEV)
    elif c["op"] == "i8":
        w = s.pop("w")
        codes = torch.empty(E, Hp, H, dtype=torch.int8, device=DEV)
        scales = torch.empty(E, Hp, device=DEV)
        for e in range(0, E, 16):
            codes[e:e + 16], scales[e:e + 16] = _i8(w[e:e + 16].transpose(1, 2).float().contiguous())
        s["w"] = (codes, scales)
    return s


# ------------------------------------------------------------------------------ one pass
def run(state):
    if own:
        return _own_i8(state) if state["case"]["op"] == "i8" else _own_ragged(state)
    return _plain_i8(state) if state["case"]["op"] == "i8" else _plain_ragged(state)


def _own_i8(s):
    bep, ctx, rows, w = s["bep"], s["ctx"], s["rows"], s["w"]
    if s["case"]["stage"] == "first":
        bep.bep_dispatch_int(ctx, s["x"], s["dest"], rows.codes, rows.scales)
    else:
        bep.bep_swiglu_int(ctx, s["h"], rows.codes, rows.scales)
    bep.bep_grouped_gemm_int(ctx, s["cu"], s["slot_expert"], rows.codes, rows.scales, w.codes, w.scales, s["y"])
    return s["y"]


def _own_ragged(s):
    bep, ctx, c = s["bep"], s["ctx"], s["case"]
    bep.bep_ragged_gemm(ctx, s["cu"], s["slot_expert"], s["x"], s["w"], s["y"], alpha=c["alpha"], add=s["add"])
    out = dict(y=s["y"])
    if c["train"]:
        bep.bep_ragged_gemm(ctx, s["cu"], s["slot_expert"], s["dy"], s["w"], s["dx"], trans=True, alpha=c["alpha"],
                            add=s["dx_add"])
        bep.bep_ragged_gemm_dw(ctx, s["cu"], s["slot_expert"], s["x"], s["dy"], s["dw"], alpha=c["alpha"])
        out.update(dx=s["dx"], dw=s["dw"])
    return out


def _padded(s, x):
    """Rows in 32 bits as [E, longest expert, width], zeros behind each expert's."""
    p = torch.zeros(s["case"]["E"], s["cap"], x.shape[-1], device=x.device)
    p[s["row_expert"], s["place"]] = x.float()
    return p


def _plain_i8(s):
    c = s["case"]
    if c["stage"] == "first":
        q, scale = _i8(s["x"].view(-1, c["H"]).float())
        q, scale = q[s["row_token"]], scale[s["row_token"]]
    else:
        gate, up = s["h"].float().chunk(2, -1)
        q, scale = _i8(gate / (1.0 + torch.exp(-gate)) * up)
    codes, w_scale = s["w"]
    y = torch.matmul(_padded(s, q), codes.float().transpose(1, 2))[s["row_expert"], s["place"]]
    return (y * w_scale[s["row_expert"]] * scale.unsqueeze(-1)).bfloat16()


def _plain_ragged(s):
    c, at = s["case"], (s["row_expert"], s["place"])
    w = s["w"].float()
    x = _padded(s, s["x"])
    y = c["alpha"] * torch.matmul(x, w)[at]
    out = dict(y=(y if s["add"] is None else y + s["add"].float()).bfloat16())
    if c["train"]:
        dy = _padded(s, s["dy"])
        dx = c["alpha"] * torch.matmul(dy, w.transpose(1, 2))[at]
        out["dx"] = (dx if s["dx_add"] is None else dx + s["dx_add"].float()).bfloat16()
        out["dw"] = c["alpha"] * torch.matmul(x.transpose(1, 2), dy)
    return out


# ------------------------------------------------------------------------------ 64 bits
def exact(case, seed):
    c = case
    # products in 64 bits run at about a TFLOP/s here
    if 2 * c["R"] * c["S"] * c["K"] * c["H"] * c["Hp"] > 4e12:
        return None
    s = _inputs(c, seed)
    bounds = torch.searchsorted(s["row_expert"].contiguous(), torch.arange(c["E"] + 1, device=DEV)).tolist()
    spans = [(e, slice(a, b)) for e, (a, b) in enumerate(zip(bounds, bounds[1:])) if b > a]
    return _exact_i8(s, spans) if c["op"] == "i8" else _exact_ragged(s, spans)


def _exact_quantised(x):
    """fp64 values on the grid of 255 integers of each row: (integers, scale)."""
    m = x.abs().max(-1, keepdim=True).values
    step = m / 127
    safe = torch.where(m > 0, m, torch.ones_like(m))
    return (127 * x / safe).round(), step


def _exact_i8(s, spans):
    c = s["case"]
    if c["stage"] == "first":
        q, step = _exact_quantised(s["x"].reshape(-1, c["H"]).double())
        q, step = q[s["row_token"]], step[s["row_token"]]
    else:
        h = s["h"].double()
        gate, up = h[:, :c["H"]], h[:, c["H"]:]
        q, step = _exact_quantised(gate * torch.sigmoid(gate) * up)
    y = torch.empty(q.shape[0], c["Hp"], dtype=torch.float64, device=DEV)
    for e, rows in spans:
        wq, w_step = _exact_quantised(s["w"][e].double().t())
        y[rows] = (q[rows] * step[rows]) @ (wq * w_step).t()
    return y


def _exact_ragged(s, spans):
    c = s["case"]
    n = s["x"].shape[0]
    out = dict(y=torch.empty(n, c["Hp"], dtype=torch.float64, device=DEV))
    if c["train"]:
        out["dx"] = torch.empty(n, c["H"], dtype=torch.float64, device=DEV)
        out["dw"] = torch.zeros(c["E"], c["H"], c["Hp"], dtype=torch.float64, device=DEV)
    for e, rows in spans:
        x, w = s["x"][rows].double() * c["alpha"], s["w"][e].double()
        out["y"][rows] = x @ w
        if c["train"]:
            dy = s["dy"][rows].double()
            out["dx"][rows] = dy @ w.t() * c["alpha"]
            out["dw"][e] = x.t() @ dy
    if c["add"]:
        out["y"] += s["add"].double()
        if c["train"]:
            out["dx"] += s["dx_add"].double()
    return out
