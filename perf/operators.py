"""Cases of the expert layer's operators: routing, experts in 4-bit microscaled floating
point, and the gated activation with its 8-bit checkpoint.

Every case is one pass of one operator, in its plain form (elementary torch operations in
32 bits) or, where ``own`` is true, through the calls a user makes of the library:

* ``route``: expert scores (softmax or sigmoid of the logits), a balance bias for the choice,
  limited groups, top-K, renormalised gates and the experts' loads; in training also the
  gradient of the logits from the gates' gradients.
* ``mx``: one projection with 4-bit expert weights. ``first``: tokens are quantised and sent to
  their expert-grouped rows, and multiplied. ``second``: the gated activation of the first
  projection's output is quantised and multiplied.
* ``act``: the gated activation of a training step: its forward, which keeps the activations in
  8 bits, and its backward from that checkpoint, which also gives the forward's output again.

4-bit and 8-bit values are microscaled: blocks of 32 share a power of two, the smallest that
keeps the block's largest magnitude inside the element type (6 for e2m1, 127 for int8), and
elements round to the nearest value, ties to even.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
BLOCK = 32


# ------------------------------------------------------------------------------ cases
def listed():
    return [
        # one token on each of 8 ranks: a decode step of the 384-expert layer; scores by sigmoid,
        # 4 of 8 groups, a bias for balance
        dict(name="route_decode", op="route", R=8, S=1, E=384, K=8, score="sigmoid", groups=8,
             top_groups=4, group_top=2, bias=True, renorm=True, scale=2.5, half=False, train=False),
        # the inference batch of the same layer, logits of a bf16 product: many equal ones
        dict(name="route_infer", op="route", R=8, S=512, E=384, K=8, score="sigmoid", groups=8,
             top_groups=4, group_top=2, bias=True, renorm=True, scale=2.5, half=True, train=False),
        # training on an odd batch of 3 ranks, groups by their best expert, bf16 logits and gradients
        dict(name="route_train_odd", op="route", R=3, S=2731, E=90, K=5, score="softmax", groups=6,
             top_groups=3, group_top=1, bias=False, renorm=False, scale=1.0, half=True, train=True),
        # the largest: 65,536 tokens over 384 experts, every logit has a gradient
        dict(name="route_train_e384", op="route", R=8, S=8192, E=384, K=8, score="softmax", groups=1,
             top_groups=1, group_top=1, bias=True, renorm=False, scale=1.0, half=False, train=True),
        # decode step, one token a rank: streams the weights of the experts that are hit
        dict(name="mx_decode", op="mx", stage="first", R=8, S=1, E=384, K=8, H=7168, Hp=2048, zipf=0.2),
        # decode batch through the second projection (1024 activations back to 7168)
        dict(name="mx_decode_second", op="mx", stage="second", R=8, S=12, E=384, K=8, H=1024, Hp=7168,
             zipf=0.2),
        # odd sizes: 3 ranks, rows of 1088 (not a multiple of 128), 576 outputs, short ragged segments
        dict(name="mx_ragged", op="mx", stage="first", R=3, S=211, E=48, K=6, H=1088, Hp=576, zipf=0.5),
        # the inference batch over 384 experts: 32,768 rows, about 85 a segment, every weight read
        dict(name="mx_infer", op="mx", stage="first", R=8, S=512, E=384, K=8, H=7168, Hp=2048, zipf=0.3),
        # the largest: 524,288 rows, long segments, bound by the products
        dict(name="mx_bench", op="mx", stage="first", R=8, S=8192, E=384, K=8, H=7168, Hp=2048, zipf=0.2),
        # smallest training layer: 256 rows of 64 + 64 activations
        dict(name="act_tiny", op="act", R=2, S=64, K=2, F=64),
        # odd row count, 15 blocks a half
        dict(name="act_odd", op="act", R=3, S=1237, K=3, F=480),
        # the bench-shaped layer: 524,288 rows of 1024 + 1024 activations
        dict(name="act_bench", op="act", R=8, S=8192, K=8, F=1024),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("route", "mx", "act"))
    if op == "route":
        R = rng.choice((1, 2, 3, 4, 8))
        G = rng.choice((1, 2, 4, 6, 8))
        E = R * G * _log(rng, 4, max(4, 384 // (R * G)))
        groups = rng.choice((1, G)) if E // G >= 4 else 1
        top = rng.randint(max(1, groups // 3), groups)
        K = rng.randint(1, min(8, E // groups * top))
        S = _log(rng, 1, min(8192, 8192 * 8 // R))
        return dict(op=op, R=R, S=S, E=E, K=K, score=rng.choice(("softmax", "sigmoid")), groups=groups,
                    top_groups=top, group_top=rng.choice((1, 2)), bias=rng.random() < 0.5,
                    renorm=rng.random() < 0.5, scale=rng.choice((1.0, 2.5)), half=rng.random() < 0.5,
                    train=rng.random() < 0.6)
    if op == "mx":
        R = rng.choice((1, 2, 4, 8))
        E = R * _log(rng, 2, 384 // R)
        K = rng.randint(1, min(8, E))
        stage = rng.choice(("first", "second"))
        H, Hp = 64 * _log(rng, 1, 112), 64 * _log(rng, 1, 112)
        while E * H * Hp > 384 * 7168 * 2048:
            H, Hp = 64 * _log(rng, 1, 112), 64 * _log(rng, 1, 112)
        # no more products than the largest listed case, nor more rows than the card holds in 32 bits
        rows = min(65536 * K, int(7e12 / (2 * H * Hp)), int((5e8 if stage == "second" else 2e9) / max(H, Hp)))
        return dict(op=op, stage=stage, R=R, S=_log(rng, 1, max(1, min(8192, rows // (R * K)))), E=E, K=K, H=H, Hp=Hp,
                    zipf=rng.choice((0.0, 0.2, 0.4)))
    R = rng.choice((1, 2, 3, 4, 8))
    K = rng.randint(1, 8)
    return dict(op=op, R=R, S=_log(rng, 1, 65536 // (R * K)), K=K, F=32 * _log(rng, 1, 64))


# ------------------------------------------------------------------------------ work
def work(case):
    c = case
    R, S, K = c["R"], c["S"], c["K"]
    T = R * S
    if c["op"] == "route":
        E, b = c["E"], 2 if c["half"] else 4
        nbytes = T * E * b + T * K * 8 + (4 * E if c["bias"] else 0) + 4 * E   # logits; choice, gates; bias, loads
        flops = T * E * 4
        if c["train"]:
            # gates' gradients and the logits' gradients; the choice and the logits are held from the forward
            nbytes += T * K * 4 + T * E * b
            flops += T * E * 4
        return dict(bytes=nbytes, flops=flops)
    if c["op"] == "mx":
        H, Hp, E = c["H"], c["Hp"], c["E"]
        # the weights of the experts that some token chose: 4 bits and 1/32 byte of scale an element
        p = _zipf(E, c["zipf"])
        hit = sum(1.0 - (1.0 - min(1.0, float(q) * K)) ** T for q in p)
        rows_in = T * H * 2 if c["stage"] == "first" else T * K * H * 4
        return dict(bytes=hit * H * Hp * (0.5 + 1 / BLOCK) + rows_in + T * K * 4 + T * K * Hp * 2,
                    flops=2 * T * K * H * Hp)
    F = c["F"]
    rows = T * K
    # forward: reads gate and up, writes the output and the checkpoint; backward: reads the checkpoint
    # and the output's gradient, writes both halves' gradients and the output again
    ckpt = 2 * F * (1 + 1 / BLOCK)
    return dict(bytes=rows * (4 * F + 2 * F + ckpt + ckpt + 2 * F + 4 * F + 2 * F), flops=rows * F * 30)


# ------------------------------------------------------------------------------ inputs
def _zipf(E, s):
    p = [(e + 1) ** -s for e in range(E)]
    z = sum(p)
    return [q / z for q in p]


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 1000003 + 12345)
    return g


def _near_tie(values, count, tol):
    """Rows whose `count` largest values, or the next one, hold two that differ by less than tol but are not equal."""
    v = values.sort(dim=-1, descending=True).values[..., :count + 1]
    gap = v[..., :-1] - v[..., 1:]
    return ((gap > 0) & (gap < tol)).any(-1)


def _logits(c, g, bias):
    """Router logits [T, E]: a popularity offset per expert and noise per token, as the product of a
    trained router leaves them. The order of two scores that differ by less than the last bits of
    32-bit arithmetic has no answer that every correct program shares, so tokens with such a pair
    among the leading scores (or groups) are drawn again; equal logits stay."""
    T, E = c["R"] * c["S"], c["E"]
    pop = torch.randn(E, device=DEV, generator=g) * 0.5
    out = torch.empty(T, E, device=DEV)
    todo = torch.arange(T, device=DEV)
    for _ in range(60):
        x = torch.randn(todo.numel(), E, device=DEV, generator=g) * 1.2 + pop
        if c["half"]:
            x = x.bfloat16().float()
        out[todo] = x
        d = x.double()
        s = torch.sigmoid(d) if c["score"] == "sigmoid" else torch.softmax(d, -1)
        key = s + bias.double() if bias is not None else s
        tol = 2e-6 if c["score"] == "sigmoid" else 4e-6 * key.abs().amax(-1, keepdim=True)
        bad = torch.zeros(todo.numel(), dtype=torch.bool, device=DEV)
        if c["groups"] > 1:
            per = key.view(-1, c["groups"], E // c["groups"])
            gs = per.sort(dim=-1, descending=True).values[..., :min(c["group_top"], E // c["groups"])].sum(-1)
            bad |= _near_tie(gs, c["top_groups"], tol)
            cut = gs.sort(dim=-1, descending=True, stable=True).indices[:, c["top_groups"]:]
            key = per.scatter(1, cut.unsqueeze(-1).expand(-1, -1, E // c["groups"]), -9.0).view(-1, E)
        bad |= _near_tie(key, c["K"], tol)
        todo = todo[bad]
        if todo.numel() == 0:
            break
    else:
        # what is left after many draws gets well-spread logits
        step = torch.arange(E, device=DEV, dtype=torch.float32) * -0.125
        out[todo] = step
    return out.bfloat16() if c["half"] else out


def _pow2(byte):
    """The power of two that an e8m0 byte stands for, 2^(byte - 127), as fp32."""
    return torch.where(byte > 0, (byte.int() << 23), torch.full_like(byte, 1 << 22, dtype=torch.int32)).view(torch.float32)


def _scale_byte(amax, top):
    """e8m0 byte of the smallest power of two with amax <= top * 2^e (top: 6 or 127; e >= -127)."""
    bits = amax.view(torch.int32)
    e = (bits >> 23) - 127
    lead = int(math.log2(top))
    limit = int((top / 2 ** lead - 1) * (1 << 23))
    e = e - lead + ((bits & 0x7FFFFF) > limit).int()
    return (e + 127).clamp(0, 254).to(torch.uint8)


def _mx4(x):
    """Blocks of 32 along the last axis of fp32 x: (twice the element values, int8; scale bytes, uint8)."""
    b = x.reshape(*x.shape[:-1], x.shape[-1] // BLOCK, BLOCK)
    byte = _scale_byte(b.abs().amax(-1), 6.0)
    v = b * (1.0 / _pow2(byte)).unsqueeze(-1)
    a = v.abs()
    # e2m1 magnitudes 0, .5, 1, 1.5, 2, 3, 4, 6; ties go to the even code
    two = ((a > 0.25).float() + (a >= 0.75).float() + (a > 1.25).float() + (a >= 1.75).float()
           + 2 * (a > 2.5).float() + 2 * (a >= 3.5).float() + 4 * (a > 5.0).float())
    return (two * torch.sign(v)).to(torch.int8).reshape(x.shape), byte


def _mx4_values(two, byte):
    b = two.reshape(*byte.shape, BLOCK).float()
    return (b * (0.5 * _pow2(byte)).unsqueeze(-1)).reshape(two.shape)


def _mx8(x):
    """As _mx4 with int8 elements: (elements, scale bytes)."""
    b = x.reshape(*x.shape[:-1], x.shape[-1] // BLOCK, BLOCK)
    byte = _scale_byte(b.abs().amax(-1), 127.0)
    return torch.round(b * (1.0 / _pow2(byte)).unsqueeze(-1)).to(torch.int8).reshape(x.shape), byte


def _mx8_values(q, byte):
    return (q.reshape(*byte.shape, BLOCK).float() * _pow2(byte).unsqueeze(-1)).reshape(q.shape)


def prepare(case, seed):
    c = case
    g = _gen(seed)
    R, S, K = c["R"], c["S"], c["K"]
    T = R * S
    s = dict(case=c)
    if c["op"] == "route":
        E = c["E"]
        top = 0.05 if c["score"] == "sigmoid" else 0.3 / E
        s["bias"] = torch.randn(E, device=DEV, generator=g) * top if c["bias"] else None
        s["logits"] = _logits(c, g, s["bias"]).view(R, S, E)
        s["load"] = torch.zeros(E, dtype=torch.int32, device=DEV)
        if c["train"]:
            s["dgates"] = torch.randn(R, S, K, device=DEV, generator=g) * 0.05
    elif c["op"] == "mx":
        E, H, Hp = c["E"], c["H"], c["Hp"]
        # K distinct experts of each token, by perturbed popularity
        logp = torch.tensor(_zipf(E, c["zipf"]), device=DEV).log()
        u = torch.rand(T, E, device=DEV, generator=g).clamp_(1e-12, 1.0)
        topk = (logp - (-u.log()).log()).sort(dim=-1, descending=True).indices[:, :K]
        # (token, k) pairs in expert order, cut into R equal ranks whose segments read home rows
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
        total = counts.sum(0)
        s["cap"] = int(total.max())                                   # longest expert: a plan's number
        s["place"] = torch.arange(T * K, device=DEV) - (total.cumsum(0) - total)[order.values]
        if c["stage"] == "first":
            s["x"] = torch.empty(R, S, H, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
        else:
            s["h"] = torch.empty(T * K, 2 * H, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
        w = torch.empty(E, H, Hp, dtype=torch.bfloat16, device=DEV).normal_(std=0.02, generator=g)
        if own:
            import moe_expert_dispatch_online_gb300 as bep
            s["bep"] = bep
            s["ctx"] = bep.Context(bep.Config(R, E, 1, K, S, H, Hp, bep.BEP_INFER))
            s["slot_expert"] = torch.full((R, 1), -1, dtype=torch.int32, device=DEV)
            s["w"] = bep.MxWeight(s["ctx"])
            bep.bep_mx_quantize_weight(s["ctx"], w, s["w"].codes, s["w"].scales)
            s["rows"] = bep.MxRows(T * K, H)
            s["y"] = torch.empty(T * K, Hp, dtype=torch.bfloat16, device=DEV)
        else:
            two = torch.empty(E, Hp, H, dtype=torch.int8, device=DEV)
            byte = torch.empty(E, Hp, H // BLOCK, dtype=torch.uint8, device=DEV)
            for e in range(0, E, 16):
                two[e:e + 16], byte[e:e + 16] = _mx4(w[e:e + 16].transpose(1, 2).float().contiguous())
            s["w"] = (two, byte)
    else:
        rows, F = T * K, c["F"]
        s["h"] = torch.empty(rows, 2 * F, dtype=torch.bfloat16, device=DEV).normal_(std=1.5, generator=g)
        s["da"] = torch.empty(rows, F, dtype=torch.bfloat16, device=DEV).normal_(std=0.02, generator=g)
    if own and c["op"] != "mx":
        import moe_expert_dispatch_online_gb300 as bep
        s["bep"] = bep
        E = c["E"] if c["op"] == "route" else R * K
        s["ctx"] = bep.Context(bep.Config(R, E, E // R, K, S, 64, 64, bep.BEP_TRAIN))
        if c["op"] == "route":
            s["rc"] = bep.RouteConfig(score=bep.BEP_SCORE_SIGMOID if c["score"] == "sigmoid" else bep.BEP_SCORE_SOFTMAX,
                                      groups=c["groups"], top_groups=c["top_groups"], group_top=c["group_top"],
                                      renorm=c["renorm"], scale=c["scale"])
            s["topk"] = torch.empty(R, S, K, dtype=torch.int32, device=DEV)
            s["gates"] = torch.empty(R, S, K, dtype=torch.float32, device=DEV)
            s["dlogits"] = torch.empty_like(s["logits"])
        else:
            s["a"] = torch.empty_like(s["da"])
            s["a_again"] = torch.empty_like(s["da"])
            s["dh"] = torch.empty_like(s["h"])
            s["ckpt"] = bep.ActCheckpoint(rows, F)
    return s


# ------------------------------------------------------------------------------ one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return {"route": _own_route, "mx": _own_mx, "act": _own_act}[op](state)
    return {"route": _plain_route, "mx": _plain_mx, "act": _plain_act}[op](state)


def _own_route(s):
    bep = s["bep"]
    s["load"].zero_()
    bep.bep_route(s["ctx"], s["rc"], s["logits"], s["topk"], s["gates"], bias=s["bias"], load=s["load"])
    out = dict(topk=s["topk"], gates=s["gates"], load=s["load"])
    if s["case"]["train"]:
        bep.bep_route_bwd(s["ctx"], s["rc"], s["logits"], s["topk"], s["dgates"], s["dlogits"])
        out["dlogits"] = s["dlogits"]
    return out


def _plain_route(s):
    c = s["case"]
    E, K, n = c["E"], c["K"], c["groups"]
    x = s["logits"].view(-1, E).float()
    if c["score"] == "sigmoid":
        p = 1.0 / (1.0 + torch.exp(-x))
    else:
        e = torch.exp(x - x.amax(-1, keepdim=True))
        p = e / e.sum(-1, keepdim=True)
    key = p + s["bias"] if c["bias"] else p
    if n > 1:
        per = key.view(-1, n, E // n)
        score = per.sort(dim=-1, descending=True).values[..., :min(c["group_top"], E // n)].sum(-1)
        best = score.sort(dim=-1, descending=True, stable=True).indices[:, :c["top_groups"]]
        keep = torch.zeros_like(score, dtype=torch.bool).scatter_(1, best, True)
        key = torch.where(keep.unsqueeze(-1), per, -math.inf).view(-1, E)
    topk = key.sort(dim=-1, descending=True, stable=True).indices[:, :K]
    chosen = p.gather(1, topk)
    total = chosen.sum(-1, keepdim=True)
    gates = c["scale"] * (chosen / total if c["renorm"] else chosen)
    load = torch.zeros(E, dtype=torch.int32, device=x.device)
    load.index_add_(0, topk.reshape(-1), torch.ones(topk.numel(), dtype=torch.int32, device=x.device))
    shape = s["logits"].shape[:2] + (K,)
    out = dict(topk=topk.int().view(shape), gates=gates.view(shape), load=load)
    if c["train"]:
        dg = s["dgates"].view(-1, K) * c["scale"]
        if c["renorm"]:
            w = chosen / total
            dg = (dg - (dg * w).sum(-1, keepdim=True)) / total
        dp = torch.zeros_like(p).scatter_(1, topk, dg)
        dx = dp * p * (1.0 - p) if c["score"] == "sigmoid" else p * (dp - (p * dp).sum(-1, keepdim=True))
        out["dlogits"] = dx.to(s["logits"].dtype).view(s["logits"].shape)
    return out


def _own_mx(s):
    bep = s["bep"]
    if s["case"]["stage"] == "first":
        bep.bep_dispatch_mx(s["ctx"], s["x"], s["dest"], s["rows"].codes, s["rows"].scales)
    else:
        bep.bep_swiglu_mx(s["ctx"], s["h"], s["rows"].codes, s["rows"].scales)
    bep.bep_grouped_gemm_mx(s["ctx"], s["cu"], s["slot_expert"], s["rows"].codes, s["rows"].scales,
                            s["w"].codes, s["w"].scales, s["y"])
    return s["y"]


def _plain_mx(s):
    c = s["case"]
    if c["stage"] == "first":
        x = s["x"].view(-1, c["H"]).float()
    else:
        gate, up = s["h"].float().chunk(2, -1)
        x = gate / (1.0 + torch.exp(-gate)) * up
    x = _mx4_values(*_mx4(x))
    if c["stage"] == "first":
        x = x[s["row_token"]]
    padded = torch.zeros(c["E"], s["cap"], c["H"], device=x.device)
    padded[s["row_expert"], s["place"]] = x
    y = torch.matmul(padded, _mx4_values(*s["w"]).transpose(1, 2))
    return y[s["row_expert"], s["place"]].bfloat16()


def _own_act(s):
    bep, k = s["bep"], s["ckpt"]
    bep.bep_swiglu(s["ctx"], s["h"], s["a"], k.codes, k.scales)
    bep.bep_swiglu_bwd(s["ctx"], s["da"], k.codes, k.scales, s["dh"], s["a_again"])
    return dict(a=s["a"], dh=s["dh"], a_again=s["a_again"])


def _plain_act(s):
    h = s["h"].float()
    gate, up = h.chunk(2, -1)
    a = gate / (1.0 + torch.exp(-gate)) * up
    gate, up = _mx8_values(*_mx8(h)).chunk(2, -1)
    sig = 1.0 / (1.0 + torch.exp(-gate))
    da = s["da"].float()
    dh = torch.cat((da * up * sig * (1.0 + gate * (1.0 - sig)), da * gate * sig), -1)
    return dict(a=a.bfloat16(), dh=dh.bfloat16(), a_again=(gate * sig * up).bfloat16())


# ------------------------------------------------------------------------------ 64 bits
def exact(case, seed):
    c = case
    # products in 64 bits run at about a TFLOP/s here
    if c["op"] == "mx" and 2 * c["R"] * c["S"] * c["K"] * c["H"] * c["Hp"] > 4e12:
        return None
    s = prepare(c, seed)
    return {"route": _exact_route, "mx": _exact_mx, "act": _exact_act}[c["op"]](s)


def _exact_route(s):
    c = s["case"]
    T, E, K = c["R"] * c["S"], c["E"], c["K"]
    x = s["logits"].view(T, E).double()
    p = torch.sigmoid(x) if c["score"] == "sigmoid" else torch.softmax(x, -1)
    key = p + (s["bias"].double() if c["bias"] else 0.0)
    ids = torch.arange(E, device=x.device)

    def leading(v, count):
        """Positions of the `count` largest, one after the other; the first position on a tie."""
        v, got = v.clone(), []
        pos = torch.arange(v.shape[-1], device=v.device)
        for _ in range(count):
            top = v.amax(-1, keepdim=True)
            at = torch.where(v == top, pos, v.shape[-1]).amin(-1, keepdim=True)
            got.append(at)
            v.scatter_(-1, at, -2e300)
        return torch.cat(got, -1)

    if c["groups"] > 1:
        n, m = c["groups"], E // c["groups"]
        per = key.view(T, n, m)
        score = per.gather(-1, leading(per, min(c["group_top"], m))).sum(-1)
        best = leading(score, c["top_groups"])
        ok = (best.unsqueeze(-1) == (ids // m)).any(1)
        key = torch.where(ok, key, -1e300)
    topk = leading(key, K)
    v = p.gather(1, topk)
    z = v.sum(-1, keepdim=True) if c["renorm"] else torch.ones_like(v[:, :1])
    shape = (c["R"], c["S"], K)
    load = (topk.reshape(-1, 1) == ids).sum(0) if T * K * E < 1 << 28 else torch.bincount(topk.reshape(-1), minlength=E)
    out = dict(topk=topk.int().view(shape), gates=(c["scale"] * v / z).view(shape), load=load.int())
    if c["train"]:
        dg = s["dgates"].view(T, K).double() * c["scale"]
        if c["renorm"]:
            # d(v_k / sum v) / d v_j, for each chosen pair
            jac = (torch.eye(K, device=x.device, dtype=torch.float64) / z.unsqueeze(-1)
                   - (v / z ** 2).unsqueeze(-1))
            dv = torch.einsum("tk,tkj->tj", dg, jac)
        else:
            dv = dg
        if c["score"] == "sigmoid":
            dx = torch.zeros_like(x)
            dx.scatter_(1, topk, dv * torch.sigmoid(x.gather(1, topk)) * torch.sigmoid(-x.gather(1, topk)))
        else:
            dx = -p * (dv * v).sum(-1, keepdim=True)
            dx.scatter_add_(1, topk, dv * v)
        out["dlogits"] = dx.view(c["R"], c["S"], E)
    return out


def _exact_round(x, values, top):
    """fp64 blocks of 32: nearest of `values` (ascending magnitudes, ties to the even position) times a power of two."""
    b = x.reshape(*x.shape[:-1], -1, BLOCK)
    amax = b.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(amax.clamp_min(2.0 ** -130) / top)).clamp_min(-127)
    # log2 rounds: settle the neighbours by comparison
    e = torch.where(torch.ldexp(torch.full_like(e, top), e - 1) >= amax, e - 1, e).clamp_min(-127)
    e = torch.where(torch.ldexp(torch.full_like(e, top), e) < amax, e + 1, e)
    v = torch.ldexp(b, -e)
    if values is None:
        r = torch.round(v)
    else:
        grid = torch.tensor(values, dtype=torch.float64, device=x.device)
        mid = (grid[1:] + grid[:-1]) / 2
        a = v.abs().contiguous()
        lo, hi = torch.searchsorted(mid, a), torch.searchsorted(mid, a, right=True)
        r = grid[torch.where(lo % 2 == 0, lo, hi)] * torch.sign(v)
    return torch.ldexp(r, e).reshape(x.shape)


_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _exact_mx(s):
    c = s["case"]
    if own:
        return None
    if c["stage"] == "first":
        x = _exact_round(s["x"].view(-1, c["H"]).double(), _E2M1, 6.0)[s["row_token"]]
    else:
        h = s["h"].double()
        gate, up = h[:, :c["H"]], h[:, c["H"]:]
        x = _exact_round(gate * torch.sigmoid(gate) * up, _E2M1, 6.0)
    two, byte = s["w"]
    y = torch.zeros(x.shape[0], c["Hp"], dtype=torch.float64, device=x.device)
    first = torch.searchsorted(s["row_expert"].contiguous(), torch.arange(c["E"] + 1, device=x.device)).tolist()
    for e in range(c["E"]):
        if first[e + 1] > first[e]:
            w = torch.ldexp(two[e].double().view(c["Hp"], -1, BLOCK), byte[e].double().unsqueeze(-1) - 128.0)
            y[first[e]:first[e + 1]] = x[first[e]:first[e + 1]] @ w.view(c["Hp"], c["H"]).t()
    return y


def _exact_act(s):
    F = s["case"]["F"]
    a, dh, again = [], [], []
    for h, da in zip(s["h"].split(16384), s["da"].split(16384)):
        h, da = h.double(), da.double()
        g, u = h[:, :F], h[:, F:]
        a.append((g * torch.sigmoid(g) * u).float())
        q = _exact_round(h, None, 127.0)
        g, u = q[:, :F], q[:, F:]
        sg = torch.sigmoid(g)
        dh.append(torch.cat((da * u * (sg + g * sg * torch.sigmoid(-g)), da * g * sg), -1).float())
        again.append((g * sg * u).float())
    return dict(a=torch.cat(a), dh=torch.cat(dh), a_again=torch.cat(again))
