"""The layer of examples/moe_layer.py served with 8-bit experts, and trained and served with adapters, against
64-bit forms."""
import numpy as np
import pytest
import torch

import experts_ref
import int8_ref as ref
from test_gpu_moe_layer import example, far  # noqa: F401

pytestmark = pytest.mark.gpu


def quantised(w):
    q, s = ref.quantise(w)
    return q * s.astype(np.float64)[..., None]


@pytest.mark.parametrize("rank", [0, 24])
def test_serving_in_8_bits(lib, example, rank):  # noqa: F811
    bep = lib
    torch.manual_seed(2)
    R, S, E, K, H, F = 4, 9, 16, 4, 320, 192
    layer = example.MoELayer(R, S, E, K, H, F, bep.RouteConfig(score=bep.BEP_SCORE_SIGMOID, groups=4, top_groups=2,
                                                               group_top=2))
    layer.quantise8()
    if rank:
        layer.adapt(rank, 0.5)
        for _, B in layer.adapters:
            B.normal_(std=rank ** -0.5)
    x = torch.randn(R, S, H, device="cuda").bfloat16()
    out = layer.serve8(x)
    layer.check()
    f64 = lambda t: t.double().cpu().numpy()  # noqa: E731
    w1, w2 = (quantised(f64(w).transpose(0, 2, 1)) for w in (layer.w1, layer.w2))
    xs = f64(x).reshape(-1, H)
    xq = quantised(xs)
    ad = [[f64(w) for w in pair] for pair in layer.adapters] if rank else None
    topk, gates = layer.topk.view(-1, K).cpu().numpy(), layer.gates.view(-1, K).cpu().numpy()
    want = np.zeros((R * S, H))
    for t in range(R * S):
        for k in range(K):
            e = topk[t, k]
            h = w1[e] @ xq[t]
            if rank:
                h = h + 0.5 * (xs[t] @ ad[0][0][e]) @ ad[0][1][e]
            a = experts_ref.swiglu(h[None])
            y = w2[e] @ quantised(a)[0]
            if rank:
                y = y + 0.5 * (a[0] @ ad[1][0][e]) @ ad[1][1][e]
            want[t] += gates[t, k] * y
    # h, the adapters' low rows and y are bf16 (2^-9 of their size each, on average less); an activation whose
    # integer rounds the other way moves by 1/127 of its row's largest, one in 100 of them
    assert far(out.view(-1, H), torch.from_numpy(want)) < 1.5e-2


def test_training_with_adapters(lib, example):  # noqa: F811
    bep = lib
    torch.manual_seed(3)
    R, S, E, K, H, F, rank = 2, 48, 8, 3, 256, 128, 8
    layer = example.MoELayer(R, S, E, K, H, F, bep.RouteConfig(score=bep.BEP_SCORE_SIGMOID))
    layer.adapt(rank, 0.5)
    for _, B in layer.adapters:
        B.normal_(std=rank ** -0.5)
    x = torch.randn(R, S, H, device="cuda").bfloat16()
    dout = torch.randn(R, S, H, device="cuda").bfloat16()
    out = layer.forward(x)
    dx, g_router, g1, g2 = layer.backward(x, dout)
    layer.check()
    leaves = [t.detach().double().cpu().requires_grad_()
              for t in (x, layer.w_router, layer.w1, layer.w2, *layer.adapters[0], *layer.adapters[1])]
    xd, wr, w1, w2, A1, B1, A2, B2 = leaves
    s = torch.sigmoid(xd.view(-1, H) @ wr)
    topk = layer.topk.view(-1, K).long().cpu()
    g = s.gather(1, topk)
    g = g / g.sum(-1, keepdim=True)
    rows = lambda v, w, e: torch.einsum("tn,tnm->tm", v, w[e])  # noqa: E731
    want = torch.zeros(R * S, H, dtype=torch.float64)
    for k in range(K):
        e = topk[:, k]
        v = xd.view(-1, H)
        h = rows(v, w1, e) + 0.5 * rows(rows(v, A1, e), B1, e)
        a = torch.nn.functional.silu(h[:, :F]) * h[:, F:]
        want = want + g[:, k:k + 1] * (rows(a, w2, e) + 0.5 * rows(rows(a, A2, e), B2, e))
    want.backward(dout.double().cpu().view(-1, H))
    # bf16 between the stages, up to ten of them (2^-8 / sqrt 3 each), and int8 activations in the backward
    assert far(out, want.view(R, S, H).detach()) < 2e-2
    got = (dx, g_router, g1, g2, *layer.adapter_grads[0], *layer.adapter_grads[1])
    for t, leaf in zip(got, leaves):
        assert far(t, leaf.grad) < 3e-2


def test_example_says_how_far_8_bits_are(example, monkeypatch, capsys):  # noqa: F811
    monkeypatch.setattr("sys.argv", ["moe_layer.py", "--steps", "2", "--rank", "24"])
    example.main()
    text = capsys.readouterr().out
    assert float(text.split("8 bits: ")[1].split()[0]) < 0.03
    assert float(text.split("8-bit experts: ")[1].split()[0]) < 0.03
