"""The whole layer of examples/moe_layer.py: a training step's outputs and gradients against
autograd in 64 bits, and a serving step against the 64-bit products of the 4-bit values."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import experts_ref as ref

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example(lib):
    spec = importlib.util.spec_from_file_location("moe_layer", os.path.join(ROOT, "examples", "moe_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def far(got, want):
    got, want = got.double().cpu(), want.double().cpu()
    return ((got - want).norm() / want.norm()).item()


@pytest.mark.parametrize("softmax,renorm", [(True, True), (True, False), (False, True), (False, False)])
def test_training_step(lib, example, softmax, renorm):
    bep = lib
    torch.manual_seed(1)
    R, S, E, K, H, F = 2, 48, 8, 3, 256, 128
    rc = bep.RouteConfig(score=bep.BEP_SCORE_SOFTMAX if softmax else bep.BEP_SCORE_SIGMOID, renorm=renorm, scale=1.5)
    layer = example.MoELayer(R, S, E, K, H, F, rc)
    x = torch.randn(R, S, H, device="cuda").bfloat16()
    dout = torch.randn(R, S, H, device="cuda").bfloat16()
    out = layer.forward(x)
    dx, g_router, g1, g2 = layer.backward(x, dout)
    layer.check()
    v = [t.detach().double().cpu().requires_grad_() for t in (x, layer.w_router, layer.w1, layer.w2)]
    xd, wr, w1, w2 = v
    logits = xd.view(-1, H) @ wr
    s = torch.softmax(logits, -1) if softmax else torch.sigmoid(logits)
    topk = layer.topk.view(-1, K).long().cpu()
    assert torch.equal(topk, s.sort(dim=-1, descending=True, stable=True).indices[:, :K])
    g = s.gather(1, topk)
    g = 1.5 * (g / g.sum(-1, keepdim=True) if renorm else g)
    want = torch.zeros(R * S, H, dtype=torch.float64)
    for k in range(K):
        h = torch.einsum("th,thf->tf", xd.view(-1, H), w1[topk[:, k]])
        a = torch.nn.functional.silu(h[:, :F]) * h[:, F:]
        want = want + g[:, k:k + 1] * torch.einsum("tf,tfh->th", a, w2[topk[:, k]])
    want.backward(dout.double().cpu().view(-1, H))
    # bf16 between the stages (2^-8 / sqrt 3 each, up to six of them) and int8 activations in the
    # backward (2^-7 of a block's largest, about 1% of its rms)
    assert far(out, want.view(R, S, H).detach()) < 2e-2
    for got, t in ((dx, xd), (g_router, wr), (g1, w1), (g2, w2)):
        assert far(got, t.grad) < 3e-2


def test_serving_step(lib, example):
    bep = lib
    torch.manual_seed(2)
    R, S, E, K, H, F = 4, 9, 16, 4, 320, 192
    layer = example.MoELayer(R, S, E, K, H, F, bep.RouteConfig(score=bep.BEP_SCORE_SIGMOID, groups=4, top_groups=2,
                                                               group_top=2))
    layer.quantise()
    x = torch.randn(R, S, H, device="cuda").bfloat16()
    out = layer.serve(x)
    layer.check()

    def values(q, Hp, n):
        return ref.mx4_values(ref.unpack4(q.codes.cpu().numpy()), ref.unblock_scales(q.scales.cpu().numpy(), Hp, n // 32))

    w1, w2 = values(layer.q1, 2 * F, H), values(layer.q2, H, F)
    xq = ref.mx4_values(*ref.mx4(x.double().cpu().numpy().reshape(-1, H)))
    topk, gates = layer.topk.view(-1, K).cpu().numpy(), layer.gates.view(-1, K).cpu().numpy()
    want = np.zeros((R * S, H))
    for t in range(R * S):
        for k in range(K):
            h = w1[topk[t, k]] @ xq[t]
            a = ref.mx4_values(*ref.mx4(ref.swiglu(h[None])))[0]
            want[t] += gates[t, k] * (w2[topk[t, k]] @ a)
    # h is rounded to bf16 before the activation is quantised: of the e2m1 values within 2^-8 of a
    # rounding boundary (about 2 in 100) half go to the neighbour, a step of a quarter of their size
    assert far(out.view(-1, H), torch.from_numpy(want)) < 4e-2


def test_example_runs(example, monkeypatch, capsys):
    monkeypatch.setattr("sys.argv", ["moe_layer.py", "--steps", "3"])
    example.main()
    text = capsys.readouterr().out
    losses = [float(line.split("loss ")[1].split(",")[0]) for line in text.splitlines() if "loss" in line]
    assert len(losses) == 3 and losses[2] < losses[0]
    assert float(text.split("4 bits: ")[1].split()[0]) < 0.4
