"""The experts with gradients (training.py) against autograd of the same layer
written plainly in 64 bits, the serving layer, and the example that trains."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def layer():
    import group_limited_routed_gb300 as pkg
    from group_limited_routed_gb300 import inputs
    cfg = inputs.CONFIGS["tiny"].replace(T=70)
    t = inputs.generate(cfg, "cuda")
    ws = pkg.Workspace(cfg, cfg.T)
    idx, w = pkg.route(cfg, t["hidden"], t["router_w"], t["corr_bias"], ws=ws)
    return pkg, cfg, t, ws, idx, w


def plain(x, idx, w, wg, wu, wd):
    out = torch.zeros_like(x)
    for e in range(wg.shape[0]):
        tok, slot = (idx == e).nonzero(as_tuple=True)
        if tok.numel() == 0:
            continue
        g, u = x[tok] @ wg[e].t(), x[tok] @ wu[e].t()
        h = w[tok, slot][:, None] * g * torch.sigmoid(g) * u
        out = out.index_add(0, tok, h @ wd[e].t())
    return out


def test_experts_and_their_gradients(layer):
    pkg, cfg, t, ws, idx, w = layer
    from group_limited_routed_gb300 import training
    names = ("w_gate", "w_up", "w_down")
    leaves = [t["hidden"].clone().requires_grad_(), w.clone().requires_grad_(),
              *(t[n].clone().requires_grad_() for n in names)]
    out = training.experts(leaves[0], idx, *leaves[1:])
    exact = [v.detach().double().requires_grad_() for v in leaves]
    ref = plain(exact[0], idx, *exact[1:])
    # the layer's own bound on its outputs is 1e-2 of their root mean square
    # (three BF16 roundings on the way: gate, up, h); the same chain, one
    # product longer, gives 2e-2 for the gradients
    rms = ref.square().mean().sqrt()
    assert ((out.double() - ref).square().mean().sqrt() / rms).item() < 1e-2
    c = torch.randn(out.shape, generator=torch.Generator(device="cuda").manual_seed(5),
                    device="cuda").bfloat16()
    out.backward(c)
    ref.backward(c.double())
    for name, a, b in zip(("hidden", "topk_w") + names, leaves, exact):
        assert a.grad is not None and a.grad.dtype == a.dtype, name
        off = ((a.grad.double() - b.grad).norm() / b.grad.norm()).item()
        assert off < 2e-2, (name, off)
    # and the serving layer on the same routing
    serve = pkg.forward_routed(cfg, t["hidden"], idx, w, *(t[n] for n in names), ws=ws)
    assert ((out.double() - serve.double()).square().mean().sqrt() / rms).item() < 2e-2


def test_experts_no_token_chose_get_zero_gradients(layer):
    pkg, cfg, t, ws, idx, w = layer
    from group_limited_routed_gb300 import training
    few = idx[:2].clone()
    wd = t["w_down"].clone().requires_grad_()
    training.experts(t["hidden"][:2], few, w[:2], t["w_gate"], t["w_up"], wd).sum().backward()
    chosen = torch.zeros(cfg.n_experts, dtype=torch.bool, device="cuda")
    chosen[few.reshape(-1).long()] = True
    assert (wd.grad[~chosen] == 0).all() and (wd.grad[chosen].abs().amax((1, 2)) > 0).all()


def test_repeated_steps_are_bit_identical(layer):
    pkg, cfg, t, ws, idx, w = layer
    from group_limited_routed_gb300 import training

    def grads():
        leaves = [t["hidden"].clone().requires_grad_(), t["w_gate"].clone().requires_grad_()]
        training.experts(leaves[0], idx, w, leaves[1], t["w_up"], t["w_down"]).sum().backward()
        return [v.grad for v in leaves]
    for a, b in zip(grads(), grads()):
        assert torch.equal(a, b)


def test_the_example_trains():
    spec = importlib.util.spec_from_file_location(
        "train_experts", os.path.join(ROOT, "examples", "train_experts.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    losses = mod.main(steps=30)
    assert losses[-1] < 0.8 * losses[0], losses
