"""The pre-norm, the few-token layer and the norm's gradient as a model runs
them: MoELayerFP8.forward_prenorm (both forms of the layer) and
ExpertFFNBackward.norm_backward behind it."""
import numpy as np
import pytest
import torch

import workloads
from oracle import moe as O
from tests.test_gpu_few import D, no_error, reference
from tests.test_gpu_norm import _check_backward, _check_forward, f64

pytestmark = pytest.mark.gpu

EPS = 1e-6


def _layer(cfg, **kw):
    from fine_grained_fp8_sigmoid_b200 import MoELayerFP8
    layer = MoELayerFP8(cfg.T, cfg.d, cfg.N_r, cfg.K_r, cfg.I, **kw)
    for slot in range(cfg.N_r + 1):
        layer.load_expert(slot, *[x.cuda() for x in workloads.expert_weights(cfg, slot)])
    return layer


def _inputs(cfg, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return dict(x=r(cfg.T, cfg.d).to(torch.bfloat16).cuda(), residual=(r(cfg.T, cfg.d) * 2).to(torch.bfloat16).cuda(),
                w=(1 + 0.1 * r(cfg.d)).cuda(), e=workloads.centroids(cfg).cuda(), b=workloads.bias(cfg).cuda())


def _as_case(layer, i):
    """What the layer was given, as test_gpu_few's plain layer takes it."""
    p = dict(dims=(layer.T, layer.d, layer.N_r, layer.K_r, layer.I), u=layer.u, e=i["e"], b=i["b"], xq=layer.xq,
             xs=layer.xs, base=layer.h)
    for n in ("gate", "up", "down"):
        p["w_" + n], p["s_" + n] = getattr(layer, "w_" + n), getattr(layer, "s_" + n)
    return p


@pytest.mark.parametrize("name,T", [("tiny", 1), ("tiny", 16), ("mid", 1), ("mid", 5), ("mid", 16)])
def test_few_tokens_behind_the_norm(lib, name, T):
    cfg = workloads.CONFIGS[name].with_tokens(T)
    layer = _layer(cfg, few=True, prenorm=True)
    i = _inputs(cfg, seed=T)
    s = f64(i["x"]) + f64(i["residual"])
    bias = i["b"].clone()
    out = layer.forward_prenorm(i["x"], i["w"], i["e"], i["b"], residual=i["residual"], eps=EPS)
    no_error()
    _check_forward(s, f64(i["w"]), EPS, layer.h, layer.u, layer.xq, layer.xs)
    i["b"], moved = bias, i["b"]
    ref, bound, idx, gates = reference(_as_case(layer, i))
    assert torch.equal(layer.topk_idx.long(), idx)
    err = (out.to(D) - ref).abs()
    assert (err <= bound + 2.0 ** -8 * (ref.abs() + bound)).all()
    counts = np.bincount(idx.cpu().numpy().ravel(), minlength=cfg.N_r)
    want, _ = O.bias_update(bias.cpu().double().numpy(), counts, cfg.T, cfg.K_r)
    assert np.array_equal(f64(moved), want)


@pytest.mark.parametrize("few", [False, True])
def test_two_layers_on_one_stream_in_a_graph(lib, few):
    """Two blocks, the second's residual the first's output, captured once and
    replayed on new inputs: the same bits as running them."""
    cfg = workloads.CONFIGS["tiny"].with_tokens(9)
    layers = [_layer(cfg, few=few, prenorm=True) for _ in range(2)]
    i, j = _inputs(cfg, 3), _inputs(cfg, 4)

    def step():
        a = layers[0].forward_prenorm(i["x"], i["w"], i["e"], i["b"], residual=i["residual"], update_bias=False)
        return layers[1].forward_prenorm(i["x"], i["w"], i["e"], i["b"], residual=a, update_bias=False)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    i["x"].copy_(j["x"])
    i["residual"].copy_(j["residual"])
    graph.replay()
    got = out.clone()
    assert torch.equal(step(), got)
    no_error()


def test_separate_steps_take_the_norms_codes(lib):
    """The ordinary layer behind the norm is its own steps on u, xq, xs with h as
    the base, and without a residual h is x."""
    from fine_grained_fp8_sigmoid_b200 import binding as B
    cfg = workloads.CONFIGS["mid"].with_tokens(200)
    layer = _layer(cfg, prenorm=True)
    i = _inputs(cfg, seed=7)
    out = layer.forward_prenorm(i["x"], i["w"], i["e"], i["b"], update_bias=False).clone()
    assert torch.equal(layer.h, i["x"])
    _check_forward(f64(i["x"]), f64(i["w"]), EPS, layer.h, layer.u, layer.xq, layer.xs)
    B.moe_route(layer.u, i["e"], i["b"], layer.K_r, layer.topk_idx, layer.gates)
    layer.permute()
    layer.experts()
    layer.combine(layer.h)
    assert torch.equal(layer.out, out)
    no_error()


def test_forward_with_few_tokens_without_a_norm(lib):
    cfg = workloads.CONFIGS["mid"].with_tokens(11)
    layer, plain = _layer(cfg, few=True), _layer(cfg)
    u, e, b = workloads.activations(cfg).cuda(), workloads.centroids(cfg).cuda(), workloads.bias(cfg).cuda()
    b2 = b.clone()
    out, ref = layer.forward(u, e, b), plain.forward(u, e, b2)
    no_error()
    assert layer.launches_per_step() == 3
    assert torch.equal(layer.topk_idx, plain.topk_idx) and torch.equal(layer.counts, plain.counts)
    assert torch.equal(b, b2)
    # the plain layer rounds each of its K + 1 rows to bf16 first (half a step of what they
    # add up to in absolute terms), and a code of an intermediate row may be the neighbour
    layer.u, layer.h = u, u
    layer.quant(u)
    _, bound, _, _ = reference(_as_case(layer, dict(e=e, b=b)))
    y = torch.cat([plain.y_perm[plain.inv.long().clamp(min=0)].abs().to(D) * plain.gates[:, :, None],
                   plain.y_shared.abs().to(D)[:, None]], 1).sum(1)
    err = (out.to(D) - ref.to(D)).abs()
    assert (err <= 2 * bound + 2.0 ** -8 * y + 2.0 ** -7 * (ref.to(D).abs() + 2 * bound)).all()


def test_few_tokens_from_host_batches(lib):
    """The pipelined host path of a few-token layer runs the few-token calls."""
    cfg = workloads.CONFIGS["tiny"].with_tokens(7)
    layer = _layer(cfg, few=True)
    e, b = workloads.centroids(cfg).cuda(), workloads.bias(cfg).cuda()
    g = torch.Generator().manual_seed(2)
    us = [torch.randn(cfg.T, cfg.d, generator=g).to(torch.bfloat16).pin_memory() for _ in range(5)]
    outs = [torch.empty_like(u).pin_memory() for u in us]
    devs = [torch.empty(cfg.T, cfg.d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    layer.forward_host_pipelined(us, e, b, outs, devs, update_bias=False)
    torch.cuda.synchronize()
    for u, o in zip(us, outs):
        assert torch.equal(layer.forward(u.cuda(), e, b, update_bias=False).cpu(), o)
    no_error()


def test_gradient_of_the_norm_behind_the_experts(lib):
    from fine_grained_fp8_sigmoid_b200.backward import ExpertFFNBackward
    cfg = workloads.CONFIGS["mid"].with_tokens(96)
    layer = _layer(cfg, prenorm=True)
    i = _inputs(cfg, seed=8)
    layer.forward_prenorm(i["x"], i["w"], i["e"], i["b"], residual=i["residual"])
    g = torch.Generator().manual_seed(1)
    dy = (torch.randn(cfg.P + cfg.T, cfg.d, generator=g) * 0.01).to(torch.bfloat16).cuda()
    dres = (torch.randn(cfg.T, cfg.d, generator=g) * 0.01).to(torch.bfloat16).cuda()
    back = ExpertFFNBackward(layer)
    du = back.backward(dy, wgrad=False)["dx"]
    got = back.norm_backward(du, i["w"], EPS, dres=dres)
    _check_backward(f64(du), f64(layer.h), f64(i["w"]), EPS, f64(dres), got["dh"], got["dw"], cfg.T)


def test_layer_refusals(lib):
    from fine_grained_fp8_sigmoid_b200 import MoELayerFP8
    from fine_grained_fp8_sigmoid_b200.backward import ExpertFFNBackward
    with pytest.raises(ValueError, match="16 tokens"):
        MoELayerFP8(17, 256, 8, 2, 128, few=True)
    layer = MoELayerFP8(4, 256, 8, 2, 256)
    x = torch.zeros(4, 256, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="prenorm=True"):
        layer.forward_prenorm(x, torch.ones(256, device="cuda"), None, None)
    with pytest.raises(ValueError, match="prenorm=True"):
        ExpertFFNBackward(layer).norm_backward(x, torch.ones(256, device="cuda"))
    with pytest.raises(ValueError, match="few=True"):
        ExpertFFNBackward(MoELayerFP8(4, 256, 8, 2, 256, few=True))
