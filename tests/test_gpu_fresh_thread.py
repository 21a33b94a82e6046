"""Calls from a host thread that has done no CUDA work before: a server's worker
threads start like that, and nothing has made a context current in them."""
import threading

import pytest
import torch

from tests.test_gpu_few import buffers, call, make, no_error

pytestmark = pytest.mark.gpu


def _in_a_fresh_thread(step):
    failed = []

    def body():
        try:
            step()
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    torch.cuda.synchronize()
    t = threading.Thread(target=body)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert failed == []


def test_few_tokens(lib):
    p = make(3, 512, 8, 2, 256, seed=1)
    call(p, want := buffers(p))
    o = buffers(p)
    _in_a_fresh_thread(lambda: call(p, o))
    no_error()
    for k in ("out", "topk_idx", "gates", "counts"):
        assert torch.equal(o[k], want[k])


def test_separate_steps(lib):
    """The router's and the grouped GEMM's calls, each the first of its thread."""
    import workloads
    from fine_grained_fp8_sigmoid_b200 import MoELayerFP8
    cfg = workloads.CONFIGS["tiny"].with_tokens(33)
    layer = MoELayerFP8(cfg.T, cfg.d, cfg.N_r, cfg.K_r, cfg.I)
    for slot in range(cfg.N_r + 1):
        layer.load_expert(slot, *[x.cuda() for x in workloads.expert_weights(cfg, slot)])
    u, e, b = (x.cuda() for x in (workloads.activations(cfg), workloads.centroids(cfg), workloads.bias(cfg)))
    want = layer.forward(u, e, b, update_bias=False).clone()
    for t in (layer.topk_idx, layer.gates, layer.y_perm, layer.y_shared, layer.out):
        t.zero_()
    for step in (lambda: layer.route(u, e, b), lambda: layer.quant(u), layer.permute, layer.experts,
                 lambda: layer.combine(u)):
        _in_a_fresh_thread(step)
    no_error()
    assert torch.equal(layer.out, want)


def test_norm_and_its_gradient(lib):
    from fine_grained_fp8_sigmoid_b200 import binding as B
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn(200, 1024, generator=g, device="cuda").to(torch.bfloat16)
    w, dw, dw2 = (torch.ones(1024, device="cuda") for _ in range(3))
    y, y2, dh, dh2 = (torch.empty_like(x) for _ in range(4))
    ws = torch.empty(B.moe_rmsnorm_backward_workspace(200, 1024), dtype=torch.uint8, device="cuda")
    B.moe_rmsnorm_quant(x, w, 1e-6, y=y)
    B.moe_rmsnorm_backward(x, y, w, 1e-6, dh, dw, ws)
    _in_a_fresh_thread(lambda: B.moe_rmsnorm_quant(x, w, 1e-6, y=y2))
    _in_a_fresh_thread(lambda: B.moe_rmsnorm_backward(x, y2, w, 1e-6, dh2, dw2, ws))
    assert torch.equal(y, y2) and torch.equal(dh, dh2) and torch.equal(dw, dw2)
