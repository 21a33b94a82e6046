"""Calls that the header allows: outputs over inputs, and kernels of several calls
on the GPU at once (each with its own workspace)."""
import pytest
import torch

from tests.test_gpu_few import buffers, call, make, no_error

pytestmark = pytest.mark.gpu


def _rows(rows, d, n, seed, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(rows, d, generator=g, device="cuda").to(dtype) for _ in range(n)]


@pytest.mark.parametrize("rows,d", [(5, 512), (700, 2048), (301, 7168)])
def test_norm_over_its_inputs(lib, rows, d):
    from fine_grained_fp8_sigmoid_b200 import binding as B
    x, res = _rows(rows, d, 2, seed=rows)
    w = 1 + 0.1 * torch.randn(d, device="cuda")
    new = lambda: (torch.empty_like(x), torch.empty_like(x), torch.empty(rows, d, dtype=torch.uint8, device="cuda"),  # noqa: E731
                   torch.empty(rows, d // 128, device="cuda"))
    h, y, q, s = new()
    B.moe_rmsnorm_quant(x, w, 1e-6, y=y, q=q, scale=s, residual=res, h=h)
    for over in ("h over x", "y over x", "h over residual and y over x"):
        x2, r2 = x.clone(), res.clone()
        h2, y2, q2, s2 = new()
        if over == "h over x":
            h2 = x2
        else:
            y2 = x2
            h2 = r2 if "residual" in over else h2
        B.moe_rmsnorm_quant(x2, w, 1e-6, y=y2, q=q2, scale=s2, residual=r2, h=h2)
        for a, b in ((h, h2), (y, y2), (q, q2), (s, s2)):
            assert torch.equal(a, b), over


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,d", [(1, 512), (700, 2048), (901, 7168)])
def test_norm_gradient_over_dres(lib, rows, d, dtype):
    from fine_grained_fp8_sigmoid_b200 import binding as B
    h, dres = _rows(rows, d, 2, seed=rows, dtype=dtype)
    dy, = _rows(rows, d, 1, seed=1)
    w = 1 + 0.1 * torch.randn(d, device="cuda")
    dh, dw, dw2 = torch.empty_like(h), torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    ws = torch.empty(B.moe_rmsnorm_backward_workspace(rows, d), dtype=torch.uint8, device="cuda")
    B.moe_rmsnorm_backward(dy, h, w, 1e-6, dh, dw, ws, dres=dres)
    B.moe_rmsnorm_backward(dy, h, w, 1e-6, dres, dw2, ws, dres=dres)
    assert torch.equal(dh, dres) and torch.equal(dw, dw2)


def test_few_tokens_with_one_tensor_as_u_base_and_out(lib):
    p = make(7, 1024, 16, 3, 256, seed=3)
    call(p, want := buffers(p))
    o = buffers(p)
    u = p["u"].clone()
    call({**p, "u": u, "base": u}, o, out=u)
    no_error()
    assert torch.equal(u, want["out"]) and torch.equal(o["topk_idx"], want["topk_idx"])


def test_replays_beside_the_separate_steps(lib):
    """Two captured few-token calls replayed on two streams while a third runs the
    layer's separate steps: all of them take whole SMs' tensor memory in turns."""
    import workloads
    from fine_grained_fp8_sigmoid_b200 import MoELayerFP8
    ps = [make(T, 1024, 32, 4, 512, seed=T) for T in (3, 12)]
    os_, graphs = [buffers(p) for p in ps], []
    for p, o in zip(ps, os_):
        call(p, o)
    want = [o["out"].clone() for o in os_]
    for p, o in zip(ps, os_):
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(p, o)
        graphs.append(graph)
    cfg = workloads.CONFIGS["mid"].with_tokens(300)
    layer = MoELayerFP8(cfg.T, cfg.d, cfg.N_r, cfg.K_r, cfg.I)
    for slot in range(cfg.N_r + 1):
        layer.load_expert(slot, *[x.cuda() for x in workloads.expert_weights(cfg, slot)])
    u, e, b = (x.cuda() for x in (workloads.activations(cfg), workloads.centroids(cfg), workloads.bias(cfg)))
    ref = layer.forward(u, e, b, update_bias=False).clone()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for o in os_:
        o["out"].zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        layer.forward(u, e, b, update_bias=False, stream=streams[2])
    torch.cuda.synchronize()
    no_error()
    assert torch.equal(layer.out, ref)
    for o, w in zip(os_, want):
        assert torch.equal(o["out"], w)
