"""moe_rmsnorm_quant and moe_rmsnorm_backward against the float64 oracle.

Tolerances. All sums and products are FP32. s = x + res is one rounding; its
squares are non-negative, so their sum (at most 32 values a thread in order,
then 5 + 32 exchanged) is off by at most 70 roundings, its mean by three more
(1/d, the product, eps), which the square root halves; the root itself is
good to two units (4 steps of 2^-24), and y takes three more. That is under
ROUND = 64 steps of 2^-24 relative.
Stored values add half a step of their type. dh adds three terms, each off by
ROUND + the 70 of the projection; dw adds over rows in order.
"""
import numpy as np
import pytest
import torch

from oracle import moe as O
from oracle.e4m3 import decode

pytestmark = pytest.mark.gpu

EPS32 = 2.0 ** -24
ROUND = 64 * EPS32
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
TINY = 2.0 ** -126                       # below it a type's steps stop shrinking


def f64(t):
    return t.detach().cpu().double().numpy()


def _inputs(rows, d, stream, wtype, seed, ld=None):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, ld or d, generator=g).to(torch.bfloat16)
    res = torch.randn(rows, d, generator=g)
    res[:, ::97] *= 30.0
    w = 1.0 + 0.2 * torch.randn(d, generator=g)
    return x.cuda(), res.to(stream).cuda(), w.to(wtype).cuda()


def _outputs(rows, d, stream, quant=True):
    dev = dict(device="cuda")
    return (torch.empty(rows, d, dtype=stream, **dev), torch.empty(rows, d, dtype=torch.bfloat16, **dev),
            torch.empty(rows, d, dtype=torch.uint8, **dev) if quant else None,
            torch.empty(rows, d // 128, dtype=torch.float32, **dev) if quant else None)


def _check_forward(s, w, eps, h, y, q, scale):
    """s: the float64 sum of the inputs."""
    if h is not None:
        assert (np.abs(f64(h) - s) <= HALF[h.dtype] * np.abs(s) * (1 + 1e-6) + TINY).all()
    ref = O.rmsnorm(s, w, eps)
    if y is not None:
        assert (np.abs(f64(y) - ref) <= (HALF[torch.bfloat16] + 2 * ROUND) * np.abs(ref) + TINY).all()
    if q is not None:
        rows, d = ref.shape
        amax = np.abs(ref).reshape(rows, d // 128, 128).max(-1)
        sc = f64(scale)
        want = np.where(amax == 0, 1.0, amax / 448.0)
        assert (np.abs(sc - want) <= 2 * ROUND * want).all()
        sr = np.repeat(sc, 128, 1)
        v = decode(q.cpu().numpy()) * sr
        # half a step of E4M3: 2^-4 relative, 2^-10 of the scale below its smallest normal value
        assert (np.abs(v - ref) <= (2.0 ** -4 + 4 * ROUND) * np.abs(ref) + 2.0 ** -10 * sr * (1 + ROUND)).all()


@pytest.mark.parametrize("rows,d", [(1, 128), (1, 7168), (3, 256), (129, 384), (37, 2048), (150, 7168), (300, 640),
                                    (5, 8192), (2, 32768), (160, 16384)])
@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
def test_norm(lib, rows, d, stream):
    from fine_grained_fp8_sigmoid_b200 import binding as B
    wtype = torch.float32 if rows % 2 else torch.bfloat16
    x, res, w = _inputs(rows, d, stream, wtype, seed=rows + d)
    h, y, q, scale = _outputs(rows, d, stream)
    B.moe_rmsnorm_quant(x, w, 1e-6, y=y, q=q, scale=scale, residual=res, h=h)
    s = f64(x) + f64(res)
    _check_forward(s, f64(w), 1e-6, h, y, q, scale)
    # each output alone, without a residual
    y2 = torch.empty_like(y)
    B.moe_rmsnorm_quant(x, w, 1e-5, y=y2)
    _check_forward(f64(x), f64(w), 1e-5, None, y2, None, None)
    B.moe_rmsnorm_quant(x, w, 1e-5, q=q, scale=scale)
    _check_forward(f64(x), f64(w), 1e-5, None, None, q, scale)


@pytest.mark.parametrize("rows,d", [(4, 8), (33, 72), (130, 1000), (2, 7176)])
def test_norm_without_quantisation_takes_any_multiple_of_8(lib, rows, d):
    from fine_grained_fp8_sigmoid_b200 import binding as B
    x, res, w = _inputs(rows, d, torch.bfloat16, torch.float32, seed=d)
    h, y, _, _ = _outputs(rows, d, torch.bfloat16, quant=False)
    B.moe_rmsnorm_quant(x, w, 1e-6, y=y, residual=res, h=h)
    _check_forward(f64(x) + f64(res), f64(w), 1e-6, h, y, None, None)


def test_norm_strided_rows_and_in_place(lib):
    from fine_grained_fp8_sigmoid_b200 import binding as B
    rows, d = 41, 512
    wide, res, w = _inputs(rows, d, torch.bfloat16, torch.float32, seed=5, ld=3 * d)
    x = wide[:, d:2 * d]
    s = f64(x) + f64(res)
    y, q, scale = _outputs(rows, d, torch.bfloat16)[1:]
    B.moe_rmsnorm_quant(x, w, 1e-6, y=y, q=q, scale=scale, residual=res, h=res)     # the stream in place
    _check_forward(s, f64(w), 1e-6, res, y, q, scale)
    x2 = wide[:, :d].contiguous()
    ref = f64(x2)
    B.moe_rmsnorm_quant(x2, w, 1e-6, y=x2)                                          # y over x
    _check_forward(ref, f64(w), 1e-6, None, x2, None, None)


def test_norm_codes_equal_the_quantiser_where_y_is_exact(lib):
    """Rows of +-1 have a mean square of one: y = w x exactly, so the codes and
    scales are moe_quant_1x128's of y bit for bit."""
    from fine_grained_fp8_sigmoid_b200 import binding as B
    rows, d = 65, 1024
    g = torch.Generator().manual_seed(0)
    x = (torch.randint(0, 2, (rows, d), generator=g) * 2 - 1).to(torch.bfloat16).cuda()
    w = torch.randn(d, generator=g).to(torch.bfloat16).cuda()
    w[:128] = 0                                                                     # an all-zero tile
    _, y, q, scale = _outputs(rows, d, torch.bfloat16)
    B.moe_rmsnorm_quant(x, w, 0.0, y=y, q=q, scale=scale)
    q2, s2 = torch.empty_like(q), torch.empty_like(scale)
    B.moe_quant_1x128(y, q2, s2)
    assert torch.equal(y, (x.float() * w.float()).to(torch.bfloat16))
    assert torch.equal(q, q2) and torch.equal(scale, s2)


def test_norm_extreme_rows_stay_in_their_rows(lib):
    from fine_grained_fp8_sigmoid_b200 import binding as B
    rows, d = 140, 256
    x, res, w = _inputs(rows, d, torch.bfloat16, torch.float32, seed=9)
    x[1], res[1] = 0.0, 0.0                          # a zero row: y = 0, scale = 1
    x[2, 7] = float("nan")
    x[3, 7] = float("inf")
    x[4], res[4] = 2.0 ** -40, 0.0                   # eps dominates
    h, y, q, scale = _outputs(rows, d, torch.bfloat16)
    B.moe_rmsnorm_quant(x, w, 1e-6, y=y, q=q, scale=scale, residual=res, h=h)
    keep = [i for i in range(rows) if i not in (2, 3)]
    _check_forward((f64(x) + f64(res))[keep], f64(w), 1e-6, h[keep], y[keep], q[keep], scale[keep])
    assert (f64(y[1]) == 0).all() and (f64(scale[1]) == 1).all()
    assert np.isnan(f64(y[2])).all() and np.isnan(f64(y[3, 7])) and (f64(y[3, 8:]) == 0).all()


def test_norm_leaves_what_is_behind_its_rows(lib):
    from fine_grained_fp8_sigmoid_b200 import binding as B
    rows, d = 7, 256
    x, res, w = _inputs(rows, d, torch.bfloat16, torch.float32, seed=3)
    y = torch.full((rows + 3, d), 7.0, dtype=torch.bfloat16, device="cuda")
    q = torch.full((rows + 3, d), 9, dtype=torch.uint8, device="cuda")
    sc = torch.full((rows + 3, 2), 5.0, device="cuda")
    B.moe_rmsnorm_quant(x, w, 1e-6, y=y[:rows], q=q[:rows], scale=sc[:rows], residual=res)
    assert (y[rows:] == 7).all() and (q[rows:] == 9).all() and (sc[rows:] == 5).all()


def _check_backward(dy, h, w, eps, dres, dh, dw, rows):
    d = h.shape[1]
    ref_h, ref_w = O.rmsnorm_backward(dy, h, w, eps, dres)
    r = 1.0 / np.sqrt((h ** 2).mean(-1, keepdims=True) + eps)
    n, g = h * r, dy * w
    # the three terms and what each is off by
    terms = (0 if dres is None else np.abs(dres)) + r * np.abs(g) + r * np.abs(n) * np.abs(g * n).mean(-1, keepdims=True)
    assert (np.abs(f64(dh) - ref_h) <= HALF[dh.dtype] * np.abs(ref_h) + 4 * ROUND * terms + TINY).all()
    assert (np.abs(f64(dw) - ref_w) <= (rows * EPS32 + 4 * ROUND) * np.abs(dy * n).sum(0) + TINY).all()


@pytest.mark.parametrize("rows,d", [(1, 128), (1, 7168), (2, 8), (37, 2048), (148, 256), (149, 256), (700, 384), (301, 7168),
                                    (3, 16384), (1500, 72), (1900, 2048), (2500, 1024), (1200, 4096)])
@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
def test_norm_backward(lib, rows, d, stream):
    from fine_grained_fp8_sigmoid_b200 import binding as B
    x, h, w = _inputs(rows, d, stream, torch.bfloat16 if rows % 2 else torch.float32, seed=rows * 3 + d)
    g = torch.Generator().manual_seed(rows)
    dres = torch.randn(rows, d, generator=g).to(stream).cuda() if rows % 3 else None
    dy = x
    dh, dw = torch.empty_like(h), torch.empty(d, device="cuda")
    ws = torch.full((B.moe_rmsnorm_backward_workspace(rows, d),), 255, dtype=torch.uint8, device="cuda")
    B.moe_rmsnorm_backward(dy, h, w, 1e-6, dh, dw, ws, dres=dres)
    ref = (f64(dy), f64(h), f64(w), 1e-6, None if dres is None else f64(dres))
    _check_backward(*ref, dh, dw, rows)
    again, dw2 = torch.empty_like(dh), torch.empty_like(dw)
    B.moe_rmsnorm_backward(dy, h, w, 1e-6, again, dw2, ws, dres=dres)
    assert torch.equal(again, dh) and torch.equal(dw2, dw)          # the same bits every time
    into = h.clone()
    B.moe_rmsnorm_backward(dy, into, w, 1e-6, into, dw2, ws, dres=dres)
    assert torch.equal(into, dh) and torch.equal(dw2, dw)           # over h


def test_norm_backward_of_no_rows_and_of_a_zero_row(lib):
    from fine_grained_fp8_sigmoid_b200 import binding as B
    d = 256
    dw = torch.full((d,), 3.0, device="cuda")
    e = torch.empty(0, d, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(d, device="cuda")
    ws = torch.empty(B.moe_rmsnorm_backward_workspace(4, d), dtype=torch.uint8, device="cuda")
    B.moe_rmsnorm_backward(e, e, w, 1e-6, e, dw, ws)
    assert (dw == 0).all()
    dy, h, _ = _inputs(4, d, torch.bfloat16, torch.float32, seed=1)
    h[2] = 0.0
    dh = torch.empty_like(h)
    B.moe_rmsnorm_backward(dy, h, w, 1e-6, dh, dw, ws)
    _check_backward(f64(dy), f64(h), f64(w), 1e-6, None, dh, dw, 4)


def test_offsets_past_32_bits(lib):
    from fine_grained_fp8_sigmoid_b200 import binding as B
    rows, d = 140001, 16384
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.empty(rows, d, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    w = torch.ones(d, device="cuda")
    y, q = torch.empty_like(x), torch.empty(rows, d, dtype=torch.uint8, device="cuda")
    scale = torch.empty(rows, d // 128, device="cuda")
    B.moe_rmsnorm_quant(x, w, 1e-6, y=y, q=q, scale=scale)
    for at in (slice(0, 3), slice(131071, 131074), slice(rows - 3, rows)):     # rows * d is 2^31 at 131072
        _check_forward(f64(x[at]), f64(w), 1e-6, None, y[at], q[at], scale[at])
    dh, dw = torch.empty_like(x), torch.empty(d, device="cuda")
    ws = torch.empty(B.moe_rmsnorm_backward_workspace(rows, d), dtype=torch.uint8, device="cuda")
    del q, scale
    B.moe_rmsnorm_backward(x, y, w, 1e-6, dh, dw, ws)
    for at in (slice(0, 3), slice(131071, 131074), slice(rows - 3, rows)):
        ref, _ = O.rmsnorm_backward(f64(x[at]), f64(y[at]), f64(w), 1e-6)
        h, dy = f64(y[at]), f64(x[at])
        r = 1.0 / np.sqrt((h ** 2).mean(-1, keepdims=True) + 1e-6)
        terms = r * np.abs(dy) + r * np.abs(h * r) * np.abs(dy * h * r).mean(-1, keepdims=True)
        assert (np.abs(f64(dh[at]) - ref) <= HALF[torch.bfloat16] * np.abs(ref) + 4 * ROUND * terms + TINY).all()


def test_norm_and_gradient_replay_in_a_graph(lib):
    from fine_grained_fp8_sigmoid_b200 import binding as B
    rows, d = 200, 1024
    x, res, w = _inputs(rows, d, torch.bfloat16, torch.float32, seed=21)
    h, y, q, scale = _outputs(rows, d, torch.bfloat16)
    dh, dw = torch.empty_like(h), torch.empty(d, device="cuda")
    ws = torch.empty(B.moe_rmsnorm_backward_workspace(rows, d), dtype=torch.uint8, device="cuda")

    def step():
        B.moe_rmsnorm_quant(x, w, 1e-6, y=y, q=q, scale=scale, residual=res, h=h)
        B.moe_rmsnorm_backward(y, h, w, 1e-6, dh, dw, ws, dres=res)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    x2, res2, _ = _inputs(rows, d, torch.bfloat16, torch.float32, seed=22)
    x.copy_(x2)
    res.copy_(res2)
    graph.replay()
    got = [t.clone() for t in (h, y, q, scale, dh, dw)]
    step()
    for a, b in zip(got, (h, y, q, scale, dh, dw)):
        assert torch.equal(a, b)
