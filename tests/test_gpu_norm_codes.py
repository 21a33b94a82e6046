"""The norm's E4M3 output bit for bit, and its gradient bit for bit past 32-bit
offsets, on inputs whose FP32 arithmetic is exact.

Rows of +-1 with eps = 0 and d a power of two have a mean square of one and a
root of one, so y = w x exactly, for any FP32 w. A tile's scale is then
fl32(amax / 448) and its codes E4M3(fl32(y / scale)), the quantiser's rule, and
w puts values at and next to the borders of that rounding, where a code formed
in any other way (a product with the reciprocal, say) goes wrong."""
import numpy as np
import pytest
import torch

from oracle.e4m3 import decode, encode

D, TILE, EPS32 = 16384, 128, 2.0 ** -24
#: midpoints of neighbouring E4M3 values: what fl32(y / scale) is rounded at
BORDERS = (decode(np.arange(0, 126)) + decode(np.arange(1, 127))) / 2


def border_weights(seed=0):
    """w [D] FP32: a tile's first value is its maximum, the others lie within two
    FP32 steps of a border times the scale. Every eighth tile is scaled so that
    its scale lies between 2^-149 and 2^-101 or is subnormal."""
    g = np.random.default_rng(seed)
    w = np.empty((D // TILE, TILE), np.float32)
    for i, t in enumerate(w):
        top = np.float32(g.uniform(1, 2) * 2.0 ** (g.integers(-130, -94) if i % 8 == 7 else g.integers(-20, 20)))
        s = top / np.float32(448)
        t[:] = (g.choice(BORDERS, TILE) * np.float64(s)).astype(np.float32)
        t[:] = (t.view(np.int32) + g.integers(-2, 3, TILE)).clip(0, top.view(np.int32)).astype(np.int32).view(np.float32)
        t[0] = top
    return w.reshape(-1)


def tile_codes(w):
    """(codes, scales) of w's tiles by the rule."""
    t = w.reshape(-1, TILE)
    s = t.max(1) / np.float32(448)
    s = np.where(s == 0, np.float32(1), s).astype(np.float32)
    return encode((t / s[:, None]).astype(np.float64)).reshape(-1), s


def test_the_borders_tell_a_division_from_other_forms():
    """What test_codes_at_rounding_borders compares with is not what a product with
    the reciprocal gives, nor either end of a bracket around it."""
    w = border_weights()
    q, s = tile_codes(w)
    t = w.reshape(-1, TILE)
    with np.errstate(over="ignore"):         # of a subnormal scale
        inv = (np.float32(1) / s)[:, None]
    fine = np.repeat(s >= 2.0 ** -100, TILE)
    assert (~fine).sum() >= 10 * TILE and (s < 2.0 ** -126).any()
    for off in (1.0, 1.0 - 2.0 ** -21, 1.0 + 2.0 ** -21):
        with np.errstate(over="ignore"):
            other = encode(((t * inv) * np.float32(off)).astype(np.float64).clip(-448, 448)).reshape(-1)
        assert (other != q)[fine].sum() >= 100


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [1, 150])
def test_codes_at_rounding_borders(lib, rows):
    """One row takes 1024 threads, more rows than SMs take 256."""
    from fine_grained_fp8_sigmoid_b200 import binding as B
    w = border_weights()
    g = torch.Generator().manual_seed(rows)
    sign = torch.randint(0, 2, (rows, D), generator=g) * 2 - 1
    x = sign.to(torch.bfloat16).cuda()
    q = torch.empty(rows, D, dtype=torch.uint8, device="cuda")
    scale = torch.empty(rows, D // TILE, device="cuda")
    B.moe_rmsnorm_quant(x, torch.from_numpy(w).cuda(), 0.0, q=q, scale=scale)
    want, s = tile_codes(w)
    assert np.array_equal(scale.cpu().numpy(), np.broadcast_to(s, (rows, D // TILE)))
    bits = want[None] | np.where(sign.numpy() < 0, 128, 0).astype(np.uint8)
    assert np.array_equal(q.cpu().numpy(), bits)


@pytest.mark.gpu
def test_codes_of_rows_that_are_not_finite(lib):
    """A NaN row is NaN codes; a row with an infinity is zeros but for that channel,
    since 1 / inf is 0. Their scales are 1: a maximum passes over NaN."""
    from fine_grained_fp8_sigmoid_b200 import binding as B
    rows, d = 6, 512
    g = torch.Generator().manual_seed(4)
    x = torch.randn(rows, d, generator=g).to(torch.bfloat16).cuda()
    w = torch.ones(d, device="cuda")
    y, q = torch.empty_like(x), torch.empty(rows, d, dtype=torch.uint8, device="cuda")
    scale = torch.empty(rows, d // 128, device="cuda")
    B.moe_rmsnorm_quant(x, w, 1e-6, q=q, scale=scale)
    q0, s0 = q.clone(), scale.clone()
    x[1, 200] = float("nan")
    x[4, 200] = float("-inf")
    B.moe_rmsnorm_quant(x, w, 1e-6, y=y, q=q, scale=scale)
    keep = [0, 2, 3, 5]
    assert torch.equal(q[keep], q0[keep]) and torch.equal(scale[keep], s0[keep])
    assert ((q[1] & 127) == 127).all() and (scale[[1, 4]] == 1).all()
    others = torch.arange(d, device="cuda") != 200
    assert (q[4, 200] & 127) == 127 and ((q[4, others] & 127) == 0).all()
    q2, s2 = torch.empty_like(q), torch.empty_like(scale)
    B.moe_quant_1x128(y, q2, s2)
    assert torch.equal(q2[[1, 4]], q[[1, 4]]) and torch.equal(s2[[1, 4]], scale[[1, 4]])


@pytest.mark.gpu
def test_every_row_of_a_gradient_past_32_bits(lib):
    """h = +-1 and small whole dy: every sum is a whole number below 2^24, so dh and
    dw are exact, whatever the order; a row that is left out, read twice or
    misplaced shows in dw."""
    from fine_grained_fp8_sigmoid_b200 import binding as B
    rows = 131072 + 301                      # rows * D is past 2^31
    g = torch.Generator(device="cuda").manual_seed(0)
    h, dy = (torch.empty(rows, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    dw_ref = torch.zeros(D, dtype=torch.float64, device="cuda")
    step = 4096
    for a in range(0, rows, step):
        n = min(step, rows - a)
        h[a:a + n] = torch.randint(0, 2, (n, D), generator=g, device="cuda", dtype=torch.int8) * 2 - 1
        dy[a:a + n] = torch.randint(-3, 4, (n, D), generator=g, device="cuda", dtype=torch.int8)
        dw_ref += (h[a:a + n] * dy[a:a + n]).sum(0, dtype=torch.float64)
    dh, dw = torch.empty_like(h), torch.empty(D, device="cuda")
    ws = torch.empty(B.moe_rmsnorm_backward_workspace(rows, D), dtype=torch.uint8, device="cuda")
    B.moe_rmsnorm_backward(dy, h, torch.ones(D, device="cuda"), 0.0, dh, dw, ws)
    assert torch.equal(dw.double(), dw_ref)
    for a in range(0, rows, step):
        hh, gg = h[a:a + step].float(), dy[a:a + step].float()
        mean = (hh * gg).sum(1, keepdim=True) / D
        assert torch.equal(dh[a:a + step], (gg - hh * mean).to(torch.bfloat16))
