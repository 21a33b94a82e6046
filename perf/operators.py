"""The operators around the expert layer that a serving or training step calls
for itself: the pre-norm with the residual's addition and E4M3 output, its
gradient, and the whole layer for a few tokens. Each case is one call.

  norm      s = x + residual, h = bf16(s) (or FP32), y = s rsqrt(mean s^2 + eps) w,
            y as bf16 for the router and as E4M3 codes with one FP32 scale per
            1x128 tile for the experts
  norm_bwd  n = h rsqrt(mean h^2 + eps), g = dy w,
            dh = dres + rsqrt(mean h^2 + eps) (g - n mean(g n)), dw = sum_t dy n
  few       s = sigmoid(u e^T), the K_r largest of s + b (equal ones by the lower
            index), gates s / sum s, and
            out = base + FFN_shared(u) + sum_k gate_k FFN_k(u)
            with FFN(u) = requant(silu(G) U) W_down^T, G = u W_gate^T, U = u W_up^T
            on E4M3 activations (1x128 scales) and weights (128x128 scales)
"""
import math

import torch

own = False

E4M3 = torch.float8_e4m3fn
TOP = 448.0
EPS = 1e-6


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token of a decode step: latency alone
        dict(name="norm_one", op="norm", rows=1, d=7168, fp32=False, residual=True, quant=True),
        # a decode batch
        dict(name="norm_decode", op="norm", rows=128, d=7168, fp32=False, residual=True, quant=True),
        # a training batch of the smaller layer: FP32 residual stream, odd number of rows
        dict(name="norm_mid_fp32", op="norm", rows=4001, d=2048, fp32=True, residual=True, quant=True),
        # a prefill batch
        dict(name="norm_prefill", op="norm", rows=8192, d=7168, fp32=False, residual=True, quant=True),
        # gradients of a ragged micro-batch
        dict(name="norm_bwd_ragged", op="norm_bwd", rows=301, d=2048, fp32=False, dres=True),
        # gradients with the FP32 stream
        dict(name="norm_bwd_mid_fp32", op="norm_bwd", rows=4096, d=2048, fp32=True, dres=True),
        # gradients of a full batch
        dict(name="norm_bwd_prefill", op="norm_bwd", rows=8192, d=7168, fp32=False, dres=True),
        # the layer for one token of the small shape, and for a few
        dict(name="few_mid_1", op="few", T=1, d=2048, N_r=64, K_r=6, I=1024, quantised=False, base=False),
        dict(name="few_mid_13", op="few", T=13, d=2048, N_r=64, K_r=6, I=1024, quantised=True, base=True),
        # the full shape: a single stream, a few streams, and the most tokens
        dict(name="few_full_1", op="few", T=1, d=7168, N_r=256, K_r=8, I=2048, quantised=True, base=True),
        dict(name="few_full_4", op="few", T=4, d=7168, N_r=256, K_r=8, I=2048, quantised=True, base=True),
        dict(name="few_full_16", op="few", T=16, d=7168, N_r=256, K_r=8, I=2048, quantised=False, base=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "few"])
    if op == "few":
        N_r = _log(rng, 2, 256)
        return dict(op="few", T=rng.randint(1, 16), d=256 * _log(rng, 1, 28), N_r=N_r, K_r=rng.randint(1, min(8, N_r)),
                    I=128 * _log(rng, 1, 16), quantised=rng.random() < 0.5, base=rng.random() < 0.5)
    rows, d, fp32 = _log(rng, 1, 8192), 128 * _log(rng, 1, 56), rng.random() < 0.3
    if fp32 and rows * d > 4096 * 7168:      # no dearer than the largest listed batch
        rows = 4096 * 7168 // d
    if op == "norm":
        return dict(op="norm", rows=rows, d=d, fp32=fp32, residual=rng.random() < 0.8, quant=rng.random() < 0.8)
    return dict(op="norm_bwd", rows=rows, d=d, fp32=fp32, dres=rng.random() < 0.8)


def work(case):
    if case["op"] == "few":
        T, d, N, K, I = (case[k] for k in ("T", "d", "N_r", "K_r", "I"))
        touched = N * (1.0 - (1.0 - K / N) ** T) + 1
        return {"bytes": touched * (3 * d * I + 3 * d * I / 128 / 128 * 4) + 2 * N * d + 2 * T * d * (2 + case["base"]),
                "flops": 6.0 * T * (K + 1) * d * I + 2.0 * T * N * d}
    n, s = case["rows"] * case["d"], 4 if case["fp32"] else 2
    if case["op"] == "norm":
        b = n * (2 + 2) + n * s * (2 if case["residual"] else 0) + n * (1 + 1 / 32) * case["quant"]
        return {"bytes": b + 4 * case["d"], "flops": 8.0 * n}
    return {"bytes": n * (2 + 2 * s + (s if case["dres"] else 0)) + 8 * case["d"], "flops": 12.0 * n}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _quantise(v):
    """E4M3 codes (as uint8) and FP32 scales of 1x128 tiles of v (FP32). The scale is
    amax / 448 rounded once: bf16 values meet exact ties, which it decides."""
    t = v.view(v.shape[0], -1, 128)
    s = (t.abs().amax(-1).double() / TOP).float()
    s = torch.where(s == 0, torch.ones_like(s), s)
    q = (t / s[..., None]).clamp(-TOP, TOP).to(E4M3)
    return q.view(v.shape).view(torch.uint8), s


def _weights(g, groups, rows, cols):
    """Codes and block scales such as quantising N(0, 0.02) weights gives."""
    q = torch.empty(groups, rows, cols, dtype=torch.uint8, device="cuda")
    for i in range(0, groups, 16):
        w = torch.randn(min(16, groups - i), rows, cols, generator=g, device="cuda")
        q[i:i + 16] = w.mul_(104.0).clamp_(-TOP, TOP).to(E4M3).view(torch.uint8)
    s = (0.9 + 0.2 * torch.rand(groups, rows // 128, cols // 128, generator=g, device="cuda")) * (0.02 / 104.0)
    return q, s


def prepare(case, seed):
    g = _gen(seed)
    bf, f32, dev = torch.bfloat16, torch.float32, "cuda"
    rand = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
    st = dict(case)
    if case["op"] == "few":
        T, d, N, K, I = (case[k] for k in ("T", "d", "N_r", "K_r", "I"))
        st["u"] = rand(T, d).to(bf)
        st["e"] = (rand(N, d) / math.sqrt(d)).to(bf)
        st["b"] = rand(N) * 0.01
        st["x0"] = (rand(T, d) * 2).to(bf) if case["base"] else None
        st["xq"], st["xs"] = _quantise(st["u"].float()) if case["quantised"] else (None, None)
        for n, r, c in (("gate", I, d), ("up", I, d), ("down", d, I)):
            st["w_" + n], st["s_" + n] = _weights(g, N + 1, r, c)
        st["out"] = torch.empty(T, d, dtype=bf, device=dev)
        st["idx"] = torch.empty(T, K, dtype=torch.int32, device=dev)
        st["gates"] = torch.empty(T, K, dtype=f32, device=dev)
        st["counts"] = torch.empty(N, dtype=torch.int32, device=dev)
        return st
    rows, d = case["rows"], case["d"]
    stream = f32 if case["fp32"] else bf
    st["w"] = 1.0 + 0.1 * rand(d)
    if case["op"] == "norm":
        st["x"] = rand(rows, d).to(bf)
        # a residual stream carries a few large channels
        st["res"] = ((rand(rows, d) * (1.0 + 20.0 * (torch.rand(d, generator=g, device=dev) < 0.002))).to(stream)
                     if case["residual"] else None)
        st["h"] = torch.empty(rows, d, dtype=stream, device=dev) if case["residual"] else None
        st["y"] = torch.empty(rows, d, dtype=bf, device=dev)
        st["q"] = torch.empty(rows, d, dtype=torch.uint8, device=dev) if case["quant"] else None
        st["scale"] = torch.empty(rows, d // 128, dtype=f32, device=dev) if case["quant"] else None
    else:
        st["dy"] = (rand(rows, d) * 0.01).to(bf)
        st["h"] = (rand(rows, d) * 2).to(stream)
        st["dres"] = (rand(rows, d) * 0.01).to(stream) if case["dres"] else None
        st["dh"] = torch.empty(rows, d, dtype=stream, device=dev)
        st["dw"] = torch.empty(d, dtype=f32, device=dev)
    return st


# ------------------------------------------------------------------ one pass

def run(state):
    return {"norm": _norm, "norm_bwd": _norm_bwd, "few": _few}[state["op"]](state)


def _norm(st):
    if own:
        from fine_grained_fp8_sigmoid_b200 import binding as B
        B.moe_rmsnorm_quant(st["x"], st["w"], EPS, residual=st["res"], h=st["h"], y=st["y"], q=st["q"],
                            scale=st["scale"])
        got = [st["h"], st["y"], None if st["q"] is None else st["q"].view(E4M3), st["scale"]]
    else:
        s = st["x"].float()
        if st["res"] is not None:
            s = s + st["res"].float()
        y = s * torch.rsqrt((s * s).mean(-1, keepdim=True) + EPS) * st["w"]
        h = None if st["res"] is None else s.to(st["res"].dtype)
        q, scale = _quantise(y) if st["quant"] else (None, None)
        got = [h, y.to(torch.bfloat16), None if q is None else q.view(E4M3), scale]
    return [t for t in got if t is not None]


def _norm_bwd(st):
    if own:
        from fine_grained_fp8_sigmoid_b200 import binding as B
        if "ws" not in st:
            st["ws"] = torch.empty(B.moe_rmsnorm_backward_workspace(st["rows"], st["d"]), dtype=torch.uint8,
                                   device="cuda")
        B.moe_rmsnorm_backward(st["dy"], st["h"], st["w"], EPS, st["dh"], st["dw"], st["ws"], dres=st["dres"])
        return [st["dh"], st["dw"]]
    h, dy = st["h"].float(), st["dy"].float()
    r = torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS)
    n, g = h * r, dy * st["w"]
    dh = r * (g - n * (g * n).mean(-1, keepdim=True))
    if st["dres"] is not None:
        dh = dh + st["dres"].float()
    return [dh.to(st["h"].dtype), (dy * n).sum(0)]


def _values(q, s):
    """FP32 values of codes [.., R, C] with one scale per 128x128 block."""
    v = q.view(E4M3).float()
    R, C = v.shape[-2:]
    v.view(*v.shape[:-2], R // 128, 128, C // 128, 128).mul_(s[..., :, None, :, None])
    return v


def _tiles(q, s):
    """FP32 values of codes [rows, C] with one scale per 1x128 tile."""
    v = q.view(E4M3).float()
    v.view(v.shape[0], -1, 128).mul_(s[..., None])
    return v


def _few(st):
    if own:
        from fine_grained_fp8_sigmoid_b200 import binding as B
        if "ws" not in st:
            st["ws"] = torch.empty(B.moe_few_tokens_workspace(st["T"], st["d"], st["N_r"], st["K_r"], st["I"]),
                                   dtype=torch.uint8, device="cuda")
        B.moe_few_tokens(st["u"], st["e"], st["b"], st["K_r"], st["w_gate"], st["w_up"], st["w_down"], st["s_gate"],
                         st["s_up"], st["s_down"], st["out"], st["idx"], st["gates"], st["ws"], xq=st["xq"],
                         xs=st["xs"], base=st["x0"], counts=st["counts"])
        return [st["out"], st["idx"], st["gates"], st["counts"]]
    T, d, N, K, I = (st[k] for k in ("T", "d", "N_r", "K_r", "I"))
    u = st["u"]
    # the selection is a border: its logits in 64 bits, the keys in 32 as defined
    s = torch.sigmoid(u.double() @ st["e"].double().t()).float()
    idx = torch.sort(s + st["b"], dim=1, descending=True, stable=True)[1][:, :K]
    sel = s.gather(1, idx)
    gates = sel / sel.sum(1, keepdim=True)
    xq, xs = (st["xq"], st["xs"]) if st["xq"] is not None else _quantise(u.float())
    x = _tiles(xq, xs)
    pick = idx.reshape(-1)
    xr = x.repeat_interleave(K, 0)[:, :, None]
    G = torch.cat([(_values(st["w_gate"][pick], st["s_gate"][pick]) @ xr).squeeze(-1),
                   x @ _values(st["w_gate"][N], st["s_gate"][N]).t()])
    U = torch.cat([(_values(st["w_up"][pick], st["s_up"][pick]) @ xr).squeeze(-1),
                   x @ _values(st["w_up"][N], st["s_up"][N]).t()])
    H = _tiles(*_quantise(G * torch.sigmoid(G) * U))
    y = (_values(st["w_down"][pick], st["s_down"][pick]) @ H[:T * K, :, None]).squeeze(-1).view(T, K, d)
    out = (u if st["x0"] is None else st["x0"]).float() + H[T * K:] @ _values(st["w_down"][N], st["s_down"][N]).t()
    out = out + (gates[:, :, None] * y).sum(1)
    counts = torch.bincount(pick, minlength=N).to(torch.int32)
    return [out.to(torch.bfloat16), idx.to(torch.int32), gates, counts]


# ------------------------------------------------------------------ in 64 bits

def _e4m3_64(v):
    """Nearest E4M3 value (ties to even) of float64 v, saturating at 448."""
    a = v.abs().clamp(max=TOP)
    _, ex = torch.frexp(a)
    step = torch.ldexp(torch.ones_like(a), (ex - 1).clamp(min=-6) - 3)
    return torch.sign(v) * (torch.round(a / step) * step).clamp(max=TOP)


def _block_64(v):
    """1x128 tiles of v (float64): E4M3 values and scales. The scale and the quotient
    are FP32 by definition: bf16 values meet exact ties, which those roundings decide."""
    t = v.reshape(v.shape[0], v.shape[1] // 128, 128)
    top = t.abs().max(dim=2, keepdim=True).values
    s = torch.where(top > 0, top / TOP, torch.ones_like(top)).float().to(v.dtype)
    return _e4m3_64((t / s).float().to(v.dtype)).reshape(v.shape), s[..., 0]


def exact(case, seed):
    st = prepare(case, seed)
    D = torch.float64
    if case["op"] == "norm":
        s = st["x"].to(D) if st["res"] is None else torch.add(st["x"].to(D), st["res"].to(D))
        rms = torch.sqrt(torch.sum(s ** 2, dim=1) / case["d"] + EPS)
        y = s / rms[:, None] * st["w"].to(D)[None]
        got = [] if st["res"] is None else [s]
        return got + [y] + (list(_block_64(y)) if case["quant"] else [])
    if case["op"] == "norm_bwd":
        h, dy, w = st["h"].to(D), st["dy"].to(D), st["w"].to(D)
        q = torch.sum(h * h, dim=1, keepdim=True) / case["d"] + EPS
        proj = torch.sum(dy * w * h, dim=1, keepdim=True) / case["d"]
        dh = dy * w / q.sqrt() - h * proj / q ** 1.5
        if st["dres"] is not None:
            dh += st["dres"].to(D)
        return [dh, torch.einsum("td,td->d", dy, h / q.sqrt())]
    T, d, N, K = (case[k] for k in ("T", "d", "N_r", "K_r"))
    u, e = st["u"].to(D), st["e"].to(D)
    aff = (1.0 / (1.0 + torch.exp(-torch.einsum("td,nd->tn", u, e)))).float()
    key = (aff + st["b"]).cpu().tolist()
    order = [sorted(range(N), key=lambda i, row=row: (-row[i], i))[:K] for row in key]
    sel = torch.stack([aff[t].to(D)[order[t]] for t in range(T)])
    gates = sel / sel.sum(dim=1, keepdim=True)
    if st["xq"] is None:
        v, s = _block_64(u)
    else:
        v, s = st["xq"].view(E4M3).to(D), st["xs"].to(D)
    x = v * s.repeat_interleave(128, dim=1)

    def weight(n, i):
        w = st["w_" + n][i].view(E4M3).to(D)
        return w * st["s_" + n][i].to(D).repeat_interleave(128, 0).repeat_interleave(128, 1)

    out = u.clone() if st["x0"] is None else st["x0"].to(D)
    counts = [0] * N
    for i in sorted({i for row in order for i in row}) + [N]:
        ts = [t for t in range(T) if i == N or i in order[t]]
        a = x[ts] @ weight("gate", i).T
        hv, hs = _block_64(a / (1.0 + torch.exp(-a)) * (x[ts] @ weight("up", i).T))
        y = (hv * hs.repeat_interleave(128, dim=1)) @ weight("down", i).T
        if i < N:
            counts[i] = len(ts)
            y = y * torch.stack([gates[t][order[t].index(i)] for t in ts])[:, None]
        out[ts] += y
    return [out, torch.tensor(order, dtype=torch.int32), gates, torch.tensor(counts, dtype=torch.int32)]
