"""moe_few_tokens, the whole layer for a few tokens in one kernel, against a
plain float64 layer (torch, on the same codes and scales).

Selection, gates and counts. The kernel sums logits in FP64 and rounds each
affinity once, so its FP32 keys are the reference's: indices are equal.

Outputs. An FP32 sum of n roundings is off by at most n 2^-24 of the sum of
its absolute terms; the tensor cores add a 128-wide block with fewer bits, for
which tests/parity.py's ROUNDINGS allows (8 (blocks + 8) in all). A code of the
intermediate may be the neighbour where its value lies within that distance of
a rounding border: such an element's whole step times its weight counts toward
the bound of every output it feeds. The output adds half a bf16 step. Where
every product is a small integer the sums are exact and only silu's few
roundings remain.
"""
import numpy as np
import pytest
import torch

from tests.parity import EPS32, ROUNDINGS

pytestmark = pytest.mark.gpu

D = torch.float64
E4M3 = torch.float8_e4m3fn


def e4m3(v):
    """The nearest E4M3 value (float64 in and out), saturating."""
    a = v.abs().clamp(max=448.0)
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    return torch.sign(v) * torch.round(a / step) * step


def blocks(q, s):
    return q.view(E4M3).to(D) * s.to(D).repeat_interleave(128, 0).repeat_interleave(128, 1)


def tiles(q, s):
    return q.view(E4M3).to(D) * s.to(D).repeat_interleave(128, 1)


def quantise(v):
    """(values, scales) of 1x128 tiles: both roundings to FP32 are the rule's."""
    t = v.view(v.shape[0], -1, 128)
    s = (t.abs().amax(-1) / 448.0).float().to(D)
    s = torch.where(s == 0, torch.ones_like(s), s)
    return e4m3((t / s[..., None]).float().to(D)).view(v.shape), s


def select(u, e, b, K):
    aff = torch.sigmoid(u.to(D) @ e.to(D).t()).float()
    key = (aff + b).cpu().numpy()
    idx = torch.from_numpy(np.argsort(-key, axis=1, kind="stable")[:, :K].copy()).cuda()
    sel = aff.to(D).gather(1, idx)
    return idx, sel / sel.sum(1, keepdim=True)


def reference(p, exact=False):
    """(out, bound, idx, gates) in float64; exact: G and U have no rounding."""
    T, d, N, K, I = p["dims"]
    idx, gates = select(p["u"], p["e"], p["b"], K)
    if p["xq"] is None:
        xv, xs = quantise(p["u"].to(D))
        x = xv * xs.repeat_interleave(128, 1)
    else:
        x = tiles(p["xq"], p["xs"])
    base = (p["u"] if p["base"] is None else p["base"]).to(D)
    out, bound, mass = base.clone(), torch.zeros(T, d, dtype=D, device="cuda"), base.abs()
    slots = sorted(set(idx.flatten().tolist())) + [N]
    rd, ri = (0.0 if exact else ROUNDINGS(d // 128)) * EPS32, ROUNDINGS(I // 128) * EPS32
    for i in slots:
        wg, wu, wd = (blocks(p["w_" + n][i], p["s_" + n][i]) for n in ("gate", "up", "down"))
        ts = list(range(T)) if i == N else [t for t in range(T) if (idx[t] == i).any()]
        g = torch.ones(len(ts), 1, dtype=D, device="cuda") if i == N else gates[ts][idx[ts] == i][:, None]
        a = x[ts]
        G, U = a @ wg.t(), a @ wu.t()
        dG, dU = rd * (a.abs() @ wg.abs().t()), rd * (a.abs() @ wu.abs().t())
        sig = torch.sigmoid(G)
        v = G * sig * U
        dv = 1.1 * dG * U.abs() + (G * sig).abs() * dU + 8 * EPS32 * v.abs()
        hv, hs = quantise(v)
        sr = hs.repeat_interleave(128, 1)
        top = v.view(len(ts), -1, 128).abs().amax(-1)
        srel = torch.where(top > 0, dv.view(len(ts), -1, 128).amax(-1) / top.clamp(min=1e-300), 0 * top) + 4 * EPS32
        srel = srel.repeat_interleave(128, 1)
        z, dz = v / sr, dv / sr + (v / sr).abs() * srel
        near = (e4m3(z + dz) - e4m3(z - dz)).abs() * sr
        H = hv * sr
        y, ya = H @ wd.t(), H.abs() @ wd.abs().t()
        out[ts] += g * y
        bound[ts] += g * ((near + H.abs() * srel) @ wd.abs().t() + ri * ya)
        mass[ts] += g * ya
    bound += (len(slots) * (I // 1024 + 1) + 32) * EPS32 * mass
    return out, bound, idx, gates


def make(T, d, N, K, I, seed, quantised=False, base=False, integers=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    p = dict(dims=(T, d, N, K, I), u=r(T, d).to(torch.bfloat16), e=(r(N, d) / d ** 0.5).to(torch.bfloat16),
             b=r(N) * 0.01, base=(r(T, d) * 2).to(torch.bfloat16) if base else None, xq=None, xs=None)
    for n, a, c in (("gate", I, d), ("up", I, d), ("down", d, I)):
        if integers:      # values in {-1, 0, 1}, power-of-two scales that differ from block to block
            w = torch.randint(-1, 2, (N + 1, a, c), generator=g, device="cuda").float()
            s = torch.exp2(torch.randint(-7, -4, (N + 1, a // 128, c // 128), generator=g, device="cuda").float())
        else:
            w = r(N + 1, a, c) * 100
            s = (0.8 + 0.4 * torch.rand(N + 1, a // 128, c // 128, generator=g, device="cuda")) * (1.5 / 100 / c ** 0.5)
        p["w_" + n], p["s_" + n] = w.clamp(-448, 448).to(E4M3).view(torch.uint8), s
    if integers:
        p["xq"] = torch.randint(-2, 3, (T, d), generator=g, device="cuda").float().to(E4M3).view(torch.uint8)
        p["xs"] = torch.exp2(torch.randint(-3, 0, (T, d // 128), generator=g, device="cuda").float())
    elif quantised:
        v, s = quantise(r(T, d).to(torch.bfloat16).to(D))
        p["xq"], p["xs"] = v.float().to(E4M3).view(torch.uint8), s.float()
    return p


def buffers(p):
    from fine_grained_fp8_sigmoid_b200 import binding as B
    T, d, N, K, I = p["dims"]
    i32 = dict(dtype=torch.int32, device="cuda")
    return dict(out=torch.full((T, d), 3.0, dtype=torch.bfloat16, device="cuda"), topk_idx=torch.full((T, K), -5, **i32),
                gates=torch.full((T, K), -1.0, device="cuda"), counts=torch.full((N,), -9, **i32),
                workspace=torch.full((B.moe_few_tokens_workspace(T, d, N, K, I),), 255, dtype=torch.uint8, device="cuda"))


def call(p, o, **kw):
    from fine_grained_fp8_sigmoid_b200 import binding as B
    o = {**o, **kw}
    B.moe_few_tokens(p["u"], p["e"], p["b"], p["dims"][3], p["w_gate"], p["w_up"], p["w_down"], p["s_gate"], p["s_up"],
                     p["s_down"], o["out"], o["topk_idx"], o["gates"], o["workspace"], xq=p["xq"], xs=p["xs"],
                     base=p["base"], counts=o["counts"], stream=o.get("stream"))


def no_error():
    from fine_grained_fp8_sigmoid_b200 import binding as B
    assert B.moe_get_error() == 0


def check(p, o, exact=False):
    T, d, N, K, I = p["dims"]
    out, bound, idx, gates = reference(p, exact)
    assert torch.equal(o["topk_idx"].long(), idx)
    assert ((o["gates"].to(D) - gates).abs() <= (K + 4) * EPS32 * gates).all()
    assert torch.equal(o["counts"].long(), torch.bincount(idx.flatten(), minlength=N))
    err = (o["out"].to(D) - out).abs()
    bad = err > bound + 2.0 ** -8 * (out.abs() + bound)
    assert not bad.any(), (int(bad.sum()), torch.nonzero(bad)[0].tolist(), float((err / bound).max()))


SIZES = [(1, 256, 2, 1, 128), (2, 512, 4, 4, 256), (16, 256, 8, 2, 128), (9, 768, 33, 5, 384), (5, 1280, 7, 3, 1152),
         (8, 2048, 64, 6, 1024), (13, 2048, 64, 6, 1024), (16, 256, 256, 16, 128), (1, 256, 1, 1, 2048),
         (3, 7168, 16, 8, 2048), (16, 7168, 12, 8, 2048), (7, 8192, 3, 2, 1280)]


@pytest.mark.parametrize("dims", SIZES)
def test_exact_sums(lib, dims):
    p = make(*dims, seed=sum(dims), integers=True, base=dims[0] % 2 == 0)
    o = buffers(p)
    call(p, o)
    no_error()
    check(p, o, exact=True)


@pytest.mark.parametrize("dims", SIZES)
def test_random(lib, dims):
    p = make(*dims, seed=sum(dims) + 1, quantised=dims[0] % 2 == 1, base=dims[1] % 512 == 0)
    o = buffers(p)
    call(p, o)
    no_error()
    check(p, o)
    first = [o[k].clone() for k in ("out", "topk_idx", "gates", "counts")]
    call(p, o)                           # the same workspace again: the same bits
    for k, v in zip(("out", "topk_idx", "gates", "counts"), first):
        assert torch.equal(o[k], v)


@pytest.mark.parametrize("T", range(1, 17))
def test_every_number_of_tokens(lib, T):
    p = make(T, 512, 24, 4, 256, seed=T, integers=True)
    o = buffers(p)
    call(p, o)
    no_error()
    check(p, o, exact=True)


@pytest.mark.parametrize("T,d,I", [(16, 8192, 8192), (8, 8192, 8192), (16, 256, 8192)])
def test_largest_sizes(lib, T, d, I):
    p = make(T, d, 3, 2, I, seed=1, integers=True)
    o = buffers(p)
    call(p, o)
    no_error()
    check(p, o, exact=True)


def test_full_shape(lib):
    """Weights past 2^31 bytes a matrix."""
    p = make(2, 7168, 256, 8, 2048, seed=2, integers=True)
    o = buffers(p)
    call(p, o)
    no_error()
    check(p, o, exact=True)


def test_ties_go_to_the_lower_expert(lib):
    p = make(11, 512, 32, 5, 128, seed=4, integers=True)
    p["e"][1::2] = p["e"][0::2]          # pairs of equal centroids
    p["b"].zero_()
    p["b"][7] = -0.0
    o = buffers(p)
    call(p, o)
    check(p, o, exact=True)
    p["e"].zero_()                       # all equal
    call(p, o)
    check(p, o, exact=True)
    assert torch.equal(o["topk_idx"].cpu(), torch.arange(5, dtype=torch.int32).expand(11, 5))


def test_every_token_on_the_same_experts(lib):
    p = make(16, 512, 64, 4, 256, seed=5, integers=True)
    p["u"][:] = p["u"][0].clone()
    o = buffers(p)
    call(p, o)
    check(p, o, exact=True)


def test_own_quantisation_equals_the_quantiser(lib):
    from fine_grained_fp8_sigmoid_b200 import binding as B
    p = make(13, 1280, 16, 3, 256, seed=6)
    p["u"][3, :128] = 0.0
    p["u"][4] *= 2.0 ** -120
    o, o2 = buffers(p), buffers(p)
    call(p, o)
    xq = torch.empty(13, 1280, dtype=torch.uint8, device="cuda")
    xs = torch.empty(13, 10, device="cuda")
    B.moe_quant_1x128(p["u"], xq, xs)
    call({**p, "xq": xq, "xs": xs}, o2)
    for k in ("out", "topk_idx", "gates", "counts"):
        assert torch.equal(o[k], o2[k])


def test_outputs_over_inputs_and_optional_ones(lib):
    p = make(6, 768, 9, 2, 256, seed=7, base=True)
    o = buffers(p)
    call(p, o)
    q = {**p, "base": p["base"].clone()}
    call(q, o2 := buffers(p), out=q["base"], counts=None)
    assert torch.equal(q["base"], o["out"]) and (o2["counts"] == -9).all()
    p["base"] = None
    call(p, o)
    q = {**p, "u": p["u"].clone()}
    call(q, buffers(p), out=q["u"])
    assert torch.equal(q["u"], o["out"])


def test_bad_values_stay_with_their_token(lib):
    p = make(10, 512, 16, 3, 256, seed=8, integers=True)
    o, o2 = buffers(p), buffers(p)
    call(p, o)
    p["u"][2, 5] = float("nan")          # its keys are NaN: any valid experts
    p["u"][7, 9] = float("inf")
    p["xs"][4, 1] = float("nan")
    call(p, o2)
    no_error()
    keep = [t for t in range(10) if t not in (2, 4, 7)]
    for k in ("out", "topk_idx", "gates"):
        assert torch.equal(o2[k][keep], o[k][keep])
    assert ((o2["topk_idx"] >= 0) & (o2["topk_idx"] < 16)).all()
    assert torch.isnan(o2["out"][4]).any()
    # an expert with a NaN weight reaches only the tokens that chose it
    p = make(10, 512, 16, 1, 256, seed=8, integers=True)
    call(p, o := buffers(p))
    e = int(o["topk_idx"][0, 0])
    p["w_down"][e] = 0x7F
    call(p, o2 := buffers(p))
    hit = (o["topk_idx"][:, 0] == e)
    assert torch.isnan(o2["out"][hit]).all() and torch.equal(o2["out"][~hit], o["out"][~hit])


def test_graph_replay_with_new_inputs(lib):
    p, p2 = make(5, 1024, 32, 4, 512, seed=9), make(5, 1024, 32, 4, 512, seed=10)
    o = buffers(p)
    call(p, o)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(p, o)
    p["u"].copy_(p2["u"])
    for _ in range(3):
        graph.replay()
    check(p, o)
    no_error()


def test_two_calls_at_once(lib):
    """Two streams, a workspace each: cooperative launches take turns."""
    ps = [make(4, 1024, 32, 4, 512, seed=s) for s in (11, 12)]
    os_ = [buffers(p) for p in ps]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for p, o, s in zip(ps, os_, streams):
            call(p, o, stream=s)
    torch.cuda.synchronize()
    for p, o in zip(ps, os_):
        check(p, o)
    no_error()


def test_no_tokens(lib):
    p = make(1, 256, 8, 2, 128, seed=0)
    counts = torch.full((8,), 4, dtype=torch.int32, device="cuda")
    a = p["u"].data_ptr()
    assert lib.moe_few_tokens(a, None, None, None, a, a, 0, 256, 8, 2, a, a, a, a, a, a, 128, a, a, a,
                              counts.data_ptr(), a, 1 << 20, torch.cuda.current_stream().cuda_stream) == 0
    assert (counts == 0).all()
