"""Two host threads, each with a stream, buffers and a workspace of its own,
call one instantiation of a kernel with different shapes at once: what one
thread sets for its launch must not take anything from the other's."""
import threading

import pytest
import torch

from fine_grained_fp8_sigmoid_b200._lib import check
from tests.test_gpu_few import buffers, call, make, no_error

pytestmark = pytest.mark.gpu

CALLS = 10000


def _together(steps):
    """Runs the steps (each takes a stream) CALLS times in a thread each; their first failures."""
    start, failed = threading.Barrier(len(steps)), []

    def loop(step, stream):
        start.wait()
        try:
            for _ in range(CALLS):
                step(stream)
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    torch.cuda.synchronize()
    threads = [threading.Thread(target=loop, args=(s, torch.cuda.Stream())) for s in steps]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return failed


def test_norm_gradients_of_two_threads(lib):
    """With and without dres a row takes more or less shared memory (84 and 56 KB a
    block). Straight calls of the C entry: they leave least between two launches."""
    from fine_grained_fp8_sigmoid_b200 import binding as B
    rows, d = 460, 7168
    g = torch.Generator(device="cuda").manual_seed(0)
    r = lambda: torch.randn(rows, d, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    steps, outs, first = [], [], []
    for with_dres in (True, False):
        dy, h, dres = r(), r(), r() if with_dres else None
        w = torch.ones(d, device="cuda")
        dh, dw = torch.empty_like(h), torch.empty(d, device="cuda")
        ws = torch.empty(B.moe_rmsnorm_backward_workspace(rows, d), dtype=torch.uint8, device="cuda")
        args = (dy.data_ptr(), h.data_ptr(), 0, w.data_ptr(), 0, 1e-6, dres.data_ptr() if with_dres else None, rows, d,
                dh.data_ptr(), dw.data_ptr(), ws.data_ptr(), ws.nbytes)

        def step(stream, args=args):
            check("moe_rmsnorm_backward", lib.moe_rmsnorm_backward(*args, stream.cuda_stream))

        step(torch.cuda.current_stream())
        steps.append(step)
        outs.append((dh, dw, dy, h, dres, w, ws))
        first.append((dh.clone(), dw.clone()))
    assert _together(steps) == []
    for got, want in zip(outs, first):
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_few_tokens_of_two_threads(lib):
    """207 and 222 KB a block, by the stages that fit beside the tokens."""
    cases = [make(1, 2048, 4, 2, 512, seed=1), make(1, 256, 2, 1, 128, seed=2)]
    outs = [buffers(p) for p in cases]
    for p, o in zip(cases, outs):
        call(p, o)
    first = [{k: o[k].clone() for k in ("out", "topk_idx", "gates", "counts")} for o in outs]
    steps = []
    for p, o in zip(cases, outs):
        T, d, N, K, I = p["dims"]
        a = {k: v.data_ptr() for k, v in {**p, **o}.items() if isinstance(v, torch.Tensor)}
        args = (a["u"], None, None, None, a["e"], a["b"], T, d, N, K, a["w_gate"], a["w_up"], a["w_down"], a["s_gate"],
                a["s_up"], a["s_down"], I, a["out"], a["topk_idx"], a["gates"], a["counts"], a["workspace"],
                o["workspace"].nbytes)
        steps.append(lambda s, args=args: check("moe_few_tokens", lib.moe_few_tokens(*args, s.cuda_stream)))
    assert _together(steps) == []
    no_error()
    for o, want in zip(outs, first):
        for k, v in want.items():
            assert torch.equal(o[k], v)
