"""moe_few_tokens with nine to fifteen experts a token, where K_r is neither a
power of two nor a divisor of a warp, up to every expert there is."""
import pytest

from tests.test_gpu_few import buffers, call, check, make, no_error

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dims", [(1, 256, 33, 9, 128), (6, 512, 10, 10, 256), (16, 256, 64, 11, 128), (9, 768, 256, 12, 128),
                                  (16, 256, 13, 13, 384), (3, 512, 40, 14, 128), (8, 256, 15, 15, 128)])
def test_nine_to_fifteen_experts_a_token(lib, dims):
    p = make(*dims, seed=sum(dims), integers=True)
    o = buffers(p)
    call(p, o)
    no_error()
    check(p, o, exact=True)
    p = make(*dims, seed=sum(dims) + 1, quantised=True, base=True)
    o = buffers(p)
    call(p, o)
    no_error()
    check(p, o)
