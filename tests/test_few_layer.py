"""MoELayerFP8(few=True) without a GPU: what its constructor and its views refuse."""
import pytest

from fine_grained_fp8_sigmoid_b200 import MoELayerFP8


@pytest.mark.parametrize("T,d,N_r,K_r,I", [(4, 384, 8, 2, 128), (4, 8448, 8, 2, 128), (4, 256, 257, 2, 128), (4, 256, 8, 9, 128),
                                           (4, 256, 64, 17, 128), (4, 256, 8, 0, 128), (4, 256, 8, 2, 192), (4, 256, 8, 2, 8320),
                                           (0, 384, 8, 2, 128)])
def test_sizes_outside_the_limits_are_refused_before_any_allocation(monkeypatch, T, d, N_r, K_r, I):
    from fine_grained_fp8_sigmoid_b200 import layer

    def allocated(*a, **k):
        raise AssertionError("allocated")

    monkeypatch.setattr(layer.torch, "empty", allocated)
    with pytest.raises(ValueError, match="few=True needs"):
        MoELayerFP8(T, d, N_r, K_r, I, device="cpu", few=True)


@pytest.mark.parametrize("T", [0, 1, 16])
def test_sizes_inside_the_limits_are_not(T):
    assert MoELayerFP8(T, 256, 8, 8, 128, device="cpu", few=True).ws_few is not None


def test_there_is_no_intermediate_to_view():
    """Its forward does not write the grouped GEMM's workspace: the views would hold whatever was there."""
    layer = MoELayerFP8(2, 256, 8, 2, 128, device="cpu", few=True)
    with pytest.raises(ValueError, match="few=True"):
        layer.intermediate()
    codes, scales = MoELayerFP8(2, 256, 8, 2, 128, device="cpu").intermediate()
    assert codes.shape == (6, 128) and scales.shape == (6, 1)
